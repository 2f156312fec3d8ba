// The power-of-two units of the chunked delta rule, exponents only: shared by
// the kernels and their test on the CPU.
//
// A value channel's state is held as S 2^un.  Everything below has to stay
// finite in fp32 for every unit: 2^-un, v 2^un, and the bound of the next state.
#pragma once

namespace sconv {

// Exponents of magnitudes are held to these; 2^(14 - kMinExp) is the largest unit.
constexpr int kMinExp = -112, kMaxExp = 127;
__host__ __device__ inline int held_exp(int e) { return e < kMinExp ? kMinExp : (e > kMaxExp ? kMaxExp : e); }

// A and T are held times 2^kTriExp, X is scaled to 2^kXExp by its own exponent xe, so z = T X comes in units of
// 2^(xe - kZExp).
constexpr int kTriExp = 6, kXExp = 12, kZExp = kXExp + kTriExp;
__host__ __device__ inline int x_exp(int e) { return e < kZExp - 126 ? kZExp - 126 : e; }

// The unit of a state whose largest element lies below 2^e: at 2^14.
__host__ __device__ inline int first_unit(int e) { return 14 - held_exp(e); }

// Up to this unit a chunk's values, and kf beta times them, may be as large as 2^80: X stays below 2^113, z below 2^(xe + 7)
// with X < 2^xe, and the next state's bound, 128 of it, below 2^127.
constexpr int kPlainUnit = 32;
// Above it (a state below 2^-18) the unit is lowered so far that the chunk's values, below 2^e, lie below 2^90, with
// kf beta up to 2^22.  What this takes from the state's operands is 2^-115 of the largest of the values.
__host__ __device__ inline int unit_for_values(int un, int e) {
    const int most = 90 - held_exp(e);
    return un < most ? un : most;
}

struct UnitStep { int up, zu; };
// From the unit un to the next one, un + up: 2^14 above a bound of the next state, below 2^e in units of un; a state of 0
// says nothing about the next chunk's values and has the unit 1.  z takes 2^zu.
__host__ __device__ inline UnitStep next_unit(int un, bool zero, int e, int xe) {
    int up = zero ? -un : 14 - held_exp(e);
    up = up < -126 - un ? -126 - un : (up > 126 - un ? 126 - un : up);
    up = up < -114 ? -114 : up;
    int zu = xe - kZExp + up;
    zu = zu < -126 ? -126 : (zu > 126 ? 126 : zu);
    return {up, zu};
}

}  // namespace sconv

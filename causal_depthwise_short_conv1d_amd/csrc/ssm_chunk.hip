// The selective state space scan of the head form over 64-token chunks: prefill
// on the matrix cores.
//
// With d_j the step sizes, G the running sum of the log decay d A inside a chunk
// and S the state before it:
//   y_i = e^G_i (S C_i) + sum_(j <= i) e^(G_i - G_j) d_j (B_j . C_i) x_j + D x_i
//   S <- e^G_last S + sum_j (e^(G_last - G_j) d_j x_j) B_j^T
//
// A wave owns 32 channels of one head: their states in its registers, the chunk's
// x in a piece of LDS of its own.  The waves of a workgroup belong to one group
// and share its B and C, which come to LDS a chunk ahead, without passing
// registers.  Two waves (w and w + W / 2, on one SIMD) hold 64 channels of a head:
// one prepares the decays and a third of the scores, the other the rest.
//
// Operands.  v_mfma_f32_32x32x16_bf16: a result has its column in the lane and
// rows (q % 4) + 8 (q / 4) + 4 (l / 32) in its registers q; an operand has its row
// or column in the lane and 8 contracted places 8 (l / 32) .. in its registers.
// Since the order of a contracted index is free, a result is the next product's
// operand as it lies: the scores P^T[j][i] meet x^T[p][j], the states S^T[n][p]
// meet C.  What is contracted over tokens comes transposed out of LDS
// (ds_read_b64_tr_b16).  Rows of S and of y are taken in the order n = r with bits
// 2 and 3 swapped, so that a lane holds 8 neighbours: 16-byte reads and writes.
//
// Precision.  x, B and C are bf16 and enter as they are; every other operand
// (e^(..) d x, S, the scores) is split into three bf16 parts, which hold all of
// its 24 bits and have fp32's range.  All sums are fp32, G is fp64.
//
// Bound by the issue of instructions: of a chunk's 19.5 K cycles the two waves of a
// SIMD have 8.1 K of matrix products (32 cycles each) and 8.6 K of vector
// instructions, mostly splits, scalings and decays (64 sequences of up to 2048
// tokens, 64 heads of 64 x 128: 38 and 51 % of all cycles, the products' issue
// among the latter; LDS 25 %, a third of it bank conflicts; 616 us for 1.4 GB).
// Hence one wave's scores and decays serve two, parts are cut off by logical
// instructions (4 cycles, v_cvt_pk_bf16_f32 6.5) and vector instructions are put
// between the products.  128 x 32 states and what a wave has in flight fill its
// 256 registers, two waves a SIMD; 64 tokens are the most whose x and B come
// beside the last ones' while C and the scores lie in the LDS.  Few long
// sequences are walked in segments, twice: 14807 tokens of 128 heads 103 us for the
// states at the segments' ends, 12 to join them, 286 for the outputs (4195
// tokens: 40, 12, 96).  128 tokens of 64 heads take 20.0 us in workgroups of two
// waves.
#include "ssm_device.h"

namespace sconv {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kC = kSsmChunk;          // tokens per chunk
constexpr int kPW = 32;                // channels a wave

// A head's factors of a chunk, per token, in LDS: those of its states, whose next chunk's come beside them, and those of its
// outputs, which take the place of the last chunk's once both waves are done with these.
struct alignas(16) Keeps {
    float w[kC];                       // e^(G_last - G) d
    float keep, last;                  // e^G_last, G_last in powers of 2
};
struct alignas(16) Factors {
    float eG[kC];                      // e^G
    float u[kC];                       // e^(G - R), R: G at the start of the token's half
    float v[kC];                       // plain: e^(R - G) d, else d
    float vx[kC / 2];                  // e^(R_1 - G) d of the first half
    float relh[kC], rell[kC];          // G - R in two parts, in powers of 2
    int plain;                         // e^(R - G) does not pass 2^64
};

// Rows of U 16-byte units in LDS, unit u of row r at u ^ swz(r): 8 neighbouring rows' like units lie in different banks, and so
// do 4 neighbouring rows' pairs of units.
template <int U>
__device__ __forceinline__ int swz(int r) {
    return U >= 8 ? ((r & 3) << 1 | ((r >> 2) & 1)) : (((r >> 1) & 1) << 1 | ((r >> 2) & 1));
}

// 16 bytes a lane from byte `at` of r to lds + 16 lane, past the registers.  What lies past r's end may or may not be written
// as zero: those places hold zeros or an earlier chunk's rows.  Written as an instruction (it has no register to be written
// late): the builtin makes the compiler wait for it before the next read of the same array, the other buffer's included, which
// is a trip to memory in every chunk.  landed() waits for it.  The compiler keeps nothing in m0.  A vector instruction (the
// v_readlane of a spilled word) may have written r just before: five wait states lie between, which the compiler does not put in
// front of what it does not know.
__device__ __forceinline__ void to_lds(const u32x4 &r, uint32_t at, void *lds) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>(lds)));   // (its place in the LDS)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(at), "s"(r), "s"(to) : "memory");
}
// A barrier for what waves exchange through ds_write: what is on its way to LDS past the registers stays on its way.
__device__ __forceinline__ void exchange() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// Reads that were written before it are issued before what comes after it.
__device__ __forceinline__ void issued() { __builtin_amdgcn_sched_barrier(0); }
// N matrix products with 6 vector instructions behind each, which take no longer than it.
template <int N>
__device__ __forceinline__ void interleave() {
    if constexpr (N > 0) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, 6, 0);
        interleave<N - 1>();
    }
}
// All but this wave's last N reads and writes of memory are done, those on their way to LDS among them.  As an instruction that
// the compiler knows: it takes its own loads for done too.
template <int N>
__device__ __forceinline__ void landed() {
    static_assert(N < 16, "the low bits of the counter");
    __builtin_amdgcn_s_waitcnt(0x0f70 | N);
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ f32x4 row4(const float *v) { return *reinterpret_cast<const f32x4 *>(v); }

// Transposed: lane l gets column l % 16 of its 16 lanes' 4 rows; it names row (l % 16) / 4, columns 4 (l % 4) ..
__device__ __forceinline__ s16x4 read_tr(const uint16_t *lds) {
    typedef __attribute__((address_space(3))) s16x4 L;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)lds);
}
// 16 tokens from t0 on (contracted: 8 (e / 4) + 4 (l / 32) + e % 4) of the 32 columns of tile i, a column (bits 2 and 3
// swapped) a lane.
template <int U>
__device__ __forceinline__ bf16x8 read_cols(const uint16_t *lds, int t0, int i, int lane) {
    const int r = ((lane & 15) >> 2) + 4 * (lane >> 5), c = lane & 3;          // (t0 is a multiple of 16: swz goes by r)
    const int u = (2 * ((lane >> 4) & 1) + (c & 1)) ^ swz<U>(r), o = 4 * (c >> 1);
    const uint16_t *base = lds + (r * U + (u ^ (4 * (i & 1)))) * 8 + o;
    union { s16x4 s[2]; bf16x8 b; } x;
    x.s[0] = read_tr(base + t0 * U * 8 + 64 * (i >> 1));
    x.s[1] = read_tr(base + (t0 + 8) * U * 8 + 64 * (i >> 1));
    return x.b;
}
// Rows r0 + l % 32, columns 16 k + 8 (l / 32) ..
template <int U>
__device__ __forceinline__ bf16x8 read_rows(const uint16_t *lds, int r0, int k, int lane) {
    const int n = lane & 31, u = ((lane >> 5) ^ swz<U>(n)) ^ (2 * (k & 3));
    return *reinterpret_cast<const bf16x8 *>(lds + (n * U + u) * 8 + r0 * U * 8 + 64 * (k >> 2));
}

__device__ __forceinline__ f32x16 mfma(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() { return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0}; }

__device__ __forceinline__ bf16x8 as_bf16(const uint32_t (&w)[4]) { return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]}); }

// The upper halves of two floats: their bf16 parts, cut off.
__device__ __forceinline__ uint32_t upper(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float below(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// x = hi + mid + lo: each takes the next 8 of its 24 bits.  (Cut off, not rounded: a conversion takes 6.5 cycles where a logical
// instruction takes 4, and a dot product with (-1, 0) in place of the two for what is left takes 8 beside another wave's matrix
// products.)
struct Parts { bf16x8 hi, mid, lo; };
__device__ __forceinline__ Parts split(const float (&x)[8]) {
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = upper(x[2 * i], x[2 * i + 1]);
        const float a = below(x[2 * i]), b = below(x[2 * i + 1]);
        m[i] = upper(a, b);
        l[i] = upper(below(a), below(b));
    }
    return {as_bf16(h), as_bf16(m), as_bf16(l)};
}

// x + the value that lane CTRL's pattern moves here (fp64, 0 where it moves none).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, uint32_t(u), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, uint32_t(u >> 32), CTRL, ROWS, 0xf, false);
    return x + __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
template <int LANE>
__device__ __forceinline__ double lane64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, uint64_t(uint32_t(__builtin_amdgcn_readlane(int(u >> 32), LANE))) << 32 |
                                          uint32_t(__builtin_amdgcn_readlane(int(u), LANE)));
}

// Eight elements of a row by elements, zero past n.
__device__ __forceinline__ u32x4 load8(const uint16_t *row, int64_t sd, int c, int32_t n) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = c + i < n ? row[(c + i) * sd] : 0u;
    u32x4 r;
    r.x = e[0] | e[1] << 16; r.y = e[2] | e[3] << 16;
    r.z = e[4] | e[5] << 16; r.w = e[6] | e[7] << 16;
    return r;
}

// What a workgroup does: chunks [c0, c1) of a sequence, for a group's heads.
struct Job {
    int32_t group;
    int32_t t0, n;                     // the sequence's first row and length
    int32_t c0, c1;
};

// A wave-uniform tensor's rows from a chunk's first on; next() goes to the next chunk's.
struct Rows {
    const char *at;
    uint32_t row;                      // bytes
    __device__ __forceinline__ Rows(const uint16_t *t, int64_t st, int64_t first) {
        at = reinterpret_cast<const char *>(t + first * st);
        row = uint32_t(st) * 2;
    }
    __device__ __forceinline__ void next() { at += uint64_t(row) * kC; }
    // A descriptor that ends behind the `left`-th row (at most a chunk's).
    __device__ __forceinline__ u32x4 words(int32_t left) const {
        const uint64_t a = reinterpret_cast<uint64_t>(at);
        return u32x4{uint32_t(a), uint32_t(a >> 32) & 0xffffu, uint32_t(left < kC ? left : kC) * row, 0x00020000u};
    }
    __device__ __forceinline__ Rsrc rsrc(int32_t left) const { return make_rsrc(at, int64_t(left < kC ? left : kC) * row); }
};

enum Mode { kWhole, kStates, kSegment };

// A tile of scores as an operand of its product with x: two steps of 16 tokens.
struct Scores { Parts k[2]; };
constexpr int kTile = 3 * 2 * 64 * 8;  // halves

template <int NT, bool VEC>
struct Wave {
    static constexpr int U = 4 * NT;   // units of a row of B and C
    const SsmParams &p;
    const Job job;
    const int lane0;
    const int32_t h, ch0;              // head, first channel
    uint32_t xo, oo[2];                // the lane's offsets in a chunk's rows of x, and of out
    f32x16 S[NT];                      // S^T: n = 32 nt + 16 (q / 8) + 8 (l / 32) + q % 8 of channel chan()

    // The lane number anew, as a value that the compiler takes for unknown: addresses computed from it stay in their phase.
    __device__ __forceinline__ int fresh() const {
        int lane = lane0;
        asm volatile("" : "+v"(lane));
        return lane;
    }
    __device__ __forceinline__ int32_t chan(int lane) const {
        const int r = lane & 31;
        return ch0 + ((r & 19) | ((r & 4) << 1) | ((r & 8) >> 1));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NT; ++i) S[i] = zero16();
    }
    template <class F>
    __device__ __forceinline__ void state_rows(int lane, F fn) {
        const int hh = lane >> 5;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) fn(i, 4 * k, 32 * i + 16 * (k >> 1) + 8 * hh + 4 * (k & 1));
    }
    __device__ __forceinline__ void load(const float *rows, bool svec) {
        const int lane = fresh();
        const int32_t c = chan(lane);
        zero();
        if (c >= p.P) return;
        const float *row = rows + c * p.s_sp;
        state_rows(lane, [&](int i, int q, int n) {
            if (svec) {
                if (n < p.N) {
                    const f32x4 v = row4(row + n);
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][q + e] = v[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) S[i][q + e] = row[(n + e) * p.s_sn];
            }
        });
    }
    __device__ __forceinline__ void save(float *rows, bool svec) {
        const int lane = fresh();
        const int32_t c = chan(lane);
        if (c >= p.P) return;
        float *row = rows + c * p.s_sp;
        state_rows(lane, [&](int i, int q, int n) {
            if (svec) {
                if (n < p.N) *reinterpret_cast<f32x4 *>(row + n) = f32x4{S[i][q], S[i][q + 1], S[i][q + 2], S[i][q + 3]};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) row[(n + e) * p.s_sn] = S[i][q + e];
            }
        });
    }
    // As the registers lie: 16 bytes a lane, 4 NT pieces.
    __device__ __forceinline__ void load_raw(const float *at) {
        const int lane = fresh();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x4 v = row4(at + ((4 * i + k) * 64 + lane) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][4 * k + e] = v[e];
            }
    }
    __device__ __forceinline__ void save_raw(float *at) {
        const int lane = fresh();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<f32x4 *>(at + ((4 * i + k) * 64 + lane) * 4) =
                    f32x4{S[i][4 * k], S[i][4 * k + 1], S[i][4 * k + 2], S[i][4 * k + 3]};
    }

    // The bits of the step size's input of a chunk's token, a token a lane (behind the sequence's end anything), loaded without
    // a branch: a bf16 is the high half.
    struct Step { uint32_t lo, hi; };
    __device__ __forceinline__ Step fetch_dt(int32_t c) const {
        const int32_t r = c * kC + lane0, w = p.dt_fp32 ? 2 : 1;
        const int64_t at = (int64_t(job.t0) + (r < job.n ? r : job.n - 1)) * p.ds.st + h * p.ds.sh;
        const uint16_t *e = static_cast<const uint16_t *>(p.dt) + at * w;
        return {e[0], e[w - 1]};
    }
    __device__ __forceinline__ void offsets(uint32_t xrow, uint32_t orow) {
        const int t = lane0 >> 2, u = (lane0 & 3) ^ swz<4>(t);
        const int32_t ch = ch0 + 8 * u;
        xo = ch < p.P ? t * xrow + uint32_t(ch) * 2 : kOob;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int32_t o = ch0 + 16 * k + 8 * (lane0 >> 5);
            oo[k] = o < p.P ? (lane0 & 31) * orow + uint32_t(o) * 2 : kOob;
        }
    }
    // Pieces [k0, k1) of the wave's x of chunk c, 16 rows each, on their way to LDS.  r: that chunk's rows.
    __device__ __forceinline__ void fetch_x(const Rows &r, int32_t c, uint16_t *to, int k0, int k1) {
        if constexpr (VEC) {
            const u32x4 words = r.words(job.n - c * kC);
            uint32_t at = xo;                          // (unknown to the compiler: it would keep every piece's in a register)
            asm volatile("" : "+v"(at));
#pragma unroll
            for (int k = k0; k < k1; ++k) to_lds(words, at + 16 * k * r.row, to + 512 * k);
        } else {
            const int lane = fresh(), t0 = lane >> 2, ch = ch0 + 8 * ((lane & 3) ^ swz<4>(t0));
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
                const int32_t t = c * kC + 16 * k + t0;
                const int64_t row = int64_t(job.t0) + (t < job.n ? t : job.n - 1);
                *reinterpret_cast<u32x4 *>(to + (64 * k + lane) * 8) = load8(p.x + row * p.xs.st + h * p.xs.sh, p.xs.sd, ch, p.P);
            }
        }
    }

    // The factors of chunk c from its dt: those of the states, and with OUT of the outputs, a token a lane.
    struct Decays { float eG, u, v, vx, relh, rell; bool plain; };
    template <bool OUT>
    __device__ __forceinline__ Decays factors(int32_t c, const Step &dt, float A, float bias, Keeps &f) {
        const int lane = fresh();
        float d = ssm_clamp(p, ssm_softplus(p, __uint_as_float(dt.hi << 16 | (p.dt_fp32 ? dt.lo : 0u)) + bias));
        if (c * kC + lane >= job.n) d = 0.0f;
        float g = d == 0.0f ? 0.0f : d * A;            // (A may be infinite)
        g = g > 0.0f ? 0.0f : (g < -200.0f ? -200.0f : g);         // e^-200 is 0, as of anything below
        double G = double(g) * 1.4426950408889634;
        G = dpp_add64<0x111, 0xf>(G);                  // row_shr 1, 2, 4, 8, then the rows' last values
        G = dpp_add64<0x112, 0xf>(G);
        G = dpp_add64<0x114, 0xf>(G);
        G = dpp_add64<0x118, 0xf>(G);
        G = dpp_add64<0x142, 0xa>(G);
        G = dpp_add64<0x143, 0xc>(G);
        const double last = lane64<63>(G);
        f.w[lane] = d * __builtin_amdgcn_exp2f(float(last - G));
        if (lane == 0) {
            f.keep = __builtin_amdgcn_exp2f(float(last));
            f.last = float(last);
        }
        Decays r = {};
        if constexpr (OUT) {
            const double mid = lane64<31>(G), rel = G - (lane < 32 ? 0.0 : mid);
            r.relh = float(rel);
            r.rell = float(rel - double(r.relh));
            r.plain = __builtin_amdgcn_ballot_w64(!(r.relh > -64.0f)) == 0;
            r.eG = __builtin_amdgcn_exp2f(float(G));
            r.u = __builtin_amdgcn_exp2f(r.relh);
            r.v = r.plain ? d * __builtin_amdgcn_exp2f(-r.relh) : d;
            r.vx = d * __builtin_amdgcn_exp2f(float(mid - G));
        }
        return r;
    }
    __device__ __forceinline__ void put(const Decays &r, Factors &f) const {
        const int lane = fresh();
        f.eG[lane] = r.eG;
        f.u[lane] = r.u;
        f.v[lane] = r.v;
        if (lane < 32) f.vx[lane] = r.vx;
        if (!r.plain) {
            f.relh[lane] = r.relh;
            f.rell[lane] = r.rell;
        }
        if (lane == 0) f.plain = r.plain;
    }

    // x^T: channel chan() a lane, 16 tokens each.
    __device__ __forceinline__ void read_x(const uint16_t *xl, bf16x8 (&x)[4]) {
        const int lane = fresh();
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = read_cols<4>(xl, 16 * k, 0, lane);
    }

    // S <- e^G_last S + sum_j w_j x_j B_j^T
    __device__ __forceinline__ void advance(const uint16_t *B, const bf16x8 (&x)[4], const Keeps &f) {
        const int lane = fresh(), hh = lane >> 5;
        const float keep = f.keep;
        f32x4 w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = row4(f.w + 8 * k + 4 * hh);
        bf16x8 b[2][NT];
        Parts xp[2];
#pragma unroll
        for (int i = 0; i < NT; ++i) b[0][i] = read_cols<U>(B, 0, i, lane);
        issued();
        const auto weigh_x = [&](int k) {
            float xw[8];
            unpack8(__builtin_bit_cast(u32x4, x[k]), xw);
#pragma unroll
            for (int e = 0; e < 8; ++e) xw[e] *= w[2 * k + (e >> 2)][e & 3];
            xp[k & 1] = split(xw);
        };
        weigh_x(0);
#pragma unroll
        for (int i = 0; i < NT; ++i) S[i] *= keep;
        // The next 16 tokens' operands are read and split between this step's products.
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < 3) {
#pragma unroll
                for (int i = 0; i < NT; ++i) b[(k + 1) & 1][i] = read_cols<U>(B, 16 * k + 16, i, lane);
                issued();
                weigh_x(k + 1);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) S[i] = mfma(b[k & 1][i], xp[k & 1].hi, S[i]);
#pragma unroll
            for (int i = 0; i < NT; ++i) S[i] = mfma(b[k & 1][i], xp[k & 1].mid, S[i]);
#pragma unroll
            for (int i = 0; i < NT; ++i) S[i] = mfma(b[k & 1][i], xp[k & 1].lo, S[i]);
            if (k < 3) interleave<3 * NT>();
        }
    }

    // B_j . C_i of NJ tiles, j = 32 (jt + 0, 1) .., i = 32 it ..; four steps' operands are read before the last four's products.
    template <int NJ>
    __device__ __forceinline__ void score(const uint16_t *B, const uint16_t *C, int jt, int it, f32x16 (&s)[NJ]) {
        constexpr int kGroup = 2 * NT < 4 ? 2 * NT : 4, kN = 2 * NT / kGroup;
        const int lane = fresh();
        bf16x8 b[2][NJ][kGroup], c[2][kGroup];
        const auto fetch = [&](int g) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                c[g & 1][k] = read_rows<U>(C, 32 * it, g * kGroup + k, lane);
#pragma unroll
                for (int j = 0; j < NJ; ++j) b[g & 1][j][k] = read_rows<U>(B, 32 * (jt + j), g * kGroup + k, lane);
            }
        };
        fetch(0);
        issued();
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[j] = zero16();
#pragma unroll
        for (int g = 0; g < kN; ++g) {
            if (g + 1 < kN) {
                fetch(g + 1);
                issued();
            }
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
#pragma unroll
                for (int j = 0; j < NJ; ++j) s[j] = mfma(b[g & 1][j][k], c[g & 1][k], s[j]);
        }
    }
    // What the scores of half `half` against their own tokens (DIAG), or against the first half's, are multiplied by: u_i v_j.
    struct Weights { float u; f32x4 v[4]; };
    template <bool DIAG>
    __device__ __forceinline__ Weights weights(int half, const Factors &f) {
        const int lane = fresh();
        Weights r;
        r.u = f.u[32 * half + (lane & 31)];
#pragma unroll
        for (int k = 0; k < 4; ++k) r.v[k] = row4((DIAG ? f.v + 32 * half : f.vx) + 8 * k + 4 * (lane >> 5));
        return r;
    }
    // The scores times e^(G_i - G_j) d_j.  DIAG: of one half (masked, D on the diagonal).  What is masked is 0, not a score
    // times 0: a later token's B may not be finite.
    template <bool DIAG>
    __device__ __forceinline__ Scores weigh(const f32x16 &s, int half, const Weights &g, bool plain, const Factors &f, float D) {
        const int lane = fresh(), n = lane & 31, hh = lane >> 5;
        float v[16];
        const int i = n - 4 * hh;                      // (token j of register q is token i at j = (q % 4) + 8 (q / 4))
        if (DIAG && !plain) {
            const float ih = f.relh[32 * half + n], il = f.rell[32 * half + n];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = 32 * half + 8 * k + 4 * hh;
                const f32x4 jh = row4(f.relh + j), jl = row4(f.rell + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = (ih - jh[e]) + (il - jl[e]), d = g.v[k][e] * __builtin_amdgcn_exp2f(a > 0.0f ? 0.0f : a);
                    v[4 * k + e] = 8 * k + e <= i ? s[4 * k + e] * d : 0.0f;
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[4 * k + e] = !DIAG || 8 * k + e <= i ? s[4 * k + e] * g.u * g.v[k][e] : 0.0f;
        }
        if constexpr (DIAG) {
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] += 8 * (q >> 2) + (q & 3) == i ? D : 0.0f;
        }
        Scores r;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = v[8 * k + e];
            r.k[k] = split(t);
        }
        return r;
    }
    static __device__ __forceinline__ void put(const Scores &s, uint16_t *at, int lane) {
        bf16x8 *o = reinterpret_cast<bf16x8 *>(at) + lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) { o[192 * k] = s.k[k].hi; o[192 * k + 64] = s.k[k].mid; o[192 * k + 128] = s.k[k].lo; }
    }
    static __device__ __forceinline__ Scores get(const uint16_t *at, int lane) {
        const bf16x8 *o = reinterpret_cast<const bf16x8 *>(at) + lane;
        Scores s;
#pragma unroll
        for (int k = 0; k < 2; ++k) s.k[k] = {o[192 * k], o[192 * k + 64], o[192 * k + 128]};
        return s;
    }

    // y = e^G_i (S C_i), tokens 32 it + l % 32 a lane
    __device__ __forceinline__ void from_state(const uint16_t *C, const Factors &f, f32x16 &y0, f32x16 &y1) {
        const int lane = fresh(), n = lane & 31;
        const float e0 = f.eG[n], e1 = f.eG[32 + n];
        bf16x8 c[2][2][2];
        const auto fetch = [&](int g) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) c[g & 1][k][i] = read_rows<U>(C, 32 * i, 2 * g + k, lane);
        };
        fetch(0);
        issued();
        Parts s[2][2];
        const auto split_s = [&](int g) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = S[g][8 * k + e];
                s[g & 1][k] = split(t);
            }
        };
        split_s(0);
        y0 = zero16();
        y1 = zero16();
#pragma unroll
        for (int g = 0; g < NT; ++g) {
            if (g + 1 < NT) {
                fetch(g + 1);
                issued();
                split_s(g + 1);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                y0 = mfma(s[g & 1][k].hi, c[g & 1][k][0], y0);
                y1 = mfma(s[g & 1][k].hi, c[g & 1][k][1], y1);
                y0 = mfma(s[g & 1][k].mid, c[g & 1][k][0], y0);
                y1 = mfma(s[g & 1][k].mid, c[g & 1][k][1], y1);
                y0 = mfma(s[g & 1][k].lo, c[g & 1][k][0], y0);
                y1 = mfma(s[g & 1][k].lo, c[g & 1][k][1], y1);
            }
            if (g + 1 < NT) interleave<12>();
        }
        y0 *= e0;
        y1 *= e1;
    }
    // y += P x of a tile
    static __device__ __forceinline__ void add(f32x16 &y, const bf16x8 &xa, const bf16x8 &xb, const Scores &s) {
        y = mfma(xa, s.k[0].hi, y);
        y = mfma(xb, s.k[1].hi, y);
        y = mfma(xa, s.k[0].mid, y);
        y = mfma(xb, s.k[1].mid, y);
        y = mfma(xa, s.k[0].lo, y);
        y = mfma(xb, s.k[1].lo, y);
    }

    // Outputs of the lane's token of half `it`: channels 8 (l / 32) .. and 16 + 8 (l / 32) .. of the wave's.  VEC: two writes,
    // whatever of them exists (landed() counts them).  r: out's rows of the chunk.
    __device__ __forceinline__ void store(const Rows &r, int32_t c, int it, const f32x16 &y, bool plain) {
        const Rsrc to = r.rsrc(job.n - c * kC);
        uint32_t at[2] = {oo[0], oo[1]};
        asm volatile("" : "+v"(at[0]), "+v"(at[1]));
        if (VEC && plain) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = y[8 * k + e];
                __builtin_amdgcn_raw_buffer_store_b128(pack8(v), to, at[k] + 32 * it * r.row, 0, 0);
            }
            return;
        }
        const int lane = fresh(), t = c * kC + 32 * it + (lane & 31);
        const int64_t row = int64_t(job.t0) + (t < job.n ? t : job.n - 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int32_t ch = ch0 + 16 * k + 8 * (lane >> 5);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = y[8 * k + e];
            if (p.D.p && p.D.sd != 0 && ch < p.P) {
                float xf[8];
                const uint16_t *xr = p.x + row * p.xs.st + h * p.xs.sh;
                unpack8(VEC ? ld16(xr + ch) : load8(xr, p.xs.sd, ch, p.P), xf);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (ch + e < p.P) v[e] = fmaf(p.D.p[h * p.D.sh + (ch + e) * p.D.sd], xf[e], v[e]);
            }
            if (p.z && ch < p.P) {
                float zf[8];
                const uint16_t *zr = p.z + row * p.zs.st + h * p.zs.sh;
                unpack8(VEC ? ld16(zr + ch) : load8(zr, p.zs.sd, ch, p.P), zf);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = ssm_gate(v[e], zf[e]);
            }
            if constexpr (VEC) {
                __builtin_amdgcn_raw_buffer_store_b128(pack8(v), to, at[k] + 32 * it * r.row, 0, 0);
            } else {
                uint16_t *o = p.out + row * p.os.st + h * p.os.sh;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (t < job.n && ch + e < p.P) o[(ch + e) * p.os.sd] = to_bf16(v[e]);
            }
        }
    }
};

// Rows of B or C of chunk c on their way to LDS, by all of a workgroup's waves: each brings pieces of 64 units.  `off`: the
// lane's offset in its wave's first piece.
template <int NT, int W>
__device__ __forceinline__ uint32_t piece_offset(uint32_t row, int32_t N, int wave, int lane) {
    constexpr int U = 4 * NT;
    const int t = wave * (64 / U) + lane / U, u = (lane % U) ^ swz<U>(t);
    return 8 * u < N ? t * row + 16 * u : kOob;
}
template <int NT, int W, bool VEC>
__device__ __forceinline__ void fetch_rows(const Rows &r, uint32_t off, const uint16_t *base, const GdrTensor &ts, int32_t N,
                                           const Job &job, int32_t c, uint16_t *lds, int wave, int lane) {
    constexpr int U = 4 * NT, kPieces = kC * U / 64, kRows = 64 / U;
    static_assert(kRows * W % 8 == 0, "a wave's pieces are swizzled alike");
    const u32x4 words = r.words(job.n - c * kC);
    asm volatile("" : "+v"(off));
#pragma unroll
    for (int k = 0; k < (kPieces + W - 1) / W; ++k) {
        const int piece = wave + k * W;
        if (kPieces % W != 0 && piece >= kPieces) break;
        if constexpr (VEC) {
            to_lds(words, off + k * (kRows * W) * r.row, lds + piece * 512);
        } else {
            const int tt = piece * kRows + lane / U, u = (lane % U) ^ swz<U>(tt);
            const int32_t at = c * kC + tt;
            const int64_t rr = int64_t(job.t0) + (at < job.n ? at : job.n - 1);
            *reinterpret_cast<u32x4 *>(lds + (piece * 64 + lane) * 8) = load8(base + rr * ts.st, ts.sd, 8 * u, N);
        }
    }
}

constexpr int kMaxRanked = 256;

// The sequence that is r-th by length, the longest first: a workgroup takes as long as its sequence, and one that starts late with a
// long one leaves the chip idle behind it.  More sequences than kMaxRanked stay in order.
template <int THREADS>
__device__ __forceinline__ int32_t ranked(const SsmParams &p, int32_t r, int32_t *len) {
    if (p.batch > kMaxRanked) return r;
    int32_t *out = len + kMaxRanked;
    for (int t = threadIdx.x; t < p.batch; t += THREADS) {
        SsmSpan sp;
        len[t] = ssm_span(p, t, sp) ? int32_t(sp.n) : 0;
    }
    __syncthreads();
    for (int t = threadIdx.x; t < p.batch; t += THREADS) {
        const int32_t n = len[t];
        int32_t before = 0;
        for (int32_t i = 0; i < p.batch; ++i) before += len[i] > n || (len[i] == n && i < t);
        if (before == r) *out = t;
    }
    __syncthreads();
    return *out;
}

// Segments of `seg` chunks: segment k of sequence i has slot floor(start_i / (64 seg)) + i + k.  No two share one, and
// floor(T / (64 seg)) + batch + 1 are enough for any offsets, so no kernel has to count them.
__device__ __forceinline__ int64_t first_slot(const SsmParams &p, int32_t b, int32_t seg) {
    int64_t a = p.qsl[b];
    a = a < 0 ? 0 : (a > p.total_T ? p.total_T : a);
    return a / (int64_t(kC) * seg) + b;
}

// PAIR: two waves a block of 64 channels of a head, which share its scores; otherwise a wave for up to 32 channels.  Eight waves
// fill a CU two to a SIMD; calls that take fewer have a CU or more a workgroup.
template <int NT, int W, bool PAIR, bool VEC, Mode MODE>
__global__ __launch_bounds__(64 * W, W == kSsmWaves ? 2 : 1) void ssm_chunk_kernel(SsmParams p, int32_t blocks, int32_t units, int32_t pbs,
                                                                          int64_t places, int32_t seg, float *states, float *decays,
                                                                          bool svec) {
    constexpr int U = 4 * NT, kBC = kC * U * 8, kUnits = PAIR ? W / 2 : W;
    constexpr bool kOut = MODE != kStates;
    // Rows come one chunk ahead; where a chunk takes little time, two.
    constexpr int kAhead = kOut ? 1 : 2, kBufs = kAhead + 1;
    // (of C one chunk where the waves meet behind its last read: the next one's comes then)
    constexpr int kCBufs = kOut && !PAIR ? kBufs : 1;
    __shared__ alignas(16) uint16_t B[kBufs][kBC], C[kCBufs][kOut ? kBC : 8];
    __shared__ alignas(16) uint16_t xl[kAhead][W][kC * kPW];
    __shared__ alignas(16) uint16_t scores[kOut && PAIR ? kUnits : 1][kOut && PAIR ? 3 * kTile : 8];
    __shared__ Keeps keeps[kUnits][2];
    __shared__ Factors factors[kOut ? kUnits : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;

    // Blocks go to the 8 XCDs in turn: those of one place and group, which read the same B and C, follow each other on one.
    const uint32_t at = blockIdx.x >> 3, pg = at / uint32_t(blocks) * 8 + (blockIdx.x & 7);
    const int32_t block = int32_t(at % uint32_t(blocks));
    const uint32_t place = pg / uint32_t(p.G);
    if (place >= places) return;
    Job job;
    job.group = int32_t(pg - place * uint32_t(p.G));
    SsmSpan sp;
    int64_t slot = 0;
    int32_t b = int32_t(place);
    if constexpr (MODE == kWhole) {
        b = __builtin_amdgcn_readfirstlane(ranked<64 * W>(p, b, reinterpret_cast<int32_t *>(&xl[0][0][0])));
        __syncthreads();
    } else {
        slot = place;
        int32_t lo = 0, hi = p.batch - 1;                          // the last sequence whose slots start at or before
        while (lo < hi) {
            const int32_t m = (lo + hi + 1) >> 1;
            if (first_slot(p, m, seg) <= slot) lo = m; else hi = m - 1;
        }
        b = lo;
    }
    if (!ssm_span(p, b, sp)) return;
    job.t0 = int32_t(sp.t0);
    job.n = int32_t(sp.n);
    const int32_t nc = int32_t((sp.n + kC - 1) / kC);
    job.c0 = 0;
    job.c1 = nc;
    if constexpr (MODE != kWhole) {
        const int64_t k = slot - first_slot(p, b, seg);
        if (k < 0 || k * seg >= nc) return;
        if (MODE == kStates && (k + 1) * seg >= nc) return;        // the last segment's end is no one's start
        job.c0 = int32_t(k * seg);
        job.c1 = job.c0 + seg < nc ? job.c0 + seg : nc;
    }

    // columns and rows that a chunk may lack
    for (int i = threadIdx.x; i < kBufs * kBC / 8; i += 64 * W) {
        reinterpret_cast<u32x4 *>(&B[0][0])[i] = u32x4{0, 0, 0, 0};
        if (kOut && i < kCBufs * kBC / 8) reinterpret_cast<u32x4 *>(&C[0][0])[i] = u32x4{0, 0, 0, 0};
    }
    for (int i = threadIdx.x; i < kAhead * W * kC * kPW / 8; i += 64 * W) reinterpret_cast<u32x4 *>(&xl[0][0][0])[i] = u32x4{0, 0, 0, 0};
    __syncthreads();

    const int half = PAIR ? wave / kUnits : 0, own = PAIR ? wave % kUnits : wave;
    const int32_t unit = block * kUnits + own;
    const bool work = unit < units, first = half == 0;
    const int32_t h = job.group * p.per_group + (work ? unit / pbs : 0), pb = work ? unit % pbs : 0;
    Wave<NT, VEC> wv{p, job, lane, h, (PAIR ? 64 : 32) * pb + 32 * half};
    uint16_t *sc = scores[kOut && PAIR ? own : 0];
    float *rows = p.state ? p.state + sp.line * p.s_sl + h * p.s_sh : nullptr;
    const int64_t per_slot = int64_t(p.G) * units * (PAIR ? 2 : 1);
    const int64_t piece = (int64_t(job.group) * units + unit) * (PAIR ? 2 : 1) + half;
    const float A = p.A.p[h * p.A.sh], bias = p.bias.p ? p.bias.p[h * p.bias.sh] : 0.0f;
    const float D = kOut && p.D.p && p.D.sd == 0 ? p.D.p[h * p.D.sh] : 0.0f;
    const uint16_t *Bg = p.B + job.group * p.bs.sh, *Cg = p.C + job.group * p.cs.sh;
    const int64_t row0 = int64_t(job.t0) + int64_t(job.c0) * kC;
    Rows xr(p.x + h * p.xs.sh, p.xs.st, row0), br(Bg, p.bs.st, row0), cr(Cg, p.cs.st, row0);
    Rows orow(p.out + h * p.os.sh, p.os.st, row0);
    wv.offsets(xr.row, orow.row);
    const uint32_t bo = piece_offset<NT, W>(br.row, p.N, wave, lane), co = piece_offset<NT, W>(cr.row, p.N, wave, lane);
    const bool as_is = !p.z && (!p.D.p || p.D.sd == 0);            // outputs are written as they come
    // the next chunk that has not been asked for
    const auto fetch_b = [&](int32_t c, int buf) {
        fetch_rows<NT, W, VEC>(br, bo, Bg, p.bs, p.N, job, c, B[buf], wave, lane);
        br.next();
    };
    const auto fetch_c = [&](int32_t c, int buf) {
        if (kOut) fetch_rows<NT, W, VEC>(cr, co, Cg, p.cs, p.N, job, c, C[kCBufs > 1 ? buf : 0], wave, lane);
        cr.next();
    };
    Factors &f = factors[kOut ? own : 0];
    typename Wave<NT, VEC>::Step dt = {0, 0};
    wv.zero();
    fetch_b(job.c0, 0);
    fetch_c(job.c0, 0);
    if (work) {
        wv.fetch_x(xr, job.c0, xl[0][wave], 0, 4);
        xr.next();
        if (kAhead == 2 && job.c0 + 1 < job.c1) wv.fetch_x(xr, job.c0 + 1, xl[kAhead - 1][wave], 0, 4);
        if (kAhead == 2) xr.next();
        if (MODE == kSegment && nc > seg) {
            wv.load_raw(states + (slot * per_slot + piece) * (NT * 1024));
        } else if (MODE != kStates) {
            if (sp.init) wv.load(rows, svec);
        }
        if (first) {
            const auto r = wv.template factors<kOut>(job.c0, wv.fetch_dt(job.c0), A, bias, keeps[own][0]);
            if (kOut) wv.put(r, f);
            dt = wv.fetch_dt(job.c0 + 1);
        }
    }
    if (kAhead == 2) {
        if (job.c0 + 1 < job.c1) fetch_b(job.c0 + 1, 1);
    }
    float total = 0.0f;
    landed<0>();
    __syncthreads();
    int cur = 0;                       // the chunk's buffer of B and C
    for (int32_t c = job.c0; c < job.c1; ++c) {
        const int odd = (c - job.c0) & 1, next = cur + kAhead < kBufs ? cur + kAhead : cur + kAhead - kBufs;
        const bool more = c + 1 < job.c1, ahead = c + kAhead < job.c1;
        const Keeps &keep = keeps[own][odd];
        uint16_t *xw = xl[kAhead == 2 ? odd : 0][wave];
        bf16x8 x[4];
        if (work) wv.read_x(xw, x);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");         // x is in registers: its place is free
        typename Wave<NT, VEC>::Step later = dt;
        if (work && first) later = wv.fetch_dt(c + 2);
        // What comes for a later chunk is asked for in pieces, all over the chunk: 64 KB at once fill the memory pipeline, and
        // the waves wait for it.
        if (ahead) fetch_b(c + kAhead, next);
        if constexpr (kOut) {
            f32x16 y0, y1;
            const uint16_t *Bc = B[cur], *Cc = C[kCBufs > 1 ? cur : 0];
            typename Wave<NT, VEC>::Decays later_f = {};
            const auto ask = [&](int part) {
                if (!ahead) return;
                if (part < 2 && work) wv.fetch_x(xr, c + kAhead, xw, 2 * part, 2 * part + 2);
                if (part == 1) xr.next();
                if (part == 2) fetch_c(c + kAhead, next);
            };
            if constexpr (PAIR) {
                if (work) {
                    if (first) {
                        const auto g = wv.template weights<true>(0, f);
                        const bool plain = __builtin_amdgcn_readfirstlane(f.plain);
                        f32x16 s[1];
                        wv.template score<1>(Bc, Cc, 0, 0, s);
                        ask(0);
                        wv.put(wv.template weigh<true>(s[0], 0, g, plain, f, D), sc, lane);
                        if (more) later_f = wv.template factors<kOut>(c + 1, dt, A, bias, keeps[own][odd ^ 1]);
                    } else {
                        const auto g = wv.template weights<false>(1, f), g1 = wv.template weights<true>(1, f);
                        const bool plain = __builtin_amdgcn_readfirstlane(f.plain);
                        f32x16 s[2];
                        wv.template score<2>(Bc, Cc, 0, 1, s);
                        ask(0);
                        wv.put(wv.template weigh<false>(s[0], 1, g, plain, f, D), sc + kTile, lane);
                        wv.put(wv.template weigh<true>(s[1], 1, g1, plain, f, D), sc + 2 * kTile, lane);
                    }
                    ask(1);
                    wv.from_state(Cc, f, y0, y1);
                }
                exchange();
                ask(2);
                if (work) {
                    if (more && first) wv.put(later_f, f);
                    const Scores s00 = wv.get(sc, lane), s01 = wv.get(sc + kTile, lane), s11 = wv.get(sc + 2 * kTile, lane);
                    issued();
                    wv.add(y0, x[0], x[1], s00);
                    wv.add(y1, x[0], x[1], s01);
                    wv.add(y1, x[2], x[3], s11);
                }
            } else {
                if (work) {
                    wv.from_state(Cc, f, y0, y1);
                    ask(0);
                    const bool plain = __builtin_amdgcn_readfirstlane(f.plain);
                    f32x16 s[1], t[2];
                    wv.template score<1>(Bc, Cc, 0, 0, s);
                    wv.add(y0, x[0], x[1], wv.template weigh<true>(s[0], 0, wv.template weights<true>(0, f), plain, f, D));
                    ask(1);
                    wv.template score<2>(Bc, Cc, 0, 1, t);
                    wv.add(y1, x[0], x[1], wv.template weigh<false>(t[0], 1, wv.template weights<false>(1, f), plain, f, D));
                    wv.add(y1, x[2], x[3], wv.template weigh<true>(t[1], 1, wv.template weights<true>(1, f), plain, f, D));
                    if (more) wv.put(wv.template factors<kOut>(c + 1, dt, A, bias, keeps[own][odd ^ 1]), f);
                }
                ask(2);
            }
            if (work) {
                wv.store(orow, c, 0, y0, as_is);
                wv.store(orow, c, 1, y1, as_is);
            }
            orow.next();
        } else if (work) {
            if (ahead) wv.fetch_x(xr, c + kAhead, xw, 0, 4);
            xr.next();
            if (more && first) wv.template factors<kOut>(c + 1, dt, A, bias, keeps[own][odd ^ 1]);
        }
        if (work) {
            wv.advance(B[cur], x, keep);
            if (MODE == kStates) total += keep.last;
        }
        dt = later;
        // The next chunk's rows are there.  Behind them a wave has asked for nothing but its 4 writes of this chunk's outputs, or
        // the rows of the chunk after it: at least a piece of B and 4 of x (waves without work: a piece of B at most).
        if (!VEC || !work || (kAhead == 2 && !ahead)) landed<0>();
        else landed<kOut ? 4 : 4 + (kC * U / 64) / W>();
        exchange();
        cur = cur + 1 < kBufs ? cur + 1 : 0;
    }
    if (!work) return;
    if constexpr (MODE == kStates) {
        wv.save_raw(states + (slot * per_slot + piece) * (NT * 1024));
        if (lane == 0) decays[slot * per_slot + piece] = __builtin_amdgcn_exp2f(total);
    } else {
        if (p.state && job.c1 == nc) wv.save(rows, svec);
    }
}

// From each segment's own states to the states that it starts from, in place: a thread takes 4 of them through a sequence's
// segments.  The first one's are among them: in the third kernel the last segment may write the line before the first has begun.
template <int NT>
__global__ __launch_bounds__(256) void ssm_pass_kernel(SsmParams p, int32_t units, int32_t pbs, int32_t seg, float *states,
                                                       const float *decays, bool svec) {
    // units and pbs count 32-channel pieces here
    const int64_t per_slot = int64_t(p.G) * units;
    const int64_t id = (int64_t(blockIdx.x) * 256 + threadIdx.x) / (NT * 256);
    if (id >= int64_t(p.batch) * per_slot) return;
    const int32_t b = int32_t(id / per_slot);
    const int64_t piece = id - b * per_slot;
    const int quad = threadIdx.x + 256 * (blockIdx.x % NT), lane = quad & 63, k = quad >> 6;
    SsmSpan sp;
    if (!ssm_span(p, b, sp)) return;
    const int32_t nc = int32_t((sp.n + kC - 1) / kC), ns = (nc + seg - 1) / seg;
    if (ns < 2) return;
    const int32_t group = int32_t(piece / units), unit = int32_t(piece - int64_t(group) * units);
    const int32_t h = group * p.per_group + unit / pbs, r = lane & 31;
    const int32_t ch = kPW * (unit % pbs) + ((r & 19) | ((r & 4) << 1) | ((r & 8) >> 1));
    const int32_t n = 32 * (k >> 2) + 16 * ((k >> 1) & 1) + 8 * (lane >> 5) + 4 * (k & 1);
    f32x4 S = {0, 0, 0, 0};
    if (sp.init && ch < p.P) {
        const float *row = p.state + sp.line * p.s_sl + h * p.s_sh + ch * p.s_sp;
        if (svec) {
            if (n < p.N) S = row4(row + n);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) S[e] = row[(n + e) * p.s_sn];
        }
    }
    const int64_t first = first_slot(p, b, seg) * per_slot + piece;
    const auto place = [&](int32_t i) { return reinterpret_cast<f32x4 *>(states + (first + i * per_slot) * (NT * 1024) + quad * 4); };
    for (int32_t i = 0; i + 1 < ns; ++i) {
        f32x4 *s = place(i);
        const f32x4 end = S * decays[first + i * per_slot] + *s;
        *s = S;
        S = end;
    }
    *place(ns - 1) = S;
}

template <int NT, bool PAIR, bool VEC>
hipError_t launch_segments(const SsmParams &p, bool svec, const SsmPlan &plan, void *workspace, int32_t blocks, int32_t units,
                           int32_t pbs, hipStream_t s) {
    constexpr int W = kSsmWaves;
    const int32_t halves = PAIR ? 2 : 1;
    const dim3 grid(uint32_t((plan.slots * p.G + 7) / 8 * 8 * blocks));
    float *states = static_cast<float *>(workspace);
    const int64_t pieces = int64_t(p.G) * units * halves;
    float *decays = states + plan.slots * pieces * (NT * 1024);
    ssm_chunk_kernel<NT, W, PAIR, VEC, kStates>
        <<<grid, dim3(64 * W), 0, s>>>(p, blocks, units, pbs, plan.slots, plan.seg, states, decays, svec);
    ssm_pass_kernel<NT><<<dim3(uint32_t(p.batch * pieces * NT)), dim3(256), 0, s>>>(p, units * halves, pbs * halves, plan.seg, states,
                                                                                    decays, svec);
    ssm_chunk_kernel<NT, W, PAIR, VEC, kSegment>
        <<<grid, dim3(64 * W), 0, s>>>(p, blocks, units, pbs, plan.slots, plan.seg, states, decays, svec);
    return hipGetLastError();
}

template <int NT, int W, bool PAIR, bool VEC>
hipError_t launch_w(const SsmParams &p, bool svec, const SsmPlan &plan, void *workspace, hipStream_t s) {
    const int32_t pbs = PAIR ? (p.P + 63) / 64 : 1, units = p.per_group * pbs, per = PAIR ? W / 2 : W;
    const int32_t blocks = (units + per - 1) / per;
    const auto grid = [&](int64_t places) { return dim3(uint32_t((places * p.G + 7) / 8 * 8 * blocks)); };
    if (!plan.seg) {
        ssm_chunk_kernel<NT, W, PAIR, VEC, kWhole>
            <<<grid(p.batch), dim3(64 * W), 0, s>>>(p, blocks, units, pbs, p.batch, 0, nullptr, nullptr, svec);
        return hipGetLastError();
    }
    if constexpr (W == kSsmWaves) return launch_segments<NT, PAIR, VEC>(p, svec, plan, workspace, blocks, units, pbs, s);
    return hipErrorInvalidValue;       // (no plan has it)
}

template <int NT, bool VEC>
hipError_t launch_nt(const SsmParams &p, bool svec, const SsmPlan &plan, void *workspace, hipStream_t s) {
    if (!plan.pair) return launch_w<NT, kSsmWaves, false, VEC>(p, svec, plan, workspace, s);
    if constexpr (VEC) {
        // a chunk takes a workgroup of two or four waves less time than one of eight, which fills its CU
        const int64_t heads = int64_t(p.batch) * p.G, units = int64_t(p.per_group) * ((p.P + 63) / 64);
        if (!plan.seg && heads * units <= kSsmCus) return launch_w<NT, 2, true, VEC>(p, svec, plan, workspace, s);
        if (!plan.seg && heads * ((units + 1) / 2) <= kSsmCus) return launch_w<NT, 4, true, VEC>(p, svec, plan, workspace, s);
    }
    return launch_w<NT, kSsmWaves, true, VEC>(p, svec, plan, workspace, s);
}

}  // namespace

hipError_t launch_ssm_chunk(const SsmParams &p, bool vec, bool svec, const SsmPlan &plan, void *workspace, hipStream_t s) {
    switch (plan.nt) {
        case 1: return vec ? launch_nt<1, true>(p, svec, plan, workspace, s) : launch_nt<1, false>(p, svec, plan, workspace, s);
        case 2: return vec ? launch_nt<2, true>(p, svec, plan, workspace, s) : launch_nt<2, false>(p, svec, plan, workspace, s);
        default: return vec ? launch_nt<4, true>(p, svec, plan, workspace, s) : launch_nt<4, false>(p, svec, plan, workspace, s);
    }
}

}  // namespace sconv

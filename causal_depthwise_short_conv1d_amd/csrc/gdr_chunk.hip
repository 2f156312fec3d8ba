// The gated delta rule over 64-token chunks: prefill on the matrix cores.
//
// With G the running sum of the log decay inside a chunk, kf_i k16_i the
// (normalised) key of token i, z_i = kf_i u_i, and S the state before the chunk:
//   X_i = kf_i beta_i (v_i - e^G_i kf_i (k16_i S))
//   A_ij = beta_i kf_i^2 e^(G_i - G_j) k16_i.k16_j   (i > j),   T = (I + A)^-1
//   z = T X
//   o_i = qf_i (e^G_i (q16_i S) + sum_(j <= i) e^(G_i - G_j) (q16_i.k16_j) z_j)
//   S <- e^G_last S + sum_j e^(G_last - G_j) k16_j z_j
// Written with z, T has entries of order 1 whenever the rule contracts
// (beta |k|^2 <= 2), whatever the keys' norms.
//
// A workgroup owns NS * NT tiles of 16 value channels of one head and walks its
// sequence.  Four producer waves prepare the chunk after the one in work
// (conversion, K K^T, Q K^T, the inverse) in one of two LDS buffers; each of
// the NS state waves holds the whole state of its NT * 16 channels in registers
// and consumes the other.  Both meet at one barrier a chunk.
// The state waves never exchange anything: an MFMA result has its channel in
// the lane and 4 rows a register quad, and the next product takes it as its
// right operand as it lies, since the order of a contracted index is free.  So
// key channel 32 kt + 8 g + 4 t + i is row 4 g + i of result tile 2 kt + t and
// slot 4 t + i of lane group g in operand tile kt; tokens are ordered likewise.
//
// Precision: the state is fp32 and every product that feeds it has 22-bit
// operands: fp16 pairs (high, low part), scaled by powers of two (a key row by
// its largest element, a state, X or z column likewise), summed in fp32 by the
// MFMA.  bf16 keys are exact in fp16 after that scaling, so K S takes 2 MFMAs
// and T X 3.  An fp32 MFMA would take 8 times as long as one of these pairs,
// and a single fp16 operand would leave the state at 11 bits.  The output is
// bf16, so the products that only feed it take single fp16 operands.
#include "gdr_device.h"

namespace sconv {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr int kC = 64;                 // tokens per chunk
constexpr int kProducers = 4;          // producer waves

// Tile-ordered operands in LDS: a 16-row x 32-column fp16 tile is 1 KiB, lane
// l's 16 bytes (row l % 16, columns 8 (l / 16) ..) at 16 l, so a wave reads a
// tile in one conflict-free access.
constexpr int kTile = 512;             // halves per tile

// Tiles of the 64 x 64 lower triangle, rows in 4 tiles, columns in 2: the rows
// of tiles 0 and 1 end before column 32.
__device__ __forceinline__ constexpr int tri_tile(int mt, int tt) { return mt < 2 ? mt : 2 + 2 * (mt - 2) + tt; }
constexpr int kTriTiles = 6;

template <int KT>
struct alignas(16) Buf {
    _Float16 k[4 * KT * kTile];        // [mt][kt] rows tokens
    _Float16 q[4 * KT * kTile];
    _Float16 kt[4 * KT * kTile];       // [2 KT channel tiles][2] rows key channels, columns tokens
    _Float16 th[kTriTiles * kTile];    // T, high and low parts
    _Float16 tl[kTriTiles * kTile];
    _Float16 p[kTriTiles * kTile];     // e^(Gi - Gj) q16.k16
    float ak[kC];                      // e^G kf
    float kb[kC];                      // kf beta
    float eg[kC];                      // e^(G_last - G)
    float qf[kC];
    float qe[kC];                      // qf e^G
    float last, ak_max, kb_max;        // e^G_last; largest of ak and of kb
};

template <int KT>
struct alignas(16) Shared {
    Buf<KT> buf[2];
    _Float16 off[6 * kTile];           // A's blocks below the diagonal: [4 rows / 4][column]: 4 high, 4 low parts
    float diag[4 * 256];               // A's diagonal blocks by columns, then T's
    float dump[4];                     // for what lies in neither
    float Gh[kC], Gl[kC];              // running log decay, in powers of 2: high and low parts
    float beta[kC], eG[kC], eg[kC], kf[kC];
    int sync;
};

// Token t of a chunk as a row: tile 2 (t / 32) + (t / 4) % 2, row 4 ((t % 32) / 8) + t % 4.
__device__ __forceinline__ int row_tile(int t) { return 2 * (t >> 5) + ((t >> 2) & 1); }
__device__ __forceinline__ int row_in(int t) { return 4 * ((t >> 3) & 3) + (t & 3); }
// ... and the token of row r of tile mt.
__device__ __forceinline__ int tok_of(int mt, int r) { return 32 * (mt >> 1) + 8 * (r >> 2) + 4 * (mt & 1) + (r & 3); }
// Offset (halves) of row r, column c (0..31) in a tile.
__device__ __forceinline__ int in_tile(int r, int c) { return (r + 16 * (c >> 3)) * 8 + (c & 7); }

// Rows of the k and q tiles are stored at r ^ (g + 4 (kt % 2)), g = column / 8, and rows of the transposed tiles at
// r ^ (d / 2): the producers' 64 lanes then write to every bank alike, and a read is a permutation of 256 bytes.
__device__ __forceinline__ int swz_rows(int r, int g, int kt) { return r ^ (g + 4 * (kt & 1)); }

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }   // -126..127
__device__ __forceinline__ int exp_of(float m) {       // m in [2^(e-1), 2^e), held to -100..127
    int e = __builtin_amdgcn_frexp_expf(m);
    e = e < -100 ? -100 : (e > 127 ? 127 : e);
    return m == 0.0f ? -100 : e;
}

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                                  0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
    const uint32_t o = __builtin_amdgcn_update_dpp(0u, v, CTRL, 0xf, 0xf, true);
    return v > o ? v : o;
}
// Over aligned groups of N lanes (8 or 16).
template <int N>
__device__ __forceinline__ float max_lanes(float v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    return N == 16 ? dpp_max<0x140>(v) : v;            // row_mirror
}
template <int N>
__device__ __forceinline__ float sum_lanes(float v) {
    v = sum8(v);
    return N == 16 ? dpp_add<0x140>(v) : v;
}
// Over the four lanes that hold one column (l, l + 16, l + 32, l + 48): two register swaps between lane rows.
__device__ __forceinline__ float max_groups(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const auto c = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return fmaxf(__uint_as_float(c[0]), __uint_as_float(c[1]));
}

__device__ __forceinline__ f16x2 cvt2(float a, float b) {
    typedef float f32x2v __attribute__((ext_vector_type(2)));
    const f32x2v v = {a, b};
    return __builtin_convertvector(v, f16x2);
}
// Eight values as a high and a low fp16 part: together 22 bits.
__device__ __forceinline__ void split8(const float (&x)[8], f16x8 &hi, f16x8 &lo) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const f16x2 h = cvt2(x[i], x[i + 1]);
        const f16x2 l = cvt2(x[i] - float(h.x), x[i + 1] - float(h.y));
        hi[i] = h.x; hi[i + 1] = h.y;
        lo[i] = l.x; lo[i + 1] = l.y;
    }
}
__device__ __forceinline__ f16x8 half8(const float (&x)[8]) {
    f16x8 r;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const f16x2 h = cvt2(x[i], x[i + 1]);
        r[i] = h.x; r[i + 1] = h.y;
    }
    return r;
}
__device__ __forceinline__ f32x4 mfma(const f16x8 &a, const f16x8 &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x8 tile_of(const _Float16 *base, int tile, int lane) {
    return *reinterpret_cast<const f16x8 *>(base + tile * kTile + lane * 8);
}
// ... of the swizzled k and q tiles (tile mt * KT + kt), and of the transposed ones (2 d + tt).
__device__ __forceinline__ f16x8 row_tile_of(const _Float16 *base, int tile, int kt, int lane) {
    const int n = lane & 15, g = lane >> 4;
    return *reinterpret_cast<const f16x8 *>(base + tile * kTile + (swz_rows(n, g, kt) + 16 * g) * 8);
}
__device__ __forceinline__ f16x8 col_tile_of(const _Float16 *base, int d, int tt, int lane) {
    return *reinterpret_cast<const f16x8 *>(base + (2 * d + tt) * kTile + (lane ^ (d >> 1)) * 8);
}

// Barrier among the producer waves alone: each adds one, then waits for the
// count that all of them reach.  They are waves of one workgroup, so all are
// resident, and each passes the same barriers.
__device__ __forceinline__ void producer_sync(int *count, int &target) {
    target += kProducers;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    if ((threadIdx.x & 63) == 0) __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    while (__hip_atomic_load(count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) < target) {}
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

struct Span64 { int64_t t0; int64_t n; };              // a sequence's first row and length

// ------------------------------------------------------------- producers --

// Eight channels of a row, zero past its end or the head's.
__device__ __forceinline__ u32x4 load8(const uint16_t *row, int64_t sd, int c, int32_t Dk, bool live) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = live && c + i < Dk ? row[(c + i) * sd] : 0u;
    u32x4 r;
    r.x = e[0] | e[1] << 16; r.y = e[2] | e[3] << 16;
    r.z = e[4] | e[5] << 16; r.w = e[6] | e[7] << 16;
    return r;
}

// Four token rows of eight channels each, as a producer thread holds them.
struct Quad { u32x4 r[4]; };

// VEC: 16-byte loads through a descriptor at the chunk's first row (what does not exist lies past its extent).
template <bool VEC>
__device__ __forceinline__ Quad load_quad(const uint16_t *head, const GdrTensor &ts, const Span64 &sp, int64_t c0,
                                          int quad, int kc, int32_t Dk) {
    Quad q;
    if constexpr (VEC) {
        const Rsrc rs = make_rsrc(head + (sp.t0 + c0) * ts.st, 0x7fffffff);
        const uint32_t row = uint32_t(ts.st) * 2;
        const int left = sp.n - c0 < kC ? int(sp.n - c0) : kC;
        const uint32_t at = 8 * kc < Dk ? uint32_t(4 * quad) * row + 16u * kc : kOob;
#pragma unroll
        for (int i = 0; i < 4; ++i) q.r[i] = buf_ld128<0>(rs, 4 * quad + i < left ? at + i * row : kOob);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = c0 + 4 * quad + i;
            const bool live = t < sp.n;
            q.r[i] = load8(head + (sp.t0 + (live ? t : 0)) * ts.st, ts.sd, 8 * kc, Dk, live);
        }
    }
    return q;
}

// Scales a row by a power of two (largest element in [1, 2)), writes it as a row of the operand tiles (and, for keys,
// transposed), and its factor: the power, times the norm's inverse and `scale`.
template <int KT, bool KEYS>
__device__ __forceinline__ void stage_quad(const Quad &in, _Float16 *rows, _Float16 *cols, float *factor, int quad,
                                           int kc, float scale, bool l2norm) {
    f16x8 h[4];
    const int kt = kc >> 2, g = kc & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // the largest element by its bits (as integers, without the sign), and the sum of squares
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 m2 = {0, 0};
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, in.r[i][j] & 0x7fff7fffu));
            const bf16x2 w = __builtin_bit_cast(bf16x2, uint32_t(in.r[i][j]));
            ss = __builtin_amdgcn_fdot2_f32_bf16(w, w, ss, false);
        }
        uint32_t m = m2.x > m2.y ? m2.x : m2.y;
        m = dpp_umax<0xB1>(m);
        m = dpp_umax<0x4E>(m);
        m = dpp_umax<0x141>(m);
        if constexpr (KT == 4) m = dpp_umax<0x140>(m);
        ss = sum_lanes<4 * KT>(ss);
        int eb = int(m >> 7);                          // biased exponent, held to 2^-100 .. 2^126
        eb = eb < 27 ? 27 : (eb > 253 ? 253 : eb);
        const float s = __uint_as_float(uint32_t(254 - eb) << 23);
        float f[8];
        unpack8(in.r[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= s;
        h[i] = half8(f);
        const int t = 4 * quad + i;
        if (kc == 0)
            factor[t] = scale * (l2norm ? __builtin_amdgcn_rsqf(ss + kL2Eps) : 1.0f) * __uint_as_float(uint32_t(eb) << 23);
        // (row, columns 8 kc ..) of tile (row tile, kt)
        *reinterpret_cast<f16x8 *>(rows + (row_tile(t) * KT + kt) * kTile + (swz_rows(row_in(t), g, kt) + 16 * g) * 8) =
            h[i];
    }
    if constexpr (KEYS) {
        // channel 8 kc + j: result tile d = 2 kt + j / 4, row 4 g + j % 4; tokens 4 quad ..
        const int c = (4 * quad) & 31;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f16x4 v = {h[0][j], h[1][j], h[2][j], h[3][j]};
            const int d = 2 * kt + (j >> 2), r = 4 * g + (j & 3);
            *reinterpret_cast<f16x4 *>(cols + (2 * d + (quad >> 3)) * kTile + in_tile(r ^ kt, c)) = v;
        }
    }
}

// x + the value that lane CTRL's pattern moves here (fp64, 0 where it moves none).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, uint32_t(u), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, uint32_t(u >> 32), CTRL, ROWS, 0xf, false);
    return x + __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// -row[j] of lane I's 16-lane row.
template <int I>
__device__ __forceinline__ float row_bcast(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + I, 0xf, 0xf, true));
}

// A 16 x 16 block product in 2 MFMAs of 32 slots: left operand [4 high | 4 low parts] of row n, columns 4 g ..; right
// operand rows 4 g .. in high and low parts.  22 bits of each, without low x low.
__device__ __forceinline__ f32x4 block_mfma(const f16x8 &a, const f16x4 &bh, const f16x4 &bl, f32x4 c) {
    const f16x8 b1 = {bh[0], bh[1], bh[2], bh[3], bh[0], bh[1], bh[2], bh[3]};
    const f16x8 b2 = {bl[0], bl[1], bl[2], bl[3], 0, 0, 0, 0};
    return mfma(a, b2, mfma(a, b1, c));
}
__device__ __forceinline__ void split4(const f32x4 &x, f16x4 &hi, f16x4 &lo) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const f16x2 h = cvt2(x[i], x[i + 1]);
        const f16x2 l = cvt2(x[i] - float(h.x), x[i + 1] - float(h.y));
        hi[i] = h.x; hi[i + 1] = h.y;
        lo[i] = l.x; lo[i + 1] = l.y;
    }
}

template <int KT, bool VEC>
struct Producer {
    const GdrParams &p;
    Shared<KT> &sh;
    const Span64 sp;
    const int lane, w, h;
    const uint16_t *qh, *kh;
    int target = 0;
    Quad nk, nq;                       // the rows of the chunk to come

    // KT = 4: 16 threads a row, each thread keys and queries.  KT = 2: 8 threads a row, waves 0 and 1 keys, 2 and 3
    // queries.
    __device__ __forceinline__ int kc() const { return KT == 4 ? lane & 15 : lane & 7; }
    __device__ __forceinline__ int quad() const { return KT == 4 ? 4 * w + (lane >> 4) : 8 * (w & 1) + (lane >> 3); }

    __device__ __forceinline__ void fetch(int64_t c0) {
        if (KT == 4 || w < 2) nk = load_quad<VEC>(kh, p.ks, sp, c0, quad(), kc(), p.Dk);
        if (KT == 4 || w >= 2) nq = load_quad<VEC>(qh, p.qs, sp, c0, quad(), kc(), p.Dk);
    }

    // Gates of a chunk, one token a lane.  The running sum is in fp64 and kept in two fp32 parts: a difference of two of
    // its values keeps every bit of a small decay behind a large one.  Every e^ below is of a difference <= 0.
    __device__ __forceinline__ void gates(int64_t c0) {
        const int64_t t = c0 + lane;
        Gates gt = {0.0f, 0.0f};
        if (t < sp.n)
            gt = gdr_gates(p, (sp.t0 + t) * p.gs.st + h * p.gs.sh, (sp.t0 + t) * p.bs.st + h * p.bs.sh, h);
        double G = (gt.g < -1e4f ? -1e4 : double(gt.g)) * 1.4426950408889634;   // e^-10000 is 0, as of anything below
        G = dpp_add64<0x111, 0xf>(G);                  // row_shr 1, 2, 4, 8, then the rows' last values
        G = dpp_add64<0x112, 0xf>(G);
        G = dpp_add64<0x114, 0xf>(G);
        G = dpp_add64<0x118, 0xf>(G);
        G = dpp_add64<0x142, 0xa>(G);
        G = dpp_add64<0x143, 0xc>(G);
        const uint64_t u = __builtin_bit_cast(uint64_t, G);
        const double last = __builtin_bit_cast(
            double, uint64_t(uint32_t(__builtin_amdgcn_readlane(int(u >> 32), 63))) << 32 |
                        uint32_t(__builtin_amdgcn_readlane(int(u), 63)));
        const float gh = float(G);
        sh.Gh[lane] = gh;
        sh.Gl[lane] = float(G - double(gh));
        sh.beta[lane] = gt.beta;
        sh.eG[lane] = __builtin_amdgcn_exp2f(float(G));
        sh.eg[lane] = __builtin_amdgcn_exp2f(float(last - G));
    }

    __device__ __forceinline__ void chunk(int64_t c0, Buf<KT> &b, bool more) {
        if (KT == 4 || w < 2) stage_quad<KT, true>(nk, b.k, b.kt, sh.kf, quad(), kc(), 1.0f, p.l2norm);
        if (KT == 4 || w >= 2) stage_quad<KT, false>(nq, b.q, nullptr, b.qf, quad(), kc(), p.scale, p.l2norm);
        if (more) fetch(c0 + kC);
        producer_sync(&sh.sync, target);
        products(b);
        if (w == 0) factors(b);
        producer_sync(&sh.sync, target);
        if (w == 3) invert_diagonal();
        producer_sync(&sh.sync, target);
        invert_rest(b);
        if (w == 0 && more) gates(c0 + kC);            // the other waves still invert
    }

    // The state waves' row factors.
    __device__ __forceinline__ void factors(Buf<KT> &b) {
        const float kf = sh.kf[lane], eG = sh.eG[lane], qf = b.qf[lane];
        const float ak = eG * kf, kb = kf * sh.beta[lane];
        b.ak[lane] = ak;
        b.kb[lane] = kb;
        b.eg[lane] = sh.eg[lane];
        b.qe[lane] = qf * eG;
        const float am = max_groups(max_lanes<16>(fabsf(ak))), bm = max_groups(max_lanes<16>(fabsf(kb)));
        if (lane == 63) { b.last = eG; b.ak_max = am; b.kb_max = bm; }
    }

    // 2^ of the decay between four rows and one token, 0 where the row comes first (rows - token < least).
    __device__ __forceinline__ f32x4 decay(const f32x4 &ah, const f32x4 &al, float bh, float bl, float sign) {
        f32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_exp2f(sign * ((ah[i] - bh) + (al[i] - bl)));
        return r;
    }

    // K K^T and Q K^T: 12 tile pairs meet the lower triangle, three a wave.  K K^T has its rows in the registers, Q K^T
    // (as its transpose) its columns: what a lane holds is then one piece of the operand that it becomes.
    __device__ __forceinline__ void products(Buf<KT> &b) {
        const int n = lane & 15, g = lane >> 4;
        f32x4 kk[3], qk[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const int pr = 3 * w + x;
            const int mt = pr < 4 ? pr >> 1 : 2 + ((pr - 4) >> 2), nt = pr < 4 ? pr & 1 : (pr - 4) & 3;
            kk[x] = f32x4{0, 0, 0, 0};
            qk[x] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const f16x8 kn = row_tile_of(b.k, nt * KT + kt, kt, lane);
                kk[x] = mfma(row_tile_of(b.k, mt * KT + kt, kt, lane), kn, kk[x]);
                qk[x] = mfma(kn, row_tile_of(b.q, mt * KT + kt, kt, lane), qk[x]);
            }
        }
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const int pr = 3 * w + x;
            const int mt = pr < 4 ? pr >> 1 : 2 + ((pr - 4) >> 2), nt = pr < 4 ? pr & 1 : (pr - 4) & 3;
            {
                const int tj = tok_of(nt, n), ti = tok_of(mt, 4 * g);
                const int bi = ti >> 4, bj = tj >> 4;
                const f32x4 d = decay(*reinterpret_cast<const f32x4 *>(sh.Gh + ti), *reinterpret_cast<const f32x4 *>(sh.Gl + ti),
                                      sh.Gh[tj], sh.Gl[tj], 1.0f);
                const f32x4 kf = *reinterpret_cast<const f32x4 *>(sh.kf + ti);
                f32x4 a = *reinterpret_cast<const f32x4 *>(sh.beta + ti) * kf * kf * d * kk[x];
                f16x4 hi, lo;
                split4(a, hi, lo);
                _Float16 *op = bi > bj ? sh.off + (bi * (bi - 1) / 2 + bj) * kTile + ((tj & 15) + 4 * (ti & 12)) * 8
                                       : reinterpret_cast<_Float16 *>(sh.dump);
                *reinterpret_cast<f16x8 *>(op) = f16x8{hi[0], hi[1], hi[2], hi[3], lo[0], lo[1], lo[2], lo[3]};
                if ((mt >> 1) == (nt >> 1))
                    *reinterpret_cast<f32x4 *>(bi == bj ? sh.diag + bi * 256 + (tj & 15) * 16 + (ti & 15) : sh.dump) = a;
            }
            {
                const int ti = tok_of(mt, n), tj = tok_of(nt, 4 * g);
                const f32x4 d = decay(*reinterpret_cast<const f32x4 *>(sh.Gh + tj), *reinterpret_cast<const f32x4 *>(sh.Gl + tj),
                                      sh.Gh[ti], sh.Gl[ti], -1.0f);
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = tj + i <= ti ? d[i] * qk[x][i] : 0.0f;
                const f16x2 lo = cvt2(v[0], v[1]), hi = cvt2(v[2], v[3]);
                *reinterpret_cast<f16x4 *>(b.p + tri_tile(mt, nt >> 1) * kTile + in_tile(n, tj & 31)) =
                    f16x4{lo.x, lo.y, hi.x, hi.y};
            }
        }
    }

    // Inverts the four diagonal blocks at once: block g in lane row g, a column a lane, by forward substitution; the
    // elements of A come from the lane that holds their column.
    __device__ __forceinline__ void invert_diagonal() {
        const int n = lane & 15, g = lane >> 4;
        float *blk = sh.diag + g * 256 + n * 16;
        float a[16], x[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const f32x4 r = *reinterpret_cast<const f32x4 *>(blk + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) { a[j + e] = -r[e]; x[j + e] = j + e == n ? 1.0f : 0.0f; }
        }
        substitute<0>(a, x);
#pragma unroll
        for (int j = 0; j < 16; j += 4) *reinterpret_cast<f32x4 *>(blk + j) = f32x4{x[j], x[j + 1], x[j + 2], x[j + 3]};
    }
    // x[j] is final: takes it out of the rows below.
    template <int J>
    static __device__ __forceinline__ void substitute(const float (&a)[16], float (&x)[16]) {
        if constexpr (J < 15) {
            below<J, J + 1>(a, x);
            substitute<J + 1>(a, x);
        }
    }
    template <int J, int I>
    static __device__ __forceinline__ void below(const float (&a)[16], float (&x)[16]) {
        if constexpr (I < 16) {
            x[I] = fmaf(row_bcast<J>(a[I]), x[J], x[I]);
            below<J, I + 1>(a, x);
        }
    }

    // Wave w fills block row w of T leftwards, T_wj = -(sum_(j < k <= w) T_wk A_kj) T_jj, as transposes: the right
    // operands are the blocks T_wk^T as they lie in registers (a row of T a lane).  Then it writes the row's two parts.
    __device__ __forceinline__ void invert_rest(Buf<KT> &b) {
        const int n = lane & 15, g = lane >> 4;
        const int ti = 16 * w + n;
        f16x4 hi[4], lo[4];
#pragma unroll
        for (int j = 3; j >= 0; --j) {
            if (j > w) continue;
            f32x4 t;
            if (j == w) {
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = sh.diag[j * 256 + (4 * g + e) * 16 + n];
            } else {
                f32x4 m = {0, 0, 0, 0};
#pragma unroll
                for (int k = 3; k >= 0; --k)
                    if (k > j && k <= w) m = block_mfma(tile_of(sh.off, k * (k - 1) / 2 + j, lane), hi[k], lo[k], m);
                f16x4 mh, ml, dh, dl;
                split4(m, mh, ml);
                const f32x4 d = -*reinterpret_cast<const f32x4 *>(sh.diag + j * 256 + n * 16 + 4 * g);
                split4(d, dh, dl);
                const f16x8 left = {dh[0], dh[1], dh[2], dh[3], dl[0], dl[1], dl[2], dl[3]};
                t = block_mfma(left, mh, ml, f32x4{0, 0, 0, 0});
            }
            split4(t, hi[j], lo[j]);
            const int tj = 16 * j + 4 * g;
            const int o = tri_tile(row_tile(ti), tj >> 5) * kTile + in_tile(row_in(ti), tj & 31);
            *reinterpret_cast<f16x4 *>(b.th + o) = hi[j];
            *reinterpret_cast<f16x4 *>(b.tl + o) = lo[j];
        }
    }
};

// ----------------------------------------------------------- state waves --

template <int KT, int NT, bool VEC>
struct Consumer {
    const GdrParams &p;
    const Span64 sp;
    const int lane;
    const uint16_t *vh;                // the head's first channel of v, row 0 of the sequence
    uint16_t *oh;
    int32_t c0;                        // first channel of the wave
    f32x4 S[NT][2 * KT];               // times 2^(14 - es)
    int es[NT];
    uint16_t v[NT][16];                // the chunk's values: [4 mt + i]

    __device__ __forceinline__ int32_t col(int nt) const { return c0 + 16 * nt + (lane & 15); }

    // Element (token, channel) accesses of the result layout: rows tok_of(mt, 4 g + i) = 8 g + a constant.  VEC: a
    // descriptor at the chunk's first row; what does not exist lies past its extent.
    template <class F>
    __device__ __forceinline__ void each(int64_t t0, const GdrTensor &ts, F f) {
        const int g = lane >> 4;
        const int left = sp.n - t0 < kC ? int(sp.n - t0) : kC;
        const uint32_t row = uint32_t(ts.st) * 2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint32_t at = col(nt) < p.Dv ? uint32_t(8 * g) * row + uint32_t(col(nt)) * uint32_t(ts.sd) * 2 : kOob;
            if (left == kC) {
#pragma unroll
                for (int r = 0; r < 16; ++r) f(nt, r, at, uint32_t(tok_of(r >> 2, r & 3)) * row);
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int t = tok_of(r >> 2, r & 3);
                    f(nt, r, 8 * g + t < left ? at : kOob, uint32_t(t) * row);
                }
            }
        }
    }

    __device__ __forceinline__ void fetch(int64_t t0) {
        const int g = lane >> 4;
        if constexpr (VEC) {
            const Rsrc rs = make_rsrc(vh + t0 * p.vs.st, 0x7fffffff);
            each(t0, p.vs, [&](int nt, int r, uint32_t off, uint32_t soff) {
                v[nt][r] = __builtin_amdgcn_raw_buffer_load_b16(rs, off, soff, 0);
            });
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t t = t0 + tok_of(r >> 2, 4 * g + (r & 3));
                    v[nt][r] = t < sp.n && col(nt) < p.Dv ? vh[t * p.vs.st + col(nt) * p.vs.sd] : uint16_t(0);
                }
        }
    }

    __device__ __forceinline__ void store(int64_t t0, const float (&o)[NT][16]) {
        const int g = lane >> 4;
        if constexpr (VEC) {
            const Rsrc rs = make_rsrc(oh + t0 * p.os.st, 0x7fffffff);
            each(t0, p.os, [&](int nt, int r, uint32_t off, uint32_t soff) {
                __builtin_amdgcn_raw_buffer_store_b16(to_bf16(o[nt][r]), rs, off, soff, 0);
            });
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t t = t0 + tok_of(r >> 2, 4 * g + (r & 3));
                    if (t < sp.n && col(nt) < p.Dv) oh[t * p.os.st + col(nt) * p.os.sd] = to_bf16(o[nt][r]);
                }
        }
    }

    __device__ __forceinline__ void chunk(int64_t t0, const Buf<KT> &b, bool more) {
        const int g = lane >> 4;
        // the state in high and low parts (its largest element is below 2^15)
        f16x8 sh[NT][KT], sl[NT][KT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = S[nt][2 * kt + (j >> 2)][j & 3];
                split8(f, sh[nt][kt], sl[nt][kt]);
            }
        // scales: of X from a bound (|k16 S| <= 2 Dk max |S|), so that it is known before X
        float inv[NT], xs[NT], back[NT], ms[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float m = 0.0f;
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S[nt][d][i]));
            uint32_t vm = 0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t u = v[nt][r] & 0x7fffu;
                vm = vm > u ? vm : u;
            }
            inv[nt] = pow2(es[nt] - 14);
            ms[nt] = max_groups(m) * inv[nt];
            const float vmax = max_groups(__uint_as_float(vm << 16));
            int ex = exp_of(b.kb_max * fmaf(b.ak_max * float(64 * KT), ms[nt], vmax));
            ex = ex > 113 ? 113 : ex;
            xs[nt] = pow2(14 - ex);
            back[nt] = pow2(ex - 14);
        }

        // K S and Q S; X
        f32x4 aq[NT][4];
        float x[NT][16];
#pragma unroll
        for (int m2 = 0; m2 < 4; m2 += 2) {
            f32x4 ak[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int m = 0; m < 2; ++m) { ak[nt][m] = f32x4{0, 0, 0, 0}; aq[nt][m2 + m] = f32x4{0, 0, 0, 0}; }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                f16x8 kf[2], qf[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    kf[m] = row_tile_of(b.k, (m2 + m) * KT + kt, kt, lane);
                    qf[m] = row_tile_of(b.q, (m2 + m) * KT + kt, kt, lane);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int m = 0; m < 2; ++m) ak[nt][m] = mfma(kf[m], sh[nt][kt], ak[nt][m]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int m = 0; m < 2; ++m) aq[nt][m2 + m] = mfma(qf[m], sh[nt][kt], aq[nt][m2 + m]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int m = 0; m < 2; ++m) ak[nt][m] = mfma(kf[m], sl[nt][kt], ak[nt][m]);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int t = tok_of(m2 + m, 4 * g);
                const f32x4 fa = *reinterpret_cast<const f32x4 *>(b.ak + t), kb = *reinterpret_cast<const f32x4 *>(b.kb + t);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[nt][4 * (m2 + m) + i] =
                            kb[i] * xs[nt] * fmaf(-fa[i] * inv[nt], ak[nt][m][i], bf_one(v[nt][4 * (m2 + m) + i]));
            }
        }
        if (more) fetch(t0 + kC);

        // z = T X
        f16x8 xh[NT][2], xl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = x[nt][8 * tt + j];
                split8(f, xh[nt][tt], xl[nt][tt]);
            }
        f32x4 z[NT][4];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            f16x8 h[4], l[4];
#pragma unroll
            for (int mt = 2 * tt; mt < 4; ++mt) {
                h[mt] = tile_of(b.th, tri_tile(mt, tt), lane);
                l[mt] = tile_of(b.tl, tri_tile(mt, tt), lane);
            }
            if (tt == 0)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) z[nt][mt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 2 * tt; mt < 4; ++mt) z[nt][mt] = mfma(h[mt], xh[nt][tt], z[nt][mt]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 2 * tt; mt < 4; ++mt) z[nt][mt] = mfma(h[mt], xl[nt][tt], z[nt][mt]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 2 * tt; mt < 4; ++mt) z[nt][mt] = mfma(l[mt], xh[nt][tt], z[nt][mt]);
        }

        // the next scale of the state, and of z: from a bound of the next state (64 tokens, |k16| < 2)
        f16x8 yh[NT][2], yl[NT][2], zh[NT][2];
        float zinv[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float m = 0.0f;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(z[nt][mt][i]));
            const int ez = exp_of(fmaf(max_groups(m) * back[nt], 2.0f * kC, b.last * ms[nt])) - 1;
            const float zs = back[nt] * pow2(14 - ez);
            zinv[nt] = pow2(ez - 14);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                float f[8], y[8];
#pragma unroll
                for (int t2 = 0; t2 < 2; ++t2) {
                    const f32x4 eg = *reinterpret_cast<const f32x4 *>(b.eg + tok_of(2 * tt + t2, 4 * g));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[4 * t2 + i] = z[nt][2 * tt + t2][i] * zs;
                        y[4 * t2 + i] = f[4 * t2 + i] * eg[i];
                    }
                }
                zh[nt][tt] = half8(f);
                split8(y, yh[nt][tt], yl[nt][tt]);
            }
            int up = es[nt] - ez;
            up = up < -126 ? -126 : (up > 127 ? 127 : up);
            const float sc = b.last * pow2(up);
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d) S[nt][d] *= sc;
            es[nt] = ez;
        }

        // S += K^T y
#pragma unroll
        for (int d0 = 0; d0 < 2 * KT; d0 += 4)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                f16x8 k[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) k[d] = col_tile_of(b.kt, d0 + d, tt, lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int d = 0; d < 4; ++d) S[nt][d0 + d] = mfma(k[d], yh[nt][tt], S[nt][d0 + d]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int d = 0; d < 4; ++d) S[nt][d0 + d] = mfma(k[d], yl[nt][tt], S[nt][d0 + d]);
            }

        // o
        float o[NT][16];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 qf = *reinterpret_cast<const f32x4 *>(b.qf + tok_of(mt, 4 * g));
            const f32x4 qe = *reinterpret_cast<const f32x4 *>(b.qe + tok_of(mt, 4 * g));
            f32x4 pz[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) pz[nt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int tt = 0; tt <= mt / 2; ++tt) {
                const f16x8 pf = tile_of(b.p, tri_tile(mt, tt), lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) pz[nt] = mfma(pf, zh[nt][tt], pz[nt]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[nt][4 * mt + i] = fmaf(qf[i] * zinv[nt], pz[nt][i], qe[i] * inv[nt] * aq[nt][mt][i]);
        }
        store(t0, o);
    }
};

// Workgroups of one sequence and key head follow each other on one XCD (blocks go to the 8 XCDs in turn), so that
// they read its keys and queries from one L2.
struct Place { int32_t b, h, cg; bool ok; };
__device__ __forceinline__ Place place_of(const GdrParams &p, int32_t groups) {
    const int32_t per = p.group * groups;
    const int64_t slot = blockIdx.x >> 3;
    const int64_t unit = slot / per * 8 + (blockIdx.x & 7);
    const int32_t r = int32_t(slot % per);
    Place pl;
    pl.ok = unit < int64_t(p.batch) * p.Hk;
    pl.b = int32_t(unit / p.Hk);
    pl.h = int32_t(unit % p.Hk) * p.group + r / groups;
    pl.cg = r % groups;
    return pl;
}

template <int KT, int NS, int NT, bool VEC>
__global__ __launch_bounds__(64 * (NS + kProducers)) void gdr_chunk_kernel(GdrParams p, int32_t groups, bool svec) {
    __shared__ Shared<KT> sh;
    const Place pl = place_of(p, groups);
    if (!pl.ok) return;
    Span64 sp;
    {
        int64_t a = p.qsl[pl.b], e = p.qsl[pl.b + 1];
        a = a < 0 ? 0 : (a > p.total_T ? p.total_T : a);
        e = e < a ? a : (e > p.total_T ? p.total_T : e);
        sp.t0 = a;
        sp.n = e - a;
    }
    if (sp.n == 0) return;
    int64_t line = pl.b;
    if (p.ci) {
        line = p.ci[pl.b];
        if (line == p.pad_slot_id) return;
    }
    if (p.state && (line < 0 || line >= p.num_lines)) return;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t nc = (sp.n + kC - 1) / kC;
    if (threadIdx.x == 0) sh.sync = 0;
    // what lies above T's diagonal blocks in its tiles is zero and stays so
    for (int i = threadIdx.x; i < kTriTiles * kTile / 2; i += 64 * (NS + kProducers))
        for (int k = 0; k < 2; ++k) {
            reinterpret_cast<uint32_t *>(sh.buf[k].th)[i] = 0u;
            reinterpret_cast<uint32_t *>(sh.buf[k].tl)[i] = 0u;
        }
    __syncthreads();

    if (wave >= NS) {
        const int hk = pl.h / p.group;
        Producer<KT, VEC> pr{p, sh, sp, lane, wave - NS, pl.h, p.q + hk * p.qs.sh, p.k + hk * p.ks.sh};
        pr.fetch(0);
        if (pr.w == 0) pr.gates(0);
        pr.chunk(0, sh.buf[0], nc > 1);
        __syncthreads();
        for (int64_t c = 0; c < nc; ++c) {
            if (c + 1 < nc) pr.chunk((c + 1) * kC, sh.buf[(c + 1) & 1], c + 2 < nc);
            __syncthreads();
        }
        return;
    }

    const int g = lane >> 4;
    Consumer<KT, NT, VEC> st{p, sp, lane};
    st.c0 = (pl.cg * NS + wave) * NT * 16;
    st.vh = p.v + sp.t0 * p.vs.st + pl.h * p.vs.sh;
    st.oh = p.out + sp.t0 * p.os.st + pl.h * p.os.sh;
    const bool init = p.state && p.has_init && p.has_init[pl.b] != 0;
    float *rows = p.state ? p.state + line * p.s_sl + pl.h * p.s_sh : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float *row = rows + st.col(nt) * p.s_sv;
        const bool ok = init && st.col(nt) < p.Dv;
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) {
            const int k = 32 * (d >> 1) + 8 * g + 4 * (d & 1);
            st.S[nt][d] = f32x4{0, 0, 0, 0};
            if (svec) {
                if (ok && k < p.Dk) st.S[nt][d] = *reinterpret_cast<const f32x4 *>(row + k);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (ok && k + i < p.Dk) st.S[nt][d][i] = row[(k + i) * p.s_sk];
            }
        }
        float m = 0.0f;
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(st.S[nt][d][i]));
        st.es[nt] = exp_of(max_groups(m));
        const float s = pow2(14 - st.es[nt]);
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) st.S[nt][d] *= s;
    }
    st.fetch(0);
    __syncthreads();
    for (int64_t c = 0; c < nc; ++c) {
        st.chunk(c * kC, sh.buf[c & 1], c + 1 < nc);
        __syncthreads();
    }
    if (!p.state) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float *row = rows + st.col(nt) * p.s_sv;
        const bool ok = st.col(nt) < p.Dv;
        const float inv = pow2(st.es[nt] - 14);
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) {
            const int k = 32 * (d >> 1) + 8 * g + 4 * (d & 1);
            const f32x4 s = st.S[nt][d] * inv;
            if (svec) {
                if (ok && k < p.Dk) *reinterpret_cast<f32x4 *>(row + k) = s;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (ok && k + i < p.Dk) row[(k + i) * p.s_sk] = s[i];
            }
        }
    }
}

template <int KT, int NS, int NT, bool VEC>
hipError_t launch_cfg(const GdrParams &p, bool svec, hipStream_t s) {
    const int32_t groups = (p.Dv + 16 * NS * NT - 1) / (16 * NS * NT);
    const int64_t units = (int64_t(p.batch) * p.Hk + 7) / 8 * 8;
    const dim3 grid(uint32_t(units * p.group * groups)), block(64 * (NS + kProducers));
    gdr_chunk_kernel<KT, NS, NT, VEC><<<grid, block, 0, s>>>(p, groups, svec);
    return hipGetLastError();
}

template <int KT, bool VEC>
hipError_t launch_kt(const GdrParams &p, bool svec, hipStream_t s) {
#ifndef CFG
#define CFG 8, 1
#endif
    return launch_cfg<KT, CFG, VEC>(p, svec, s);
}

}  // namespace

hipError_t launch_gdr_chunk(const GdrParams &p, bool vec, bool svec, hipStream_t s) {
    if (p.Dk <= 64) return vec ? launch_kt<2, true>(p, svec, s) : launch_kt<2, false>(p, svec, s);
    return vec ? launch_kt<4, true>(p, svec, s) : launch_kt<4, false>(p, svec, s);
}

}  // namespace sconv

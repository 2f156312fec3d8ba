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
// The rule by itself is some 100 K fp32 operations a token and head, each token
// waiting for the one before.  Here the same work is matrix products, 64 tokens
// at a time: 64 sequences of up to 2048 tokens, 32 heads of 128 x 128, take
// 0.76 ms where a token at a time takes 18.7 ms.
//
// One kernel (many heads).  A workgroup of 8 waves owns 128 value channels of
// one head and walks its sequence.  Per chunk it prepares the operands in LDS
// (conversion, K K^T, Q K^T, the inverse: phases between barriers), then each
// wave takes its 16 channels through the chunk with the state in its
// registers.  Two workgroups share a CU (128 registers, 79 KB), so that one's
// matrix products run beside the other's conversions and waits (waves that only
// prepare beside waves that only consume, one workgroup a CU, took 13 % more when
// both were at 1.1 ms).  What bounds it now: a chunk is a chain of phases, 8.3 us
// for a workgroup alone on its CU (7.6 with few on the chip) and 12.6 for two
// sharing it, with the VALU 78 % busy (conversions, scaling, addresses: 1200
// instructions a wave and chunk) and the MFMAs 31 %; a twentieth less VALU work
// alone changes nothing.  Bytes would take 0.29 ms.
//
// Two kernels (few heads): a walk is a chain of chunks, so everything that does
// not depend on the state is prepared before it by the whole chip.  At 4195
// tokens, 32 heads: 29 us and 132 us for 66 chunks, 2.0 us each, a chain of
// products and of the conversions between them; at 14807 tokens 74 and 452 us.
//
// Waves of one state never exchange anything: an MFMA result has its channel in
// the lane and 4 rows a register quad, and the next product takes it as its
// right operand as it lies, since the order of a contracted index is free.  So
// key channel 32 kt + 8 g + 4 t + i is row 4 g + i of result tile 2 kt + t and
// slot 4 t + i of lane group g in operand tile kt; tokens are ordered likewise.
//
// Precision: the state is fp32 and every product that feeds it has 22-bit
// operands: fp16 pairs (high, low part), scaled by powers of two (a key row to
// a norm near 1, a state, X or z column by its largest element), summed in fp32
// by the MFMA.  A key is one fp16 part: its bf16 elements are exact down to 2^-16
// of the row's norm, and off by less than 2^-24 of it below that.  So K S takes 2
// MFMAs and T X 3.  An fp32 MFMA would take 8 times as long as one of these
// pairs, and a single fp16 operand would leave the state at 11 bits.  The output
// is bf16, so the products that only feed it (Q S, P z) take operands of 11 bits:
// its error against 64 bits is 0.00168 of its size where fp32 operands and the
// same last rounding have 0.00166.  S and z in two parts there give 0.00167 and
// take 815 us for the 64 sequences (771).
#include "gdr_device.h"
#include "gdr_units.h"

namespace sconv {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kC = 64;                 // tokens per chunk
constexpr int kWaves = 8;              // waves per workgroup, 16 value channels each
static_assert(64 * kWaves == kGdrThreads, "the host's launch checks");

// Tile-ordered operands in LDS: a 16-row x 32-column fp16 tile is 1 KiB, lane
// l's 16 bytes (row l % 16, columns 8 (l / 16) ..) at 16 l, so a wave reads a
// tile in one conflict-free access.
constexpr int kTile = 512;             // halves per tile

// Tiles of the 64 x 64 lower triangle, rows in 4 tiles, columns in 2: the rows
// of tiles 0 and 1 end before column 32.
__device__ __forceinline__ constexpr int tri_tile(int mt, int tt) { return mt < 2 ? mt : 2 + 2 * (mt - 2) + tt; }
constexpr int kTriTiles = 6;

// What decays between two tokens is small, and fp16 has no step below 2^-24: the triangles are held times powers of two.  A
// and T, 4 at most where the rule contracts, then have steps of 2^-30 (and may reach 1023); P, at most 2, of 2^-38.  Without,
// a state that decays by 2^-17 inside a chunk was off by 2^-23 of the chunk's largest value.
constexpr float kTriScale = 1 << kTriExp, kTriInv = 1.0f / kTriScale;
constexpr float kPScale = 1 << 14;

template <int KT>
struct alignas(16) KeyTiles {          // of a chunk's keys and queries
    _Float16 k[4 * KT * kTile];        // [mt][kt] rows tokens
    _Float16 q[4 * KT * kTile];
    _Float16 kt[4 * KT * kTile];       // [2 KT channel tiles][2] rows key channels, columns tokens
};
struct alignas(16) HeadTiles {         // ... with a value head's gates
    _Float16 th[kTriTiles * kTile];    // T kTriScale, high and low parts
    _Float16 tl[kTriTiles * kTile];
    _Float16 p[kTriTiles * kTile];     // e^(Gi - Gj) q16.k16 kPScale
    float kb[kC];                      // kf beta
    float ka[kC];                      // kf beta e^G kf
    float eg[kC];                      // e^(G_last - G)
    float qf[kC];                      // qf / kPScale
    float qe[kC];                      // qf e^G
    float last;                        // e^G_last
};
template <int KT>
struct Tiles : KeyTiles<KT>, HeadTiles {};

struct alignas(16) Scratch {           // of the preparation
    _Float16 off[6 * kTile];           // A's blocks below the diagonal, times kTriScale: [4 rows / 4][column]: 4 high, 4 low parts
    float diag[4 * 256];               // A's diagonal blocks by columns, then T's, times kTriScale
    float dump[4];                     // for what lies in neither
    float Gh[kC], Gl[kC];              // running log decay, in powers of 2: high and low parts
    float beta[kC], eG[kC], eg[kC], kf[kC], qf[kC];
};
static_assert(sizeof(Tiles<4>) + sizeof(Scratch) <= 80 * 1024, "two workgroups of the one-kernel form per CU");

// Token t of a chunk as a row: tile 2 (t / 32) + (t / 4) % 2, row 4 ((t % 32) / 8) + t % 4.
__device__ __forceinline__ int row_tile(int t) { return 2 * (t >> 5) + ((t >> 2) & 1); }
__device__ __forceinline__ int row_in(int t) { return 4 * ((t >> 3) & 3) + (t & 3); }
// ... and the token of row r of tile mt.
__device__ __forceinline__ int tok_of(int mt, int r) { return 32 * (mt >> 1) + 8 * (r >> 2) + 4 * (mt & 1) + (r & 3); }
// Offset (halves) of row r, column c (0..31) in a tile.
__device__ __forceinline__ int in_tile(int r, int c) { return (r + 16 * (c >> 3)) * 8 + (c & 7); }

// Rows of the k and q tiles are stored at r ^ (g + 4 (kt % 2)), g = column / 8, and rows of the transposed tiles at
// r ^ (d / 2): the staging waves' 64 lanes then write to every bank alike, and a read is a permutation of 256 bytes.
__device__ __forceinline__ int swz_rows(int r, int g, int kt) { return r ^ (g + 4 * (kt & 1)); }

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }   // -126..127
__device__ __forceinline__ int exp_of(float m) {       // m in [2^(e-1), 2^e)
    return m == 0.0f ? kMinExp : held_exp(__builtin_amdgcn_frexp_expf(m));
}

// The lane number anew, as a value that the compiler takes for unknown: what is computed from it stays in its phase.
// (Every phase has its own addresses; kept in registers over the whole loop they would spill.)
__device__ __forceinline__ int fresh(int lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}

// Over aligned groups of N lanes (8 or 16).
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
// A factor of 1 that the compiler does not know: x - h in fp16 is then one instruction (a multiplication and addition of
// mixed types) instead of a conversion, a subtraction and half a conversion.
__device__ __forceinline__ float opaque_one() {
    float one = 1.0f;
    asm("" : "+s"(one));
    return one;
}
// ... as they are.
__device__ __forceinline__ void split8(const float (&x)[8], f16x8 &hi, f16x8 &lo) {
    const float one = opaque_one();
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const f16x2 h = cvt2(x[i], x[i + 1]);
        hi[i] = h.x; hi[i + 1] = h.y;
        lo[i] = _Float16(fmaf(x[i], one, -float(h.x)));
        lo[i + 1] = _Float16(fmaf(x[i + 1], one, -float(h.y)));
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

struct Span32 { int32_t t0, n; };      // a sequence's first row and length

// A head's rows of one tensor, from the sequence's first on.  VEC reads and writes them through a descriptor over a
// chunk's rows, each longer than the head's channels, so that what does not exist lies past its end.
struct Rows {
    const uint16_t *base;
    uint32_t row;                      // bytes (VEC)
    const GdrTensor *ts;
};
__device__ __forceinline__ Rows rows_of(const uint16_t *t, const GdrTensor &ts, int32_t t0, int32_t h) {
    return {t + t0 * ts.st + h * ts.sh, uint32_t(ts.st) * 2, &ts};
}
__device__ __forceinline__ Rsrc chunk_rsrc(const Rows &r, const Span32 &sp, int32_t c0) {
    const int32_t left = sp.n - c0 < kC ? sp.n - c0 : kC;
    const char *a = reinterpret_cast<const char *>(r.base) + uint64_t(uint32_t(c0)) * r.row;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(a), short(0), left <= 0 ? 0 : int(left * r.row), 0x00020000);
}

// --------------------------------------------------- preparing the chunk --

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

// Four token rows of eight channels each, as a staging thread holds them.
struct Quad { u32x4 r[4]; };

template <bool VEC>
__device__ __forceinline__ Quad load_quad(const Rows &r, const Span32 &sp, int32_t c0, int quad, int kc, int32_t Dk) {
    Quad q;
    if constexpr (VEC) {
        const Rsrc rs = chunk_rsrc(r, sp, c0);
        const uint32_t at = 8 * kc < Dk ? uint32_t(4 * quad) * r.row + 16u * kc : kOob;
#pragma unroll
        for (int i = 0; i < 4; ++i) q.r[i] = buf_ld128<0>(rs, at + i * r.row);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t t = c0 + 4 * quad + i;
            const bool live = t < sp.n;
            q.r[i] = load8(r.base + (live ? t : 0) * r.ts->st, r.ts->sd, 8 * kc, Dk, live);
        }
    }
    return q;
}

// Scales a row by a power of two (to a norm of 2^-0.5 .. 2^0.5), writes it as a row of the operand tiles (and, for
// keys, transposed), and its factor: the power, times the norm's inverse and `scale`.
// `cols` or `factor` may be null: not wanted.
template <int KT>
__device__ __forceinline__ void stage_quad(const Quad &in, _Float16 *rows, _Float16 *cols, float *factor, int quad, int kc,
                                           float scale, bool l2norm) {
    f16x8 h[4];
    const int kt = kc >> 2, g = kc & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x2 w = __builtin_bit_cast(bf16x2, uint32_t(in.r[i][j]));
            ss = __builtin_amdgcn_fdot2_f32_bf16(w, w, ss, false);
        }
        ss = sum_lanes<4 * KT>(ss);
        // 2^(63 - e) with e half of the sum's biased exponent brings the norm to 2^-0.5 .. 2^0.5
        const uint32_t e = __float_as_uint(ss) >> 24;
        const float s = __uint_as_float((190u - e) << 23);
        float f[8];
        unpack8(in.r[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= s;
        h[i] = half8(f);
        const int t = 4 * quad + i;
        if (factor && kc == i)
            factor[t] = scale * (l2norm ? __builtin_amdgcn_rsqf(ss + kL2Eps) : 1.0f) * __uint_as_float((64u + e) << 23);
        // (row, columns 8 kc ..) of tile (row tile, kt)
        const int at = (row_tile(t) * KT + kt) * kTile + (swz_rows(row_in(t), g, kt) + 16 * g) * 8;
        *reinterpret_cast<f16x8 *>(rows + at) = h[i];
    }
    if (cols) {
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

// What lane I of the 16-lane row holds.
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
    const float one = opaque_one();
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const f16x2 h = cvt2(x[i], x[i + 1]);
        hi[i] = h.x; hi[i + 1] = h.y;
        lo[i] = _Float16(fmaf(x[i], one, -float(h.x)));
        lo[i + 1] = _Float16(fmaf(x[i + 1], one, -float(h.y)));
    }
}

template <int KT, bool VEC>
struct Prepare {
    const GdrParams &p;
    Scratch &sh;
    _Float16 *k, *q, *cols;            // the chunk's rows as tiles, and the keys' transposed or null, in LDS
    HeadTiles *ht;                     // in LDS or in memory
    const Span32 sp;
    const int lane0, w;
    int h;                             // value head
    const Rows qr, kr;

    // The first waves stage the keys, as many after them the queries: 4 KT threads a row, four rows a thread.
    static constexpr int kStage = KT;  // waves
    __device__ __forceinline__ int quad_of(int lane) const { return (64 * (w & (kStage - 1)) + lane) / (4 * KT); }

    __device__ __forceinline__ Quad load(int32_t c0) const {
        const int lane = fresh(lane0), kc = lane & (4 * KT - 1), quad = quad_of(lane);
        return load_quad<VEC>(w < kStage ? kr : qr, sp, c0, quad, kc, p.Dk);
    }
    __device__ __forceinline__ void stage(const Quad &in) {
        const int lane = fresh(lane0), kc = lane & (4 * KT - 1), quad = quad_of(lane);
        if (w < kStage) stage_quad<KT>(in, k, cols, sh.kf, quad, kc, 1.0f, p.l2norm);
        else if (w < 2 * kStage) stage_quad<KT>(in, q, nullptr, sh.qf, quad, kc, p.scale, p.l2norm);
    }

    // From the chunk's staged rows and its gates in LDS to its tiles.  `ahead` runs in wave 7 once the gates' place is free.
    template <class F>
    __device__ __forceinline__ void tiles(F ahead) {
        __syncthreads();
        key_products();
        if (w == 7) factors();
        __syncthreads();
        if (w == 0) invert_diagonal();
        else if (w < 7) query_products();              // (the inverse waits for one wave)
        __syncthreads();
        if (w < 4) invert_rest();
        else if (w == 7) ahead();
        __syncthreads();
    }

    // Gates of a chunk, one token a lane.  The running sum is in fp64 and kept in two fp32 parts: a difference of two of
    // its values keeps every bit of a small decay behind a large one.  Every e^ below is of a difference <= 0.
    __device__ __forceinline__ void gates(int32_t c0) {
        const int lane = fresh(lane0);
        const int32_t t = c0 + lane;
        Gates gt = {0.0f, 0.0f};
        if (t < sp.n)
            gt = gdr_gates(p, int64_t(sp.t0 + t) * p.gs.st + h * p.gs.sh, int64_t(sp.t0 + t) * p.bs.st + h * p.bs.sh, h);
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

    // The row factors of the chunk.
    __device__ __forceinline__ void factors() {
        const int lane = fresh(lane0);
        const float kf = sh.kf[lane], qf = sh.qf[lane], eG = sh.eG[lane], kb = kf * sh.beta[lane];
        ht->qf[lane] = qf * (1.0f / kPScale);
        ht->kb[lane] = kb;
        ht->ka[lane] = kb * eG * kf;
        ht->eg[lane] = sh.eg[lane];
        ht->qe[lane] = qf * eG;
        if (lane == 63) ht->last = eG;
    }

    // 2^(running decays of four tokens less that of one, or the reverse).
    template <bool REV>
    __device__ __forceinline__ f32x4 decay(int t4, int t) {
        const f32x4 ah = *reinterpret_cast<const f32x4 *>(sh.Gh + t4), al = *reinterpret_cast<const f32x4 *>(sh.Gl + t4);
        const float bh = sh.Gh[t], bl = sh.Gl[t];
        f32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = __builtin_amdgcn_exp2f(REV ? (bh - ah[i]) + (bl - al[i]) : (ah[i] - bh) + (al[i] - bl));
        return r;
    }

    // K K^T and Q K^T: 12 tile pairs meet the lower triangle, one or two a wave.  K K^T has its rows in the registers, Q K^T
    // (as its transpose) its columns: what a lane holds is then one piece of the operand that it becomes.
    static __device__ __forceinline__ void pair(int pr, int &mt, int &nt) {
        mt = pr < 4 ? pr >> 1 : 2 + ((pr - 4) >> 2);
        nt = pr < 4 ? pr & 1 : (pr - 4) & 3;
    }
    __device__ __forceinline__ void key_products() {
        const int lane = fresh(lane0), n = lane & 15, g = lane >> 4;
        for (int pr = w; pr < 12; pr += 8) {
            int mt, nt;
            pair(pr, mt, nt);
            f32x4 kk = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KT; ++i) kk = mfma(row_tile_of(k, mt * KT + i, i, lane), row_tile_of(k, nt * KT + i, i, lane), kk);
            const int tj = tok_of(nt, n), ti = tok_of(mt, 4 * g);
            const int bi = ti >> 4, bj = tj >> 4;
            const f32x4 kf = *reinterpret_cast<const f32x4 *>(sh.kf + ti);
            const f32x4 a = *reinterpret_cast<const f32x4 *>(sh.beta + ti) * kf * kf * decay<false>(ti, tj) * kk;
            f16x4 hi, lo;
            split4(a * kTriScale, hi, lo);
            _Float16 *op = bi > bj ? sh.off + (bi * (bi - 1) / 2 + bj) * kTile + ((tj & 15) + 4 * (ti & 12)) * 8
                                   : reinterpret_cast<_Float16 *>(sh.dump);
            *reinterpret_cast<f16x8 *>(op) = f16x8{hi[0], hi[1], hi[2], hi[3], lo[0], lo[1], lo[2], lo[3]};
            if ((mt >> 1) == (nt >> 1))
                *reinterpret_cast<f32x4 *>(bi == bj ? sh.diag + bi * 256 + (tj & 15) * 16 + (ti & 15) : sh.dump) = a;
        }
    }
    // Waves 1 to 6.
    __device__ __forceinline__ void query_products() {
        const int lane = fresh(lane0), n = lane & 15, g = lane >> 4;
        f32x4 qk[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            int mt, nt;
            pair(2 * (w - 1) + x, mt, nt);
            qk[x] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KT; ++i)
                qk[x] = mfma(row_tile_of(k, nt * KT + i, i, lane), row_tile_of(q, mt * KT + i, i, lane), qk[x]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            int mt, nt;
            pair(2 * (w - 1) + x, mt, nt);
            const int ti = tok_of(mt, n), tj = tok_of(nt, 4 * g);
            const f32x4 d = decay<true>(tj, ti);
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = tj + i <= ti ? d[i] * (qk[x][i] * kPScale) : 0.0f;
            const f16x2 lo = cvt2(v[0], v[1]), hi = cvt2(v[2], v[3]);
            *reinterpret_cast<f16x4 *>(ht->p + tri_tile(mt, nt >> 1) * kTile + in_tile(n, tj & 31)) =
                f16x4{lo.x, lo.y, hi.x, hi.y};
        }
    }

    // Inverts the four diagonal blocks at once: block g in lane row g, a column a lane, by forward substitution; the
    // elements of A come from the lane that holds their column.
    __device__ __forceinline__ void invert_diagonal() {
        const int lane = fresh(lane0), n = lane & 15, g = lane >> 4;
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
        for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<f32x4 *>(blk + j) = f32x4{x[j], x[j + 1], x[j + 2], x[j + 3]} * kTriScale;
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
    __device__ __forceinline__ void invert_rest() {
        const int lane = fresh(lane0), n = lane & 15, g = lane >> 4;
        const int ti = 16 * w + n;
        // every operand at once, used or not: what is left is a chain of products
        f16x8 off[6], left[3];
#pragma unroll
        for (int i = 0; i < 6; ++i) off[i] = tile_of(sh.off, i, lane);
        f32x4 d[3], t;
#pragma unroll
        for (int j = 0; j < 3; ++j) d[j] = -*reinterpret_cast<const f32x4 *>(sh.diag + j * 256 + n * 16 + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = sh.diag[w * 256 + (4 * g + e) * 16 + n];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            f16x4 dh, dl;
            split4(d[j], dh, dl);
            left[j] = f16x8{dh[0], dh[1], dh[2], dh[3], dl[0], dl[1], dl[2], dl[3]};
        }
        f16x4 hi[4], lo[4];
#pragma unroll
        for (int j = 3; j >= 0; --j) {
            if (j > w) continue;
            if (j < w) {
                f32x4 m = {0, 0, 0, 0};
#pragma unroll
                for (int k = 3; k >= 0; --k)
                    if (k > j && k <= w) m = block_mfma(off[k * (k - 1) / 2 + j], hi[k], lo[k], m);
                f16x4 mh, ml;
                split4(m * kTriInv, mh, ml);
                t = block_mfma(left[j < 3 ? j : 0], mh, ml, f32x4{0, 0, 0, 0}) * kTriInv;
            }
            split4(t, hi[j], lo[j]);
            const int tj = 16 * j + 4 * g;
            const int o = tri_tile(row_tile(ti), tj >> 5) * kTile + in_tile(row_in(ti), tj & 31);
            *reinterpret_cast<f16x4 *>(ht->th + o) = hi[j];
            *reinterpret_cast<f16x4 *>(ht->tl + o) = lo[j];
        }
        if (!(w & 1)) {                                // the block to the right shares the tile: zero
            const int o = tri_tile(row_tile(ti), ti >> 5) * kTile + in_tile(row_in(ti), (16 * (w + 1) + 4 * g) & 31);
            *reinterpret_cast<f16x4 *>(ht->th + o) = f16x4{0, 0, 0, 0};
            *reinterpret_cast<f16x4 *>(ht->tl + o) = f16x4{0, 0, 0, 0};
        }
    }
};

// ---------------------------------------------------- the state's passage --

// What a state wave hands to the wave that computes its channels' output: the state before the chunk and z as fp16
// operands, and 2^-unit of both.  `ready` counts the halves handed over, two a chunk.
template <int KT>
struct alignas(16) Exchange {
    f16x8 s[KT * 64];
    f16x8 z[2 * 64];
    float oinv[16], ninv[16];
};

__device__ __forceinline__ void hand_over(int *ready) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    if ((threadIdx.x & 63) == 0) __hip_atomic_fetch_add(ready, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
// Both waves are of one workgroup, so both are resident, and the state wave waits for no one between two barriers.
__device__ __forceinline__ void await(int *ready, int count) {
    while (__hip_atomic_load(ready, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) < count) __builtin_amdgcn_s_sleep(1);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

template <int KT, bool VEC>
struct Consumer {
    const GdrParams &p;
    const Span32 sp;
    const int lane0;
    const Rows vr, out;
    int32_t c0;                        // the wave's first channel; lane l has c0 + l % 16
    f32x4 S[2 * KT];                   // the state times 2^un
    int un;

    // The state's rows in memory: this lane has channels 8 g + 4 t .. of each 32 of its value channel's row.
    template <class F>
    __device__ __forceinline__ void state_rows(float *rows, F f) {
        const int lane = fresh(lane0), g = lane >> 4;
        const int32_t c = c0 + (lane & 15);
        float *row = rows + c * p.s_sv;
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) f(d, row, 32 * (d >> 1) + 8 * g + 4 * (d & 1), c < p.Dv);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) S[d] = f32x4{0, 0, 0, 0};
        un = 0;
    }
    __device__ __forceinline__ void load(float *rows, bool svec) {
        zero();
        float m = 0.0f;
        state_rows(rows, [&](int d, const float *row, int k, bool ok) {
            if (svec) {
                if (ok && k < p.Dk) S[d] = *reinterpret_cast<const f32x4 *>(row + k);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (ok && k + i < p.Dk) S[d][i] = row[(k + i) * p.s_sk];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S[d][i]));
        });
        m = max_groups(m);
        un = m == 0.0f ? 0 : first_unit(exp_of(m));
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) S[d] *= pow2(un);
    }
    __device__ __forceinline__ void save(float *rows, bool svec) {
        const float inv = pow2(-un);
        state_rows(rows, [&](int d, float *row, int k, bool ok) {
            const f32x4 s = S[d] * inv;
            if (svec) {
                if (ok && k < p.Dk) *reinterpret_cast<f32x4 *>(row + k) = s;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (ok && k + i < p.Dk) row[(k + i) * p.s_sk] = s[i];
            }
        });
    }

    // The chunk's values as left operands: tile mt has token tok_of(mt, n) in row n, the wave's 16 channels in its first
    // columns.  Times the identity they become results, a channel a lane, like everything they meet (with bf16 values
    // nothing is rounded; it takes 4 loads where that layout would take 16).
    __device__ __forceinline__ void fetch(int32_t t0, u32x4 (&v)[4]) {
        const int lane = fresh(lane0), n = lane & 15, g = lane >> 4;
        const int32_t c = c0 + 8 * g;
        if constexpr (VEC) {
            const Rsrc rs = chunk_rsrc(vr, sp, t0);
            const uint32_t row = vr.row;
            const uint32_t at = g < 2 && c < p.Dv ? uint32_t(tok_of(0, n)) * row + uint32_t(c) * 2 : kOob;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) v[mt] = buf_ld128<0>(rs, at + uint32_t(tok_of(mt, 0)) * row);
        } else {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const int32_t t = t0 + tok_of(mt, n);
                const bool live = g < 2 && t < sp.n;
                v[mt] = load8(vr.base + (live ? t : 0) * p.vs.st, p.vs.sd, c, p.Dv, live);
            }
        }
    }
    // The identity as a right operand, times the column's unit (a power of two, within bf16's range).
    static __device__ __forceinline__ bf16x8 identity(int lane, int unit) {
        const uint32_t one = uint32_t(unit + 127) << 7;
        u32x4 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = 8 * (lane >> 4) + 2 * j - (lane & 15);
            r[j] = at == 0 ? one : at == -1 ? one << 16 : 0u;
        }
        return __builtin_bit_cast(bf16x8, r);
    }
    static __device__ __forceinline__ f32x4 values(const u32x4 &v, const bf16x8 &id) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), id, f32x4{0, 0, 0, 0}, 0, 0, 0);
    }

    // The output of tile mt comes as a transpose: token tok_of(mt, n) in the lane, channels 4 g .. in its registers.
    __device__ __forceinline__ void store(int32_t t0, const f32x4 (&o)[4]) {
        const int lane = fresh(lane0), n = lane & 15, g = lane >> 4;
        const int32_t c = c0 + 4 * g;
        if constexpr (VEC) {
            const Rsrc rs = chunk_rsrc(out, sp, t0);
            const uint32_t row = out.row;
            const uint32_t at = c < p.Dv ? uint32_t(tok_of(0, n)) * row + uint32_t(c) * 2 : kOob;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const u32x2 w = {pack_bf16x2(o[mt][0], o[mt][1]), pack_bf16x2(o[mt][2], o[mt][3])};
                __builtin_amdgcn_raw_buffer_store_b64(w, rs, at + uint32_t(tok_of(mt, 0)) * row, 0, 0);
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const int32_t t = t0 + tok_of(mt, n);
                uint16_t *row = const_cast<uint16_t *>(out.base) + t * p.os.st;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t < sp.n && c + i < p.Dv) row[(c + i) * p.os.sd] = to_bf16(o[mt][i]);
            }
        }
    }

    // The units of the next state: 2^14 above a bound of it (64 tokens, |k16| < 1.5, so the chunk adds at most 2^7 max |z|
    // to what is left of the last one).  z comes in its own unit, 2^(xe - kZExp) of the state's.
    struct Units { float zs, sc, ninv; };
    __device__ __forceinline__ Units next_unit(const f32x4 (&z)[4], float ms, float last, int xe) {
        float zm = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) zm = fmaxf(zm, fabsf(z[mt][i]));
        const float bound = max_groups(fmaf(zm * pow2(xe - kZExp), 128.0f, ms * last));
        const UnitStep st = sconv::next_unit(un, bound == 0.0f, exp_of(bound), xe);
        un += st.up;
        return {pow2(st.zu), last * pow2(st.up), pow2(-un)};
    }
    // A column whose unit is high (its state is small) takes one that its chunk's values allow; v: those values.  Hardly any
    // chunk has such a column.
    __device__ __forceinline__ bool high_unit() const { return __builtin_amdgcn_ballot_w64(un > kPlainUnit) != 0; }
    __device__ __forceinline__ void lower_unit(const u32x4 (&v)[4]) {
        const int lane = fresh(lane0);
        const bf16x8 id = identity(lane, 0);
        float m = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 vv = values(v[mt], id);
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(vv[i]));
        }
        m = max_groups(m);
        const int to = un > kPlainUnit ? unit_for_values(un, exp_of(m)) : un;
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[d][i] = ldexpf(S[d][i], to - un);
        un = to;
    }
    __device__ __forceinline__ void split_state(int kt, f16x8 &hi, f16x8 &lo) const {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = S[2 * kt + (j >> 2)][j & 3];
        split8(f, hi, lo);
    }
    __device__ __forceinline__ float largest() const {
        float m = 0.0f;
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S[d][i]));
        return m;
    }
    // z of tiles 2 tt and 2 tt + 1 as an fp16 operand, and y = e^(G_last - G) z.
    static __device__ __forceinline__ f16x8 scaled(const f32x4 (&z)[4], int tt, float zs, const f32x4 (&eg)[2], float (&y)[8]) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = z[2 * tt + (j >> 2)][j & 3] * zs;
            y[j] = f[j] * eg[j >> 2][j & 3];
        }
        return half8(f);
    }
    static __device__ __forceinline__ f32x4 row4(const float *v, int t) { return *reinterpret_cast<const f32x4 *>(v + t); }

    // The state and the output through one chunk, in 128 registers: four waves a SIMD hide what each waits for.
    template <class F>
    __device__ __forceinline__ void chunk(int32_t t0, const Tiles<KT> &b, F ahead) {
        const int lane = fresh(lane0), g = lane >> 4;
        f32x4 ak[4], aq[4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) { ak[mt] = f32x4{0, 0, 0, 0}; aq[mt] = f32x4{0, 0, 0, 0}; }
        const float ms = largest(), oinv = pow2(-un);
        u32x4 v[4];
        // K S and Q S, the state split on the way (its largest element is below 2^15)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            f16x8 hi, lo;
            if (kt == KT - 1) fetch(t0, v);            // (from L2)
            split_state(kt, hi, lo);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const f16x8 kf = row_tile_of(b.k, mt * KT + kt, kt, lane), qf = row_tile_of(b.q, mt * KT + kt, kt, lane);
                ak[mt] = mfma(kf, hi, ak[mt]);
                aq[mt] = mfma(hi, qf, aq[mt]);         // (transposed, as the output is)
                ak[mt] = mfma(kf, lo, ak[mt]);
            }
        }
        // X, scaled to 2^kXExp
        float x[16], xm = 0.0f;
        const bf16x8 id = identity(lane, un);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 ka = row4(b.ka, tok_of(mt, 4 * g)), kb = row4(b.kb, tok_of(mt, 4 * g)), vv = values(v[mt], id);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[4 * mt + i] = fmaf(-ka[i], ak[mt][i], kb[i] * vv[i]);
                xm = fmaxf(xm, fabsf(x[4 * mt + i]));
            }
        }
        const int xe = x_exp(exp_of(max_groups(xm)));
        const float xs = pow2(kXExp - xe);
        // z = T X
        f32x4 z[4];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            float f[8];
            f16x8 xh, xl;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = x[8 * tt + j] * xs;
            split8(f, xh, xl);
#pragma unroll
            for (int mt = 2 * tt; mt < 4; ++mt) {
                const f16x8 h = tile_of(b.th, tri_tile(mt, tt), lane), l = tile_of(b.tl, tri_tile(mt, tt), lane);
                if (tt == 0) z[mt] = f32x4{0, 0, 0, 0};
                z[mt] = mfma(h, xh, z[mt]);
                z[mt] = mfma(h, xl, z[mt]);
                z[mt] = mfma(l, xh, z[mt]);
            }
        }
        const Units u = next_unit(z, ms, b.last, xe);
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) S[d] *= u.sc;
        // S += K^T y
        f16x8 zh[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const f32x4 eg[2] = {row4(b.eg, tok_of(2 * tt, 4 * g)), row4(b.eg, tok_of(2 * tt + 1, 4 * g))};
            float y[8];
            f16x8 yh, yl;
            zh[tt] = scaled(z, tt, u.zs, eg, y);
            split8(y, yh, yl);
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d) {
                const f16x8 k = col_tile_of(b.kt, d, tt, lane);
                S[d] = mfma(k, yh, S[d]);
                S[d] = mfma(k, yl, S[d]);
            }
        }
        ahead();                                       // (the next chunk's rows are under way while the output is computed)
        __builtin_amdgcn_sched_barrier(0x7cf);         // VMEM reads stay here
        // o
        f32x4 o[4], oi, ni;
#pragma unroll
        for (int i = 0; i < 4; ++i) { oi[i] = __shfl(oinv, 4 * g + i); ni[i] = __shfl(u.ninv, 4 * g + i); }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            f32x4 pz = {0, 0, 0, 0};
#pragma unroll
            for (int tt = 0; tt <= mt / 2; ++tt) pz = mfma(zh[tt], tile_of(b.p, tri_tile(mt, tt), lane), pz);
            const int t = tok_of(mt, lane & 15);
            o[mt] = b.qf[t] * ni * pz + b.qe[t] * oi * aq[mt];
        }
        store(t0, o);
    }

    // The state alone through one chunk, one wave a SIMD: what a product needs beside the last one's result is read and
    // computed before that result is there.  v comes in and goes out with the next chunk's.
    __device__ __forceinline__ void advance(int32_t t0, const Tiles<KT> &b, u32x4 (&v)[4], Exchange<KT> *ex, int *ready) {
        if (high_unit()) lower_unit(v);
        const int lane = fresh(lane0), g = lane >> 4;
        f16x8 sh[KT], sl[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            split_state(kt, sh[kt], sl[kt]);
            ex->s[kt * 64 + lane] = sh[kt];
        }
        if (lane < 16) ex->oinv[lane] = pow2(-un);
        // K S
        f32x4 ak[4];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            f16x8 k[4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) k[mt] = row_tile_of(b.k, mt * KT + kt, kt, lane);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) ak[mt] = mfma(k[mt], sh[kt], kt ? ak[mt] : f32x4{0, 0, 0, 0});
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) ak[mt] = mfma(k[mt], sl[kt], ak[mt]);
        }
        hand_over(ready);
        f32x4 ka[4], xv[4];
        const bf16x8 id = identity(lane, un);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            ka[mt] = row4(b.ka, tok_of(mt, 4 * g));
            xv[mt] = row4(b.kb, tok_of(mt, 4 * g)) * values(v[mt], id);
        }
        f16x8 th[kTriTiles], tl[kTriTiles];
#pragma unroll
        for (int i = 0; i < kTriTiles; ++i) { th[i] = tile_of(b.th, i, lane); tl[i] = tile_of(b.tl, i, lane); }
        __builtin_amdgcn_sched_barrier(0);
        // X, scaled to 2^kXExp
        float xm = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xv[mt][i] = fmaf(-ka[mt][i], ak[mt][i], xv[mt][i]);
                xm = fmaxf(xm, fabsf(xv[mt][i]));
            }
        const int xe = x_exp(exp_of(max_groups(xm)));
        const float xs = pow2(kXExp - xe);
        // z = T X
        f32x4 z[4];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            float f[8];
            f16x8 xh, xl;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = xv[2 * tt + (j >> 2)][j & 3] * xs;
            split8(f, xh, xl);
#pragma unroll
            for (int mt = 2 * tt; mt < 4; ++mt) z[mt] = mfma(th[tri_tile(mt, tt)], xh, tt ? z[mt] : f32x4{0, 0, 0, 0});
#pragma unroll
            for (int mt = 2 * tt; mt < 4; ++mt) z[mt] = mfma(th[tri_tile(mt, tt)], xl, z[mt]);
#pragma unroll
            for (int mt = 2 * tt; mt < 4; ++mt) z[mt] = mfma(tl[tri_tile(mt, tt)], xh, z[mt]);
        }
        fetch(t0 + kC, v);                             // (rows behind the end read as zero)
        const float last = b.last, ms = largest();
        f32x4 eg[4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) eg[mt] = row4(b.eg, tok_of(mt, 4 * g));
        f16x8 kc[2 * KT];
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) kc[d] = col_tile_of(b.kt, d, 0, lane);
        __builtin_amdgcn_sched_barrier(0);
        const Units u = next_unit(z, ms, last, xe);
        float y[2][8];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const f32x4 e[2] = {eg[2 * tt], eg[2 * tt + 1]};
            ex->z[tt * 64 + lane] = scaled(z, tt, u.zs, e, y[tt]);
        }
        if (lane < 16) ex->ninv[lane] = u.ninv;
        hand_over(ready);
        // S += K^T y
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d) S[d] *= u.sc;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            f16x8 yh, yl;
            split8(y[tt], yh, yl);
            if (tt)
#pragma unroll
                for (int d = 0; d < 2 * KT; ++d) kc[d] = col_tile_of(b.kt, d, 1, lane);
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d) S[d] = mfma(kc[d], yh, S[d]);
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d) S[d] = mfma(kc[d], yl, S[d]);
        }
    }

    // The output of one chunk from what the state wave hands over; `done` halves came before.  All but z's own product
    // is ready when z comes.
    __device__ __forceinline__ void emit(int32_t t0, const Tiles<KT> &b, const Exchange<KT> *ex, int *ready, int done) {
        const int lane = fresh(lane0), n = lane & 15, g = lane >> 4;
        f32x4 aq[4];
        f16x8 q[4], pt[kTriTiles];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) q[mt] = row_tile_of(b.q, mt * KT, 0, lane);
        await(ready, done + 1);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const f16x8 s = ex->s[kt * 64 + lane];
            if (kt)
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) q[mt] = row_tile_of(b.q, mt * KT + kt, kt, lane);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) aq[mt] = mfma(s, q[mt], kt ? aq[mt] : f32x4{0, 0, 0, 0});
        }
        const f32x4 oinv = row4(ex->oinv, 4 * g);
        float qf[4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            qf[mt] = b.qf[tok_of(mt, n)];
            aq[mt] *= b.qe[tok_of(mt, n)] * oinv;
        }
#pragma unroll
        for (int i = 0; i < kTriTiles; ++i) pt[i] = tile_of(b.p, i, lane);
        __builtin_amdgcn_sched_barrier(0);
        await(ready, done + 2);
        const f16x8 zh[2] = {ex->z[lane], ex->z[64 + lane]};
        const f32x4 ninv = row4(ex->ninv, 4 * g);
        f32x4 o[4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) o[mt] = mfma(zh[0], pt[tri_tile(mt, 0)], f32x4{0, 0, 0, 0});
#pragma unroll
        for (int mt = 2; mt < 4; ++mt) o[mt] = mfma(zh[1], pt[tri_tile(mt, 1)], o[mt]);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) o[mt] = qf[mt] * ninv * o[mt] + aq[mt];
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

// Sequence b's rows and line; false when nothing is to be done for it.
__device__ __forceinline__ bool sequence(const GdrParams &p, int32_t b, Span32 &sp, int64_t &line) {
    int64_t a = p.qsl[b], e = p.qsl[b + 1];
    a = a < 0 ? 0 : (a > p.total_T ? p.total_T : a);
    e = e < a ? a : (e > p.total_T ? p.total_T : e);
    sp.t0 = int32_t(a);
    sp.n = int32_t(e - a);
    if (sp.n == 0) return false;
    line = b;
    if (p.ci) {
        line = p.ci[b];
        if (line == p.pad_slot_id) return false;
    }
    return !(p.state && (line < 0 || line >= p.num_lines));
}

constexpr int kMaxRanked = 64 * kWaves;

// The sequence that is r-th by length (the longest first): a workgroup takes as long as its sequence, and one that starts
// late with a long one leaves the chip idle behind it.  A thread a sequence counts those before it.  More sequences than
// threads stay in order.
__device__ __forceinline__ int32_t ranked(const GdrParams &p, int32_t r, int32_t *len, int32_t *out) {
    if (p.batch > kMaxRanked) return r;
    const int t = threadIdx.x;
    Span32 sp;
    int64_t line;
    int32_t n = 0;
    if (t < p.batch) {
        n = sequence(p, t, sp, line) ? sp.n : 0;
        len[t] = n;
    }
    __syncthreads();
    if (t < p.batch) {
        int32_t before = 0;
        for (int32_t i = 0; i < p.batch; ++i) before += len[i] > n || (len[i] == n && i < t);
        if (before == r) *out = t;
    }
    __syncthreads();
    return *out;
}

template <int KT, bool VEC>
__device__ __forceinline__ Consumer<KT, VEC> consumer(const GdrParams &p, const Span32 &sp, int lane, int32_t h, int32_t tile) {
    Consumer<KT, VEC> st{p, sp, lane, rows_of(p.v, p.vs, sp.t0, h), rows_of(p.out, p.os, sp.t0, h)};
    st.c0 = tile * 16;
    return st;
}

template <int KT, bool VEC>
__global__ __launch_bounds__(64 * kWaves, 4) void gdr_chunk_kernel(GdrParams p, int32_t groups, bool svec) {
    __shared__ Tiles<KT> tiles;
    __shared__ Scratch sh;
    Place pl = place_of(p, groups);
    if (!pl.ok) return;
    pl.b = __builtin_amdgcn_readfirstlane(
        ranked(p, pl.b, reinterpret_cast<int32_t *>(sh.diag), reinterpret_cast<int32_t *>(sh.diag) + kMaxRanked));
    Span32 sp;
    int64_t line;
    if (!sequence(p, pl.b, sp, line)) return;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int32_t nc = int32_t((int64_t(sp.n) + kC - 1) / kC);
    const int hk = pl.h / p.group;
    Prepare<KT, VEC> pr{p, sh, tiles.k, tiles.q, tiles.kt, &tiles, sp, lane, wave, pl.h, rows_of(p.q, p.qs, sp.t0, hk),
                        rows_of(p.k, p.ks, sp.t0, hk)};
    if (wave == 7) pr.gates(0);

    const int32_t tile = pl.cg * kWaves + wave;
    auto st = consumer<KT, VEC>(p, sp, lane, pl.h, tile);
    const bool work = tile * 16 < p.Dv;                            // this wave has channels
    float *rows = p.state ? p.state + line * p.s_sl + pl.h * p.s_sh : nullptr;
    if (p.state && p.has_init && p.has_init[pl.b] != 0) st.load(rows, svec);
    else st.zero();

    Quad rows4 = pr.load(0);
    for (int32_t c = 0; c < nc; ++c) {
        const bool more = c + 1 < nc;
        // The preparation's waves, few at a time and one chain, go before the other workgroup's products: 204 us for 384
        // workgroups of 16 chunks (215), 1 % where the chip is full.
        __builtin_amdgcn_s_setprio(2);
        pr.stage(rows4);
        if (work && st.high_unit()) {                  // (here it costs nothing; before the products 2 to 4 %)
            u32x4 v[4];
            st.fetch(c * kC, v);
            st.lower_unit(v);
        }
        pr.tiles([&]() { if (more) pr.gates((c + 1) * kC); });
        __builtin_amdgcn_s_setprio(0);
        if (work) st.chunk(c * kC, tiles, [&]() { rows4 = pr.load((c + 1) * kC); });
        else rows4 = pr.load((c + 1) * kC);            // (rows behind the end read as zero)
        __syncthreads();
    }
    if (p.state) st.save(rows, svec);
}

// ------------------------------------------------------------ two kernels --
//
// The tiles of all chunks are prepared into a workspace, [slots][Hv] HeadTiles (19 KB each).  Chunk j of sequence i has
// slot floor(start_i / 64) + i + j: no two chunks share one, and floor(T / 64) + batch + 2 of them are enough for any
// offsets, so no kernel has to count chunks.

__device__ __forceinline__ int64_t first_slot(const GdrParams &p, int32_t b) {
    int64_t a = p.qsl[b];
    a = a < 0 ? 0 : (a > p.total_T ? p.total_T : a);
    return (a >> 6) + b;
}

// A workgroup prepares one chunk of one key head, for `per` of the value heads that share it.
template <int KT, bool VEC>
__global__ __launch_bounds__(64 * kWaves, 4) void gdr_prepare_kernel(GdrParams p, HeadTiles *heads, int32_t per) {
    __shared__ _Float16 k[4 * KT * kTile], q[4 * KT * kTile];
    __shared__ Scratch sh;
    const uint32_t units = uint32_t(p.Hv / per);
    const int64_t slot = blockIdx.x / units;
    const int32_t h0 = int32_t(blockIdx.x - uint32_t(slot) * units) * per, hk = h0 / p.group;
    int32_t lo = 0, hi = p.batch - 1;                              // the last sequence whose slots start at or before
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (first_slot(p, mid) <= slot) lo = mid; else hi = mid - 1;
    }
    Span32 sp;
    int64_t line;
    if (!sequence(p, lo, sp, line)) return;
    const int64_t chunk = slot - first_slot(p, lo);
    if (chunk < 0 || chunk * kC >= sp.n) return;
    const int32_t c = int32_t(chunk);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    HeadTiles *ht = heads + slot * p.Hv + h0;
    Prepare<KT, VEC> pr{p, sh, k, q, nullptr, ht, sp, lane, wave, h0, rows_of(p.q, p.qs, sp.t0, hk),
                        rows_of(p.k, p.ks, sp.t0, hk)};
    if (wave == 7) pr.gates(c * kC);
    pr.stage(pr.load(c * kC));
    for (int32_t x = 0; x < per; ++x) {
        pr.tiles([&]() {
            if (x + 1 < per) {
                ++pr.h;
                pr.gates(c * kC);
            }
        });
        pr.h = h0 + x + 1;
        ++pr.ht;
    }
}

constexpr int kWalkers = 2;            // state waves of a walking workgroup
constexpr int kLoaders = 4;
constexpr int kWalkWaves = 2 * kWalkers + kLoaders;
static_assert(64 * kWalkWaves == kGdrThreads, "the host's launch checks");

// Walks a sequence over prepared tiles: four waves bring the next chunk's through registers into one of two buffers (and
// convert its keys and queries again, which costs less than their tiles in memory: 168 against 192 us at 4195 tokens),
// two take the state of 16 channels each through the present one, two compute those channels' output beside them.  Four
// state waves ask more of the LDS than it gives, 174 against 150 us at 4195 tokens; one, with
// twice the workgroups, saves 2 % of the whole and is slower where these fill the chip.
template <int KT, bool VEC>
__global__ __launch_bounds__(64 * kWalkWaves, kWalkWaves / 4) void gdr_walk_kernel(GdrParams p, const HeadTiles *heads,
                                                                                   int32_t groups, bool svec) {
    __shared__ Tiles<KT> buf[2];
    __shared__ Exchange<KT> exchange[kWalkers];
    __shared__ int ready[kWalkers];
    const Place pl = place_of(p, groups);
    if (!pl.ok) return;
    Span32 sp;
    int64_t line;
    if (!sequence(p, pl.b, sp, line)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int32_t nc = int32_t((int64_t(sp.n) + kC - 1) / kC);
    const int64_t slot = first_slot(p, pl.b);
    if (threadIdx.x < kWalkers) ready[threadIdx.x] = 0;

    if (wave >= 2 * kWalkers) {
        constexpr int kN = 64 * kLoaders, kHead = sizeof(HeadTiles) / 16, kPer = (kHead + kN - 1) / kN;
        const int lw = wave - 2 * kWalkers, t = lw * 64 + lane, kc = t % (4 * KT), hk = pl.h / p.group;
        // 16 quads of rows: with 128 channels every wave has four of keys and of queries, else two waves the keys
        const bool keys = KT == 4 || lw < 2, queries = KT == 4 || lw >= 2;
        const int quad = t / (4 * KT) & 15;
        const Rows kr = rows_of(p.k, p.ks, sp.t0, hk), qr = rows_of(p.q, p.qs, sp.t0, hk);
        u32x4 rh[kPer];
        Quad k, q;
        const auto load = [&](int32_t c) {
            const u32x4 *h = reinterpret_cast<const u32x4 *>(heads + (slot + c) * p.Hv + pl.h);
#pragma unroll
            for (int i = 0; i < kPer; ++i) rh[i] = h[t + i * kN < kHead ? t + i * kN : 0];
            if (keys) k = load_quad<VEC>(kr, sp, c * kC, quad, kc, p.Dk);
            if (queries) q = load_quad<VEC>(qr, sp, c * kC, quad, kc, p.Dk);
        };
        const auto put = [&](Tiles<KT> &b) {
            u32x4 *h = reinterpret_cast<u32x4 *>(static_cast<HeadTiles *>(&b));
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (t + i * kN < kHead) h[t + i * kN] = rh[i];
            if (keys) stage_quad<KT>(k, b.k, b.kt, nullptr, quad, kc, 1.0f, false);
            if (queries) stage_quad<KT>(q, b.q, nullptr, nullptr, quad, kc, 1.0f, false);
        };
        load(0);
        put(buf[0]);
        load(nc > 1 ? 1 : 0);
        __syncthreads();
        for (int32_t c = 0; c < nc; ++c) {
            put(buf[(c + 1) & 1]);
            load(c + 2 < nc ? c + 2 : nc - 1);
            __syncthreads();
        }
        return;
    }

    const int unit = wave & (kWalkers - 1);
    const int32_t tile = pl.cg * kWalkers + unit;
    auto st = consumer<KT, VEC>(p, sp, lane, pl.h, tile);
    const bool work = tile * 16 < p.Dv;
    if (wave >= kWalkers) {
        __syncthreads();
        for (int32_t c = 0; c < nc; ++c) {
            if (work) st.emit(c * kC, buf[c & 1], &exchange[unit], &ready[unit], 2 * c);
            __syncthreads();
        }
        return;
    }
    float *rows = p.state ? p.state + line * p.s_sl + pl.h * p.s_sh : nullptr;
    if (p.state && p.has_init && p.has_init[pl.b] != 0) st.load(rows, svec);
    else st.zero();
    u32x4 v[4];
    st.fetch(0, v);
    __syncthreads();
    for (int32_t c = 0; c < nc; ++c) {
        if (work) st.advance(c * kC, buf[c & 1], v, &exchange[unit], &ready[unit]);
        __syncthreads();
    }
    if (p.state) st.save(rows, svec);
}

template <int KT>
hipError_t launch_one(const GdrParams &p, bool svec, hipStream_t s) {
    const int32_t groups = (p.Dv + 16 * kWaves - 1) / (16 * kWaves);
    const dim3 grid(uint32_t(gdr_walk_grid(p.batch, p.Hk, p.Hv, groups)));
    gdr_chunk_kernel<KT, true><<<grid, dim3(64 * kWaves), 0, s>>>(p, groups, svec);
    return hipGetLastError();
}

// Value heads that a preparing workgroup takes one after the other: they share the rows' conversion, but a call of few
// workgroups is over sooner when each takes fewer.  As many as leave two workgroups a CU: 32 heads and 7, 19, 35, 68
// and 131 chunks took 9, 13, 19, 33 and 54 us with one (of 8) together, 12, 15, 17, 30 and 44 with two, 17, 20, 19, 30 and
// 42 with four, 27, 29, 29, 39 and 43 with eight.
int32_t heads_together(const GdrParams &p, int64_t slots) {
    int32_t per = p.group;
    if (per > 64) return per;          // (and no launch grows past the host's check)
    while (per > 1 && (p.group % per || slots * (p.Hv / per) < 512)) --per;
    return per;
}

template <int KT, bool VEC>
hipError_t launch_walk(const GdrParams &p, bool svec, void *workspace, hipStream_t s) {
    const int64_t slots = gdr_slots(p.total_T, p.batch);
    HeadTiles *heads = static_cast<HeadTiles *>(workspace);
    const int32_t per = heads_together(p, slots);
    gdr_prepare_kernel<KT, VEC><<<dim3(uint32_t(slots * (p.Hv / per))), dim3(64 * kWaves), 0, s>>>(p, heads, per);
    const int32_t groups = (p.Dv + 16 * kWalkers - 1) / (16 * kWalkers);
    const dim3 grid(uint32_t(gdr_walk_grid(p.batch, p.Hk, p.Hv, groups)));
    gdr_walk_kernel<KT, VEC><<<grid, dim3(64 * kWalkWaves), 0, s>>>(p, heads, groups, svec);
    return hipGetLastError();
}

}  // namespace

int64_t gdr_workspace_bytes(int64_t T, int64_t batch, int32_t Hv) {
    return gdr_slots(T, batch) * Hv * int64_t(sizeof(HeadTiles));
}

hipError_t launch_gdr_chunk(const GdrParams &p, bool vec, bool svec, void *workspace, hipStream_t s) {
    if (workspace) {
        if (p.Dk <= 64) return vec ? launch_walk<2, true>(p, svec, workspace, s) : launch_walk<2, false>(p, svec, workspace, s);
        return vec ? launch_walk<4, true>(p, svec, workspace, s) : launch_walk<4, false>(p, svec, workspace, s);
    }
    return p.Dk <= 64 ? launch_one<2>(p, svec, s) : launch_one<4>(p, svec, s);
}

}  // namespace sconv

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
    float eG[kC];
};

template <int KT>
struct alignas(16) Shared {
    Buf<KT> buf[2];
    float a[10 * 256];                 // A in 16 x 16 blocks of the lower triangle; then the diagonal ones of T
    double G[kC];
    float kf[kC];
    float beta[kC];
    int sync;
};

// Token t of a chunk as a row: tile 2 (t / 32) + (t / 4) % 2, row 4 ((t % 32) / 8) + t % 4.
__device__ __forceinline__ int row_tile(int t) { return 2 * (t >> 5) + ((t >> 2) & 1); }
__device__ __forceinline__ int row_in(int t) { return 4 * ((t >> 3) & 3) + (t & 3); }
// ... and the token of row r of tile mt.
__device__ __forceinline__ int tok_of(int mt, int r) { return 32 * (mt >> 1) + 8 * (r >> 2) + 4 * (mt & 1) + (r & 3); }
// Offset (halves) of row r, column c (0..31) in a tile.
__device__ __forceinline__ int in_tile(int r, int c) { return (r + 16 * (c >> 3)) * 8 + (c & 7); }

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
// Over the four lanes that hold one column (l, l + 16, l + 32, l + 48).
__device__ __forceinline__ float max_groups(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
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
__device__ __forceinline__ f32x4 mfma4(float a, float b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x8 tile_of(const _Float16 *base, int tile, int lane) {
    return *reinterpret_cast<const f16x8 *>(base + tile * kTile + lane * 8);
}

// Barrier among the producer waves alone: each adds one, then waits for the
// count that all of them reach.  They are waves of one workgroup, so all are
// resident, and each passes the same barriers.
__device__ __forceinline__ void producer_sync(int *count, int &target) {
    target += kProducers;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    if ((threadIdx.x & 63) == 0) __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    while (__hip_atomic_load(count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) < target)
        __builtin_amdgcn_s_sleep(1);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

struct Span64 { int64_t t0; int64_t n; };              // a sequence's first row and length

// ------------------------------------------------------------- producers --

// Eight channels of a row, zero past its end or the head's.
template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t *row, int64_t sd, int c, int32_t Dk, bool live) {
    u32x4 r = {0u, 0u, 0u, 0u};
    if constexpr (VEC) {
        if (live && c < Dk) r = ld16(row + c);
    } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = live && c + i < Dk ? row[(c + i) * sd] : 0u;
        r.x = e[0] | e[1] << 16; r.y = e[2] | e[3] << 16;
        r.z = e[4] | e[5] << 16; r.w = e[6] | e[7] << 16;
    }
    return r;
}

// Four token rows of eight channels each, as a producer thread holds them.
struct Quad { u32x4 r[4]; };

template <bool VEC>
__device__ __forceinline__ Quad load_quad(const uint16_t *head, const GdrTensor &ts, const Span64 &sp, int64_t c0,
                                          int quad, int kc, int32_t Dk) {
    Quad q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = c0 + 4 * quad + i;
        const bool live = t < sp.n;
        q.r[i] = load8<VEC>(head + (sp.t0 + (live ? t : 0)) * ts.st, ts.sd, 8 * kc, Dk, live);
    }
    return q;
}

// Scales a row by a power of two (largest element in [1, 2)), writes it as a
// row of the operand tiles (and, for keys, transposed), and its factor: the
// power, times the norm's inverse and `scale`.
template <int KT, bool KEYS>
__device__ __forceinline__ void stage_quad(const Quad &in, _Float16 *rows, _Float16 *cols, float *factor, int quad,
                                           int kc, float scale, bool l2norm) {
    f16x8 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[8];
        unpack8(in.r[i], f);
        float m = 0.0f, ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) { m = fmaxf(m, fabsf(f[j])); ss = fmaf(f[j], f[j], ss); }
        m = max_lanes<4 * KT>(m);
        ss = sum_lanes<4 * KT>(ss);
        const int e = exp_of(m);
        const float s = pow2(1 - e);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= s;
        h[i] = half8(f);
        const int t = 4 * quad + i;
        if (kc == 0) factor[t] = scale * (l2norm ? 1.0f / sqrtf(ss + kL2Eps) : 1.0f) * pow2(e - 1);
        // (row, columns 8 kc ..) of tile (row tile, kc / 4)
        *reinterpret_cast<f16x8 *>(rows + (row_tile(t) * KT + (kc >> 2)) * kTile + (row_in(t) + 16 * (kc & 3)) * 8) = h[i];
    }
    if constexpr (KEYS) {
        // channel 8 kc + j: result tile 2 (kc / 4) + j / 4, row 4 (kc % 4) + j % 4; tokens 4 quad ..
        const int c = (4 * quad) & 31;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f16x4 v = {h[0][j], h[1][j], h[2][j], h[3][j]};
            const int d = 2 * (kc >> 2) + (j >> 2), r = 4 * (kc & 3) + (j & 3);
            *reinterpret_cast<f16x4 *>(cols + (d * 2 + (quad >> 3)) * kTile + in_tile(r, c)) = v;
        }
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

    __device__ __forceinline__ void chunk(int64_t c0, Buf<KT> &b, bool more) {
        // gates: one token a lane, the running sum in fp64 (a difference of two of its values keeps every bit of
        // a small decay behind a large one); every e^ below is of a difference <= 0
        if (w == 3) {
            const int64_t t = c0 + lane;
            Gates gt = {0.0f, 0.0f};
            if (t < sp.n)
                gt = gdr_gates(p, (sp.t0 + t) * p.gs.st + h * p.gs.sh, (sp.t0 + t) * p.bs.st + h * p.bs.sh, h);
            double G = gt.g < -1e4f ? -1e4 : double(gt.g);         // e^-10000 is 0 like that of anything below
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double o = __shfl_up(G, m);
                if (lane >= m) G += o;
            }
            const double last = __shfl(G, 63);
            sh.G[lane] = G;
            sh.beta[lane] = gt.beta;
            b.eG[lane] = __builtin_amdgcn_exp2f(float(G * 1.4426950408889634));
            b.eg[lane] = __builtin_amdgcn_exp2f(float((last - G) * 1.4426950408889634));
        }
        if (KT == 4 || w < 2) stage_quad<KT, true>(nk, b.k, b.kt, sh.kf, quad(), kc(), 1.0f, p.l2norm);
        if (KT == 4 || w >= 2) stage_quad<KT, false>(nq, b.q, nullptr, b.qf, quad(), kc(), p.scale, p.l2norm);
        if (more) fetch(c0 + kC);
        producer_sync(&sh.sync, target);

        if (w == 0) {
            const float kf = sh.kf[lane];
            b.ak[lane] = b.eG[lane] * kf;
            b.kb[lane] = kf * sh.beta[lane];
        }
        products(b);
        producer_sync(&sh.sync, target);
        invert_diagonal();
        producer_sync(&sh.sync, target);
        invert_rest(b);
    }

    // K K^T and Q K^T: 12 tile pairs meet the lower triangle, three a wave.
    __device__ __forceinline__ void products(Buf<KT> &b) {
        const int n = lane & 15, g = lane >> 4;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const int pr = 3 * w + x;
            const int mt = pr < 4 ? pr >> 1 : 2 + ((pr - 4) >> 2), nt = pr < 4 ? pr & 1 : (pr - 4) & 3;
            f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const f16x8 right = tile_of(b.k, nt * KT + kt, lane);
                kk = mfma(tile_of(b.k, mt * KT + kt, lane), right, kk);
                qk = mfma(tile_of(b.q, mt * KT + kt, lane), right, qk);
            }
            const int tj = tok_of(nt, n), ti0 = tok_of(mt, 4 * g);
            const double Gj = sh.G[tj];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ti = ti0 + i;
                const float d = ti >= tj ? __builtin_amdgcn_exp2f(float((sh.G[ti] - Gj) * 1.4426950408889634)) : 0.0f;
                const float kf = sh.kf[ti];
                if (ti > tj) {
                    const int bi = ti >> 4, bj = tj >> 4;
                    sh.a[(bi * (bi + 1) / 2 + bj) * 256 + (ti & 15) * 16 + (tj & 15)] = sh.beta[ti] * kf * kf * d * kk[i];
                }
                b.p[tri_tile(mt, nt >> 1) * kTile + in_tile(4 * g + i, tj & 31)] =
                    _Float16(ti >= tj ? d * qk[i] : 0.0f);
            }
        }
    }

    // Wave w inverts diagonal block w by forward substitution, a column a lane.
    __device__ __forceinline__ void invert_diagonal() {
        const int n = lane & 15, g = lane >> 4;
        float *blk = sh.a + (w * (w + 1) / 2 + w) * 256;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == n ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
            for (int j4 = 0; j4 < i; j4 += 4) {
                const f32x4 r = *reinterpret_cast<const f32x4 *>(blk + i * 16 + j4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j4 + e < i) {
                        if (e & 1) s1 = fmaf(-r[e], x[j4 + e], s1);
                        else s0 = fmaf(-r[e], x[j4 + e], s0);
                    }
            }
            x[i] = s0 + s1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = g == 0 ? x[i] : g == 1 ? x[4 + i] : g == 2 ? x[8 + i] : x[12 + i];
            blk[(4 * g + i) * 16 + n] = v;
        }
    }

    // Wave w fills block column w of T downwards: T_iw = -T_ii sum_k A_ik T_kw, in fp32 MFMAs whose right operands are
    // the blocks above as they lie in registers; then it writes the column's two fp16 parts.
    __device__ __forceinline__ void invert_rest(Buf<KT> &b) {
        const int n = lane & 15, g = lane >> 4;
        const int at = n * 16 + 4 * g;                 // left operand: row n, columns 4 g ..
        f32x4 col[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < w) continue;
            if (i == w) {
                const float *d = sh.a + (i * (i + 1) / 2 + i) * 256;
#pragma unroll
                for (int e = 0; e < 4; ++e) col[i][e] = d[(4 * g + e) * 16 + n];
                continue;
            }
            f32x4 m = {0, 0, 0, 0}, t = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k < w || k >= i) continue;
                const f32x4 a = *reinterpret_cast<const f32x4 *>(sh.a + (i * (i + 1) / 2 + k) * 256 + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) m = mfma4(a[e], col[k][e], m);
            }
            const f32x4 d = *reinterpret_cast<const f32x4 *>(sh.a + (i * (i + 1) / 2 + i) * 256 + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) t = mfma4(d[e], m[e], t);
#pragma unroll
            for (int e = 0; e < 4; ++e) col[i][e] = -t[e];
        }
        const int tj = 16 * w + n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < w) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ti = 16 * i + 4 * g + e;
                const int o = tri_tile(row_tile(ti), tj >> 5) * kTile + in_tile(row_in(ti), tj & 31);
                const _Float16 hi = _Float16(col[i][e]);
                b.th[o] = hi;
                b.tl[o] = _Float16(col[i][e] - float(hi));
            }
        }
    }
};

// ----------------------------------------------------------- state waves --

template <int KT, int NT>
struct Consumer {
    const GdrParams &p;
    const Span64 sp;
    const int lane;
    const uint16_t *vh;                // this lane's first channel of v, row 0 of the sequence
    uint16_t *oh;
    int32_t c0;                        // first channel of the wave
    f32x4 S[NT][2 * KT];               // times 2^(14 - es)
    int es[NT];
    float v[NT][16];                   // the chunk's values: [4 mt + i]

    __device__ __forceinline__ bool col_ok(int nt) const { return c0 + 16 * nt + (lane & 15) < p.Dv; }

    __device__ __forceinline__ void fetch(int64_t t0) {
        const int g = lane >> 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t t = t0 + tok_of(mt, 4 * g + i);
                    v[nt][4 * mt + i] =
                        t < sp.n && col_ok(nt) ? bf_one(vh[t * p.vs.st + 16 * nt * p.vs.sd]) : 0.0f;
                }
    }

    __device__ __forceinline__ void chunk(int64_t t0, const Buf<KT> &b, bool more) {
        const int g = lane >> 4;
        float x[NT][16];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 16; ++i) x[nt][i] = v[nt][i];
        if (more) fetch(t0 + kC);

        // the state's columns, rescaled to 2^14 and split
        f16x8 sh[NT][KT], sl[NT][KT];
        float inv[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float m = 0.0f;
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S[nt][d][i]));
            m = max_groups(m);
            int e = exp_of(m) - 14 + es[nt];           // of the true values
            e = e < -100 ? -100 : e;
            int up = es[nt] - e;                       // S * 2^up has its largest near 2^14
            up = up > 120 ? 120 : (up < -120 ? -120 : up);
            const float s = pow2(up);
            es[nt] = es[nt] - up;
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d) S[nt][d] *= s;
            inv[nt] = pow2(es[nt] - 14);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = S[nt][2 * kt + (j >> 2)][j & 3];
                split8(f, sh[nt][kt], sl[nt][kt]);
            }
        }

        // K S and Q S
        f32x4 aq[NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            f32x4 ak[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) { ak[nt] = f32x4{0, 0, 0, 0}; aq[nt][mt] = f32x4{0, 0, 0, 0}; }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const f16x8 kf = tile_of(b.k, mt * KT + kt, lane), qf = tile_of(b.q, mt * KT + kt, lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    ak[nt] = mfma(kf, sh[nt][kt], ak[nt]);
                    aq[nt][mt] = mfma(qf, sh[nt][kt], aq[nt][mt]);
                    ak[nt] = mfma(kf, sl[nt][kt], ak[nt]);
                }
            }
            const int t = tok_of(mt, 4 * g);
            const f32x4 fa = *reinterpret_cast<const f32x4 *>(b.ak + t), kb = *reinterpret_cast<const f32x4 *>(b.kb + t);
            const f32x4 eG = *reinterpret_cast<const f32x4 *>(b.eG + t);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[nt][4 * mt + i] = kb[i] * fmaf(-fa[i] * inv[nt], ak[nt][i], x[nt][4 * mt + i]);
                    aq[nt][mt][i] *= eG[i] * inv[nt];
                }
        }

        // z = T X
        f16x8 yh[NT][2], yl[NT][2], zh[NT][2];
        float zinv[NT];
        const float last = b.eG[kC - 1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[nt][i]));
            const int ex = exp_of(max_groups(m));
            const float s = pow2(14 - ex), back = pow2(ex - 14);
            f16x8 xh[2], xl[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = x[nt][8 * tt + j] * s;
                split8(f, xh[tt], xl[tt]);
            }
            f32x4 z[4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                z[mt] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int tt = 0; tt <= mt / 2; ++tt) {
                    const f16x8 h = tile_of(b.th, tri_tile(mt, tt), lane), l = tile_of(b.tl, tri_tile(mt, tt), lane);
                    z[mt] = mfma(h, xh[tt], z[mt]);
                    z[mt] = mfma(h, xl[tt], z[mt]);
                    z[mt] = mfma(l, xh[tt], z[mt]);
                }
            }
            m = 0.0f;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) { z[mt][i] *= back; m = fmaxf(m, fabsf(z[mt][i])); }
            // z may be small beside the state, but no further down than counts in it (and S must not overflow in
            // z's scale)
            int ez = exp_of(max_groups(m));
            ez = ez < es[nt] - 40 ? es[nt] - 40 : ez;
            const float zs = pow2(14 - ez);
            zinv[nt] = pow2(ez - 14);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                float f[8], y[8];
#pragma unroll
                for (int t2 = 0; t2 < 2; ++t2) {
                    const f32x4 eg = *reinterpret_cast<const f32x4 *>(b.eg + tok_of(2 * tt + t2, 4 * g));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[4 * t2 + i] = z[2 * tt + t2][i] * zs;
                        y[4 * t2 + i] = f[4 * t2 + i] * eg[i];
                    }
                }
                zh[nt][tt] = half8(f);
                split8(y, yh[nt][tt], yl[nt][tt]);
            }
            // S to z's scale, decayed
            int up = es[nt] - ez;
            up = up < -120 ? -120 : up;
            const float sc = last * pow2(up);
#pragma unroll
            for (int d = 0; d < 2 * KT; ++d) S[nt][d] *= sc;
            es[nt] = ez;
        }

        // S += K^T y
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const f16x8 k = tile_of(b.kt, 2 * d + tt, lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    S[nt][d] = mfma(k, yh[nt][tt], S[nt][d]);
                    S[nt][d] = mfma(k, yl[nt][tt], S[nt][d]);
                }
            }

        // o
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 qf = *reinterpret_cast<const f32x4 *>(b.qf + tok_of(mt, 4 * g));
            f32x4 o[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) o[nt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int tt = 0; tt <= mt / 2; ++tt) {
                const f16x8 pf = tile_of(b.p, tri_tile(mt, tt), lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) o[nt] = mfma(pf, zh[nt][tt], o[nt]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t t = t0 + tok_of(mt, 4 * g + i);
                    const float r = qf[i] * fmaf(o[nt][i], zinv[nt], aq[nt][mt][i]);
                    if (t < sp.n && col_ok(nt)) oh[t * p.os.st + 16 * nt * p.os.sd] = to_bf16(r);
                }
        }
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
        pr.chunk(0, sh.buf[0], nc > 1);
        __syncthreads();
        for (int64_t c = 0; c < nc; ++c) {
            if (c + 1 < nc) pr.chunk((c + 1) * kC, sh.buf[(c + 1) & 1], c + 2 < nc);
            __syncthreads();
        }
        return;
    }

    const int g = lane >> 4;
    Consumer<KT, NT> st{p, sp, lane};
    st.c0 = (pl.cg * NS + wave) * NT * 16;
    const int32_t col = st.c0 + (lane & 15);
    st.vh = p.v + sp.t0 * p.vs.st + pl.h * p.vs.sh + int64_t(col) * p.vs.sd;
    st.oh = p.out + sp.t0 * p.os.st + pl.h * p.os.sh + int64_t(col) * p.os.sd;
    const bool init = p.state && p.has_init && p.has_init[pl.b] != 0;
    float *rows = p.state ? p.state + line * p.s_sl + pl.h * p.s_sh : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        st.es[nt] = 14;
        const float *row = rows + (col + 16 * nt) * p.s_sv;
        const bool ok = init && st.col_ok(nt);
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
        float *row = rows + (col + 16 * nt) * p.s_sv;
        const bool ok = st.col_ok(nt);
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
    return launch_cfg<KT, 4, 2, VEC>(p, svec, s);
}

}  // namespace

hipError_t launch_gdr_chunk(const GdrParams &p, bool vec, bool svec, hipStream_t s) {
    if (p.Dk <= 64) return vec ? launch_kt<2, true>(p, svec, s) : launch_kt<2, false>(p, svec, s);
    return vec ? launch_kt<4, true>(p, svec, s) : launch_kt<4, false>(p, svec, s);
}

}  // namespace sconv

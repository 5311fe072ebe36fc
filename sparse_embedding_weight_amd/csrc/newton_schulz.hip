// Orthogonalising an update by Newton-Schulz steps, and the optimiser step
// built on it (include/muon.h).
//
// With X the update scaled to Frobenius norm 1 (its shorter side first), a
// step is
//     A = X X^T,  B = b A + c A A,  X <- a X + B X
// which maps every singular value s of X to a s + b s^3 + c s^5 and leaves the
// singular vectors alone. Three products a step; A and B are symmetric, so
// only the tiles on and below the diagonal are computed and the others
// mirrored.
//
// The state X is held in 32 bits. The products read 16-bit copies of X, A and
// B in half precision, scaled by powers of two that keep their entries well
// inside its range (|X| <= ~1.2, |A| <= ~1.5, |B| <= ~6), and add up in
// 32 bits. Half precision rather than bfloat16 because its three more bits
// matter here: the steps amplify what rounding puts into the small singular
// directions (by up to 3.4 a step), and the result differs from the 64-bit
// one by 0.03-0.1 % of its norm instead of 1-5 %. Two choices keep rounding
// out of what the steps amplify most:
//   - a X is taken from the 32-bit state: from the half copy, the error of an
//     update with a few strong directions is 0.6 % instead of 0.04 %;
//   - the diagonals of A and B, their largest entries, are held apart in 32
//     bits (A = D + O: A A = O O + D O + O D + D D, where only O O is a matrix
//     product, and B X = E X + (B - E) X with E X from the state): 0.04-0.07 %
//     instead of 0.12-0.19 % for updates without strong directions.
#include "newton_schulz.h"

#include <hip/hip_fp16.h>

#include "ewg_device.h"
#include "muon.h"

namespace ewg {

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));

// Powers of two of the half copies of A and B.
constexpr float kGramScale = 256.0f;

// ---- 1. momentum and the sum of squares ---------------------------------------

// What the update is made of. Plain: u = update. Momentum: m' = beta m + g is
// written, and u = g + beta m' (Nesterov) or m'.
struct NsSource {
    const void *g;             // the update, or main_grad
    int64_t g_batch, g_row;
    const float *m;            // momentum, or null
    float *m_out;
    int64_t m_batch, m_row;
    float beta;
    int nesterov;
};

template <class G>
__device__ __forceinline__ float load_g(const NsSource &s, int b, int r, int c) {
    return G::widen(static_cast<const typename G::T *>(s.g)[b * s.g_batch + r * s.g_row + c]);
}

// the update's value once m_out holds the new momentum
template <class G, bool MOM>
__device__ __forceinline__ float load_u(const NsSource &s, int b, int r, int c) {
    const float g = load_g<G>(s, b, r, c);
    if constexpr (!MOM) return g;
    const float m = s.m_out[b * s.m_batch + r * s.m_row + c];
    return s.nesterov ? __builtin_fmaf(s.beta, m, g) : m;
}

// Sums u^2 in 64 bits (squares of 1e-25 or 1e25 neither vanish nor overflow),
// a fixed share of the rows and a fixed order for every workgroup. One pass
// over main_grad and momentum; bound by HBM.
template <class G, bool MOM>
__global__ __launch_bounds__(256) void ns_norm_kernel(NsSource s, int rows, int cols,
                                                      double *__restrict__ partials) {
    const int b = blockIdx.y, parts = gridDim.x;
    double sum = 0.0;
    const int64_t total = (int64_t)rows * cols;
    const int64_t share = ((total + parts - 1) / parts + 255) / 256 * 256;
    const int64_t first = (int64_t)blockIdx.x * share;
    const int64_t last = first + share < total ? first + share : total;
    for (int64_t i = first + threadIdx.x; i < last; i += 256) {
        const int r = (int)(i / cols), c = (int)(i - (int64_t)r * cols);
        float u;
        if constexpr (MOM) {
            const float g = load_g<G>(s, b, r, c);
            const int64_t at = b * s.m_batch + r * s.m_row + c;
            const float m = __builtin_fmaf(s.beta, s.m[at], g);
            s.m_out[at] = m;
            u = s.nesterov ? __builtin_fmaf(s.beta, m, g) : m;
        } else {
            u = load_g<G>(s, b, r, c);
        }
        sum += (double)u * (double)u;
    }
    __shared__ double part[256];
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int n = 128; n > 0; n >>= 1) {
        if ((int)threadIdx.x < n) part[threadIdx.x] += part[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) partials[(int64_t)b * kNsMaxPartials + blockIdx.x] = part[0];
}

// ---- 2. X = u / (|u| + eps) in its three layouts ----------------------------

template <class G, bool MOM>
__global__ __launch_bounds__(256) void ns_layout_kernel(NsSource s, NsShape sh, int parts, float eps,
                                                        float x_scale,
                                                        const double *__restrict__ partials,
                                                        float *__restrict__ x,
                                                        _Float16 *__restrict__ xh,
                                                        _Float16 *__restrict__ xt) {
    __shared__ float t[64][65];
    __shared__ double part[256];
    const int b = blockIdx.z, tid = threadIdx.x;
    part[tid] = tid < parts ? partials[(int64_t)b * kNsMaxPartials + tid] : 0.0;
    __syncthreads();
    for (int n = 128; n > 0; n >>= 1) {
        if (tid < n) part[tid] += part[tid + n];
        __syncthreads();
    }
    // Division by the norm in 64 bits: 1 / norm need not fit 32 bits for tiny updates.
    const double inverse = 1.0 / (sqrt(part[0]) + (double)eps);
    const int i0 = blockIdx.x * 64, j0 = blockIdx.y * 64;   // X tile: rows i0.., columns j0..
    const int lane = tid & 63, w = tid >> 6;
    for (int q = w; q < 64; q += 4) {
        // one source row of the tile: X row i0+q, or X column j0+q of a tall update
        const int r = (sh.tall ? j0 : i0) + q, c = (sh.tall ? i0 : j0) + lane;
        float v = 0.0f;
        if (r < sh.rows && c < sh.cols) v = (float)((double)load_u<G, MOM>(s, b, r, c) * inverse);
        if (sh.tall)
            t[lane][q] = v;
        else
            t[q][lane] = v;
    }
    __syncthreads();
    const int64_t base = (int64_t)b * sh.kp * sh.lp;
    for (int q = w; q < 64; q += 4) {
        const int64_t at = base + (int64_t)(i0 + q) * sh.lp + j0 + lane;
        const float v = t[q][lane];
        x[at] = v;
        xh[at] = (_Float16)(v * x_scale);
        xt[base + (int64_t)(j0 + q) * sh.kp + i0 + lane] = (_Float16)(t[lane][q] * x_scale);
    }
}

// ---- 3. the products ----------------------------------------------------------

// Where the last product's X goes: the caller's output, or the weight.
struct NsSink {
    void *out;                 // bf16 update, or the new weight
    int64_t out_batch, out_row;
    const void *weight;        // old weight (same layout as out), or null
    float keep, take;          // weight * keep - take * X
};

struct NsProduct {
    const _Float16 *p, *q;     // C = P Q^T, both [rows][depth]
    int64_t p_batch, q_batch;
    int depth;                 // padded, a multiple of 64
    int tiles_p, tiles_q;
    // epilogue
    float factor;              // on the 32-bit sums
    const _Float16 *gram;      // for B: A without its diagonal
    float *diag_a, *diag_b;    // [batch][kp]: kGramScale times A's diagonal, B's diagonal
    float b_coef, c_coef;
    float a_coef, x_scale;     // for X
    _Float16 *out;             // A, B or the half copy of X
    _Float16 *out_t;           // its transpose (X)
    float *x;
    NsShape sh;
};

enum NsEpilogue { kGram, kPoly, kState, kLast };

// XOR swizzle of the 16-byte pieces of a 128-byte tile row: 32 lanes reading
// one piece column of 32 rows then touch every bank group equally.
__device__ __forceinline__ int swizzled(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

template <class S, bool WEIGHT>
__device__ __forceinline__ void sink_one(const NsSink &k, int64_t at, float v) {
    typename S::T *out = static_cast<typename S::T *>(k.out);
    if constexpr (WEIGHT) {
        const float w = S::widen(static_cast<const typename S::T *>(k.weight)[at]);
        v = __builtin_fmaf(-k.take, v, w * k.keep);
    }
    out[at] = S::narrow(v);
}

// One tile of C = P Q^T. Tiles of 64 halves of depth go through LDS twice
// buffered, written by direct-to-LDS loads; each of the WP x WQ waves keeps
// (TP/WP) x (TQ/WQ) of C in registers as 32x32 blocks. The matrix
// instruction takes Q as its first operand: a lane then holds four
// consecutive columns of one row of C.
template <int TP, int TQ, int WP, int WQ, int EPI, class S, bool WEIGHT>
__global__ __launch_bounds__(WP *WQ * 64) void ns_product_kernel(NsProduct a, NsSink sink) {
    constexpr int WAVES = WP * WQ;
    constexpr int FP = TP / WP / 32, FQ = TQ / WQ / 32;
    constexpr int PIECES = (TP + TQ) / 8;            // 1 KiB wave loads a tile
    static_assert(PIECES % WAVES == 0 && TP % 8 == 0, "whole loads");
    constexpr int LOADS = PIECES / WAVES;
    constexpr int BYTES = (TP + TQ) * 128;
    constexpr bool SYM = EPI == kGram || EPI == kPoly;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * BYTES];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int batch = blockIdx.y;
    int ti, tj;
    if constexpr (SYM) {
        // blocks count the tiles of the lower triangle row by row
        const int n = blockIdx.x;
        ti = (int)((sqrtf(8.0f * (float)n + 1.0f) - 1.0f) * 0.5f);
        while ((ti + 1) * (ti + 2) / 2 <= n) ++ti;
        while (ti * (ti + 1) / 2 > n) --ti;
        tj = n - ti * (ti + 1) / 2;
    } else {
        ti = blockIdx.x % a.tiles_p;
        tj = blockIdx.x / a.tiles_p;
    }
    const _Float16 *p = a.p + batch * a.p_batch + (int64_t)ti * TP * a.depth;
    const _Float16 *q = a.q + batch * a.q_batch + (int64_t)tj * TQ * a.depth;

    // lane l of a load brings row l/8 of eight, piece (l%8) ^ (l/8) of it
    const int row8 = lane >> 3, piece = (lane & 7) ^ row8;
    const _Float16 *from[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = (i * WAVES + wave) * 8;
        from[i] = (row < TP ? p + (int64_t)(row + row8) * a.depth : q + (int64_t)(row - TP + row8) * a.depth) + piece * 8;
    }
    auto stage = [&](int buffer, int kt) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)(from[i] + kt * 64),
                (__attribute__((address_space(3))) void *)(lds + buffer * BYTES + (i * WAVES + wave) * 1024), 16, 0, 0);
    };

    const int wp = wave % WP, wq = wave / WP;
    const int r32 = lane & 31, h = lane >> 5;
    float16v acc[FP][FQ] = {};
    const int steps = a.depth / 64;
    stage(0, 0);
    for (int kt = 0; kt < steps; ++kt) {
        // this tile has arrived for every wave, and every wave has read the one before
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __syncthreads();
        const uint8_t *tile = lds + (kt & 1) * BYTES;
        half8 pf[4][FP], qf[4][FQ];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int i = 0; i < FP; ++i)
                pf[s][i] = *reinterpret_cast<const half8 *>(tile + swizzled(wp * FP * 32 + i * 32 + r32, s * 2 + h));
#pragma unroll
            for (int j = 0; j < FQ; ++j)
                qf[s][j] = *reinterpret_cast<const half8 *>(tile + TP * 128 + swizzled(wq * FQ * 32 + j * 32 + r32, s * 2 + h));
        }
        if (kt + 1 < steps) stage((kt + 1) & 1, kt + 1);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(qf[s][j], pf[s][i], acc[i][j], 0, 0, 0);
    }

    const int kp = a.sh.kp, lp = a.sh.lp;
    float *diag_a = a.diag_a + (int64_t)batch * kp, *diag_b = a.diag_b + (int64_t)batch * kp;
#pragma unroll
    for (int i = 0; i < FP; ++i) {
        const int row = ti * TP + (wp * FP + i) * 32 + r32;
        // a + e for X's row; A's diagonal for B's
        float of_row = 0.0f;
        if constexpr (EPI == kPoly) of_row = diag_a[row];
        if constexpr (EPI == kState || EPI == kLast) of_row = a.a_coef + diag_b[row];
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int col = tj * TQ + (wq * FQ + j) * 32 + g * 8 + h * 4;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][g * 4 + e] * a.factor;
                if constexpr (SYM) {
                    _Float16 *out = a.out + (int64_t)batch * kp * kp;
                    if constexpr (EPI == kPoly) {
                        const half4 gram = *reinterpret_cast<const half4 *>(a.gram + (int64_t)batch * kp * kp + (int64_t)row * kp + col);
                        const float4 of_col = *reinterpret_cast<const float4 *>(diag_a + col);
                        const float dc[4] = {of_col.x, of_col.y, of_col.z, of_col.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (row == col + e)
                                diag_b[row] = (v[e] + of_row * __builtin_fmaf(of_row, a.c_coef / kGramScale, a.b_coef)) / kGramScale;
                            v[e] = __builtin_fmaf(__builtin_fmaf(of_row + dc[e], a.c_coef / kGramScale, a.b_coef), (float)gram[e], v[e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (row == col + e) diag_a[row] = v[e];
                    }
                    half4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = row == col + e ? (_Float16)0.0f : (_Float16)v[e];
                    *reinterpret_cast<half4 *>(out + (int64_t)row * kp + col) = o;
                    if (ti != tj) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) out[(int64_t)(col + e) * kp + row] = o[e];
                    }
                } else {
                    const int64_t base = (int64_t)batch * kp * lp;
                    const int64_t at = base + (int64_t)row * lp + col;
                    const float4 old = *reinterpret_cast<const float4 *>(a.x + at);
                    v[0] = __builtin_fmaf(of_row, old.x, v[0]);
                    v[1] = __builtin_fmaf(of_row, old.y, v[1]);
                    v[2] = __builtin_fmaf(of_row, old.z, v[2]);
                    v[3] = __builtin_fmaf(of_row, old.w, v[3]);
                    if constexpr (EPI == kState) {
                        *reinterpret_cast<float4 *>(a.x + at) = make_float4(v[0], v[1], v[2], v[3]);
                        half4 o;
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = (_Float16)(v[e] * a.x_scale);
                        *reinterpret_cast<half4 *>(a.out + at) = o;
#pragma unroll
                        for (int e = 0; e < 4; ++e) a.out_t[base + (int64_t)(col + e) * kp + row] = o[e];
                    } else {
                        const int64_t to = batch * sink.out_batch;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = col + e;
                            if (row < a.sh.k && c < a.sh.len)
                                sink_one<S, WEIGHT>(sink, to + (a.sh.tall ? (int64_t)c * sink.out_row + row : (int64_t)row * sink.out_row + c), v[e]);
                        }
                    }
                }
            }
        }
    }
}

int round_to(int64_t v, int t) { return (int)((v + t - 1) / t * t); }

template <int TP, int TQ, int WP, int WQ, int EPI, class S = BF16, bool WEIGHT = false>
hipError_t launch_product(const NsProduct &a, const NsSink &sink, hipStream_t stream) {
    const int64_t tiles = EPI == kGram || EPI == kPoly ? (int64_t)a.tiles_p * (a.tiles_p + 1) / 2 : (int64_t)a.tiles_p * a.tiles_q;
    ns_product_kernel<TP, TQ, WP, WQ, EPI, S, WEIGHT><<<dim3((unsigned)tiles, a.sh.batch), WP * WQ * 64, 0, stream>>>(a, sink);
    return hipGetLastError();
}

template <int EPI>
hipError_t launch_tiled(const NsProduct &a, const NsSink &sink, hipStream_t stream) {
    return a.sh.tile == 256 ? launch_product<256, 256, 2, 4, EPI>(a, sink, stream)
                            : launch_product<128, 128, 2, 2, EPI>(a, sink, stream);
}

template <class S, bool WEIGHT>
hipError_t launch_last(const NsProduct &a, const NsSink &sink, hipStream_t stream) {
    return a.sh.tile == 256 ? launch_product<256, 256, 2, 4, kLast, S, WEIGHT>(a, sink, stream)
                            : launch_product<128, 128, 2, 2, kLast, S, WEIGHT>(a, sink, stream);
}

template <class G, bool MOM>
hipError_t launch_prepare(const NsSource &src, const NsShape &sh, const NsLayout &l, uint8_t *ws, float eps,
                          float x_scale, hipStream_t stream) {
    const int64_t total = (int64_t)sh.rows * sh.cols;
    int parts = (int)((total + 4095) / 4096);
    if (parts > kNsMaxPartials) parts = kNsMaxPartials;
    double *partials = reinterpret_cast<double *>(ws + l.partials);
    ns_norm_kernel<G, MOM><<<dim3(parts, sh.batch), 256, 0, stream>>>(src, sh.rows, sh.cols, partials);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ns_layout_kernel<G, MOM><<<dim3(sh.kp / 64, sh.lp / 64, sh.batch), 256, 0, stream>>>(
        src, sh, parts, eps, x_scale, partials, reinterpret_cast<float *>(ws + l.x),
        reinterpret_cast<_Float16 *>(ws + l.xh), reinterpret_cast<_Float16 *>(ws + l.xt0));
    return hipGetLastError();
}

hipError_t run(const NsSource &src, bool g_bf16, const NsSink &sink, bool out_bf16, const NsShape &sh, int steps,
               const float *coef, float eps, uint8_t *ws, hipStream_t stream) {
    const NsLayout l = ns_layout(sh);
    // power of two near sqrt(len): a typical entry of X is then about 1
    float x_scale = 1.0f;
    while (4.0f * x_scale * x_scale <= (float)sh.len) x_scale *= 2.0f;
    const bool mom = src.m != nullptr;
    hipError_t e = g_bf16 ? (mom ? launch_prepare<BF16, true>(src, sh, l, ws, eps, x_scale, stream)
                                 : launch_prepare<BF16, false>(src, sh, l, ws, eps, x_scale, stream))
                          : (mom ? launch_prepare<F32, true>(src, sh, l, ws, eps, x_scale, stream)
                                 : launch_prepare<F32, false>(src, sh, l, ws, eps, x_scale, stream));
    if (e != hipSuccess) return e;
    _Float16 *xh = reinterpret_cast<_Float16 *>(ws + l.xh);
    _Float16 *xt[2] = {reinterpret_cast<_Float16 *>(ws + l.xt0), reinterpret_cast<_Float16 *>(ws + l.xt1)};
    _Float16 *am = reinterpret_cast<_Float16 *>(ws + l.a), *bm = reinterpret_cast<_Float16 *>(ws + l.b);
    const int64_t kl = (int64_t)sh.kp * sh.lp, kk = (int64_t)sh.kp * sh.kp;
    for (int s = 0; s < steps; ++s) {
        NsProduct a = {};
        a.sh = sh;
        a.tiles_p = sh.kp / sh.tile;
        a.tiles_q = a.tiles_p;
        a.p = a.q = xh;
        a.p_batch = a.q_batch = kl;
        a.depth = sh.lp;
        a.diag_a = reinterpret_cast<float *>(ws + l.diag_a);
        a.diag_b = reinterpret_cast<float *>(ws + l.diag_b);
        a.factor = kGramScale / (x_scale * x_scale);
        a.out = am;
        if ((e = launch_tiled<kGram>(a, sink, stream)) != hipSuccess) return e;
        a.p = a.q = am;
        a.p_batch = a.q_batch = kk;
        a.depth = sh.kp;
        a.factor = coef[2] / kGramScale;
        a.gram = am;
        a.b_coef = coef[1];
        a.c_coef = coef[2];
        a.out = bm;
        if ((e = launch_tiled<kPoly>(a, sink, stream)) != hipSuccess) return e;
        a.p = bm;
        a.q = xt[s & 1];
        a.p_batch = kk;
        a.q_batch = kl;
        a.tiles_q = sh.lp / sh.tile;
        a.factor = 1.0f / (kGramScale * x_scale);
        a.a_coef = coef[0];
        a.x_scale = x_scale;
        a.x = reinterpret_cast<float *>(ws + l.x);
        a.out = xh;
        a.out_t = xt[(s + 1) & 1];
        if (s + 1 < steps)
            e = launch_tiled<kState>(a, sink, stream);
        else if (!sink.weight)
            e = launch_last<BF16, false>(a, sink, stream);
        else
            e = out_bf16 ? launch_last<BF16, true>(a, sink, stream) : launch_last<F32, true>(a, sink, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

bool sizes_ok(int64_t batch, int64_t rows, int64_t cols) {
    return batch >= 0 && rows >= 0 && cols >= 0 && batch <= kNsMaxBatch && rows <= kNsMaxSide && cols <= kNsMaxSide;
}

bool is_float(int d) { return d == EWG_BF16 || d == EWG_FP32; }
bool is_known(int d) { return d >= EWG_INT32 && d <= EWG_FP32; }

// rows of one matrix do not overlap, nor do matrices of one batch
bool strides_ok(int64_t batch, int64_t rows, int64_t cols, int64_t batch_stride, int64_t row_stride) {
    return row_stride >= cols && (batch <= 1 || batch_stride >= (rows - 1) * row_stride + cols);
}

int check_ns(int64_t batch, int64_t rows, int64_t cols, int steps, float a, float b, float c, float eps,
             const void *workspace, size_t workspace_bytes) {
    if (!sizes_ok(batch, rows, cols) || steps < 1 || steps > EWG_MUON_MAX_STEPS) return EWG_UNSUPPORTED;
    if (!(eps >= 0.0f) || !(a - a == 0.0f) || !(b - b == 0.0f) || !(c - c == 0.0f) || !(eps - eps == 0.0f))
        return EWG_INVALID_ARGUMENT;
    if (batch == 0 || rows == 0 || cols == 0) return EWG_OK;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return EWG_INVALID_ARGUMENT;
    if (workspace_bytes < ns_layout(ns_shape(batch, rows, cols)).total) return EWG_WORKSPACE_TOO_SMALL;
    return EWG_OK;
}

}  // namespace

NsShape ns_shape(int64_t batch, int64_t rows, int64_t cols) {
    NsShape s;
    s.batch = (int)batch;
    s.rows = (int)rows;
    s.cols = (int)cols;
    s.tall = rows > cols;
    s.k = (int)(rows < cols ? rows : cols);
    s.len = (int)(rows < cols ? cols : rows);
    s.tile = s.k >= 2048 ? 256 : 128;
    s.kp = round_to(s.k, s.tile);
    s.lp = round_to(s.len, s.tile);
    return s;
}

NsLayout ns_layout(const NsShape &s) {
    NsLayout l;
    const size_t kl = (size_t)s.batch * s.kp * s.lp, kk = (size_t)s.batch * s.kp * s.kp;
    l.partials = 0;
    l.x = round_up(l.partials + sizeof(double) * kNsMaxPartials * s.batch, 256);
    l.xh = round_up(l.x + 4 * kl, 256);
    l.xt0 = round_up(l.xh + 2 * kl, 256);
    l.xt1 = round_up(l.xt0 + 2 * kl, 256);
    l.a = round_up(l.xt1 + 2 * kl, 256);
    l.b = round_up(l.a + 2 * kk, 256);
    l.diag_a = round_up(l.b + 2 * kk, 256);
    l.diag_b = round_up(l.diag_a + 4 * (size_t)s.batch * s.kp, 256);
    l.total = round_up(l.diag_b + 4 * (size_t)s.batch * s.kp, 256);
    return l;
}

}  // namespace ewg

extern "C" {

size_t orthogonalize_update_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    using namespace ewg;
    if (!sizes_ok(batch, rows, cols) || batch == 0 || rows == 0 || cols == 0) return 0;
    return ns_layout(ns_shape(batch, rows, cols)).total;
}

int orthogonalize_update(const void *update, void *out, int64_t batch, int64_t rows, int64_t cols,
                         int64_t update_batch_stride, int64_t update_row_stride,
                         int64_t out_batch_stride, int64_t out_row_stride, int update_dtype,
                         int steps, float a, float b, float c, float eps, void *workspace,
                         size_t workspace_bytes, hipStream_t stream) {
    using namespace ewg;
    if (!is_known(update_dtype)) return EWG_INVALID_ARGUMENT;
    if (!is_float(update_dtype)) return EWG_UNSUPPORTED;
    int st = check_ns(batch, rows, cols, steps, a, b, c, eps, workspace, workspace_bytes);
    if (st != EWG_OK || batch == 0 || rows == 0 || cols == 0) return st;
    if (!update || !out) return EWG_INVALID_ARGUMENT;
    if (!strides_ok(batch, rows, cols, update_batch_stride, update_row_stride) ||
        !strides_ok(batch, rows, cols, out_batch_stride, out_row_stride))
        return EWG_INVALID_ARGUMENT;
    NsSource src = {};
    src.g = update;
    src.g_batch = update_batch_stride;
    src.g_row = update_row_stride;
    NsSink sink = {};
    sink.out = out;
    sink.out_batch = out_batch_stride;
    sink.out_row = out_row_stride;
    const float coef[3] = {a, b, c};
    (void)hipGetLastError();
    return run(src, update_dtype == EWG_BF16, sink, true, ns_shape(batch, rows, cols), steps, coef, eps,
               static_cast<uint8_t *>(workspace), stream) == hipSuccess ? EWG_OK : EWG_HIP_ERROR;
}

int muon_step(const void *weight, void *out_weight, const void *main_grad, const float *momentum,
              float *out_momentum, int64_t batch, int64_t rows, int64_t cols,
              int64_t weight_batch_stride, int64_t weight_row_stride,
              int64_t main_grad_batch_stride, int64_t main_grad_row_stride,
              int64_t momentum_batch_stride, int64_t momentum_row_stride, int weight_dtype,
              int main_grad_dtype, float lr, float beta, int nesterov, float weight_decay, float scale,
              int steps, float a, float b, float c, float eps, void *workspace,
              size_t workspace_bytes, hipStream_t stream) {
    using namespace ewg;
    if (!is_known(weight_dtype) || !is_known(main_grad_dtype)) return EWG_INVALID_ARGUMENT;
    if (!is_float(weight_dtype) || !is_float(main_grad_dtype)) return EWG_UNSUPPORTED;
    if (nesterov != 0 && nesterov != 1) return EWG_INVALID_ARGUMENT;
    int st = check_ns(batch, rows, cols, steps, a, b, c, eps, workspace, workspace_bytes);
    if (st != EWG_OK || batch == 0 || rows == 0 || cols == 0) return st;
    if (!weight || !out_weight || !main_grad || !momentum || !out_momentum) return EWG_INVALID_ARGUMENT;
    if (!strides_ok(batch, rows, cols, weight_batch_stride, weight_row_stride) ||
        !strides_ok(batch, rows, cols, main_grad_batch_stride, main_grad_row_stride) ||
        !strides_ok(batch, rows, cols, momentum_batch_stride, momentum_row_stride))
        return EWG_INVALID_ARGUMENT;
    NsSource src = {main_grad, main_grad_batch_stride, main_grad_row_stride, momentum, out_momentum,
                    momentum_batch_stride, momentum_row_stride, beta, nesterov};
    NsSink sink = {out_weight, weight_batch_stride, weight_row_stride, weight, 1.0f - lr * weight_decay, lr * scale};
    const float coef[3] = {a, b, c};
    (void)hipGetLastError();
    return run(src, main_grad_dtype == EWG_BF16, sink, weight_dtype == EWG_BF16, ns_shape(batch, rows, cols), steps,
               coef, eps, static_cast<uint8_t *>(workspace), stream) == hipSuccess ? EWG_OK : EWG_HIP_ERROR;
}

}  // extern "C"

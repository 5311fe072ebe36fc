// Log probabilities of given tokens with entropy and top alternatives, and
// their gradient (include/token_logprobs.h).
//
// Forward, one pass over the logits. With y = x / T, a lane keeps the largest
// logit m it has seen, s = sum 2^d and w = sum 2^d d over d = (x - m) log2(e) / T,
// and rescales both when m grows; lanes, waves and workgroups join the same
// way. Then
//     logsumexp = m / T + ln s,   entropy = ln s - ln2 w / s,
//     logprob   = (x_t - m) / T - ln s.
// w holds distances to the maximum, not the logits themselves, so nothing
// cancels in the entropy of a peaked row.
//
// The pass reads rows in groups of 64 16-byte pieces (one wave load). For the
// alternatives it keeps nothing per element: only each group's maximum, in
// LDS. The top_k largest elements lie in the top_k groups with the largest
// maxima (equal ones by the lower index: groups are contiguous, so that is
// the order of their first largest elements too), and by the same argument in
// the top_k largest pieces of those groups; these few are read again.
//
// Backward, one pass that reads the logits and writes the gradient.
#include <hip/hip_runtime.h>

#include <atomic>

#include "ewg_device.h"
#include "ewg_internal.h"
#include "token_logprobs.h"

namespace ewg {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnroll = 4;             // groups a wave has in flight
constexpr int kMaxGroups = 1024;       // group maxima one workgroup keeps
constexpr int kMaxSplits = 64;         // parts of a row: one lane each in the join
constexpr int kMaxTopK = EWG_MAX_TOP_LOGPROBS;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kMasked = -1e38f;      // logits at or below are masked, the types' lowest values among them
constexpr float kNegInf = -__builtin_inff();

// Grids: parts of a row along x, rows along y and z (y holds at most 65535).
constexpr int kRowsY = 32768;
__device__ __forceinline__ int64_t row_of_block() { return (int64_t)blockIdx.z * kRowsY + blockIdx.y; }
dim3 grid_of(int parts, int64_t rows) {
    return dim3((unsigned)parts, (unsigned)(rows < kRowsY ? rows : kRowsY), (unsigned)((rows + kRowsY - 1) / kRowsY));
}

// log-sum state of some logits, in units of 2
struct Stat {
    float m, s, w;
};

template <class T>
constexpr int kPiece = 16 / (int)sizeof(typename T::T);    // elements of a 16-byte piece

// The 16-byte pieces of a row start at the 16-byte boundary at or before its
// first element: piece q holds elements q * E - lead ... of the row.
template <class T>
__device__ __forceinline__ int lead_of(const typename T::T *row) {
    return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(typename T::T));
}

// Elements of piece q as fp32; -inf where it lies outside the row. Masked
// logits become -inf too.
template <class T>
__device__ __forceinline__ void load_piece(const typename T::T *row, int64_t first, int vocab,
                                           float (&v)[kPiece<T>]) {
    constexpr int E = kPiece<T>;
    if (first >= 0 && first + E <= vocab) {
        typename T::T raw[E];
        load_vec<typename T::T, E>(row + first, raw);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = T::widen(raw[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t at = first + e;
            v[e] = at >= 0 && at < vocab ? T::widen(row[at]) : kNegInf;
        }
    }
}

__device__ __forceinline__ float max2(float a, float b) { return __builtin_fmaxf(a, b); }

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp(int v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, ROWS, 0xf, false);
}

// maximum / minimum over the wave, the same in every lane
__device__ __forceinline__ float wave_max(float v) {
    v = max2(v, dpp<0x128>(v));
    v = max2(v, dpp<0x124>(v));
    v = max2(v, dpp<0x122>(v));
    v = max2(v, dpp<0x121>(v));
    v = max2(v, dpp<0x142, 0xa>(v));
    v = max2(v, dpp<0x143, 0xc>(v));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ int wave_min(int v) {
    v = min(v, dpp<0x128>(v));
    v = min(v, dpp<0x124>(v));
    v = min(v, dpp<0x122>(v));
    v = min(v, dpp<0x121>(v));
    v = min(v, dpp<0x142, 0xa>(v));
    v = min(v, dpp<0x143, 0xc>(v));
    return __builtin_amdgcn_readlane(v, 63);
}

// Joins two states. A state of nothing has m = -inf and s = w = 0.
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = max2(a.m, b.m);
    const float da = a.m == kNegInf ? 0.0f : (a.m - m) * c, db = b.m == kNegInf ? 0.0f : (b.m - m) * c;
    const float ea = exp2f(da), eb = exp2f(db);
    return {m, __builtin_fmaf(a.s, ea, b.s * eb),
            __builtin_fmaf(ea, __builtin_fmaf(a.s, da, a.w), eb * __builtin_fmaf(b.s, db, b.w))};
}

__device__ __forceinline__ Stat join_wave(Stat a, float c) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const Stat b = {__shfl_xor(a.m, o), __shfl_xor(a.s, o), __shfl_xor(a.w, o)};
        a = join(a, b, c);
    }
    return a;
}

struct RowOut {
    float *logprobs, *entropy, *logsumexp, *top_logprobs;
    int64_t *top_ids;
};

// The numbers of a row from its joined state. Returns logsumexp; ln_s is 0
// for a row with nothing left.
template <class T>
__device__ __forceinline__ float finish_row(const RowOut &o, int64_t row, Stat t, const typename T::T *x,
                                            int64_t target, int64_t vocab, float inv_t, float &ln_s) {
    ln_s = t.m == kNegInf && t.s == 0.0f ? 0.0f : kLn2 * log2f(t.s);
    float lse = t.m * inv_t + ln_s;
    float entropy = t.s == 0.0f ? 0.0f : __builtin_fmaf(-kLn2, t.w / t.s, ln_s);
    // the largest logit's term is 1; a NaN or +inf leaves NaN in the sum
    const bool bad = !(t.s >= 1.0f || (t.m == kNegInf && t.s == 0.0f)) || !(t.s < __builtin_inff());
    float lp;
    if (target < 0) {
        lp = 0.0f;
    } else if (target >= vocab) {
        lp = __builtin_nanf("");
    } else {
        const float xt = T::widen(x[target]);
        lp = xt <= kMasked ? kNegInf : __builtin_fmaf(xt - t.m, inv_t, -ln_s);
    }
    if (bad) {
        lse = entropy = __builtin_nanf("");
        if (target >= 0) lp = lse;
    }
    o.logprobs[row] = lp;
    o.entropy[row] = entropy;
    o.logsumexp[row] = lse;
    return lse;
}

// Marks the k largest of n values (n <= 64 * kept) in LDS, equal ones by the
// lower index first, by setting bit 0 of flags; values are consumed. One wave.
__device__ __forceinline__ void select_top(float *values, uint8_t *flags, int n, int k) {
    const int lane = threadIdx.x & 63;
    float best = kNegInf;
    int at = n;
    auto scan = [&]() {
        best = kNegInf;
        at = 0x7fffffff;
        for (int i = lane; i < n; i += 64) {
            const float v = values[i];
            if (v > best) {
                best = v;
                at = i;
            }
        }
    };
    for (int i = lane; i < n; i += 64) flags[i] = 0;
    scan();
    for (int r = 0; r < k; ++r) {
        const float top = wave_max(best);
        if (top == kNegInf) break;
        const int first = wave_min(best == top ? at : 0x7fffffff);
        if (at == first) {
            values[first] = kNegInf;
            flags[first] = 1;
            scan();
        }
    }
}

// Indexes of the set flags, ascending, into list; returns how many.
__device__ __forceinline__ int collect(const uint8_t *flags, int n, uint16_t *list) {
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int base = 0; base < n; base += 64) {
        const bool on = base + lane < n && flags[base + lane];
        const uint64_t who = __ballot(on);
        if (on) list[count + __popcll(who & ((1ull << lane) - 1))] = (uint16_t)(base + lane);
        count += __popcll(who);
    }
    return count;
}

struct TopScratch {
    float group_max[kMaxGroups];
    float piece_max[kMaxTopK * 64];
    uint8_t flags[kMaxTopK * 64];
    uint16_t list[kMaxTopK * 64];
    uint16_t groups[kMaxTopK];
};
static_assert(kMaxGroups <= kMaxTopK * 64, "flags and list hold either");

// The top_k largest of groups [g0, g0 + n), in order; lane r of wave 0 ends
// with the r-th (value -inf where there is none). Wave 0 only, after a
// barrier behind the group maxima.
template <class T>
__device__ __forceinline__ void top_of_part(TopScratch &t, const typename T::T *row, int lead, int vocab, int g0, int n,
                                            int k, float &value, int &index) {
    constexpr int E = kPiece<T>;
    const int lane = threadIdx.x & 63;
    // the k-th largest group maximum bounds the k-th largest element from below
    int picked;
    if (n > k) {
        select_top(t.group_max, t.flags, n, k);
        picked = collect(t.flags, n, t.list);
    } else {
        for (int i = lane; i < n; i += 64) t.list[i] = (uint16_t)i;
        picked = n;
    }
    if (lane < picked) t.groups[lane] = t.list[lane];
    // maxima of the 64 pieces of each picked group, in index order
    for (int j = 0; j < picked; ++j) {
        float v[E];
        load_piece<T>(row, ((int64_t)(g0 + t.groups[j]) * 64 + lane) * E - lead, vocab, v);
        float m = v[0];
#pragma unroll
        for (int e = 1; e < E; ++e) m = max2(m, v[e]);
        t.piece_max[j * 64 + lane] = m > kMasked ? m : kNegInf;
    }
    select_top(t.piece_max, t.flags, picked * 64, k);
    const int pieces = collect(t.flags, picked * 64, t.list);
    // at most one piece a lane: its elements
    float v[E];
    int64_t first = 0;
    if (lane < pieces) {
        const int p = t.list[lane];
        first = ((int64_t)(g0 + t.groups[p >> 6]) * 64 + (p & 63)) * E - lead;
        load_piece<T>(row, first, vocab, v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] > kMasked ? v[e] : kNegInf;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = kNegInf;
    }
    value = kNegInf;
    index = -1;
    for (int r = 0; r < k; ++r) {
        float best = v[0];
        int e_best = 0;
#pragma unroll
        for (int e = 1; e < E; ++e)
            if (v[e] > best) {
                best = v[e];
                e_best = e;
            }
        const float top = wave_max(best);
        if (top == kNegInf) break;
        const uint64_t who = __ballot(best == top);
        const int owner = __ffsll((unsigned long long)who) - 1;     // pieces are in index order
        const int at = (int)first + e_best;
        const int won = __builtin_amdgcn_readlane(at, owner);
        if (lane == owner) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e == e_best) v[e] = kNegInf;
        }
        if (lane == r) {
            value = top;
            index = won;
        }
    }
}

struct Forward {
    const void *logits;
    int64_t row_stride;
    const void *targets;
    int targets64;
    int64_t rows;
    int vocab, splits, groups_per_split, top_k;
    float c, inv_t;            // log2(e) / T and 1 / T
    RowOut out;
    Stat *stats;               // [rows][splits] where splits > 1
    float *part_values;        // [rows][splits][top_k]
    int *part_ids;
};

__device__ __forceinline__ int64_t target_of(const void *targets, int is64, int64_t row) {
    return is64 ? static_cast<const int64_t *>(targets)[row] : static_cast<const int32_t *>(targets)[row];
}

template <class T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(Forward f) {
    constexpr int E = kPiece<T>;
    using V = typename T::T;
    __shared__ Stat stats[kWaves];
    __shared__ typename std::conditional<TOP, TopScratch, int>::type scratch;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = row_of_block();
    if (row >= f.rows) return;
    const int split = blockIdx.x;
    const V *x = static_cast<const V *>(f.logits) + row * f.row_stride;
    const int lead = lead_of<T>(x);
    const int groups = (int)(((int64_t)lead + f.vocab + 64 * E - 1) / (64 * E));
    const int g0 = split * f.groups_per_split;
    int n = groups - g0;
    if (n > f.groups_per_split) n = f.groups_per_split;

    Stat t = {kNegInf, 0.0f, 0.0f};
    // a set: kUnroll groups a wave, one after another
    for (int g = wave * kUnroll; g < n; g += kWaves * kUnroll) {
        float v[kUnroll][E];
        const int64_t from = (int64_t)(g0 + g) * 64 * E - lead;
        if (g + kUnroll <= n && from >= 0 && from + kUnroll * 64 * E <= f.vocab) {
            // inside the row, the same for the whole wave: the loads go out back to back
            V raw[kUnroll][E];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) load_vec<V, E>(x + from + (u * 64 + lane) * E, raw[u]);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) v[u][e] = T::widen(raw[u][e]);
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (g + u < n) {
                    load_piece<T>(x, from + (u * 64 + lane) * E, f.vocab, v[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) v[u][e] = kNegInf;
                }
            }
        }
        float top = t.m;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float m = v[u][0];
#pragma unroll
            for (int e = 1; e < E; ++e) m = max2(m, v[u][e]);
            m = m > kMasked ? m : kNegInf;
            top = max2(top, m);
            if constexpr (TOP) {
                const float all = wave_max(m);
                if (lane == 0 && g + u < n) scratch.group_max[g + u] = all;
            }
        }
        const float d = t.m == kNegInf ? 0.0f : (t.m - top) * f.c;
        const float scale = exp2f(d);
        t.w = scale * __builtin_fmaf(t.s, d, t.w);
        t.s *= scale;
        t.m = top;
        // Subtracted before it is scaled: the largest logit's term is then 1 whatever its
        // size, where one fused multiply-add would leave the rounding of m log2(e) / T in it.
        const float base = top == kNegInf ? 0.0f : top;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // the clamp keeps 0 * -inf out of w; it passes NaN to exp2 and so to s
                const float y = (v[u][e] - base) * f.c;
                const float p = __builtin_amdgcn_exp2f(y);
                t.s += p;
                t.w = __builtin_fmaf(p, max2(y, -3.0e38f), t.w);
            }
    }
    t = join_wave(t, f.c);
    if (lane == 0) stats[wave] = t;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) t = join(t, stats[i], f.c);

    float value = kNegInf;
    int index = -1;
    if constexpr (TOP) top_of_part<T>(scratch, x, lead, f.vocab, g0, n, f.top_k, value, index);
    if (f.splits > 1) {
        if (lane == 0) f.stats[row * f.splits + split] = t;
        if (TOP && lane < f.top_k) {
            f.part_values[(row * f.splits + split) * f.top_k + lane] = value;
            f.part_ids[(row * f.splits + split) * f.top_k + lane] = index;
        }
        return;
    }
    float ln_s = 0.0f, lse = 0.0f;
    if (lane == 0) lse = finish_row<T>(f.out, row, t, x, target_of(f.targets, f.targets64, row), f.vocab, f.inv_t, ln_s);
    if constexpr (TOP) {
        ln_s = __shfl(ln_s, 0);
        lse = __shfl(lse, 0);
        if (lane < f.top_k) {
            const bool none = index < 0 || lse != lse;
            f.out.top_logprobs[row * f.top_k + lane] =
                lse != lse ? lse : none ? kNegInf : __builtin_fmaf(value - t.m, f.inv_t, -ln_s);
            f.out.top_ids[row * f.top_k + lane] = none ? -1 : index;
        }
    }
}

// Joins the parts of a row: one wave a row, one lane a part.
template <class T, bool TOP>
__global__ __launch_bounds__(64) void logprobs_join_kernel(Forward f) {
    using V = typename T::T;
    const int lane = threadIdx.x;
    const int64_t row = row_of_block();
    if (row >= f.rows) return;
    Stat t = {kNegInf, 0.0f, 0.0f};
    if (lane < f.splits) t = f.stats[row * f.splits + lane];
    t = join_wave(t, f.c);
    const V *x = static_cast<const V *>(f.logits) + row * f.row_stride;
    float ln_s = 0.0f, lse = 0.0f;
    if (lane == 0) lse = finish_row<T>(f.out, row, t, x, target_of(f.targets, f.targets64, row), f.vocab, f.inv_t, ln_s);
    if constexpr (TOP) {
        ln_s = __shfl(ln_s, 0);
        lse = __shfl(lse, 0);
        // every part's alternatives are in order; parts are in index order
        const int64_t base = (row * f.splits + lane) * f.top_k;
        int taken = 0;
        float head = lane < f.splits ? f.part_values[base] : kNegInf;
        float value = kNegInf;
        int index = -1;
        for (int r = 0; r < f.top_k; ++r) {
            const float top = wave_max(head);
            if (top == kNegInf) break;
            const int owner = __ffsll((unsigned long long)__ballot(head == top)) - 1;
            int id = 0;
            if (lane == owner) {
                id = f.part_ids[base + taken];
                ++taken;
                head = taken < f.top_k ? f.part_values[base + taken] : kNegInf;
            }
            id = __builtin_amdgcn_readlane(id, owner);
            if (lane == r) {
                value = top;
                index = id;
            }
        }
        if (lane < f.top_k) {
            const bool none = index < 0 || lse != lse;
            f.out.top_logprobs[row * f.top_k + lane] =
                lse != lse ? lse : none ? kNegInf : __builtin_fmaf(value - t.m, f.inv_t, -ln_s);
            f.out.top_ids[row * f.top_k + lane] = none ? -1 : index;
        }
    }
}

// ---- backward -----------------------------------------------------------------

struct Backward {
    const void *logits;
    void *grad;
    int64_t row_stride, grad_stride;
    const void *targets;
    int targets64;
    const float *logsumexp, *entropy, *grad_logprobs, *grad_entropy;
    int64_t rows;
    int vocab, chunks;         // workgroups a row
    float inv_t;
};

constexpr int kBackUnroll = 4;         // pieces a lane has in flight

// With logp = x / T - logsumexp and p = e^logp,
//     grad = (g [j = target] - p (g + h (logp + H))) / T
// for the gradients g of the log probability and h of the entropy H. PIECES:
// logits and gradient rows share their offset in 16 bytes; otherwise one
// element at a time.
template <class T, bool PIECES>
__global__ __launch_bounds__(kThreads) void logprobs_backward_kernel(Backward f) {
    constexpr int E = PIECES ? kPiece<T> : 1;
    using V = typename T::T;
    const int64_t row = row_of_block();
    if (row >= f.rows) return;
    const int chunk = blockIdx.x;
    const V *x = static_cast<const V *>(f.logits) + row * f.row_stride;
    V *out = static_cast<V *>(f.grad) + row * f.grad_stride;
    const int lead = PIECES ? lead_of<T>(x) : 0;
    const int64_t target = target_of(f.targets, f.targets64, row);
    float lse = f.logsumexp[row];
    float g = f.grad_logprobs && target >= 0 ? f.grad_logprobs[row] : 0.0f;
    if (target >= f.vocab) g = __builtin_nanf("");
    const float h = f.grad_entropy ? f.grad_entropy[row] : 0.0f;
    const float hh = f.grad_entropy ? h * f.entropy[row] : 0.0f;
    const bool empty = lse == kNegInf;          // nothing left: no probabilities, no gradient
    if (empty) lse = 0.0f;
    // p (a + b logp)
    const float a = empty ? 0.0f : -(g + hh) * f.inv_t, b = empty ? 0.0f : -h * f.inv_t;
    const float at_target = empty ? 0.0f : g * f.inv_t;
    const int64_t hit = target >= 0 ? target + lead : -1;   // in pieces' elements
    const int64_t pieces = ((int64_t)lead + f.vocab + E - 1) / E;
    const int64_t q0 = (int64_t)chunk * kThreads * kBackUnroll;
    // the gradient of one piece, in place
    auto grad_piece = [&](float (&v)[E], int64_t q, V (&o)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            // x / T - logsumexp first, rounded once: near 0, where it matters, nothing is lost
            const float logp = __builtin_fmaf(v[e], f.inv_t, -lse);
            const float p = __builtin_amdgcn_exp2f(logp * kLog2e);
            v[e] = p * __builtin_fmaf(b, max2(logp, -3.0e38f), a);
        }
        if (hit >= q * E && hit < q * E + E) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (hit == q * E + e) v[e] += at_target;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = T::narrow(v[e]);
    };
    const int64_t from = q0 * E - lead;
    if (from >= 0 && from + kThreads * kBackUnroll * E <= f.vocab) {
        // inside the row, the same for the whole workgroup
        V raw[kBackUnroll][E];
#pragma unroll
        for (int u = 0; u < kBackUnroll; ++u) load_vec<V, E>(x + from + (u * kThreads + (int)threadIdx.x) * E, raw[u]);
#pragma unroll
        for (int u = 0; u < kBackUnroll; ++u) {
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = T::widen(raw[u][e]);
            grad_piece(v, q0 + u * kThreads + threadIdx.x, raw[u]);
            store_vec<V, E>(out + from + (u * kThreads + (int)threadIdx.x) * E, raw[u]);
        }
        return;
    }
    for (int u = 0; u < kBackUnroll; ++u) {
        const int64_t q = q0 + u * kThreads + threadIdx.x;
        if (q >= pieces) break;
        const int64_t first = q * E - lead;
        float v[E];
        V o[E];
        if constexpr (PIECES) {
            load_piece<T>(x, first, f.vocab, v);
        } else {
            v[0] = T::widen(x[q]);
        }
        grad_piece(v, q, o);
        if (first >= 0 && first + E <= f.vocab) {
            store_vec<V, E>(out + first, o);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (first + e >= 0 && first + e < f.vocab) out[first + e] = o[e];
        }
    }
}

// ---- host ---------------------------------------------------------------------

struct Plan {
    int splits, groups_per_split;
    size_t stats, values, ids, total;
};

int compute_units() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

// Parts of a row: about four workgroups a compute unit in all when there are
// few rows, but no part below one set of a workgroup's waves (four groups),
// and no part above the group maxima a workgroup keeps. cus: the device's.
Plan plan_for(int64_t rows, int64_t vocab, int elem, int top_k, int cus) {
    const int64_t per = 64 * (16 / elem);
    const int64_t groups = (vocab + 16 / elem - 1 + per - 1) / per;     // the most any lead gives
    int64_t splits = rows > 0 ? (4 * (int64_t)cus + rows - 1) / rows : 1;
    if (splits > (groups + kWaves - 1) / kWaves) splits = (groups + kWaves - 1) / kWaves;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits < (groups + kMaxGroups - 1) / kMaxGroups) splits = (groups + kMaxGroups - 1) / kMaxGroups;
    if (splits < 1) splits = 1;
    Plan p;
    p.groups_per_split = (int)((groups + splits - 1) / splits);
    p.splits = (int)((groups + p.groups_per_split - 1) / p.groups_per_split);
    p.stats = 0;
    p.values = p.splits > 1 ? round_up(sizeof(Stat) * (size_t)rows * p.splits, 256) : 0;
    p.ids = p.splits > 1 ? round_up(p.values + 4 * (size_t)rows * p.splits * top_k, 256) : 0;
    p.total = p.splits > 1 ? round_up(p.ids + 4 * (size_t)rows * p.splits * top_k, 256) : 0;
    return p;
}

bool is_float(int d) { return d == EWG_BF16 || d == EWG_FP32; }
bool is_index(int d) { return d == EWG_INT32 || d == EWG_INT64; }
bool is_known(int d) { return d >= EWG_INT32 && d <= EWG_FP32; }

int check_sizes(int64_t rows, int64_t vocab, int64_t stride, int logits_dtype, int targets_dtype, float temperature) {
    if (!is_known(logits_dtype) || !is_known(targets_dtype)) return EWG_INVALID_ARGUMENT;
    if (!is_float(logits_dtype) || !is_index(targets_dtype)) return EWG_UNSUPPORTED;
    if (rows < 0 || rows > EWG_LOGPROBS_MAX_ROWS || vocab < 1 || vocab > EWG_LOGPROBS_MAX_VOCAB) return EWG_UNSUPPORTED;
    if (!(temperature >= 1e-4f && temperature <= 1e4f)) return EWG_INVALID_ARGUMENT;
    if (rows > 1 && stride < vocab) return EWG_INVALID_ARGUMENT;
    return EWG_OK;
}

template <class T, bool TOP>
hipError_t launch_forward(const Forward &f, hipStream_t stream) {
    logprobs_kernel<T, TOP><<<grid_of(f.splits, f.rows), kThreads, 0, stream>>>(f);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || f.splits == 1) return e;
    logprobs_join_kernel<T, TOP><<<grid_of(1, f.rows), 64, 0, stream>>>(f);
    return hipGetLastError();
}

template <class T>
hipError_t launch_backward(const Backward &f, bool pieces, hipStream_t stream) {
    const dim3 grid = grid_of(f.chunks, f.rows);
    if (pieces)
        logprobs_backward_kernel<T, true><<<grid, kThreads, 0, stream>>>(f);
    else
        logprobs_backward_kernel<T, false><<<grid, kThreads, 0, stream>>>(f);
    return hipGetLastError();
}

}  // namespace
}  // namespace ewg

extern "C" {

size_t token_logprobs_workspace_bytes(int64_t num_rows, int64_t vocab, int logits_dtype, int top_k) {
    using namespace ewg;
    if (num_rows < 1 || num_rows > EWG_LOGPROBS_MAX_ROWS || vocab < 1 || vocab > EWG_LOGPROBS_MAX_VOCAB ||
        !is_float(logits_dtype) || top_k < 0 || top_k > EWG_MAX_TOP_LOGPROBS)
        return 0;
    return plan_for(num_rows, vocab, logits_dtype == EWG_BF16 ? 2 : 4, top_k, compute_units()).total;
}

int token_logprobs(const void *logits, const void *targets, int64_t num_rows, int64_t vocab,
                   int64_t row_stride, int logits_dtype, int targets_dtype, float temperature, int top_k,
                   float *logprobs, float *entropy, float *logsumexp, float *top_logprobs,
                   int64_t *top_ids, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace ewg;
    int st = check_sizes(num_rows, vocab, row_stride, logits_dtype, targets_dtype, temperature);
    if (st != EWG_OK) return st;
    if (top_k < 0 || top_k > EWG_MAX_TOP_LOGPROBS) return EWG_UNSUPPORTED;
    if (num_rows == 0) return EWG_OK;
    const int elem = logits_dtype == EWG_BF16 ? 2 : 4;
    if (!logits || !targets || !logprobs || !entropy || !logsumexp || (top_k > 0 && (!top_logprobs || !top_ids)))
        return EWG_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(logits) % elem) return EWG_INVALID_ARGUMENT;
    const Plan p = plan_for(num_rows, vocab, elem, top_k, compute_units());
    if (p.splits > 1) {
        if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return EWG_INVALID_ARGUMENT;
        if (workspace_bytes < p.total) return EWG_WORKSPACE_TOO_SMALL;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Forward f = {};
    f.logits = logits;
    f.row_stride = row_stride;
    f.targets = targets;
    f.targets64 = targets_dtype == EWG_INT64;
    f.rows = num_rows;
    f.vocab = (int)vocab;
    f.splits = p.splits;
    f.groups_per_split = p.groups_per_split;
    f.top_k = top_k;
    f.inv_t = 1.0f / temperature;
    f.c = kLog2e / temperature;
    f.out = {logprobs, entropy, logsumexp, top_logprobs, top_ids};
    if (p.splits > 1) {
        f.stats = reinterpret_cast<Stat *>(ws + p.stats);
        f.part_values = reinterpret_cast<float *>(ws + p.values);
        f.part_ids = reinterpret_cast<int *>(ws + p.ids);
    }
    (void)hipGetLastError();
    hipError_t e;
    if (logits_dtype == EWG_BF16)
        e = top_k ? launch_forward<BF16, true>(f, stream) : launch_forward<BF16, false>(f, stream);
    else
        e = top_k ? launch_forward<F32, true>(f, stream) : launch_forward<F32, false>(f, stream);
    return e == hipSuccess ? EWG_OK : EWG_HIP_ERROR;
}

int token_logprobs_backward(const void *logits, const void *targets, const float *logsumexp,
                            const float *entropy, const float *grad_logprobs,
                            const float *grad_entropy, void *grad_logits, int64_t num_rows,
                            int64_t vocab, int64_t row_stride, int64_t grad_row_stride,
                            int logits_dtype, int targets_dtype, float temperature,
                            hipStream_t stream) {
    using namespace ewg;
    int st = check_sizes(num_rows, vocab, row_stride, logits_dtype, targets_dtype, temperature);
    if (st != EWG_OK) return st;
    if (num_rows > 1 && grad_row_stride < vocab) return EWG_INVALID_ARGUMENT;
    if (num_rows == 0) return EWG_OK;
    const int elem = logits_dtype == EWG_BF16 ? 2 : 4;
    if (!logits || !targets || !logsumexp || !grad_logits || (grad_entropy && !entropy)) return EWG_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(logits) % elem || reinterpret_cast<uintptr_t>(grad_logits) % elem)
        return EWG_INVALID_ARGUMENT;
    Backward f = {};
    f.logits = logits;
    f.grad = grad_logits;
    f.row_stride = row_stride;
    f.grad_stride = grad_row_stride;
    f.targets = targets;
    f.targets64 = targets_dtype == EWG_INT64;
    f.logsumexp = logsumexp;
    f.entropy = entropy;
    f.grad_logprobs = grad_logprobs;
    f.grad_entropy = grad_entropy;
    f.rows = num_rows;
    f.vocab = (int)vocab;
    f.inv_t = 1.0f / temperature;
    // 16-byte pieces where both rows start at the same place in 16 bytes, for every row
    const bool pieces = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(grad_logits)) % 16 == 0 &&
                        (num_rows == 1 || (row_stride - grad_row_stride) * elem % 16 == 0);
    const int64_t per = pieces ? 16 / elem : 1;
    f.chunks = (int)((vocab + per - 1 + (int64_t)per * kThreads * kBackUnroll - 1) / (per * kThreads * kBackUnroll));
    (void)hipGetLastError();
    const hipError_t e = logits_dtype == EWG_BF16 ? launch_backward<BF16>(f, pieces, stream)
                                                  : launch_backward<F32>(f, pieces, stream);
    return e == hipSuccess ? EWG_OK : EWG_HIP_ERROR;
}

}  // extern "C"

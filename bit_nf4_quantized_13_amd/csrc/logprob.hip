// Token log-probabilities over rows of logits x [M x V], and their gradient:
//   lse = log sum_v e^x_v       logp = x_t - lse       p = e^(x - lse)
//   H = -sum_v p_v log p_v = log l - (sum_v e^d_v d_v) / l,  d = x - max x, l = sum e^d
//   the `top` largest x, equal ones in ascending order of index
//   dx_v = g (delta_vt - p_v) - h p_v (log p_v + H)      g, h the gradients of logp and H
// A logit of -inf is a forbidden token: p = 0, no part in H, gradient 0.  A row
// of -inf only has lse = -inf, logp = -inf, H = 0 and gradient 0.  A NaN or +inf
// makes its row's results NaN.  A target outside [0, V) is no target: logp = 0 and
// g is not used.
//
// All sums in fp32.  H is taken from the deviations d, not as lse - sum p x:
// that difference would lose digits in rows of large logits, and so would
// x - lse: log p is d - log l.  The gradient has lse alone; where |lse| is so
// large that its last digit matters (kLargeLse; a row masked with -1e9 or the
// type's lowest value throughout is one), it adds up the row's e^(x - lse) again
// and divides by it.
//
// Bound: HBM (V elements read once; the gradient reads and writes them), with
// the vector unit close behind for bf16: e^d is a quarter-rate operation.  A
// workgroup holds its piece of a row in registers, 32 elements a thread: the
// maximum first, then the exponentials against it, with no running rescale.
// Rows are cut into chunks of at most 8192 for 256 threads, whose (max, l, sum
// e^d d) and best candidates go to the workspace, and a wave a row joins them in
// chunk order in a second launch; of few rows, one of up to 32768 elements is a
// workgroup's of 1024 threads, which writes its results.
//
// The best `top`: keys order value and index in 64 bits, all distinct.  A group of
// 8 threads (2 where a thread has 8 elements) owns up to 256 in a row; the top-th
// best of these groups by (maximum, then place) bounds the candidates: an element
// below its maximum, or equal to it in a later group, has top better ones.  So at
// most top 256 elements remain, usually some dozen; they are collected in LDS and
// each counts the larger ones (of thousands of equal ones, the best are taken one
// by one).
//
// Measured, bf16: 2048 x 131071 with 8 alternatives 142 + 9 us for 537 MB, 92 in
// all without them (5.8 TB/s); one row of 32000 with 5 alternatives 8.0 us;
// gradient of 4096 x 32000 81 to 92 us for 524 MB.
#include "elem8.hpp"
#include "launch.hpp"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;                     // of a chunk, and of the gradient
constexpr int kRowThreads = 1024;                 // of a whole row
constexpr int kVecs = 4;                          // groups of 8 a thread
constexpr int kHeld = kVecs * 8;                  // elements a thread
constexpr int kChunk = kThreads * kHeld;          // 8192
constexpr int64_t kWholeRow = kRowThreads * kHeld;  // 32768
constexpr int kGroupElems = 256;                  // most elements of a group
constexpr int kCandBytes = kGroupElems * 12 + kGroupElems / 8 * 4;  // their keys, values and vectors' places
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLargeLse = 4096.0f;              // half a last digit of lse is 2.4e-4 of p there
constexpr float kLargeMax = 1048576.0f;           // half a last digit of max x log2 e is 0.06 there

typedef unsigned long long u64;

// Ascending with the value (-0 taken as +0), then descending with the index.
__device__ __forceinline__ u64 key_of(float x, uint32_t index) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t up = b & 0x80000000u ? ~b : b | 0x80000000u;
    return ((u64)up << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(u64 k) {
    const uint32_t up = (uint32_t)(k >> 32);
    return __uint_as_float(up & 0x80000000u ? up & 0x7FFFFFFFu : ~up);
}
__device__ __forceinline__ uint32_t key_index(u64 k) { return ~(uint32_t)k; }

__device__ __forceinline__ u64 max_key(u64 a, u64 b) { return a > b ? a : b; }

// Chunks of a row and the elements of one (a multiple of 8; the last may be shorter).
struct Cut {
    int chunks;
    int64_t len;
};
__host__ __device__ inline Cut cut_of(int64_t V) {
    const int64_t c = (V + kChunk - 1) / kChunk;
    const int64_t len = ((V + c - 1) / c + 7) / 8 * 8;
    return Cut{(int)((V + len - 1) / len), len};
}

// A row of -inf only; a NaN, which no maximum shows, is in l.
__device__ __forceinline__ bool none_left(float mx, float l) { return mx == -INFINITY && l == 0.0f; }

// What a row's sums come to, written by one thread.
struct RowOut {
    const int64_t *targets;
    float *logp, *entropy, *lse, *top_logp;
    int32_t *top_ids;
};
template <typename T>
__device__ __forceinline__ void write_row(const RowOut &o, int64_t row, const T *xr, int64_t V, float mx, float base,
                                          float l, float a) {
    const bool none = none_left(mx, l);
    const float log_l = logf(l);
    if (o.lse) o.lse[row] = none ? -INFINITY : base + log_l;
    if (o.entropy) o.entropy[row] = none ? 0.0f : log_l - a / l;
    if (o.logp) {
        const int64_t t = o.targets[row];
        o.logp[row] = t < 0 || t >= V ? 0.0f : none ? -INFINITY : load1(xr + t) - base - log_l;
    }
}

// Two sums over the workgroup, on every thread, in wave order.
template <int THREADS>
__device__ __forceinline__ void group_totals(float &l, float &a, float (*red)[THREADS / 64]) {
    l = wave_sum(l);
    a = wave_sum(a);
    if ((threadIdx.x & 63) == 0) {
        red[0][threadIdx.x >> 6] = l;
        red[1][threadIdx.x >> 6] = a;
    }
    __syncthreads();
    l = a = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
        l += red[0][i];
        a += red[1][i];
    }
}

// One piece of a row.  ROW: the whole row, its results to `out`; otherwise chunk
// blockIdx.x % chunks of row blockIdx.x / chunks, its sums to stats and best.
// LDS beyond the static: top kCandBytes.
template <typename T, bool TOP, int THREADS, bool ROW>
__global__ __launch_bounds__(THREADS) void logprob_piece_kernel(const T *__restrict__ x, int64_t V, int64_t ld,
                                                                int chunks, int64_t len, int top,
                                                                float *__restrict__ stats, u64 *__restrict__ best,
                                                                RowOut out) {
    __shared__ float red[3][THREADS / 64];
    __shared__ float gmax[TOP ? THREADS / 2 : 1];
    __shared__ int nvec, ncand, thr_group;
    extern __shared__ __attribute__((aligned(16))) u64 cand[];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t row = ROW ? blockIdx.x : blockIdx.x / chunks;
    const int64_t c0 = ROW ? 0 : blockIdx.x % chunks * len;
    const int left = (int)(V - c0 < len ? V - c0 : len);
    const T *xr = x + row * ld + c0;
    // groups of gt threads, nv vectors of 8 a thread, side by side
    const int nv = (left + THREADS * 8 - 1) / (THREADS * 8), gt = nv == 1 ? 2 : 8, gshift = nv == 1 ? 1 : 3;
    const int group = tid >> gshift, per = 8 * nv * gt, groups = (left + per - 1) / per;
    const int first = group * per + (tid & (gt - 1)) * 8, step = 8 * gt;
    F8 v[kVecs];
    float vmax[kVecs], mx = -INFINITY;
    auto at = [&](int i) { return i < nv ? first + i * step : left; };
    RowLoad<T, kVecs> in_flight;
    in_flight.request(xr, left, at);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = in_flight.get(xr, left, at, i, -INFINITY);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        vmax[i] = v[i].v[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) vmax[i] = fmaxf(vmax[i], v[i].v[e]);
        mx = fmaxf(mx, vmax[i]);
    }
    if (TOP) {
        float g = fmaxf(mx, dpp_or<0xB1, 0xF>(mx, mx));  // the neighbour's; then the pair's and the four's beside it
        if (gt == 8) {
            g = fmaxf(g, dpp_or<0x4E, 0xF>(g, g));
            g = fmaxf(g, dpp_or<0x141, 0xF>(g, g));
        }
        if ((tid & (gt - 1)) == 0) gmax[group] = g;
        if (tid == 0) {
            nvec = ncand = thr_group = 0;
        }
    }
    mx = wave_max(mx);
    if ((tid & 63) == 0) red[2][wave] = mx;
    __syncthreads();
    mx = red[2][0];
#pragma unroll
    for (int i = 1; i < THREADS / 64; ++i) mx = fmaxf(mx, red[2][i]);
    if (TOP && tid < groups && groups >= top) {
        const float g = gmax[tid];
        int better = 0;
#pragma unroll 8
        for (int i = 0; i < groups; ++i) better += gmax[i] > g || (gmax[i] == g && i < tid);
        if (better == top - 1) thr_group = tid;
    }
    // e^d with d = x - mx, to the base 2: one fma an element from shift = mx log2 e, whose
    // rounding, off, is the same in every d and taken out of the sums
    const float base = mx == -INFINITY ? 0.0f : mx;
    const bool large = !(fabsf(base) < kLargeMax);
    const float shift = base * kLog2e, off = fmaf(base, kLog2e, -shift);
    float l = 0.0f, a = 0.0f;
    if (!large) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int n = i < nv ? left - first - i * step : 0;
            if (n <= 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float d = fmaf(v[i].v[e], kLog2e, -shift);
                if (n < 8 && e >= n) d = -200.0f;
                const float ex = __builtin_amdgcn_exp2f(d);
                l += ex;
                a = fmaf(ex, d, a);
            }
        }
    }
    group_totals<THREADS>(l, a, red);
    if (large || a != a) {
        // ruled-out tokens (0 times -inf above): d held above the underflow of e^d, so that
        // their part is 0, and a NaN kept; the same for the whole workgroup
        l = a = 0.0f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float d = (v[i].v[e] - base) * kLog2e;
                d = d < -200.0f ? -200.0f : d;
                const float ex = __builtin_amdgcn_exp2f(d);
                l += ex;
                a = fmaf(ex, d, a);
            }
        __syncthreads();  // red is read above
        group_totals<THREADS>(l, a, red);
    } else {
        const float f = __builtin_amdgcn_exp2f(-off);
        a = (a - off * l) * f;
        l *= f;
    }
    a *= kLn2;
    if (tid == 0) {
        if (ROW) {
            write_row(out, row, xr, V, mx, base, l, a);
        } else {
            float *o = stats + (int64_t)blockIdx.x * 4;
            o[0] = mx;
            o[1] = l;
            o[2] = a;
        }
    }
    if (!TOP) return;
    const bool all = groups < top;       // fewer groups than places: every element is a candidate
    const float thr = gmax[thr_group];
    const bool in = group <= thr_group;  // of groups with the threshold's maximum, these hold candidates
    // the vectors that reach the threshold, as they are; then a key for each of their elements that does
    float *vals = reinterpret_cast<float *>(cand + top * kGroupElems);
    int *at_c = reinterpret_cast<int *>(vals + top * kGroupElems);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = at(i);
        if (!(c < left && (all || vmax[i] > thr || (in && vmax[i] == thr)))) continue;
        const int j = atomicAdd(&nvec, 1);
        at_c[j] = c;
        *reinterpret_cast<f32x4 *>(vals + 8 * j) = f32x4{v[i].v[0], v[i].v[1], v[i].v[2], v[i].v[3]};
        *reinterpret_cast<f32x4 *>(vals + 8 * j + 4) = f32x4{v[i].v[4], v[i].v[5], v[i].v[6], v[i].v[7]};
    }
    __syncthreads();
    u64 *list = ROW ? nullptr : best + (int64_t)blockIdx.x * top;
    for (int i = tid; i < 8 * nvec; i += THREADS) {
        const float x1 = vals[i];
        const int c = at_c[i >> 3] + (i & 7);
        if (c < left && (all || x1 >= thr)) cand[atomicAdd(&ncand, 1)] = key_of(x1, (uint32_t)(c0 + c));
    }
    __syncthreads();
    const int n = ncand;
    const float log_l = logf(l);
    auto place = [&](int rank, u64 k) {
        if (ROW) {
            out.top_logp[row * top + rank] = none_left(mx, l) ? -INFINITY : key_value(k) - base - log_l;
            out.top_ids[row * top + rank] = (int32_t)key_index(k);
        } else {
            list[rank] = k;
        }
    };
    if (n <= THREADS) {
        if (tid < n) {
            const u64 k = cand[tid];
            int larger = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) larger += cand[j] > k;
            if (larger < top) place(larger, k);
        }
    } else {  // many equal logits: one after the other, each the largest below the last
        __shared__ u64 wave_best[THREADS / 64];
        u64 last = ~(u64)0;
        for (int rank = 0; rank < top; ++rank) {
            u64 k = 0;
            for (int i = tid; i < n; i += THREADS) k = cand[i] < last ? max_key(k, cand[i]) : k;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) k = max_key(k, __shfl_xor(k, o));
            if ((tid & 63) == 0) wave_best[wave] = k;
            __syncthreads();
            last = wave_best[0];
#pragma unroll
            for (int i = 1; i < THREADS / 64; ++i) last = max_key(last, wave_best[i]);
            if (tid == 0) place(rank, last);
            __syncthreads();
        }
    }
    for (int i = n + tid; i < top; i += THREADS) place(i, 0);  // a chunk of fewer elements, or NaN
}

// One wave a row: the chunks' sums against the row's maximum, lane i holding
// chunk i, and the chunks' best lists (descending) merged from their heads.
template <typename T>
__global__ __launch_bounds__(64) void logprob_join_kernel(const T *__restrict__ x, int64_t V, int64_t ld, int chunks,
                                                          const float *__restrict__ stats, const u64 *__restrict__ best,
                                                          int top, RowOut out) {
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x;
    const bool mine = lane < chunks;
    const float *s = stats + (row * chunks + lane) * 4;
    const float m = mine ? s[0] : -INFINITY, mx = wave_max(m), base = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f, a = 0.0f;
    if (mine && !none_left(m, s[1])) {
        const float d = fmaxf(m - base, -150.0f), f = expf(d);
        l = s[1] * f;
        a = (s[2] + s[1] * d) * f;
    }
    l = wave_sum(l);
    a = wave_sum(a);
    if (lane == 0) write_row(out, row, x + row * ld, V, mx, base, l, a);
    if (top == 0) return;
    const float log_l = logf(l);
    const u64 *list = best + (row * chunks + lane) * top;
    int at = 0;
    u64 head = mine ? list[0] : 0;
    for (int i = 0; i < top; ++i) {
        u64 k = head;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) k = max_key(k, __shfl_xor(k, o));
        if (head == k && k != 0) {
            ++at;
            head = at < top ? list[at] : 0;
        }
        if (lane == 0) {
            out.top_logp[row * top + i] = none_left(mx, l) ? -INFINITY : key_value(k) - base - log_l;
            out.top_ids[row * top + i] = (int32_t)key_index(k);
        }
    }
}

// The gradient: `split` workgroups a row, each every split-th chunk of it, a
// chunk held as in the forward.  In place, a row belongs to one workgroup (split
// = 1): its sum over the row is done before it overwrites any of it.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprob_bwd_kernel(const T *x, int64_t V, int64_t ld, int split,
                                                               int chunks, int64_t len,
                                                               const int64_t *__restrict__ targets,
                                                               const float *__restrict__ lse_in,
                                                               const float *__restrict__ entropy,
                                                               const float *__restrict__ dlogp,
                                                               const float *__restrict__ dent, T *dx, int64_t ldd) {
    const int64_t row = blockIdx.x / split;
    const int64_t t = targets ? targets[row] : -1;
    const bool has = t >= 0 && t < V;
    const float lse = lse_in[row], h = dent ? dent[row] : 0.0f, ent = dent ? entropy[row] : 0.0f;
    const bool none = lse == -INFINITY;
    const float g = has && !none ? dlogp[row] : 0.0f;
    const float base = none ? 0.0f : lse;
    const T *xr = x + row * ld;
    T *dr = dx + row * ldd;
    float scale = base == base ? 1.0f : base, log_s = 0.0f;  // p = scale e^(x - lse), log p = x - lse - log_s
    if (fabsf(base) > kLargeLse) {     // the same for the whole workgroup
        __shared__ float red[kThreads / 64];
        float s = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < V; c += kThreads * 8) {
            const F8 w = load8(xr + c, V - c, -INFINITY);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += __builtin_amdgcn_exp2f(fmaxf(w.v[e] - base, -150.0f) * kLog2e);
        }
        s = wave_sum(s);
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.0f;
        for (int i = 0; i < kThreads / 64; ++i) s += red[i];
        scale = 1.0f / s;
        log_s = logf(s);
    }
    const float c1 = -(g + h * (ent - log_s)) * scale, c2 = -h * scale;
    for (int chunk = (int)(blockIdx.x % split); chunk < chunks; chunk += split) {
        const int64_t c0 = chunk * len;
        const int left = (int)(V - c0 < len ? V - c0 : len);
        const int hot = has && t >= c0 && t < c0 + left ? (int)(t - c0) : -1;
        F8 v[kVecs];
        auto at = [&](int i) { return (i * kThreads + (int)threadIdx.x) * 8; };
        RowLoad<T, kVecs> in_flight;
        in_flight.request(xr + c0, left, at);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = in_flight.get(xr + c0, left, at, i);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = at(i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // -inf (and a difference below e's underflow) gives p = 0 and a finite log
                const float lp = fmaxf(v[i].v[e] - base, -150.0f);
                const float p = __builtin_amdgcn_exp2f(lp * kLog2e);
                v[i].v[e] = none ? 0.0f : p * fmaf(c2, lp, c1);
                if (c + e == hot) v[i].v[e] += g;
            }
            if (c < left) store8(dr + c0 + c, left - c, v[i]);
        }
    }
}

}  // namespace

// Rows that go whole to a workgroup each, with one launch and no join: those of one chunk,
// and longer ones where there are no more of them than CUs (one row of 32000 with 5
// alternatives 9.7 against 11.6 us, 128 rows 10.9 against 12.6); with more, the chunks'
// smaller workgroups overlap better (4096 rows 84 against 147 us).
bool whole_rows(int64_t M, int64_t V) { return V <= kChunk || (M <= 256 && V <= kWholeRow); }

size_t logprob_stats_bytes(int64_t M, int64_t V) {
    return whole_rows(M, V) ? 0 : sizeof(float) * 4 * (size_t)M * cut_of(V).chunks;
}
size_t logprob_best_bytes(int64_t M, int64_t V, int top) {
    return whole_rows(M, V) ? 0 : sizeof(u64) * (size_t)top * (size_t)M * cut_of(V).chunks;
}
int64_t logprob_groups(int64_t M, int64_t V) { return M * cut_of(V).chunks; }

hipError_t launch_logprob_fwd(const void *x, bool f32, int64_t M, int64_t V, int64_t ld, const int64_t *targets,
                              int top, float *logp, float *entropy, float *lse, float *top_logp, int32_t *top_ids,
                              float *stats, void *best, hipStream_t s) {
    const RowOut out{targets, logp, entropy, lse, top_logp, top_ids};
    const size_t lds = (size_t)top * kCandBytes;  // up to 50 KiB
    auto run = [&](auto *p) {
        using T = std::remove_pointer_t<decltype(p)>;
        const T *xt = (const T *)x;
        const Cut cut = cut_of(V);
        const bool whole = whole_rows(M, V), small = V <= kChunk;
        const unsigned groups = (unsigned)(whole ? M : M * cut.chunks);
        auto *kernel = whole ? small ? top > 0 ? logprob_piece_kernel<T, true, kThreads, true>
                                               : logprob_piece_kernel<T, false, kThreads, true>
                               : top > 0 ? logprob_piece_kernel<T, true, kRowThreads, true>
                                         : logprob_piece_kernel<T, false, kRowThreads, true>
                       : top > 0 ? logprob_piece_kernel<T, true, kThreads, false>
                                 : logprob_piece_kernel<T, false, kThreads, false>;
        kernel<<<groups, whole && !small ? kRowThreads : kThreads, lds, s>>>(xt, V, ld, cut.chunks, whole ? V : cut.len, top,
                                                                           stats, (u64 *)best, out);
        if (whole) return hipGetLastError();
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        logprob_join_kernel<T><<<(unsigned)M, 64, 0, s>>>(xt, V, ld, cut.chunks, stats, (const u64 *)best, top, out);
        return hipGetLastError();
    };
    return f32 ? run((float *)nullptr) : run((uint16_t *)nullptr);
}

hipError_t launch_logprob_bwd(const void *x, bool f32, int64_t M, int64_t V, int64_t ld, const int64_t *targets,
                              const float *lse, const float *entropy, const float *dlogp, const float *dent, void *dx,
                              int64_t ldd, hipStream_t s) {
    const Cut cut = cut_of(V);
    const int split = x == dx ? 1 : cut.chunks;
    const unsigned groups = (unsigned)(M * split);
    if (f32)
        logprob_bwd_kernel<float><<<groups, kThreads, 0, s>>>((const float *)x, V, ld, split, cut.chunks, cut.len,
                                                              targets, lse, entropy, dlogp, dent, (float *)dx, ldd);
    else
        logprob_bwd_kernel<uint16_t><<<groups, kThreads, 0, s>>>((const uint16_t *)x, V, ld, split, cut.chunks, cut.len,
                                                                 targets, lse, entropy, dlogp, dent, (uint16_t *)dx, ldd);
    return hipGetLastError();
}

}  // namespace qnf4

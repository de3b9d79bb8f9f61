// Token log-probabilities over rows of logits x [M x V], and their gradient:
//   lse = log sum_v e^x_v       logp = x_t - lse       p = e^(x - lse)
//   H = -sum_v p_v log p_v = log l - (sum_v e^d_v d_v) / l,  d = x - max x, l = sum e^d
//   the `top` largest x, equal ones in ascending order of index
//   dx_v = g (delta_vt - p_v) - h p_v (log p_v + H)      g, h the gradients of logp and H
// A logit of -inf is a forbidden token: p = 0, no part in H, gradient 0.  A row
// of -inf only has lse = -inf, logp = -inf, H = 0 and gradient 0.  A target
// outside [0, V) is no target: logp = 0 and g is not used.
//
// All sums in fp32.  H is taken from the deviations d, not as lse - sum p x:
// that difference would lose digits in rows of large logits, and so would
// x - lse: log p is d - log l.  The gradient has lse alone; where |lse| is so
// large that its last digit matters (kLargeLse; a row masked with -1e9 or the
// type's lowest value throughout is one), it adds up the row's e^(x - lse) again
// and divides by it.
//
// Bound: HBM (V elements read once; the gradient reads and writes them), with
// the vector unit close behind for bf16: e^d is a quarter-rate operation.  Every
// row is cut into chunks of at most kChunk elements that one workgroup holds in
// registers: the maximum first, then the exponentials against it, with no
// running rescale; few rows still fill the GPU, and long rows need no loop.
// The chunks' (max, l, sum e^d d) and best candidates go to the workspace and a
// wave a row joins them in chunk order.
//
// The best `top` of a chunk: keys order value and index in 64 bits, all
// distinct.  The top-th largest of the 64 largest keys of 4 threads each is a
// lower bound for the chunk's top-th largest key; at most (top - 1) 128 + 1
// keys reach it (only the top - 1 groups above it can hold several), usually
// some dozen.  They are collected in LDS and each counts the larger ones.
#include "elem8.hpp"
#include "launch.hpp"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                          // groups of 8 a thread
constexpr int kChunk = kThreads * kVecs * 8;      // 8192 elements
constexpr int kGroupThreads = 4;                  // threads of a threshold group
constexpr int kGroups = kThreads / kGroupThreads;
constexpr int kMaxCand = (kMaxTop - 1) * kGroupThreads * kVecs * 8 + 1;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLargeLse = 4096.0f;              // half a last digit of lse is 2.4e-4 of p there

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

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprob_chunk_kernel(const T *__restrict__ x, int64_t V, int64_t ld,
                                                                 int chunks, int64_t len, int top,
                                                                 float *__restrict__ stats, u64 *__restrict__ best) {
    __shared__ float redf[3][kThreads / 64];
    __shared__ u64 gkey[TOP ? kGroups : 1], thr_s;
    __shared__ u64 cand[TOP ? kMaxCand : 1];
    __shared__ int ncand;
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t row = blockIdx.x / chunks;
    const int chunk = (int)(blockIdx.x % chunks);
    const int64_t c0 = chunk * len, left = V - c0 < len ? V - c0 : len;
    const T *xr = x + row * ld + c0;
    F8 v[kVecs];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = (i * kThreads + tid) * 8;
        v[i] = load8(xr + c, left - c, -INFINITY);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, v[i].v[e]);
    if (TOP) {
        // the thread's largest key: its first element equal to mx
        int at = 0;
#pragma unroll
        for (int i = kVecs - 1; i >= 0; --i)
#pragma unroll
            for (int e = 7; e >= 0; --e)
                if (v[i].v[e] == mx) at = i * kThreads * 8 + e;
        u64 k = at + tid * 8 < left ? key_of(mx, (uint32_t)(c0 + at + tid * 8)) : 0;
        k = max_key(k, __shfl_xor(k, 1));
        k = max_key(k, __shfl_xor(k, 2));
        if ((tid & 3) == 0) gkey[tid >> 2] = k;
        if (tid == 0) ncand = 0;
    }
    mx = wave_max(mx);
    if ((tid & 63) == 0) redf[0][wave] = mx;
    __syncthreads();
    mx = redf[0][0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) mx = fmaxf(mx, redf[0][i]);
    if (TOP && tid < kGroups) {
        const u64 k = gkey[tid];
        int larger = 0;
        for (int i = 0; i < kGroups; ++i) larger += gkey[i] > k || (gkey[i] == k && i < tid);
        if (larger == top - 1) thr_s = k;
    }
    // e^d with d = x - mx; d is held above the fp32 underflow of e^d so that 0 d is 0
    const float base = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f, a = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = fmaxf((v[i].v[e] - base) * kLog2e, -200.0f);
            const float ex = __builtin_amdgcn_exp2f(d);
            l += ex;
            a = fmaf(ex, d, a);
        }
    l = wave_sum(l);
    a = wave_sum(a);
    if ((tid & 63) == 0) {
        redf[1][wave] = l;
        redf[2][wave] = a;
    }
    __syncthreads();
    if (tid == 0) {
        l = a = 0.0f;
        for (int i = 0; i < kThreads / 64; ++i) {
            l += redf[1][i];
            a += redf[2][i];
        }
        float *o = stats + (int64_t)blockIdx.x * 4;
        o[0] = mx;
        o[1] = l;
        o[2] = a * kLn2;
    }
    if (!TOP) return;
    const u64 thr = thr_s;
    const float thr_v = key_value(thr);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = (i * kThreads + tid) * 8 + e;
            if (v[i].v[e] >= thr_v || thr == 0) {
                const u64 k = key_of(v[i].v[e], (uint32_t)(c0 + c));
                if (k >= thr && c < left) cand[atomicAdd(&ncand, 1)] = k;
            }
        }
    __syncthreads();
    const int n = ncand;
    u64 *out = best + (int64_t)blockIdx.x * top;
    for (int i = tid; i < n; i += kThreads) {
        const u64 k = cand[i];
        int larger = 0;
        for (int j = 0; j < n; ++j) larger += cand[j] > k;
        if (larger < top) out[larger] = k;
    }
    for (int i = n + tid; i < top; i += kThreads) out[i] = 0;  // fewer elements than asked for
}

// One wave a row: the chunks' sums against the row's maximum, lane i holding
// chunk i, and the chunks' best lists (descending) merged from their heads.
template <typename T>
__global__ __launch_bounds__(64) void logprob_join_kernel(const T *__restrict__ x, int64_t V, int64_t ld, int chunks,
                                                          const float *__restrict__ stats, const u64 *__restrict__ best,
                                                          int top, const int64_t *__restrict__ targets,
                                                          float *__restrict__ logp, float *__restrict__ entropy,
                                                          float *__restrict__ lse_out, float *__restrict__ top_logp,
                                                          int32_t *__restrict__ top_ids) {
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x;
    const bool mine = lane < chunks;
    const float *s = stats + (row * chunks + lane) * 4;
    const float m = mine ? s[0] : -INFINITY, mx = wave_max(m), base = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f, a = 0.0f;
    if (mine && m > -INFINITY) {
        const float d = fmaxf(m - base, -150.0f), f = expf(d);
        l = s[1] * f;
        a = (s[2] + s[1] * d) * f;
    }
    l = wave_sum(l);
    a = wave_sum(a);
    const bool none = mx == -INFINITY;
    const float log_l = logf(l), lse = none ? -INFINITY : base + log_l;
    if (lane == 0) {
        if (lse_out) lse_out[row] = lse;
        if (entropy) entropy[row] = none ? 0.0f : log_l - a / l;
        if (logp) {
            const int64_t t = targets[row];
            logp[row] = t < 0 || t >= V ? 0.0f : none ? -INFINITY : load1(x + row * ld + t) - base - log_l;
        }
    }
    if (top == 0) return;
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
            top_logp[row * top + i] = none ? -INFINITY : key_value(k) - base - log_l;
            top_ids[row * top + i] = (int32_t)key_index(k);
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
    float scale = 1.0f, log_s = 0.0f;  // p = scale e^(x - lse), log p = x - lse - log_s
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
        const int64_t c0 = chunk * len, left = V - c0 < len ? V - c0 : len;
        const int hot = has && t >= c0 && t < c0 + left ? (int)(t - c0) : -1;
        F8 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = (i * kThreads + threadIdx.x) * 8;
            v[i] = load8(xr + c0 + c, left - c);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = (i * kThreads + threadIdx.x) * 8;
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

size_t logprob_stats_bytes(int64_t M, int64_t V) { return sizeof(float) * 4 * (size_t)M * cut_of(V).chunks; }
size_t logprob_best_bytes(int64_t M, int64_t V, int top) { return sizeof(u64) * (size_t)top * (size_t)M * cut_of(V).chunks; }
int64_t logprob_groups(int64_t M, int64_t V) { return M * cut_of(V).chunks; }

hipError_t launch_logprob_fwd(const void *x, bool f32, int64_t M, int64_t V, int64_t ld, const int64_t *targets,
                              int top, float *logp, float *entropy, float *lse, float *top_logp, int32_t *top_ids,
                              float *stats, void *best, hipStream_t s) {
    const Cut cut = cut_of(V);
    const unsigned groups = (unsigned)(M * cut.chunks);
    auto run = [&](auto *p) {
        using T = std::remove_pointer_t<decltype(p)>;
        if (top > 0)
            logprob_chunk_kernel<T, true>
                <<<groups, kThreads, 0, s>>>((const T *)x, V, ld, cut.chunks, cut.len, top, stats, (u64 *)best);
        else
            logprob_chunk_kernel<T, false>
                <<<groups, kThreads, 0, s>>>((const T *)x, V, ld, cut.chunks, cut.len, 0, stats, (u64 *)best);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        logprob_join_kernel<T><<<(unsigned)M, 64, 0, s>>>((const T *)x, V, ld, cut.chunks, stats, (const u64 *)best, top,
                                                          targets, logp, entropy, lse, top_logp, top_ids);
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

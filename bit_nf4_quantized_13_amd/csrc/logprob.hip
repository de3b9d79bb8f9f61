// Token log-probabilities over rows of logits x [M x V], and their gradient:
//   lse = log sum_v e^x_v       logp = x_t - lse       p = e^(x - lse)
//   H = -sum_v p_v log p_v = log l - (sum_v e^d_v d_v) / l,  d = x - max x, l = sum e^d
//   the `top` largest x, equal ones in ascending order of index
//   dx_v = g (delta_vt - p_v) - h p_v (log p_v + H)      g, h the gradients of logp and H
// A logit of -inf is a forbidden token: p = 0, no part in H, gradient 0 (g if it is the target).  A row
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
// e^d d) and groups' maxima go to the workspace, and a wave a row joins them in
// chunk order in a second launch; of few rows, one of up to 32768 elements is a
// workgroup's of 1024 threads, which writes its results.
//
// The best `top`: keys order value and index in 64 bits, all distinct.  A group of
// 8 threads (2 where a thread has 8 elements) owns up to 256 in a row; the top-th
// best of these groups by (maximum, then place) bounds the candidates: an element
// below its maximum, or equal to it in a later group, has top better ones.  So at
// most top 256 elements remain, usually some dozen (the join reads their groups
// again, 0.1 to 1 % of the row); they are collected in LDS and each counts the larger
// ones (of thousands of equal ones, the best are taken one by one).
//
// Measured, bf16: 2048 x 131071 with 8 alternatives 94 + 11 us for 537 MB (the first
// kernel 5.7 TB/s; 142 + 9 with the chunks' own search for them); one row of 32000 with 5
// alternatives 8.0 us; gradient of 4096 x 32000 81 to 92 us for 524 MB.
#include "elem8.hpp"
#include "launch.hpp"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;                     // of a chunk, and of the gradient
constexpr int kRowThreads = 1024;                 // of a whole row
constexpr int64_t kLaunchGroups = 1 << 23;        // workgroups of a launch: its threads stay below 2^32
constexpr int kVecs = 4;                          // groups of 8 a thread
constexpr int kHeld = kVecs * 8;                  // elements a thread
constexpr int kChunk = kThreads * kHeld;          // 8192
constexpr int64_t kWholeRow = kRowThreads * kHeld;  // 32768
constexpr int kGroupElems = 256;                  // most elements of a group
constexpr int kChunkGroups = kThreads / 8;        // of a chunk, when its row's best are looked for
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
// The target's logit, asked for before the row's sums are known.
struct Target {
    bool has;
    float x;
};
template <typename T>
__device__ __forceinline__ Target target_of(const RowOut &o, int64_t row, const T *xr, int64_t V) {
    const int64_t t = o.logp ? o.targets[row] : -1;
    const bool has = t >= 0 && t < V;
    return Target{has, load1(xr + (has ? t : 0))};
}
__device__ __forceinline__ void write_row(const RowOut &o, int64_t row, const Target &t, float mx, float base, float l,
                                          float a) {
    const bool none = none_left(mx, l);
    const float log_l = logf(l);
    if (o.lse) o.lse[row] = none ? -INFINITY : base + log_l;
    if (o.entropy) o.entropy[row] = none ? 0.0f : log_l - a / l;
    if (o.logp) o.logp[row] = !t.has ? 0.0f : none ? -INFINITY : t.x - base - log_l;
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

// One piece of a row.  ROW: the whole row, its results to `out` (LDS beyond the static:
// top kCandBytes); otherwise chunk blockIdx.x % chunks of row blockIdx.x / chunks, its
// sums to stats and its groups' maxima.
template <typename T, bool TOP, int THREADS, bool ROW>
__global__ __launch_bounds__(THREADS) void logprob_piece_kernel(const T *__restrict__ x, int64_t V, int64_t ld,
                                                                int chunks, int64_t len, int top,
                                                                float *__restrict__ stats, float *__restrict__ maxima,
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
    const int nv = (int)((len + THREADS * 8 - 1) / (THREADS * 8)), gt = nv == 1 ? 2 : 8, gshift = nv == 1 ? 1 : 3;
    const int group = tid >> gshift, per = 8 * nv * gt, groups = (left + per - 1) / per;
    const int first = group * per + (tid & (gt - 1)) * 8, step = 8 * gt;
    F8 v[kVecs];
    float vmax[kVecs], mx = -INFINITY;
    auto at = [&](int i) { return i < nv ? first + i * step : left; };
    RowLoad<T, kVecs> in_flight;
    in_flight.request(xr, left, at);
    Target target{};
    if (ROW && tid == 0) target = target_of(out, row, xr, V);
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
        if ((tid & (gt - 1)) == 0) {
            if (ROW) gmax[group] = g;
            else maxima[(int64_t)blockIdx.x * kChunkGroups + group] = g;
        }
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
    if (TOP && ROW && tid < groups && groups >= top) {
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
            write_row(out, row, target, mx, base, l, a);
        } else {
            float *o = stats + (int64_t)blockIdx.x * 4;
            o[0] = mx;
            o[1] = l;
            o[2] = a;
        }
    }
    if (!TOP || !ROW) return;
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
    for (int i = tid; i < 8 * nvec; i += THREADS) {
        const float x1 = vals[i];
        const int c = at_c[i >> 3] + (i & 7);
        if (c < left && (all ? x1 == x1 : x1 >= thr)) cand[atomicAdd(&ncand, 1)] = key_of(x1, (uint32_t)(c0 + c));  // no NaN
    }
    __syncthreads();
    const int n = ncand;
    const float log_l = logf(l);
    auto place = [&](int rank, u64 k) {
        out.top_logp[row * top + rank] = none_left(mx, l) ? -INFINITY : key_value(k) - base - log_l;
        out.top_ids[row * top + rank] = (int32_t)key_index(k);
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
    for (int i = n + tid; i < top; i += THREADS) place(i, 0);  // NaN are none
}

// Four consecutive elements as they are in memory.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
__device__ __forceinline__ u32x2 raw4(const uint16_t *p) { return *reinterpret_cast<const u32x2_any *>(p); }
__device__ __forceinline__ u32x4 raw4(const float *p) { return *reinterpret_cast<const u32x4_any *>(p); }
__device__ __forceinline__ f32x4 widen4(u32x2 w) {
    return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                 __uint_as_float(w[1] & 0xFFFF0000u)};
}
__device__ __forceinline__ f32x4 widen4(u32x4 w) { return __builtin_bit_cast(f32x4, w); }

// Largest over the wave, on every lane, without a trip through LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = dpp_max<0x111, 0xF>(v);  // the steps of wave_max
    v = dpp_max<0x112, 0xF>(v);
    v = dpp_max<0x114, 0xF>(v);
    v = dpp_max<0x118, 0xF>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ u64 wave_max_key(u64 k) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) k = max_key(k, __shfl_xor(k, o));
    return k;
}

// One wave a row: the chunks' sums against the row's maximum, lane i holding
// chunk i.  The best MOST at most (0: none are asked for): the top best groups by
// (maximum, then place), KEYS a lane, hold them; these groups, 4 elements a lane
// each, are read again.  LDS: top kGroupElems keys.
template <typename T, int KEYS, int MOST>
__global__ __launch_bounds__(64) void logprob_join_kernel(const T *__restrict__ x, int64_t V, int64_t ld, int chunks,
                                                          int64_t len, const float *__restrict__ stats,
                                                          const float *__restrict__ maxima, int top, RowOut out) {
    extern __shared__ __attribute__((aligned(16))) u64 cand[];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x;
    const T *xr = x + row * ld;
    const Target target = target_of(out, row, xr, V);
    const int total = chunks * kChunkGroups;
    float g[KEYS];
    if (MOST > 0) {
        const float *gm = maxima + row * total;
#pragma unroll
        for (int i = 0; i < KEYS; ++i) g[i] = gm[min(i * 64 + lane, total - 1)];
    }
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
    if (lane == 0) write_row(out, row, target, mx, base, l, a);
    if (MOST > 0 && none_left(mx, l)) {  // all equal: the lowest indices, without the search
        if (lane < top) {
            out.top_logp[row * top + lane] = -INFINITY;
            out.top_ids[row * top + lane] = lane;
        }
    } else if constexpr (MOST > 0) {
        const int per = (int)((len + kThreads * 8 - 1) / (kThreads * 8)) * 64;
        uint32_t up[KEYS];  // ascending with the maximum; 0: no group, or taken
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int n = i * 64 + lane, c = n / kChunkGroups, first = n % kChunkGroups * per;
            up[i] = n < total && c * len + first < V && first < len ? (uint32_t)(key_of(g[i], 0) >> 32) : 0;
        }
        uint32_t best = 0;
        int chosen = 0, number = 0;  // lane i: the i-th best group
        for (int i = 0; i < top; ++i) {
            uint32_t own = 0, place = 0;
#pragma unroll
            for (int j = 0; j < KEYS; ++j) own = up[j] > own ? up[j] : own;
            own = wave_max_u32(own);
            if (own == 0) break;
            best = own;
#pragma unroll
            for (int j = KEYS - 1; j >= 0; --j) place = up[j] == best ? ~(uint32_t)(j * 64 + lane) : place;
            place = ~wave_max_u32(place);  // the first of equal ones
#pragma unroll
            for (int j = 0; j < KEYS; ++j) up[j] = j * 64 + lane == (int)place ? 0 : up[j];
            if (lane == i) chosen = (int)place;
            ++number;
        }
        const float thr = number < top ? -INFINITY : key_value((u64)best << 32);  // fewer groups than places: all count
        decltype(raw4((const T *)nullptr)) raw[MOST];
        int at[MOST], left[MOST];
        int64_t c0[MOST];
#pragma unroll
        for (int i = 0; i < MOST; ++i) {  // all requested before the first is used
            const int n = __builtin_amdgcn_readlane(chosen, i < number ? i : 0), c = n / kChunkGroups;
            c0[i] = c * len;
            left[i] = (int)(V - c0[i] < len ? V - c0[i] : len);
            at[i] = n % kChunkGroups * per + lane * 4;
            raw[i] = raw4(xr + c0[i] + min(at[i], left[i] - 4));  // a chunk has thousands of elements
        }
        int n = 0;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            if (i >= number) continue;
            f32x4 v = widen4(raw[i]);
            const bool cut = at[i] + 4 > left[i];
            if (__ballot(cut) && cut) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = at[i] + e < left[i] ? load1(xr + c0[i] + at[i] + e) : NAN;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = v[e] >= thr && lane * 4 < per;
                const u64 who = __ballot(in);
                if (who == 0) continue;
                if (in) cand[n + __popcll(who & (((u64)1 << lane) - 1))] = key_of(v[e], (uint32_t)(c0[i] + at[i] + e));
                n += __popcll(who);
            }
        }
        __syncthreads();
        const float log_l = logf(l);
        auto place = [&](int rank, u64 k) {
            out.top_logp[row * top + rank] = key_value(k) - base - log_l;
            out.top_ids[row * top + rank] = (int32_t)key_index(k);
        };
        if (n <= 64) {
            const u64 k = lane < n ? cand[lane] : 0;
            int larger = 0;
            for (int j = 0; j < n; ++j) larger += cand[j] > k;
            if (lane < n && larger < top) place(larger, k);
        } else {  // many equal logits: one after the other, each the largest below the last
            u64 last = ~(u64)0;
            for (int i = 0; i < top; ++i) {
                u64 k = 0;
#pragma unroll 8
                for (int j = lane; j < n; j += 64) k = cand[j] < last ? max_key(k, cand[j]) : k;
                last = wave_max_key(k);
                if (lane == 0) place(i, last);
            }
        }
        for (int i = n + lane; i < top; i += 64) place(i, 0);  // NaN are none
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
// and longer ones where there are no more of them than CUs (bf16, 32000 logits, 5 alternatives: one
// row 8.7 us against 9.3, 256 rows 9.6 against 11.9); with more, the chunks' smaller
// workgroups overlap better (512 rows 15.2 against 18.0, 4096 rows 57 against 128).
bool whole_rows(int64_t M, int64_t V) { return V <= kChunk || (M <= 256 && V <= kWholeRow); }

size_t logprob_stats_bytes(int64_t M, int64_t V) {
    return whole_rows(M, V) ? 0 : sizeof(float) * 4 * (size_t)M * cut_of(V).chunks;
}
size_t logprob_best_bytes(int64_t M, int64_t V, int top) {
    return whole_rows(M, V) || top == 0 ? 0 : sizeof(float) * kChunkGroups * (size_t)M * cut_of(V).chunks;
}
int64_t logprob_groups(int64_t M, int64_t V) { return M * cut_of(V).chunks; }

hipError_t launch_logprob_fwd(const void *x, bool f32, int64_t M, int64_t V, int64_t ld, const int64_t *targets,
                              int top, float *logp, float *entropy, float *lse, float *top_logp, int32_t *top_ids,
                              float *stats, void *best, hipStream_t s) {
    const bool whole = whole_rows(M, V), small = V <= kChunk;
    const Cut cut = whole ? Cut{1, V} : cut_of(V);
    auto run = [&](auto *p) {
        using T = std::remove_pointer_t<decltype(p)>;
        auto *kernel = whole ? small ? top > 0 ? logprob_piece_kernel<T, true, kThreads, true>
                                               : logprob_piece_kernel<T, false, kThreads, true>
                               : top > 0 ? logprob_piece_kernel<T, true, kRowThreads, true>
                                         : logprob_piece_kernel<T, false, kRowThreads, true>
                       : top > 0 ? logprob_piece_kernel<T, true, kThreads, false>
                                 : logprob_piece_kernel<T, false, kThreads, false>;
        const bool wide = cut.chunks > 16;
        auto *join = top == 0   ? logprob_join_kernel<T, 1, 0>
                     : top <= 8 ? wide ? logprob_join_kernel<T, 32, 8> : logprob_join_kernel<T, 8, 8>
                                : wide ? logprob_join_kernel<T, 32, 16> : logprob_join_kernel<T, 8, 16>;
        const int threads = whole && !small ? kRowThreads : kThreads;
        const size_t lds = whole ? (size_t)top * kCandBytes : 0;  // up to 50 KiB
        const int64_t most = kLaunchGroups / cut.chunks;          // rows of a launch
        for (int64_t r = 0; r < M; r += most) {
            const unsigned rows = (unsigned)(M - r < most ? M - r : most);
            const T *xr = (const T *)x + r * ld;
            auto from = [&](auto *q, int64_t each) { return q ? q + r * each : nullptr; };
            const RowOut out{from(targets, 1), from(logp, 1), from(entropy, 1), from(lse, 1), from(top_logp, top), from(top_ids, top)};
            kernel<<<rows * cut.chunks, threads, lds, s>>>(xr, V, ld, cut.chunks, cut.len, top, stats, (float *)best, out);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            if (whole) continue;
            join<<<rows, 64, sizeof(u64) * kGroupElems * (size_t)top, s>>>(xr, V, ld, cut.chunks, cut.len, stats,
                                                                          (const float *)best, top, out);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    return f32 ? run((float *)nullptr) : run((uint16_t *)nullptr);
}

hipError_t launch_logprob_bwd(const void *x, bool f32, int64_t M, int64_t V, int64_t ld, const int64_t *targets,
                              const float *lse, const float *entropy, const float *dlogp, const float *dent, void *dx,
                              int64_t ldd, hipStream_t s) {
    const Cut cut = cut_of(V);
    const int split = x == dx ? 1 : cut.chunks;
    const int64_t most = kLaunchGroups / split;  // rows of a launch
    auto run = [&](auto *p) {
        using T = std::remove_pointer_t<decltype(p)>;
        for (int64_t r = 0; r < M; r += most) {
            const unsigned rows = (unsigned)(M - r < most ? M - r : most);
            auto from = [&](auto *q) { return q ? q + r : nullptr; };
            logprob_bwd_kernel<T><<<rows * split, kThreads, 0, s>>>((const T *)x + r * ld, V, ld, split, cut.chunks, cut.len,
                                                                   from(targets), lse + r, from(entropy), from(dlogp),
                                                                   from(dent), (T *)dx + r * ldd, ldd);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    return f32 ? run((float *)nullptr) : run((uint16_t *)nullptr);
}

}  // namespace qnf4

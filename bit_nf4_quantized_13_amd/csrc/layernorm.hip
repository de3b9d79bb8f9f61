// Layer norm over the rows of x [M x n], and its backward:
//   mu = sum(x) / n      rstd = (sum((x - mu)^2) / n + eps)^-1/2
//   y  = (x - mu) rstd w + b
//   xh = (x - mu) rstd   g = dy w
//   dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh      db = sum over rows of dy
//
// Statistics and sums in fp32 whatever x's type: mu first, then the squares of
// the deviations from it (both from registers), so a row whose mean is far
// larger than its spread keeps its variance; one rounding at the store.
//
// Bound: HBM (8 to 14 flops an element).  x (and dy) are read once and held in
// registers over the reductions: a row is spread over TPR threads of 8 elements
// each, TPR the smallest that holds n (16 lanes up to 128 columns: 131072 x 128 forward
// 15 us, 42 with a wave a row); 256 threads take 256 / TPR rows at a time.
// Rows wider than kMaxHeld go through a kernel that reads them again for each
// reduction, from L2 (a thread with 16 elements held is slower: 4096 x 12288
// forward 62 us against 44, backward 72 against 69).
//
// dw and db add over all rows: a workgroup of up to 1024 threads walks the rows
// with its columns' sums in registers, adds its row groups' sums in LDS and
// writes one partial row, and a second kernel adds the partial rows: fixed
// orders, so the same bits on every run.  For rows wider than kMaxHeld a kernel
// of its own reads x and dy by columns (4096 x 6144: 43 us in one pass, 64 in two).
//
// Measured: 4096 x 8192 bf16 with dw and db 37 + 4.9 us for 201 MB (5.4 TB/s in
// the main kernel; a copy reaches 5.2); 1531 x 2753 fp32 dx alone 11.2 us for 51 MB; one row
// of 4096 forward 2.4 us.
#include "elem8.hpp"
#include "launch.hpp"

namespace qnf4 {
namespace {

constexpr int64_t kMaxHeld = 8192;     // widest row held in registers
constexpr int kGradThreads = 1024;     // workgroup of the backward with parameter gradients
constexpr int kMaxPartials = 256;      // its partial rows: one workgroup a CU (128: 8192 x 4096 58 us against 43)
// The backward without them: workgroups that walk over rows as well, the next row's loads
// under way (8192 x 4096 bf16: 34 us; a workgroup a row 45), two a CU.  The forward, with one load
// less to wait for, is as fast or faster with a workgroup a row (4096 x 8192: 29 us against 35).
constexpr int kRowThreads = 512;
constexpr int kMaxRowGroups = 512;
constexpr int64_t kLaunchRows = 1 << 21;  // of a launch with a workgroup a row: its threads stay below 2^32
constexpr int kStreamThreads = 1024;   // workgroup of a row wider than kMaxHeld

// Sum of v over the 16 or 32 lanes of a row group, or over the wave, on every lane:
// 16 lanes by rotations within them.
template <int TPR>
__device__ __forceinline__ float lanes_sum(float v) {
    if (TPR >= 64) return wave_sum(v);
    v += dpp_or<0x128, 0xF>(v, v);
    v += dpp_or<0x124, 0xF>(v, v);
    v += dpp_or<0x122, 0xF>(v, v);
    v += dpp_or<0x121, 0xF>(v, v);
    if (TPR == 32) v += __shfl_xor(v, 16);
    return v;
}

// Sum of v over the TPR threads of a row group (16, 32 or a multiple of 64); every
// thread of the workgroup calls it.  red: one float for each wave, not written
// again before another barrier.
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float *red) {
    v = lanes_sum<TPR>(v);
    if (TPR <= 64) return v;
    const int wave = threadIdx.x >> 6, w0 = threadIdx.x / TPR * (TPR / 64);
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) s += red[w0 + i];
    return s;
}

template <typename T>
__device__ __forceinline__ F8 param8(const T *p, int64_t c, int64_t n, float fill) {
    F8 r;
    if (p) return load8(p + c, n - c, fill);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = fill;
    return r;
}

template <typename T, typename W, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(
    const T *__restrict__ x, int64_t M, int64_t n, int64_t ldx, const W *__restrict__ w, const W *__restrict__ b,
    float eps, T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd) {
    constexpr int kThreads = TPR > 256 ? TPR : 256;
    __shared__ float red[2][kThreads / 64];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    const bool live = row < M;
    const float inv_n = 1.0f / (float)n;
    const int len = (int)n, c = t * 8;
    const T *xr = x + (live ? row : 0) * ldx;
    auto at = [&](int) { return c; };
    RowLoad<T, 1> xl;
    RowLoad<W, 1> wl, bl;
    xl.request(xr, len, at);
    if (w) wl.request(w, len, at);
    if (b) bl.request(b, len, at);
    F8 v = xl.get(xr, len, at, 0);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v.v[e];
    const float mu = group_sum<TPR>(s, red[0]) * inv_n;
    float q = 0.0f;
    if (c < len) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v.v[e] -= mu;
            if (c + 8 <= len || c + e < len) q += v.v[e] * v.v[e];
        }
    }
    const float rs = 1.0f / sqrtf(group_sum<TPR>(q, red[1]) * inv_n + eps);
    if (!live) return;
    if (t == 0 && mean) mean[row] = mu;
    if (t == 0 && rstd) rstd[row] = rs;
    if (c >= len) return;
    F8 wv, bv;
    if (w) wv = wl.get(w, len, at, 0);
    if (b) bv = bl.get(b, len, at, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] = v.v[e] * rs * (w ? wv.v[e] : 1.0f) + (b ? bv.v[e] : 0.0f);
    store8(y + row * n + c, n - c, v);
}

// Rows wider than the registers hold: one workgroup a row, read three times.
template <typename T, typename W>
__global__ __launch_bounds__(kStreamThreads) void norm_fwd_stream_kernel(
    const T *__restrict__ x, int64_t n, int64_t ldx, const W *__restrict__ w, const W *__restrict__ b, float eps,
    T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd) {
    __shared__ float red[2][kStreamThreads / 64];
    const int64_t row = blockIdx.x;
    const T *xr = x + row * ldx;
    const float inv_n = 1.0f / (float)n;
    float s = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < n; c += kStreamThreads * 8) {
        const F8 v = load8(xr + c, n - c);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v.v[e];
    }
    const float mu = group_sum<kStreamThreads>(s, red[0]) * inv_n;
    float q = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < n; c += kStreamThreads * 8) {
        const F8 v = load8(xr + c, n - c, mu);
#pragma unroll
        for (int e = 0; e < 8; ++e) q += (v.v[e] - mu) * (v.v[e] - mu);
    }
    const float rs = 1.0f / sqrtf(group_sum<kStreamThreads>(q, red[1]) * inv_n + eps);
    if (threadIdx.x == 0 && mean) mean[row] = mu;
    if (threadIdx.x == 0 && rstd) rstd[row] = rs;
    for (int64_t c = threadIdx.x * 8; c < n; c += kStreamThreads * 8) {
        F8 v = load8(xr + c, n - c);
        const F8 wv = param8(w, c, n, 1.0f), bv = param8(b, c, n, 0.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = (v.v[e] - mu) * rs * wv.v[e] + bv.v[e];
        store8(y + row * n + c, n - c, v);
    }
}

// dX (which may be written over dy), and with GRAD the workgroup's partial row of dw and db ([2][n] at
// part + blockIdx.x 2 n).  Row group g of the workgroup takes the rows
// blockIdx.x GROUPS + g, then every gridDim.x GROUPS-th.
template <typename T, typename W, int THREADS, int TPR, bool GRAD>
__global__ __launch_bounds__(THREADS) void norm_bwd_kernel(
    const T *__restrict__ x, const T *dy, int64_t M, int64_t n, int64_t ldx,
    const float *__restrict__ mean, const float *__restrict__ rstd, const W *__restrict__ w, T *dx,
    float *__restrict__ part, float *__restrict__ dweight, float *__restrict__ dbias) {
    constexpr int kGroups = THREADS / TPR, kWavesRow = TPR / 64;
    __shared__ float red[2][2][THREADS / 64];  // of the two sums, in turn from one pass over the rows to the next
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const int len = (int)n, c = t * 8;
    const float inv_n = 1.0f / (float)n;
    auto at = [&](int) { return c; };
    RowLoad<W, 1> wl;  // the weight stays in registers
    if (w) wl.request(w, len, at);
    F8 dw, db;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw.v[e] = db.v[e] = 0.0f;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    RowLoad<T, 1> xl, yl;
    float mu, rs;
    auto request = [&](int64_t row) {
        const int64_t r = row < M ? row : 0;
        xl.request(x + r * ldx, len, at);
        yl.request(dy + r * n, len, at);
        mu = mean[r];
        rs = rstd[r];
    };
    request((int64_t)blockIdx.x * kGroups + g);
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < M; r0 += step, turn ^= 1) {
        const int64_t row = r0 + g;
        const bool live = row < M;
        float s1 = 0.0f, s2 = 0.0f;
        const float rs0 = rs;
        F8 xh = xl.get(x + (live ? row : 0) * ldx, len, at, 0, mu), gr = yl.get(dy + (live ? row : 0) * n, len, at, 0), wv;
        if (w) wv = wl.get(w, len, at, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float h = (xh.v[e] - mu) * rs, d = live ? gr.v[e] : 0.0f;
            if (GRAD) {
                dw.v[e] += d * h;
                db.v[e] += d;
            }
            xh.v[e] = h;
            gr.v[e] = w ? d * wv.v[e] : d;
            s1 += gr.v[e];
            s2 += gr.v[e] * h;
        }
        // the rows of the next pass are requested before this one's sums are waited for
        if (r0 + step < M) request(row + step);
        s1 = lanes_sum<TPR>(s1);
        s2 = lanes_sum<TPR>(s2);
        if (TPR > 64) {
            const int wave = threadIdx.x >> 6, w0 = g * kWavesRow;
            if ((threadIdx.x & 63) == 0) {
                red[turn][0][wave] = s1;
                red[turn][1][wave] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < kWavesRow; ++i) {
                s1 += red[turn][0][w0 + i];
                s2 += red[turn][1][w0 + i];
            }
        }
        const float c1 = s1 * inv_n, c2 = s2 * inv_n;
        if (live && c < len) {
            F8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o.v[e] = rs0 * (gr.v[e] - c1 - xh.v[e] * c2);
            store8(dx + row * n + c, n - c, o);
        }
    }
    if (!GRAD) return;
    // the row groups' sums: those of one wave first, then the others' in order, by the
    // last one's threads (one after the other, each adding to LDS, cost 8 us a launch)
    constexpr int kSums = TPR < 64 ? THREADS / 64 : kGroups;
    const int sum = TPR < 64 ? threadIdx.x >> 6 : g;
#pragma unroll
    for (int o = TPR; o < 64; o *= 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw.v[e] += __shfl_xor(dw.v[e], o);
            db.v[e] += __shfl_xor(db.v[e], o);
        }
    }
    const bool holds = c < len && (TPR >= 64 || (threadIdx.x & 63) < TPR);
    extern __shared__ __attribute__((aligned(16))) float sums[];  // [kSums - 1][2][pitch]
    const int pitch = (len + 7) / 8 * 8;
    if (holds && sum + 1 < kSums) {
        f32x4 *to = reinterpret_cast<f32x4 *>(sums + sum * 2 * pitch + c);
        to[0] = f32x4{dw.v[0], dw.v[1], dw.v[2], dw.v[3]};
        to[1] = f32x4{dw.v[4], dw.v[5], dw.v[6], dw.v[7]};
        to += pitch / 4;
        to[0] = f32x4{db.v[0], db.v[1], db.v[2], db.v[3]};
        to[1] = f32x4{db.v[4], db.v[5], db.v[6], db.v[7]};
    }
    if (kSums > 1) __syncthreads();
    if (!holds || sum + 1 < kSums) return;
    f32x4 w0 = {}, w1 = {}, b0 = {}, b1 = {};
    // all 15 at once spill the 128 registers that 1024 threads have: 131072 x 128 29 us against 24, 64 x 128 8.3
    // against 5.8
#pragma unroll 4
    for (int k = 0; k + 1 < kSums; ++k) {
        const f32x4 *from = reinterpret_cast<const f32x4 *>(sums + k * 2 * pitch + c);
        w0 += from[0];
        w1 += from[1];
        b0 += from[pitch / 4];
        b1 += from[pitch / 4 + 1];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        dw.v[e] += w0[e];
        dw.v[4 + e] += w1[e];
        db.v[e] += b0[e];
        db.v[4 + e] += b1[e];
    }
    float *out_w = part + (int64_t)blockIdx.x * 2 * n, *out_b = out_w + n;
    if (gridDim.x == 1) {  // nothing to add to
        out_w = dweight;
        out_b = dbias;
    }
    if (out_w) store8(out_w + c, n - c, dw);
    if (out_b) store8(out_b + c, n - c, db);
}

// Wide rows' dX: one workgroup a row, read twice.
template <typename T, typename W>
__global__ __launch_bounds__(kStreamThreads) void norm_bwd_stream_kernel(
    const T *__restrict__ x, const T *dy, int64_t n, int64_t ldx, const float *__restrict__ mean,
    const float *__restrict__ rstd, const W *__restrict__ w, T *dx) {
    __shared__ float red1[kStreamThreads / 64], red2[kStreamThreads / 64];
    const int64_t row = blockIdx.x;
    const T *xr = x + row * ldx, *dr = dy + row * n;
    const float mu = mean[row], rs = rstd[row], inv_n = 1.0f / (float)n;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < n; c += kStreamThreads * 8) {
        const F8 xv = load8(xr + c, n - c, mu), dv = load8(dr + c, n - c), wv = param8(w, c, n, 1.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float gv = dv.v[e] * wv.v[e];
            s1 += gv;
            s2 += gv * ((xv.v[e] - mu) * rs);
        }
    }
    const float c1 = group_sum<kStreamThreads>(s1, red1) * inv_n, c2 = group_sum<kStreamThreads>(s2, red2) * inv_n;
    for (int64_t c = threadIdx.x * 8; c < n; c += kStreamThreads * 8) {
        const F8 xv = load8(xr + c, n - c, mu), dv = load8(dr + c, n - c), wv = param8(w, c, n, 1.0f);
        F8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = rs * (dv.v[e] * wv.v[e] - c1 - (xv.v[e] - mu) * rs * c2);
        store8(dx + row * n + c, n - c, o);
    }
}

// Wide rows' dw and db: a workgroup takes 8 columns a thread and every
// gridDim.y-th row, into partial row blockIdx.y.
template <typename T>
__global__ __launch_bounds__(256) void norm_cols_kernel(const T *__restrict__ x, const T *__restrict__ dy, int64_t M,
                                                        int64_t n, int64_t ldx, const float *__restrict__ mean,
                                                        const float *__restrict__ rstd, float *__restrict__ part) {
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= n) return;
    F8 dw, db;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw.v[e] = db.v[e] = 0.0f;
    for (int64_t row = blockIdx.y; row < M; row += gridDim.y) {
        const float mu = mean[row], rs = rstd[row];
        const F8 xv = load8(x + row * ldx + c, n - c), dv = load8(dy + row * n + c, n - c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw.v[e] += dv.v[e] * ((xv.v[e] - mu) * rs);
            db.v[e] += dv.v[e];
        }
    }
    float *out = part + (int64_t)blockIdx.y * 2 * n;
    store8(out + c, n - c, dw);
    store8(out + n + c, n - c, db);
}

// dw and db from the partial rows: 64 columns of [dw | db] a workgroup, its 16
// waves a sixteenth of the rows each, added in wave order.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float *__restrict__ part, int parts, int64_t n,
                                                           float *__restrict__ dw, float *__restrict__ db) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < 2 * n) {
        // kMaxPartials / 16 loads at once
        float v[kMaxPartials / 16];
#pragma unroll
        for (int i = 0; i < kMaxPartials / 16; ++i) v[i] = wave + 16 * i < parts ? part[(int64_t)(wave + 16 * i) * 2 * n + c] : 0.0f;
#pragma unroll
        for (int i = 0; i < kMaxPartials / 16; ++i) s += v[i];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= 2 * n) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sums[i][lane];
    if (c < n) {
        if (dw) dw[c] = s;
    } else if (db) {
        db[c - n] = s;
    }
}

// The threads a row of n takes, passed on as a template value.
template <typename F>
hipError_t held_shape(int64_t n, F f) {
    if (n <= 128) return f(std::integral_constant<int, 16>());
    if (n <= 256) return f(std::integral_constant<int, 32>());
    if (n <= 512) return f(std::integral_constant<int, 64>());
    if (n <= 1024) return f(std::integral_constant<int, 128>());
    if (n <= 2048) return f(std::integral_constant<int, 256>());
    if (n <= 4096) return f(std::integral_constant<int, 512>());
    if (n <= 6144) return f(std::integral_constant<int, 768>());
    return f(std::integral_constant<int, 1024>());
}

template <typename T, typename W>
hipError_t norm_fwd(const T *x, int64_t M, int64_t n, int64_t ldx, const W *w, const W *b, float eps, T *y,
                    float *mean, float *rstd, hipStream_t s) {
    if (n > kMaxHeld) {
        norm_fwd_stream_kernel<T, W><<<(unsigned)M, kStreamThreads, 0, s>>>(x, n, ldx, w, b, eps, y, mean, rstd);
        return hipGetLastError();
    }
    return held_shape(n, [&](auto tpr) {
        constexpr int kTpr = decltype(tpr)::value, kThreads = kTpr > 256 ? kTpr : 256, kRows = kThreads / kTpr;
        norm_fwd_kernel<T, W, kTpr>
            <<<(unsigned)((M + kRows - 1) / kRows), kThreads, 0, s>>>(x, M, n, ldx, w, b, eps, y, mean, rstd);
        return hipGetLastError();
    });
}

template <typename T, typename W>
hipError_t norm_bwd(const T *x, const T *dy, int64_t M, int64_t n, int64_t ldx, const float *mean, const float *rstd,
                    const W *w, T *dx, float *dw, float *db, float *part, hipStream_t s) {
    const bool grad = dw || db, fused = grad && n <= kMaxHeld;
    int parts = 0;
    hipError_t e;
    if (fused) {
        e = held_shape(n, [&](auto tpr) {
            constexpr int kTpr = decltype(tpr)::value, kThreads = kTpr > 512 ? kTpr : kGradThreads, kRows = kThreads / kTpr;
            const int64_t groups = (M + kRows - 1) / kRows;
            parts = groups < kMaxPartials ? (int)groups : kMaxPartials;
            constexpr int kSums = kTpr < 64 ? kThreads / 64 : kRows;
            const size_t lds = 2 * sizeof(float) * (size_t)(kSums - 1) * (size_t)((n + 7) / 8 * 8);  // up to 60 KiB
            norm_bwd_kernel<T, W, kThreads, kTpr, true>
                <<<parts, kThreads, lds, s>>>(x, dy, M, n, ldx, mean, rstd, w, dx, part, dw, db);
            return hipGetLastError();
        });
    } else if (n <= kMaxHeld) {
        e = held_shape(n, [&](auto tpr) {
            constexpr int kTpr = decltype(tpr)::value, kThreads = kTpr > kRowThreads ? kTpr : kRowThreads, kRows = kThreads / kTpr;
            const int64_t groups = (M + kRows - 1) / kRows;
            norm_bwd_kernel<T, W, kThreads, kTpr, false><<<(unsigned)(groups < kMaxRowGroups ? groups : kMaxRowGroups), kThreads, 0, s>>>(
                x, dy, M, n, ldx, mean, rstd, w, dx, nullptr, nullptr, nullptr);
            return hipGetLastError();
        });
    } else {
        e = hipSuccess;
        if (grad) {  // before dx, which may overwrite dy
            parts = M < kMaxPartials ? (int)M : kMaxPartials;
            norm_cols_kernel<T><<<dim3((unsigned)((n + 2047) / 2048), parts), 256, 0, s>>>(x, dy, M, n, ldx, mean, rstd, part);
            e = hipGetLastError();
        }
        for (int64_t r = 0; r < M && e == hipSuccess; r += kLaunchRows) {
            const int64_t rows = M - r < kLaunchRows ? M - r : kLaunchRows;
            norm_bwd_stream_kernel<T, W><<<(unsigned)rows, kStreamThreads, 0, s>>>(x + r * ldx, dy + r * n, n, ldx, mean + r, rstd + r,
                                                                                  w, dx + r * n);
            e = hipGetLastError();
        }
    }
    if (!grad || e != hipSuccess || (fused && parts == 1)) return e;
    norm_reduce_kernel<<<(unsigned)((2 * n + 63) / 64), 1024, 0, s>>>(part, parts, n, dw, db);
    return hipGetLastError();
}

// f with x's and the weight's element types.
template <typename F>
hipError_t typed(bool x_f32, bool w_f32, F f) {
    if (x_f32) return w_f32 ? f((float *)nullptr, (float *)nullptr) : f((float *)nullptr, (uint16_t *)nullptr);
    return w_f32 ? f((uint16_t *)nullptr, (float *)nullptr) : f((uint16_t *)nullptr, (uint16_t *)nullptr);
}

}  // namespace

size_t layernorm_part_bytes(int64_t M, int64_t n) {
    return sizeof(float) * 2 * (size_t)n * (size_t)(M < kMaxPartials ? M : kMaxPartials);
}

hipError_t launch_layernorm_fwd(const void *x, bool x_f32, int64_t M, int64_t n, int64_t ldx, const void *w,
                                const void *b, bool w_f32, float eps, void *y, float *mean, float *rstd,
                                hipStream_t s) {
    return typed(x_f32, w_f32, [&](auto *tx, auto *tw) {
        using T = std::remove_pointer_t<decltype(tx)>;
        using W = std::remove_pointer_t<decltype(tw)>;
        for (int64_t r = 0; r < M; r += kLaunchRows) {
            const hipError_t e = norm_fwd<T, W>((const T *)x + r * ldx, M - r < kLaunchRows ? M - r : kLaunchRows, n, ldx,
                                                (const W *)w, (const W *)b, eps, (T *)y + r * n, mean ? mean + r : nullptr,
                                                rstd ? rstd + r : nullptr, s);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    });
}

hipError_t launch_layernorm_bwd(const void *x, const void *dy, bool x_f32, int64_t M, int64_t n, int64_t ldx,
                                const float *mean, const float *rstd, const void *w, bool w_f32, void *dx, float *dw,
                                float *db, float *part, hipStream_t s) {
    return typed(x_f32, w_f32, [&](auto *tx, auto *tw) {
        using T = std::remove_pointer_t<decltype(tx)>;
        using W = std::remove_pointer_t<decltype(tw)>;
        return norm_bwd<T, W>((const T *)x, (const T *)dy, M, n, ldx, mean, rstd, (const W *)w, (T *)dx, dw, db, part, s);
    });
}

}  // namespace qnf4

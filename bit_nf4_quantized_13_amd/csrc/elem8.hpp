// Rows of bf16 or fp32 taken 8 consecutive elements at a time, widened to
// fp32.  A full group is read or written with 16-byte accesses at any element
// alignment (gfx950 takes unaligned global accesses; an odd row pitch or a
// view that starts mid-buffer needs no second code path).  Nothing outside the row
// is touched: the group that its end falls into is stored element by element, and
// read the same way or (RowLoad) as the row's last 8 elements.
#pragma once
#include "common.hpp"

namespace qnf4 {

// A 16-byte global access at the alignment of the element.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

struct F8 {
    float v[8];
};

__device__ __forceinline__ void unpack8(u32x4 w, float *v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ F8 load8(const uint16_t *p) {
    F8 r;
    unpack8(*reinterpret_cast<const u32x4_any *>(p), r.v);
    return r;
}
__device__ __forceinline__ F8 load8(const float *p) {
    const u32x4 a = *reinterpret_cast<const u32x4_any *>(p), b = *reinterpret_cast<const u32x4_any *>(p + 4);
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[i] = __uint_as_float(a[i]);
        r.v[4 + i] = __uint_as_float(b[i]);
    }
    return r;
}

__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float load1(const float *p) { return *p; }

// A group as it is in memory: its load can be under way while others are issued.
struct Raw16 {
    u32x4 w;
};
struct Raw32 {
    u32x4 w[2];
};
__device__ __forceinline__ Raw16 raw8(const uint16_t *p) { return Raw16{*reinterpret_cast<const u32x4_any *>(p)}; }
__device__ __forceinline__ Raw32 raw8(const float *p) {
    Raw32 r;
    r.w[0] = *reinterpret_cast<const u32x4_any *>(p);
    r.w[1] = *reinterpret_cast<const u32x4_any *>(p + 4);
    return r;
}
__device__ __forceinline__ F8 widen(const Raw16 &r) {
    F8 f;
    unpack8(r.w, f.v);
    return f;
}
__device__ __forceinline__ F8 widen(const Raw32 &r) {
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.v[i] = __uint_as_float(r.w[0][i]);
        f.v[4 + i] = __uint_as_float(r.w[1][i]);
    }
    return f;
}
template <typename T>
using RawOf = decltype(raw8((const T *)nullptr));

// A group moved down by k elements, 0 <= k <= 8.
__device__ __forceinline__ Raw16 moved(const Raw16 &r, int k) {
    uint64_t lo = r.w[0] | (uint64_t)r.w[1] << 32, hi = r.w[2] | (uint64_t)r.w[3] << 32;
    if (k & 4) {
        lo = hi;
        hi = 0;
    }
    const int s = 16 * (k & 3);
    lo = lo >> s | (hi << 1) << (63 - s);
    hi >>= s;
    return Raw16{u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)}};
}
__device__ __forceinline__ Raw32 moved(Raw32 r, int k) {
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) {
        if (!(k & s)) continue;
#pragma unroll
        for (int i = 0; i + s < 8; ++i) r.w[i >> 2][i & 3] = r.w[(i + s) >> 2][(i + s) & 3];
    }
    return r;
}

// N groups of a row of n elements, group i at element at(i): all are requested
// before the first is used, each whole and inside the row; the one that would
// cross the row's end takes the row's last 8 elements and moves them down.
// `fill` past the end.
template <typename T, int N>
struct RowLoad {
    RawOf<T> r[N];
    template <typename At>
    __device__ __forceinline__ void request(const T *row, int n, At at) {
        if (n < 8) return;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = raw8(row + (at(i) + 8 <= n ? at(i) : n - 8));
    }
    template <typename At>
    __device__ __forceinline__ F8 get(const T *row, int n, At at, int i, float fill = 0.0f) const {
        const int c = at(i), left = n - c;
        F8 f;
        if (n < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] = e < left ? load1(row + c + e) : fill;
            return f;
        }
        f = widen(r[i]);
        if (__ballot(left < 8)) {  // only the wave that the row's end falls into
            const F8 g = widen(moved(r[i], left > 0 && left < 8 ? 8 - left : 0));
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] = e < left ? g.v[e] : fill;
        }
        return f;
    }
};

// The first cnt elements from p (any cnt; none for cnt <= 0), `fill` beyond.
template <typename T>
__device__ __forceinline__ F8 load8(const T *p, int64_t cnt, float fill = 0.0f) {
    if (cnt >= 8) return load8(p);
    F8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < cnt ? load1(p + i) : fill;
    return r;
}

__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

__device__ __forceinline__ void store8(uint16_t *p, const F8 &r) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(r.v[2 * i], r.v[2 * i + 1]);
    *reinterpret_cast<u32x4_any *>(p) = w;
}
__device__ __forceinline__ void store8(float *p, const F8 &r) {
    u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = __float_as_uint(r.v[i]);
        b[i] = __float_as_uint(r.v[4 + i]);
    }
    *reinterpret_cast<u32x4_any *>(p) = a;
    *reinterpret_cast<u32x4_any *>(p + 4) = b;
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int64_t cnt, const F8 &r) {
    if (cnt >= 8) {
        store8(p, r);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < cnt) store1(p + i, r.v[i]);
}

// Sum and maximum over the wave's 64 lanes, on every lane: rows of 16 by shifted
// adds, then the rows' totals passed on (DPP operands: no trip through LDS).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float other, float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(other), __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_or<0x111, 0xF>(0.0f, v);  // from 1, 2, 4, 8 lanes down the row
    v += dpp_or<0x112, 0xF>(0.0f, v);
    v += dpp_or<0x114, 0xF>(0.0f, v);
    v += dpp_or<0x118, 0xF>(0.0f, v);
    v += dpp_or<0x142, 0xA>(0.0f, v);  // lane 15 of rows 0 and 2 to rows 1 and 3
    v += dpp_or<0x143, 0xC>(0.0f, v);  // lane 31 to rows 2 and 3
    return last_lane(v);
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_or<0x111, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x112, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x114, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x118, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x142, 0xA>(v, v));
    v = fmaxf(v, dpp_or<0x143, 0xC>(v, v));
    return last_lane(v);
}

}  // namespace qnf4

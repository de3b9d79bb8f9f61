// Rows of bf16 or fp32 taken 8 consecutive elements at a time, widened to
// fp32.  A full group is read or written with 16-byte accesses at any element
// alignment (gfx950 takes unaligned global accesses; an odd row pitch or a
// view that starts mid-buffer needs no second code path), the last group of a
// row element by element, so nothing outside the row is touched.
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

// Sum and maximum over the wave's 64 lanes, on every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

}  // namespace qnf4

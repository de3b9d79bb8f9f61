// One AdamW step over a list of tensors, element by element:
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) (1 - b2^t)^-1/2 + eps)
// with g the stored gradient times grad_scale.  Everything is fp32 between the
// load and the store; a bf16 p (without a master) is rounded to nearest even.
//
// States in 8 bits, in blocks of 256 elements with one fp32 scale s each:
//   m = sign(c) c^2 s   s = fp32(max|m| fp32(127^-2))   c = rint(sqrt(fp32(|m| fp32(1/s)))), |c| <= 127
//   v = c^4 s           s = fp32(max v fp32(255^-4))    c = rint(sqrt(sqrt(fp32(v fp32(1/s))))), c >= 1 where v > 0
// (c^2, c^4 in fp32 as (c c) (c c)).  The square and the fourth power spend the
// codes evenly over the roots: the steps shrink with the value, v spans 9
// decades, and sqrt(v), which divides, has the resolution of m.  v > 0 never
// becomes 0, so m is never divided by eps alone.  A block whose scale would be
// below the smallest normal number is stored as zeros.  All of it is fixed
// IEEE arithmetic: the codes are reproducible bit for bit.  An element whose new m or v is
// not finite is left out of the maxima, so that its block keeps its scales; m's code -128
// marks it (v's is 0) and reads as NaN for both, as fp32 states would hold the damage.
//
// Bound: HBM, 24 bytes an element with fp32 states, 12 with 8-bit states (bf16
// p, fp32 g).  Each thread takes 8 consecutive elements of every array (16-byte
// accesses), a block of 256 is half a wave, its maxima 5 lane exchanges.
// Tensors go to the kernel as arguments, up to kMaxAdamwTensors a launch: nothing
// about them is kept anywhere between calls.  Measured: 20 M elements in 56 tensors,
// 8-bit states, 45 us (12.06 bytes each: 5.4 TB/s), their moments 34 us (10.06 bytes each);
// 65,536 elements with fp32 states 3.6 us.
#include "elem8.hpp"
#include "launch.hpp"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;   // elements a workgroup takes

struct TensorList {
    AdamwTensor t[kMaxAdamwTensors];
    uint32_t first[kMaxAdamwTensors + 1];  // the tensors' first workgroups
    int count;
};

static_assert(sizeof(TensorList) + sizeof(AdamwHyper) <= 4096, "kernel arguments");

constexpr float kFastEps = 1e-15f;  // beside it the root of a v below the normal numbers, 1e-19, is nothing
constexpr float kMUnit = 1.0f / 16129.0f;       // 127^-2
constexpr float kVUnit = 1.0f / 4228250625.0f;  // 255^-4, from 255^4 rounded to fp32

// The tensor that a workgroup belongs to (first is ascending).
__device__ __forceinline__ int tensor_of(const TensorList &list, uint32_t wg) {
    int lo = 0, hi = list.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list.first[mid] <= wg) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

struct U8x8 {
    uint32_t w[2];
};
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

__device__ __forceinline__ U8x8 load_codes(const uint8_t *p, int64_t cnt) {
    U8x8 r;
    if (cnt >= 8) {
        const u32x2 w = *reinterpret_cast<const u32x2_any *>(p);
        r.w[0] = w.x;
        r.w[1] = w.y;
        return r;
    }
    r.w[0] = r.w[1] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < cnt) r.w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return r;
}
__device__ __forceinline__ void store_codes(uint8_t *p, int64_t cnt, const U8x8 &r) {
    if (cnt >= 8) {
        *reinterpret_cast<u32x2_any *>(p) = u32x2{r.w[0], r.w[1]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < cnt) p[i] = (uint8_t)(r.w[i >> 2] >> (8 * (i & 3)));
}

// Whether a byte of w is -128, m's code of an element whose states are not finite.
__device__ __forceinline__ bool has_lost(uint32_t w) {
    const uint32_t y = w ^ 0x80808080u;
    return ((y - 0x01010101u) & ~y & 0x80808080u) != 0;
}
__device__ __forceinline__ void decode(const U8x8 &mc, const U8x8 &vc, float m_scale, float v_scale, F8 &m, F8 &v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = (float)(int8_t)(mc.w[i >> 2] >> (8 * (i & 3))), d = (float)(uint8_t)(vc.w[i >> 2] >> (8 * (i & 3)));
        m.v[i] = c * fabsf(c) * m_scale;
        v.v[i] = d * d * (d * d) * v_scale;
    }
    if (has_lost(mc.w[0]) || has_lost(mc.w[1])) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((mc.w[i >> 2] >> (8 * (i & 3)) & 0xFFu) == 0x80u) m.v[i] = v.v[i] = NAN;
    }
}

// Maximum over the half wave that holds a block.
__device__ __forceinline__ float block_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float block_scale_of(float top, float unit) {
    const float s = top * unit;
    return s >= 1.17549435e-38f ? s : 0.0f;
}

// rint of a root that the fast square root gives to 2 units in its last place:
// exact unless the root lies so near to a half that these could matter; then
// `near` is set, for the IEEE root to decide.
__device__ __forceinline__ float root_code(float root, float band, bool &near) {
    const float r = rintf(root);
    near |= fabsf(fabsf(root - r) - 0.5f) < band;
    return r;
}

// The step of 8 elements at `at`, cnt of them there.  FULL: all 8, with every
// load requested before the first is used.
template <bool PF32, bool GF32, bool BITS8, bool MASTER, bool FULL>
__device__ __forceinline__ void adamw_group(const AdamwTensor &t, const AdamwHyper &h, int64_t at, int64_t cnt) {
    using P = std::conditional_t<PF32, float, uint16_t>;
    using G = std::conditional_t<GF32, float, uint16_t>;
    P *p = (P *)t.param + at;
    float *master = MASTER ? t.master + at : nullptr;
    F8 g, m, v, w;
    U8x8 mc, vc;
    float ms0 = 0.0f, vs0 = 0.0f;
    if (FULL) {
        const auto gr = raw8((const G *)t.grad + at);
        RawOf<P> pr;
        RawOf<float> wr, mr, vr;
        if (MASTER) wr = raw8((const float *)master);
        else pr = raw8((const P *)p);
        if (BITS8) {
            mc = load_codes((const uint8_t *)t.m + at, 8);
            vc = load_codes((const uint8_t *)t.v + at, 8);
            ms0 = t.m_scale[at >> 8];
            vs0 = t.v_scale[at >> 8];
        } else {
            mr = raw8((const float *)t.m + at);
            vr = raw8((const float *)t.v + at);
        }
        g = widen(gr);
        w = MASTER ? widen(wr) : widen(pr);
        if (!BITS8) {
            m = widen(mr);
            v = widen(vr);
        }
    } else {
        g = load8((const G *)t.grad + at, cnt);
        w = MASTER ? load8((const float *)master, cnt) : load8((const P *)p, cnt);
        if (BITS8) {
            mc = load_codes((const uint8_t *)t.m + at, cnt);
            vc = load_codes((const uint8_t *)t.v + at, cnt);
            if (cnt > 0) {
                ms0 = t.m_scale[at >> 8];
                vs0 = t.v_scale[at >> 8];
            }
        } else {
            m = load8((const float *)t.m + at, cnt);
            v = load8((const float *)t.v + at, cnt);
        }
    }
    if (BITS8) decode(mc, vc, ms0, vs0, m, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = g.v[i] * h.grad_scale;
        m.v[i] = m.v[i] * h.beta1 + gi * h.one_minus_beta1;
        v.v[i] = v.v[i] * h.beta2 + gi * gi * h.one_minus_beta2;
    }
    if (h.eps >= kFastEps) {
        // root and reciprocal to the last place each: the update's own error stays below 3 units of it
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = __builtin_amdgcn_sqrtf(v.v[i]) * h.v_correction + h.eps;
            w.v[i] = w.v[i] * h.decay - h.step_size * (m.v[i] * __builtin_amdgcn_rcpf(d));
        }
    } else {  // a v below the normal numbers counts: these take it as 0
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w.v[i] = w.v[i] * h.decay - h.step_size * (m.v[i] / (sqrtf(v.v[i]) * h.v_correction + h.eps));
    }
    if (MASTER) store8(master, FULL ? 8 : cnt, w);
    store8(p, FULL ? 8 : cnt, w);
    if (!BITS8) {
        store8((float *)t.m + at, FULL ? 8 : cnt, m);
        store8((float *)t.v + at, FULL ? 8 : cnt, v);
        return;
    }
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) z = fmaf(m.v[i], 0.0f, fmaf(v.v[i], 0.0f, z));
    const bool lost = z != z;  // one of them
    if (lost) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (fabsf(m.v[i]) < INFINITY && v.v[i] < INFINITY) continue;
            m.v[i] = NAN;  // which fmaxf leaves out
            v.v[i] = 0.0f;
        }
    }
    float mtop = 0.0f, vtop = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mtop = fmaxf(mtop, fabsf(m.v[i]));
        vtop = fmaxf(vtop, v.v[i]);
    }
    const float ms = block_scale_of(block_max(mtop), kMUnit), vs = block_scale_of(block_max(vtop), kVUnit);
    const float mi = ms > 0.0f ? 1.0f / ms : 0.0f, vi = vs > 0.0f ? 1.0f / vs : 0.0f;
    float cm[8], cv[8];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cm[i] = root_code(__builtin_amdgcn_sqrtf(fabsf(m.v[i]) * mi), 0x1p-15f, near);  // roots up to 127: 2 units are 2^-16
        cv[i] = root_code(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(v.v[i] * vi)), 0x1p-14f, near);  // up to 255
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cm[i] = rintf(sqrtf(fabsf(m.v[i]) * mi));
            cv[i] = rintf(sqrtf(sqrtf(v.v[i] * vi)));
        }
    }
    mc.w[0] = mc.w[1] = vc.w[0] = vc.w[1] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int c = (int)fminf(cm[i], 127.0f);
        c = m.v[i] < 0.0f ? -c : c;
        mc.w[i >> 2] |= (uint32_t)(uint8_t)c << (8 * (i & 3));
        int d = (int)fminf(cv[i], 255.0f);
        if (v.v[i] > 0.0f && vs > 0.0f && d < 1) d = 1;
        vc.w[i >> 2] |= (uint32_t)d << (8 * (i & 3));
    }
    if (lost) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (m.v[i] != m.v[i]) mc.w[i >> 2] ^= 0xFFu << (8 * (i & 3));  // 127, as fminf takes NaN, to -128
    }
    store_codes((uint8_t *)t.m + at, FULL ? 8 : cnt, mc);
    store_codes((uint8_t *)t.v + at, FULL ? 8 : cnt, vc);
    if ((threadIdx.x & 31) == 0 && cnt > 0) {
        t.m_scale[at >> 8] = ms;
        t.v_scale[at >> 8] = vs;
    }
}

template <bool PF32, bool GF32, bool BITS8, bool MASTER>
__global__ __launch_bounds__(kThreads) void adamw_kernel(TensorList list, AdamwHyper h) {
    const int k = tensor_of(list, blockIdx.x);
    const AdamwTensor &t = list.t[k];
    const int64_t first = (int64_t)(blockIdx.x - list.first[k]) * kChunk, at = first + threadIdx.x * 8;
    if (first + kChunk <= t.n) adamw_group<PF32, GF32, BITS8, MASTER, true>(t, h, at, 8);
    else adamw_group<PF32, GF32, BITS8, MASTER, false>(t, h, at, t.n - at);  // a tensor's last workgroup
}

// The values that 8-bit states stand for; here param and grad are the fp32
// arrays that receive m and v.
__global__ __launch_bounds__(kThreads) void adamw_moments_kernel(TensorList list) {
    const int k = tensor_of(list, blockIdx.x);
    const AdamwTensor &t = list.t[k];
    const int64_t at = (int64_t)(blockIdx.x - list.first[k]) * kChunk + threadIdx.x * 8, cnt = t.n - at;
    if (cnt <= 0) return;
    const U8x8 mc = load_codes((const uint8_t *)t.m + at, cnt), vc = load_codes((const uint8_t *)t.v + at, cnt);
    const float ms = t.m_scale[at >> 8], vs = t.v_scale[at >> 8];
    F8 m, v;
    decode(mc, vc, ms, vs, m, v);
    store8((float *)t.param + at, cnt, m);
    store8((float *)const_cast<void *>(t.grad) + at, cnt, v);
}

// f(list, workgroups) for each launch's part of the tensors; empty ones are left out.
template <typename F>
hipError_t in_lists(const AdamwTensor *t, int count, F f) {
    TensorList list;
    list.count = 0;
    uint32_t wgs = 0;
    for (int i = 0; i <= count; ++i) {
        const uint32_t need = i < count ? (uint32_t)((t[i].n + kChunk - 1) / kChunk) : 0;
        if (list.count > 0 && (i == count || list.count == kMaxAdamwTensors || wgs + need > kMaxAdamwGroups)) {
            list.first[list.count] = wgs;
            f(list, wgs);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            list.count = 0;
            wgs = 0;
        }
        if (need == 0) continue;
        list.t[list.count] = t[i];
        list.first[list.count++] = wgs;
        wgs += need;
    }
    return hipSuccess;
}

template <bool PF32, bool GF32, bool BITS8, bool MASTER>
hipError_t step(const AdamwTensor *t, int count, const AdamwHyper &h, hipStream_t s) {
    return in_lists(t, count, [&](const TensorList &list, uint32_t wgs) {
        adamw_kernel<PF32, GF32, BITS8, MASTER><<<wgs, kThreads, 0, s>>>(list, h);
    });
}

template <bool PF32, bool MASTER>
hipError_t step_typed(const AdamwTensor *t, int count, bool g_f32, bool bits8, const AdamwHyper &h, hipStream_t s) {
    if (g_f32)
        return bits8 ? step<PF32, true, true, MASTER>(t, count, h, s) : step<PF32, true, false, MASTER>(t, count, h, s);
    return bits8 ? step<PF32, false, true, MASTER>(t, count, h, s) : step<PF32, false, false, MASTER>(t, count, h, s);
}

}  // namespace

hipError_t launch_adamw(const AdamwTensor *t, int count, bool p_f32, bool g_f32, bool bits8, bool master,
                        const AdamwHyper &h, hipStream_t s) {
    if (p_f32) return step_typed<true, false>(t, count, g_f32, bits8, h, s);
    return master ? step_typed<false, true>(t, count, g_f32, bits8, h, s)
                  : step_typed<false, false>(t, count, g_f32, bits8, h, s);
}

hipError_t launch_adamw_moments(const AdamwTensor *t, int count, hipStream_t s) {
    return in_lists(t, count, [&](const TensorList &list, uint32_t wgs) {
        adamw_moments_kernel<<<wgs, kThreads, 0, s>>>(list);
    });
}

}  // namespace qnf4

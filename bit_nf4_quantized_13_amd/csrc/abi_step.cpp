// The C ABI of the operators around the linear layer in a fine-tuning step
// (include/qlora_nf4.h): layer norm, attention, token log-probabilities, AdamW.  As in
// abi.cpp every check runs before the first launch; no allocation, no
// synchronisation, no state.
#include "qlora_nf4.h"

#include <cmath>

#include "abi_util.hpp"
#include "launch.hpp"

using namespace qnf4;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxNormWidth = int64_t(1) << 26;   // a launch over its columns stays below 2^32 threads
constexpr int64_t kMaxGroups = (int64_t(1) << 23) - 1;  // workgroups of up to 512 threads of a launch: the same

bool known_type(int32_t t) { return t == QLORA_BF16 || t == QLORA_F32; }
uintptr_t type_bytes(int32_t t) { return t == QLORA_F32 ? 4 : 2; }
bool aligned_or_null(const void *p, uintptr_t a) { return !p || aligned(p, a); }

// The checks that both layer norm calls share.
int check_norm(const void *x, int32_t x_type, int64_t M, int64_t n, int64_t ldx, const void *weight, int32_t w_type) {
    if (!x || M <= 0 || n <= 0 || ldx < n) return QLORA_EINVAL;
    if (!known_type(x_type) || !known_type(w_type)) return QLORA_ENOTSUP;
    if (M > kMaxRows || n > kMaxNormWidth) return QLORA_ENOTSUP;
    if (!aligned(x, type_bytes(x_type)) || !aligned_or_null(weight, type_bytes(w_type))) return QLORA_EALIGN;
    return QLORA_OK;
}

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // row numbers and tile ends stay below 2^31
constexpr float kMinScale = 0x1p-64f;             // lse / scale stays far from overflow

// A matrix of `width` values a row: pitch and alignment of 16-byte accesses.
int check_pitch(int64_t ld, int64_t width) {
    if (ld < width) return QLORA_EINVAL;
    return ld % 8 == 0 && ld <= kMaxPitch ? QLORA_OK : QLORA_ENOTSUP;
}

int check_attention(const qlora_attention_shape *s, AttentionShape *a) {
    if (!s) return QLORA_EINVAL;
    if (s->T <= 0 || s->sequences <= 0 || s->heads <= 0 || s->kv_heads <= 0 || s->dim <= 0) return QLORA_EINVAL;
    if (s->heads % s->kv_heads != 0 || !(s->scale > 0.0f) || std::isinf(s->scale)) return QLORA_EINVAL;
    if (s->scale < kMinScale) return QLORA_ENOTSUP;
    if (s->dim % 8 != 0 || s->dim > 128 || s->T > kMaxTokens || s->sequences > kMaxTokens) return QLORA_ENOTSUP;
    const int64_t wide = (int64_t)s->heads * s->dim, narrow = (int64_t)s->kv_heads * s->dim;
    if (wide > kMaxPitch) return QLORA_ENOTSUP;  // the dense rows of o
    int st = check_pitch(s->ldq, wide);
    if (st == QLORA_OK) st = check_pitch(s->ldk, narrow);
    if (st == QLORA_OK) st = check_pitch(s->ldv, narrow);
    if (st != QLORA_OK) return st;
    *a = AttentionShape{(int)s->T, s->sequences, s->heads, s->kv_heads, s->dim, s->ldq, s->ldk, s->ldv, s->scale};
    return attention_groups(*a) <= kMaxGroups ? QLORA_OK : QLORA_ENOTSUP;
}

int check_logits(const void *logits, int32_t type, int64_t M, int64_t V, int64_t ld) {
    if (!logits || M <= 0 || V <= 0 || ld < V) return QLORA_EINVAL;
    if (!known_type(type)) return QLORA_ENOTSUP;
    if (V > kMaxVocab || M > kMaxRows || logprob_groups(M, V) > kMaxRows) return QLORA_ENOTSUP;
    return aligned(logits, type_bytes(type)) ? QLORA_OK : QLORA_EALIGN;
}

static_assert(sizeof(AdamwTensor) == sizeof(qlora_adamw_tensor), "the kernels' view of a tensor");

// The tensors' pointers for the given types (param / grad only where `all`).
int check_tensors(const qlora_adamw_tensor *t, int32_t count, const qlora_adamw_config *c, bool all) {
    if (!t || count < 0) return QLORA_EINVAL;
    const bool bits8 = c->state_type == QLORA_STATE_8BIT;
    const uintptr_t ab = type_bytes(c->param_type), gb = type_bytes(c->grad_type), sb = bits8 ? 1 : 4;
    for (int32_t i = 0; i < count; ++i) {
        if (t[i].n < 0) return QLORA_EINVAL;
        if (t[i].n == 0) continue;
        if (t[i].n > kMaxAdamwElems) return QLORA_ENOTSUP;
        if (!t[i].m || !t[i].v || (bits8 && (!t[i].m_scale || !t[i].v_scale))) return QLORA_EINVAL;
        if (all && (!t[i].param || !t[i].grad)) return QLORA_EINVAL;
        if (all && (c->use_master != 0) != (t[i].master != nullptr)) return QLORA_EINVAL;
        if (!aligned(t[i].m, sb) || !aligned(t[i].v, sb)) return QLORA_EALIGN;
        if (bits8 && (!aligned(t[i].m_scale, 4) || !aligned(t[i].v_scale, 4))) return QLORA_EALIGN;
        if (all && (!aligned(t[i].param, ab) || !aligned(t[i].grad, gb) || !aligned_or_null(t[i].master, 4)))
            return QLORA_EALIGN;
    }
    return QLORA_OK;
}

}  // namespace

extern "C" {

size_t qlora_layernorm_workspace(int64_t M, int64_t n) {
    if (M <= 0 || n <= 0 || M > kMaxRows || n > kMaxNormWidth) return 0;
    return round_up(layernorm_part_bytes(M, n), 256);
}

int qlora_layernorm_fwd(const void *x, int32_t x_type, int64_t M, int64_t n, int64_t ldx, const void *weight,
                        const void *bias, int32_t w_type, float eps, void *y, float *mean, float *rstd,
                        void *stream) {
    const int st = check_norm(x, x_type, M, n, ldx, weight, w_type);
    if (st != QLORA_OK) return st;
    if (!y || !(eps >= 0.0f) || std::isinf(eps)) return QLORA_EINVAL;
    if (!aligned_or_null(bias, type_bytes(w_type)) || !aligned(y, type_bytes(x_type)) || !aligned_or_null(mean, 4) ||
        !aligned_or_null(rstd, 4))
        return QLORA_EALIGN;
    (void)hipGetLastError();
    return hip_status(launch_layernorm_fwd(x, x_type == QLORA_F32, M, n, ldx, weight, bias, w_type == QLORA_F32, eps, y,
                                           mean, rstd, static_cast<hipStream_t>(stream)));
}

int qlora_layernorm_bwd(const void *x, const void *dy, int32_t x_type, int64_t M, int64_t n, int64_t ldx,
                        const float *mean, const float *rstd, const void *weight, int32_t w_type, void *dx,
                        float *dweight, float *dbias, void *ws, size_t ws_bytes, void *stream) {
    const int st = check_norm(x, x_type, M, n, ldx, weight, w_type);
    if (st != QLORA_OK) return st;
    if (!dy || !mean || !rstd || !dx) return QLORA_EINVAL;
    if (!aligned(dy, type_bytes(x_type)) || !aligned(dx, type_bytes(x_type)) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned_or_null(dweight, 4) || !aligned_or_null(dbias, 4))
        return QLORA_EALIGN;
    if (dweight || dbias) {
        if (!ws || ws_bytes < qlora_layernorm_workspace(M, n)) return QLORA_EWORKSPACE;
        if (!aligned(ws, 16)) return QLORA_EALIGN;
    }
    (void)hipGetLastError();
    return hip_status(launch_layernorm_bwd(x, dy, x_type == QLORA_F32, M, n, ldx, mean, rstd, weight,
                                           w_type == QLORA_F32, dx, dweight, dbias, static_cast<float *>(ws),
                                           static_cast<hipStream_t>(stream)));
}

int qlora_attention_fwd(const qlora_attention_shape *shape, const qlora_bf16 *q, const qlora_bf16 *k,
                        const qlora_bf16 *v, const int32_t *cu_seqlens, qlora_bf16 *o, qlora_bf16 *residual,
                        float *lse, void *stream) {
    AttentionShape a;
    const int st = check_attention(shape, &a);
    if (st != QLORA_OK) return st;
    if (!q || !k || !v || !cu_seqlens || !o || !lse) return QLORA_EINVAL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned_or_null(residual, 16) ||
        !aligned(cu_seqlens, 4) || !aligned(lse, 4))
        return QLORA_EALIGN;
    (void)hipGetLastError();
    return hip_status(launch_attention_fwd(a, q, k, v, cu_seqlens, o, residual, lse, static_cast<hipStream_t>(stream)));
}

size_t qlora_attention_workspace(const qlora_attention_shape *shape) {
    AttentionShape a;
    if (check_attention(shape, &a) != QLORA_OK) return 0;
    return round_up(attention_bwd_bytes(a), 256);
}

int qlora_attention_bwd(const qlora_attention_shape *shape, const qlora_bf16 *q, const qlora_bf16 *k,
                        const qlora_bf16 *v, const qlora_bf16 *o, const qlora_bf16 *residual, const float *lse,
                        const qlora_bf16 *dout, const int32_t *cu_seqlens, qlora_bf16 *dq, int64_t lddq,
                        qlora_bf16 *dk, int64_t lddk, qlora_bf16 *dv, int64_t lddv, void *ws, size_t ws_bytes,
                        void *stream) {
    AttentionShape a;
    int st = check_attention(shape, &a);
    if (st != QLORA_OK) return st;
    if (!q || !k || !v || !o || !lse || !dout || !cu_seqlens || !dq || !dk || !dv) return QLORA_EINVAL;
    const int64_t wide = (int64_t)a.H * a.D, narrow = (int64_t)a.Hk * a.D;
    st = check_pitch(lddq, wide);
    if (st == QLORA_OK) st = check_pitch(lddk, narrow);
    if (st == QLORA_OK) st = check_pitch(lddv, narrow);
    if (st != QLORA_OK) return st;
    for (const void *p : {(const void *)q, (const void *)k, (const void *)v, (const void *)o, (const void *)residual,
                          (const void *)dout, (const void *)dq, (const void *)dk, (const void *)dv})
        if (!aligned_or_null(p, 16)) return QLORA_EALIGN;
    if (!aligned(cu_seqlens, 4) || !aligned(lse, 4)) return QLORA_EALIGN;
    if (!ws || ws_bytes < qlora_attention_workspace(shape)) return QLORA_EWORKSPACE;
    if (!aligned(ws, 16)) return QLORA_EALIGN;
    (void)hipGetLastError();
    return hip_status(launch_attention_bwd(a, q, k, v, o, residual, lse, dout, cu_seqlens, dq, lddq, dk, lddk, dv, lddv,
                                           ws, static_cast<hipStream_t>(stream)));
}

size_t qlora_logprob_workspace(int64_t M, int64_t V, int32_t top) {
    if (M <= 0 || V <= 0 || V > kMaxVocab || M > kMaxRows || top < 0 || top > kMaxTop) return 0;
    return 16 + round_up(logprob_stats_bytes(M, V), 256) + round_up(logprob_best_bytes(M, V, top), 256);
}

int qlora_logprob_fwd(const void *logits, int32_t type, int64_t M, int64_t V, int64_t ld, const int64_t *targets,
                      int32_t top, float *logp, float *entropy, float *lse, float *top_logp, int32_t *top_ids,
                      void *ws, size_t ws_bytes, void *stream) {
    const int st = check_logits(logits, type, M, V, ld);
    if (st != QLORA_OK) return st;
    if (top < 0 || top > V || (logp != nullptr) != (targets != nullptr)) return QLORA_EINVAL;
    if (top > kMaxTop) return QLORA_ENOTSUP;
    if (top > 0 && (!top_logp || !top_ids)) return QLORA_EINVAL;
    if (!aligned_or_null(targets, 8) || !aligned_or_null(logp, 4) || !aligned_or_null(entropy, 4) ||
        !aligned_or_null(lse, 4) || (top > 0 && (!aligned(top_logp, 4) || !aligned(top_ids, 4))))
        return QLORA_EALIGN;
    if (!ws || ws_bytes < qlora_logprob_workspace(M, V, top)) return QLORA_EWORKSPACE;
    if (!aligned(ws, 16)) return QLORA_EALIGN;
    (void)hipGetLastError();
    char *best = static_cast<char *>(ws) + round_up(logprob_stats_bytes(M, V), 256);
    return hip_status(launch_logprob_fwd(logits, type == QLORA_F32, M, V, ld, targets, top, logp, entropy, lse, top_logp,
                                         top_ids, static_cast<float *>(ws), best, static_cast<hipStream_t>(stream)));
}

int qlora_logprob_bwd(const void *logits, int32_t type, int64_t M, int64_t V, int64_t ld, const int64_t *targets,
                      const float *lse, const float *entropy, const float *dlogp, const float *dentropy,
                      void *dlogits, int64_t ldd, void *stream) {
    const int st = check_logits(logits, type, M, V, ld);
    if (st != QLORA_OK) return st;
    if (!lse || !dlogits || ldd < V) return QLORA_EINVAL;
    if ((dlogp != nullptr) != (targets != nullptr) || (dentropy && !entropy) || (!dlogp && !dentropy))
        return QLORA_EINVAL;
    if (dlogits == logits && ldd != ld) return QLORA_EINVAL;  // in place: the same rows
    if (!aligned_or_null(targets, 8) || !aligned(lse, 4) || !aligned_or_null(entropy, 4) ||
        !aligned_or_null(dlogp, 4) || !aligned_or_null(dentropy, 4) || !aligned(dlogits, type_bytes(type)))
        return QLORA_EALIGN;
    (void)hipGetLastError();
    return hip_status(launch_logprob_bwd(logits, type == QLORA_F32, M, V, ld, targets, lse, entropy, dlogp, dentropy,
                                         dlogits, ldd, static_cast<hipStream_t>(stream)));
}

int qlora_adamw_step(const qlora_adamw_tensor *tensors, int32_t count, const qlora_adamw_config *config,
                     void *stream) {
    if (!config) return QLORA_EINVAL;
    const qlora_adamw_config &c = *config;
    if (!known_type(c.param_type) || !known_type(c.grad_type) ||
        (c.state_type != QLORA_STATE_F32 && c.state_type != QLORA_STATE_8BIT))
        return QLORA_ENOTSUP;
    if (c.use_master && c.param_type != QLORA_BF16) return QLORA_EINVAL;
    if (c.step < 1 || !(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0)) return QLORA_EINVAL;
    if (!(c.eps >= 0.0) || std::isinf(c.eps) || !std::isfinite(c.lr) || !std::isfinite(c.weight_decay) ||
        !std::isfinite(c.grad_scale))
        return QLORA_EINVAL;
    const int st = check_tensors(tensors, count, config, true);
    if (st != QLORA_OK) return st;
    // 1 - b^t in fp64 (t as a power: b^t underflows to 0 for a long run, leaving 1)
    const double bias1 = 1.0 - std::pow(c.beta1, (double)c.step), bias2 = 1.0 - std::pow(c.beta2, (double)c.step);
    AdamwHyper h;
    h.beta1 = (float)c.beta1;
    h.one_minus_beta1 = (float)(1.0 - c.beta1);
    h.beta2 = (float)c.beta2;
    h.one_minus_beta2 = (float)(1.0 - c.beta2);
    h.eps = (float)c.eps;
    h.decay = (float)(1.0 - c.lr * c.weight_decay);
    h.step_size = (float)(c.lr / bias1);
    h.v_correction = (float)(1.0 / std::sqrt(bias2));
    h.grad_scale = (float)c.grad_scale;
    (void)hipGetLastError();
    return hip_status(launch_adamw(reinterpret_cast<const AdamwTensor *>(tensors), count, c.param_type == QLORA_F32,
                                   c.grad_type == QLORA_F32, c.state_type == QLORA_STATE_8BIT, c.use_master != 0, h,
                                   static_cast<hipStream_t>(stream)));
}

int qlora_adamw_moments(const qlora_adamw_tensor *tensors, int32_t count, float *const *m_out, float *const *v_out,
                        void *stream) {
    qlora_adamw_config c{};
    c.state_type = QLORA_STATE_8BIT;
    const int st = check_tensors(tensors, count, &c, false);
    if (st != QLORA_OK) return st;
    if (!m_out || !v_out) return QLORA_EINVAL;
    for (int32_t i = 0; i < count; ++i) {
        if (tensors[i].n == 0) continue;
        if (!m_out[i] || !v_out[i]) return QLORA_EINVAL;
        if (!aligned(m_out[i], 4) || !aligned(v_out[i], 4)) return QLORA_EALIGN;
    }
    (void)hipGetLastError();
    AdamwTensor batch[kMaxAdamwTensors];  // a launch's tensors, handed on from the stack
    for (int32_t i = 0; i < count; i += kMaxAdamwTensors) {
        const int n = count - i < kMaxAdamwTensors ? count - i : kMaxAdamwTensors;
        for (int j = 0; j < n; ++j) {
            const qlora_adamw_tensor &t = tensors[i + j];
            batch[j] = AdamwTensor{m_out[i + j], v_out[i + j], t.m, t.v, t.m_scale, t.v_scale, nullptr, t.n};
        }
        const int e = hip_status(launch_adamw_moments(batch, n, static_cast<hipStream_t>(stream)));
        if (e != QLORA_OK) return e;
    }
    return QLORA_OK;
}

}  // extern "C"

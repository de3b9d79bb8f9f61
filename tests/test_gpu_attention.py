"""Causal attention over packed sequences against the 64-bit oracle: lengths
around the tiles (32, 64, 128), empty and single-row sequences, rows that belong
to no sequence, grouped heads, head dimensions, row pitches.

Bounds: P and dS are rounded to bf16 (2^-8 of each at most) for products that
sum them with fp32 accumulation, and results are stored in bf16, so with the
sums of magnitudes taken by the oracle's own formulas
  |o error|  <= 2^-8 (sum_j p |v|) + 2^-8 |o|          and so on for dq, dk, dv,
where dS inherits also delta's and p's fp32 errors (under 2^-12 of the sums
together, for scores below 100), through delta = do o the forward's rounding of P
(2^-8 sum_j p |do| |v|) and, without the forward's residual, the bf16 rounding of
o (2^-8 sum_d |do| |o|)."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.helpers import say

pytestmark = pytest.mark.gpu

R = 2.0 ** -8          # largest relative rounding to bf16
SMALL = 2.0 ** -12     # fp32 effects: exponentials of scores below 100, sums of a few thousand


def host(t):
    return t.detach().double().cpu().numpy()


def make(lens, tail, h, hk, d, seed, fused=False, head=0):
    g = torch.Generator().manual_seed(seed)
    t = head + sum(lens) + tail
    draw = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    if fused:
        both = draw(t, (h + 2 * hk) * d + 8)
        q, k, v = (both[:, a * d:b * d].view(t, b - a, d) for a, b in ((0, h), (h, h + hk), (h + hk, h + 2 * hk)))
    else:
        q, k, v = draw(t, h, d), draw(t, hk, d), draw(t, hk, d)
    starts = np.cumsum([head] + list(lens)).astype(np.int32)
    return q, k, v, draw(t, h, d), starts, torch.from_numpy(starts).cuda()


def bounds(q, k, v, do, starts, scale, residual):
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    bo, bq, bk, bv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, b in zip(starts[:-1], starts[1:]):
        if b <= a:
            continue
        later = np.triu(np.ones((b - a, b - a), dtype=bool), 1)
        for h in range(heads):
            g = h // group
            s = np.where(later, -np.inf, scale * q[a:b, h] @ k[a:b, g].T)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = p @ v[a:b, g]
            bo[a:b, h] = p @ np.abs(v[a:b, g])
            dp = do[a:b, h] @ v[a:b, g].T
            size = np.abs(do[a:b, h]) @ np.abs(v[a:b, g]).T   # of dp's and delta's own sums
            delta = (p * dp).sum(1, keepdims=True)
            ds = R * p * np.abs(dp - delta) + p * (SMALL * size + (R + SMALL) * (p * size).sum(1, keepdims=True))
            if not residual:
                ds = ds + R * p * (np.abs(do[a:b, h]) * np.abs(o)).sum(1, keepdims=True)
            bq[a:b, h] = scale * ds @ np.abs(k[a:b, g])
            bk[a:b, g] += scale * ds.T @ np.abs(q[a:b, h])
            bv[a:b, g] += (R + SMALL) * p.T @ np.abs(do[a:b, h])
    return (R + SMALL) * bo, bq, bk, bv


def check(lens, tail, h, hk, d, seed, fused=False, head=0, scale=None):
    import bit_nf4_quantized_13_amd as q_
    say(f"attention lens={lens[:12]} tail={tail} heads={h}/{hk} dim={d} fused={fused} head={head}")
    q, k, v, do, starts, cu = make(lens, tail, h, hk, d, seed, fused, head)
    sc = d ** -0.5 if scale is None else scale
    o, lse, none = q_.qlora_attention_fwd(q, k, v, cu, scale)
    o2, lse2, res = q_.qlora_attention_fwd(q, k, v, cu, scale, save_residual=True)
    torch.cuda.synchronize()
    assert none is None and torch.equal(o, o2) and torch.equal(lse, lse2)
    qh, kh, vh, dh = host(q), host(k), host(v), host(do)
    ro, rl, rq, rk, rv = step.attention(qh, kh, vh, starts, sc, dh)
    outside = np.ones(q.shape[0], dtype=bool)
    outside[starts[0]:starts[-1]] = False
    assert np.all(host(o)[outside] == 0) and np.all(host(lse)[:, outside] == -np.inf)
    inside = ~outside
    assert np.all(np.abs(host(lse)[:, inside] - rl[:, inside]) <= SMALL * (1 + np.abs(rl[:, inside])))
    for r in (None, res):
        bo, bq, bk, bv = bounds(qh, kh, vh, dh, starts, sc, r is not None)
        assert np.all(np.abs(host(o) - ro) <= bo + R * np.abs(ro))
        grads = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, scale, residual=r)
        for got, ref, b, name in zip(grads, (rq, rk, rv), (bq, bk, bv), ("dq", "dk", "dv")):
            got = host(got)
            assert np.all(np.isfinite(got)), name
            assert np.all(got[outside] == 0), name
            excess = np.abs(got - ref) - (b * (1 + R) + R * np.abs(ref))
            assert excess.max() <= 1e-30, f"{name}: {excess.max():.3e} beyond the bound"
        again = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, scale, residual=r)
        assert all(torch.equal(s, t) for s, t in zip(grads, again))
    # what the residual is: o and it together are o to 2^-16
    both = host(o) + host(res)
    assert np.all(np.abs(both - ro)[inside] <= (bo + SMALL * np.abs(ro))[inside])


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 257, 500])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(n, d):
    check([n], 0, 2, 2, d, n)


@pytest.mark.parametrize("d", [8, 16, 40, 56, 72, 80, 96, 112, 120])
def test_head_dimensions(d):
    check([70, 1, 150], 3, 2, 1, d, d, fused=True)


@pytest.mark.parametrize("h,hk", [(1, 1), (3, 1), (4, 2), (6, 3), (8, 8), (16, 8), (5, 5)])
def test_heads(h, hk):
    check([129, 40], 2, h, hk, 64, h)
    check([130], 0, h, hk, 128, h, fused=True)


@pytest.mark.parametrize("d", [64, 128])
def test_packed_sequences(d):
    """Empty ones first, inside and last; rows before the first and after the last sequence."""
    check([0, 5, 0, 0, 128, 1, 1, 64, 257, 0, 3, 130, 0], 77, 4, 2, d, 3, fused=True)
    check([0, 0], 5, 2, 1, d, 4)
    check([10, 300], 0, 2, 2, d, 5, head=140)
    check([200], 260, 2, 2, d, 6, head=1)


@pytest.mark.parametrize("lens,h,hk,d", [
    ([384], 2, 2, 64), ([385], 2, 1, 128), ([449, 703], 2, 2, 128), ([512, 1, 1040], 3, 1, 64), ([1027, 130, 0, 545], 4, 2, 72),
    ([800], 1, 1, 40), ([480, 480], 2, 2, 112), ([430, 450], 14, 7, 64), ([700], 28, 28, 128), ([600, 1, 3], 2, 1, 64),
    ([3, 640, 1], 2, 2, 128), ([600, 1, 3, 2, 0], 2, 1, 64), ([3, 640, 1, 1], 2, 2, 128), ([620, 0, 1300], 28, 7, 64)])
def test_few_long_sequences(lens, h, hk, d):
    """Sequences whose rows one, two or four parts of a workgroup share."""
    check(lens, 7, h, hk, d, len(lens), fused=True, head=5)


def test_few_long_sequences_keep_apart():
    """NaN and infinity in one of them and around them leave the others' bits alone; the same bits on every run."""
    import bit_nf4_quantized_13_amd as q_
    say("attention long neighbours")
    for d in (64, 128):
        q, k, v, do, starts, cu = make([450, 391, 500], 9, 2, 1, d, 21, fused=True, head=3)
        clean = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
        grads = q_.qlora_attention_bwd(q, k, v, clean[0], clean[1], do, cu, residual=clean[2])
        bad = np.r_[0:3, starts[1]:starts[2], starts[3]:q.shape[0]]
        keep = np.setdiff1d(np.arange(q.shape[0]), bad)
        for t in (q, k, v, do):
            t[bad] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0] * (d // 4)).cuda().bfloat16()
        o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
        got = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res)
        assert torch.equal(o[keep], clean[0][keep]) and torch.equal(lse[:, keep], clean[1][:, keep])
        assert all(torch.equal(s[keep], t[keep]) for s, t in zip(got, grads))


def test_many_short_sequences():
    """More sequences than the 64 and the 4096 that one and two steps of the look-up cover."""
    check([1 + i % 7 for i in range(150)], 3, 2, 1, 64, 7)
    check([i % 2 for i in range(4500)], 0, 1, 1, 64, 8)


def test_scales():
    check([180], 0, 2, 2, 64, 9, scale=1.0)
    check([180], 0, 2, 2, 128, 9, scale=1e-3)


def test_neighbours_do_not_leak():
    """NaN and infinity in the rows of one sequence (and outside of all) leave the others' bits alone."""
    import bit_nf4_quantized_13_amd as q_
    say("attention neighbours")
    for d in (64, 128, 72):
        q, k, v, do, starts, cu = make([70, 61, 200], 9, 2, 1, d, 11, fused=True, head=3)
        clean = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
        grads = q_.qlora_attention_bwd(q, k, v, clean[0], clean[1], do, cu, residual=clean[2])
        bad = np.r_[0:3, starts[1]:starts[2], starts[3]:q.shape[0]]
        keep = np.setdiff1d(np.arange(q.shape[0]), bad)
        for t in (q, k, v, do):
            t[bad] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0] * (d // 4)).cuda().bfloat16()
        o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
        got = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res)
        assert torch.equal(o[keep], clean[0][keep]) and torch.equal(lse[:, keep], clean[1][:, keep])
        assert all(torch.equal(s[keep], t[keep]) for s, t in zip(got, grads))
        outside = np.r_[0:3, starts[3]:q.shape[0]]
        assert all(bool((s[outside] == 0).all()) for s in (o, *got))


def test_growing_scores():
    """Maxima that rise tile after tile, and scores far apart: the running maximum moves."""
    import bit_nf4_quantized_13_amd as q_
    say("attention growing scores")
    q, k, v, do, starts, cu = make([400], 0, 1, 1, 64, 12)
    q.fill_(1.0)
    k.copy_((torch.arange(400).view(400, 1, 1) * 0.01).expand(400, 1, 64))
    o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, 1.0, save_residual=True)
    ro, rl, rq, rk, rv = step.attention(host(q), host(k), host(v), starts, 1.0, host(do))
    assert np.all(np.abs(host(lse) - rl) <= SMALL * (1 + np.abs(rl)))
    bo, bq, bk, bv = bounds(host(q), host(k), host(v), host(do), starts, 1.0, True)
    # scores reach 256: an exponential's argument is off by 2^-24 of that, 4 times the small term's share
    assert np.all(np.abs(host(o) - ro) <= 2 * bo + R * np.abs(ro))


def test_slices_of_one_gradient_matrix():
    import bit_nf4_quantized_13_amd as q_
    say("attention gradients into one matrix")
    h, hk, d = 4, 2, 64
    q, k, v, do, starts, cu = make([100, 33], 4, h, hk, d, 13, fused=True)
    o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
    want = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res)
    both = torch.full((q.shape[0], (h + 2 * hk) * d), 7.0, dtype=torch.bfloat16, device="cuda")
    outs = tuple(both[:, a * d:b * d].view(-1, b - a, d) for a, b in ((0, h), (h, h + hk), (h + hk, h + 2 * hk)))
    q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res, outs=outs)
    assert all(torch.equal(s, t) for s, t in zip(outs, want))


def test_gradients_against_differences():
    """The oracle's gradients (which the kernels are held to) against differences of its forward."""
    g = np.random.default_rng(0)
    q, k, v, do = (g.standard_normal((7, n, 4)) for n in (2, 1, 1, 2))
    starts, sc = [0, 4, 7], 0.5
    grads = step.attention(q, k, v, starts, sc, do)[2:]
    for t, grad in zip((q, k, v), grads):
        for i in np.ndindex(*t.shape):
            both = []
            for sign in (1, -1):
                t[i] += sign * 1e-6
                both.append((do * step.attention(q, k, v, starts, sc)[0]).sum())
                t[i] -= sign * 1e-6
            assert abs((both[0] - both[1]) / 2e-6 - grad[i]) <= 1e-7


def test_bad_starts_stay_in_bounds():
    """Starts beyond the rows or descending give wrong rows, never an access outside (they are clamped)."""
    import bit_nf4_quantized_13_amd as q_
    say("attention odd starts")
    q, k, v, do, _, _ = make([300], 0, 2, 2, 64, 14)
    for bad in ([0, 1000], [-5, 300], [0, 200, 100, 300]):
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
        q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res)
    torch.cuda.synchronize()


def test_other_stream_and_graph():
    import bit_nf4_quantized_13_amd as q_
    say("attention graph")
    q, k, v, do, starts, cu = make([90, 200], 0, 2, 2, 64, 15)
    o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
    want = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2, res2 = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
        got = q_.qlora_attention_bwd(q, k, v, o2, lse2, do, cu, residual=res2)
    side.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(s, t) for s, t in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3, res3 = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
        got3 = q_.qlora_attention_bwd(q, k, v, o3, lse3, do, cu, residual=res3)
    for _ in range(3):
        o3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o3) and all(torch.equal(s, t) for s, t in zip(want, got3))

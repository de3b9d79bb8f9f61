"""Token log-probabilities, entropies, alternatives and their gradient against
the 64-bit oracle: vocabularies around the chunk sizes, ties, ruled-out tokens,
rows with nothing left, missing targets, row pitches.

Bounds (u = 2^-24): an exponential's argument is rounded to 2 u of itself and
its value to 2 u, sums are trees less than 64 deep; lse is stored to u of
itself (the gradient's p carries that up to |lse| = 4096, where it is
normalised anew).  bf16 gradients add 2^-8 of the value."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


def host(t):
    return t.detach().double().cpu().numpy()


def logits(rows, v, dtype, seed, pitch=None, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    store = torch.full((rows, pitch or v), float("nan"))
    store[:, :v] = spread * torch.randn(rows, v, generator=g)
    return store.to(dtype).cuda()[:, :v]


def log_p(xh):
    with np.errstate(invalid="ignore", over="ignore"):
        d = xh - xh.max(1, keepdims=True)
        return np.where(np.isnan(d), -INF, d - np.log(np.exp(d).sum(1, keepdims=True)))


def check(x, targets, top, seed=0):
    import bit_nf4_quantized_13_amd as q
    rows, v = x.shape
    logp, entropy, lse, top_logp, top_ids = q.qlora_logprob_fwd(x, targets, top=top)
    torch.cuda.synchronize()
    xh, th = host(x), targets.cpu().numpy()
    r_logp, r_ent, r_lse, r_top, r_ids = step.logprob(xh, th, top)
    live = np.isfinite(r_lse)
    assert np.array_equal(np.isfinite(host(lse)), live)
    fin = np.where(np.isfinite(xh), np.abs(xh), 0).max(1)
    off = U * (2 * fin + 200)                       # of lse, absolutely: both roundings and the sum
    assert np.all(np.abs(host(lse)[live] - r_lse[live]) <= off[live])
    got, ok = host(logp), np.isfinite(r_logp)
    assert np.array_equal(got[~ok], r_logp[~ok])
    assert np.all(np.abs(got[ok] - r_logp[ok]) <= (off + U * np.where(ok, np.abs(r_logp), 0) + U * fin)[ok])
    # log l and the mean deviation, each up to log V + 100, each to 64 u
    assert np.all(np.abs(host(entropy) - r_ent) <= 128 * U * (np.log(v) + 8))
    if top:
        assert np.array_equal(top_ids.cpu().numpy(), r_ids)
        fine = np.isfinite(r_top)
        assert np.array_equal(np.isfinite(host(top_logp)), fine)
        assert np.all((np.abs(host(top_logp) - np.where(fine, r_top, 0)) <= (off + 2 * U * fin)[:, None] + U * np.abs(r_top))[fine])
    else:
        assert top_logp is None and top_ids is None
    g = torch.Generator().manual_seed(seed)
    dlogp, dent = torch.randn(rows, generator=g).cuda(), torch.randn(rows, generator=g).cuda()
    for de in (None, dent):
        d = q.qlora_logprob_bwd(x, targets, lse, entropy if de is not None else None, dlogp, de)
        ref = step.logprob_backward(xh, th, host(dlogp), host(de) if de is not None else None)
        lp = log_p(xh)
        p = np.exp(lp)
        lp = np.where(lp > -np.inf, lp, 0)
        gs = np.abs(host(dlogp))[:, None]
        hs = (np.abs(host(dent))[:, None] * (np.abs(lp) + r_ent[:, None] + 1)) if de is not None else 0
        bound = U * (80 + 8 * np.abs(lp) + np.minimum(fin, 4200)[:, None]) * p * (gs + hs) + 4 * U * np.abs(ref)
        if x.dtype == torch.bfloat16:
            bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
        got = host(d)
        assert np.all(np.isfinite(got))
        # a p below 2^-126 may be taken as 0, and so may a result
        assert np.all(np.abs(got - ref) <= bound + 2.0 ** -126 * (1 + gs + hs))
        assert np.all(got[(xh == -INF) & (np.arange(v)[None] != th[:, None])] == 0) and np.all(got[~live] == 0)


@pytest.mark.parametrize("v", [1, 2, 5, 8, 9, 255, 2048, 2049, 8191, 8192, 8193, 16384, 16392, 32000, 50001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_vocabularies(v, dtype):
    rows = 4
    say(f"logprob V={v} {dtype}")
    x = logits(rows, v, dtype, v)
    t = torch.tensor([0, v - 1, v // 2, v // 3]).cuda()
    for top in sorted({0, 1, min(5, v), min(16, v)}):
        check(x, t, top, v)


@pytest.mark.parametrize("v,pitch", [(31, 32), (1001, 1003), (8193, 8200), (32000, 32007)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_pitch(v, pitch, dtype):
    """The padding holds NaN: nothing of it is read into a row."""
    say(f"logprob pitch V={v} pitch={pitch}")
    check(logits(5, v, dtype, 7, pitch), torch.tensor([1, 2, 3, 4, v - 1]).cuda(), min(7, v), 3)


def test_many_rows_and_the_largest_vocabulary():
    say("logprob many rows")
    check(logits(700, 129, torch.bfloat16, 2), torch.arange(700).cuda() % 129, 5, 1)
    say("logprob 2^19")
    v = 1 << 19
    check(logits(2, v, torch.bfloat16, 4), torch.tensor([5, v - 1]).cuda(), 16, 2)


@pytest.mark.parametrize("top", [1, 16])
def test_ties_go_to_the_lowest_index(top):
    """All equal, few levels, and +0 beside -0 (equal): more candidates than the usual dozens."""
    for v in (16, 300, 8192, 20000):
        say(f"logprob ties V={v} top={top}")
        x = torch.zeros(4, v, dtype=torch.bfloat16, device="cuda")
        x[1] = torch.arange(v, device="cuda") % 2 * -0.0
        x[2] = (torch.arange(v, device="cuda") % 3).bfloat16()
        x[3] = torch.arange(v, device="cuda").flip(0).bfloat16() / v
        check(x, torch.tensor([0, 1, 2, v - 1]).cuda(), top, top)


def test_best_candidates_in_one_place():
    """The largest values side by side in one thread's, one group's and one chunk's elements, ascending."""
    for v, n in ((20000, 8), (20000, 40), (9000, 3000)):
        say(f"logprob neighbours V={v} n={n}")
        x = logits(3, v, torch.float32, n)
        x[0, 4096:4096 + n] = 50 + torch.arange(n, device="cuda") / 64
        x[1, -n:] = 50 + torch.arange(n, device="cuda") / 64
        x[2] = torch.arange(v, device="cuda") / 1024
        check(x, torch.tensor([4096, 7, -1]).cuda(), 16, n)


def test_ruled_out_tokens():
    """Rows with one token, few tokens, none; a ruled-out target; the type's lowest value as a mask."""
    for v in (40, 8500):
        for dtype in (torch.bfloat16, torch.float32):
            say(f"logprob masks V={v} {dtype}")
            x = logits(7, v, dtype, 9)
            low = torch.finfo(dtype).min
            x[0] = -INF                         # nothing allowed
            x[1, 1:] = -INF                     # one token
            x[2, 3:] = -INF
            x[3, :-2] = -INF                    # only the last chunk holds something
            x[4] = low                          # all at the lowest finite value: uniform
            x[5, ::2] = low
            x[6, 5] = -INF
            t = torch.tensor([2, 0, 7, v - 1, 3, 1, 5]).cuda()
            check(x, t, 5, 1)


def test_rows_without_target():
    say("logprob targets outside the vocabulary")
    x = logits(5, 77, torch.bfloat16, 1)
    check(x, torch.tensor([-100, 77, 1 << 40, -(1 << 60), 3]).cuda(), 2, 1)


def test_large_and_close_logits():
    """Entropy of logits near 1000 and of a nearly certain row."""
    say("logprob large logits")
    x = logits(3, 5000, torch.float32, 6, spread=1.0)
    x[0] += 1000.0
    x[1] -= 1000.0
    x[2, 17] = 40.0
    check(x, torch.tensor([1, 2, 17]).cuda(), 3, 1)
    x = logits(3, 20000, torch.float32, 7, spread=1.0)
    x[0] = -1e9                             # a finite mask over everything: uniform, whatever lse can hold
    x[1] += 1e6
    x[2] -= 3e4
    check(x, torch.tensor([1, 2, 17]).cuda(), 3, 1)


def test_a_row_with_nan_or_infinity():
    """Its results are NaN, its gradient too; the other rows keep their bits and the indices stay in range."""
    import bit_nf4_quantized_13_amd as q
    for v, rows in ((40, 6), (9000, 6), (9000, 300), (40000, 6)):
        say(f"logprob NaN V={v} rows={rows}")
        x = logits(rows, v, torch.bfloat16, v)
        t = torch.arange(rows).cuda() % 7
        clean = q.qlora_logprob_fwd(x, t, top=5)
        dl, de = torch.ones(rows, device="cuda"), torch.ones(rows, device="cuda")
        want = q.qlora_logprob_bwd(x, t, clean[2], clean[1], dl, de)
        x[1, v - 2] = float("nan")
        x[2, :] = float("nan")
        x[3, 17] = INF
        x[4, :] = -INF
        x[4, 3] = float("nan")
        logp, ent, lse, tl, ti = q.qlora_logprob_fwd(x, t, top=5)
        d = q.qlora_logprob_bwd(x, t, lse, None, dl, None)
        d2 = q.qlora_logprob_bwd(x, t, lse, ent, dl, de)
        bad, keep = [1, 2, 3, 4], [0, *range(5, rows)]
        for r in (logp, ent, lse, tl, d, d2):
            assert bool(r[bad].isnan().all())
        assert bool(((ti >= -1) & (ti < v)).all())
        for a, b in zip((logp, ent, lse, tl, ti, d2), (*clean, want)):
            assert torch.equal(a[keep], b[keep])


def test_in_place_gradient_and_reruns():
    import bit_nf4_quantized_13_amd as q
    say("logprob in place")
    x = logits(33, 20007, torch.bfloat16, 12, pitch=20010)
    x[3] = torch.finfo(torch.bfloat16).min      # normalised anew before it is overwritten
    x[4] += 30000.0
    t = torch.arange(33).cuda() * 17
    logp, ent, lse, tl, ti = q.qlora_logprob_fwd(x, t, top=4)
    again = q.qlora_logprob_fwd(x, t, top=4)
    assert all(torch.equal(a, b) for a, b in zip((logp, ent, lse, tl, ti), again))
    dl, de = torch.randn(33, device="cuda"), torch.randn(33, device="cuda")
    want = q.qlora_logprob_bwd(x, t, lse, ent, dl, de)
    got = q.qlora_logprob_bwd(x, t, lse, ent, dl, de, out=x)
    assert got is x and torch.equal(x, want)


def test_gradient_against_differences():
    import bit_nf4_quantized_13_amd as q
    say("logprob differences")
    x = logits(3, 11, torch.float32, 31, spread=1.0)
    t = torch.tensor([3, 10, -1]).cuda()
    logp, ent, lse, _, _ = q.qlora_logprob_fwd(x, t)
    dl, de = torch.tensor([0.7, -1.3, 2.0]).cuda(), torch.tensor([0.5, 0.25, -1.0]).cuda()
    got = host(q.qlora_logprob_bwd(x, t, lse, ent, dl, de))
    xh, h = host(x), 1e-5
    diff = np.zeros_like(xh)
    for i in np.ndindex(*xh.shape):
        both = []
        for sign in (1, -1):
            m = xh.copy()
            m[i] += sign * h
            a, b = step.logprob(m, t.cpu().numpy())[:2]
            both.append((host(dl) * a + host(de) * b).sum())
        diff[i] = (both[0] - both[1]) / (2 * h)
    assert np.abs(got - diff).max() <= 1e-5

"""Layer norm's forward and backward against the 64-bit oracle: widths around
every change of layout (64, 256, 512 and 1024 threads a row, rows that are read
again), odd widths and pitches, rows that start at no 16-byte boundary.

Bounds: a sum of the kernel is a tree of at most 64 fp32 additions deep, so its
error is within 64 u of the sum of magnitudes (u = 2^-24); a stored bf16 adds
2^-8 of the value, its largest rounding (8 significant bits)."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
WIDTHS = [1, 7, 8, 9, 64, 511, 512, 513, 1024, 1031, 2048, 2049, 4096, 4100, 8192, 8195, 16384, 16385, 20011]


def tensors(rows, n, dtype, wdtype, seed, pitch=None, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    store = torch.zeros(rows, pitch or n)
    store[:, :n] = torch.randn(rows, n, generator=g) + offset
    x = store.to(dtype).cuda()[:, :n]
    dy = torch.randn(rows, n, generator=g).to(dtype).cuda()
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(wdtype).cuda()
    b = (0.2 * torch.randn(n, generator=g)).to(wdtype).cuda()
    return x, dy, w, b


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    assert np.all(np.isfinite(got)), what
    excess = np.abs(got - want) - bound
    assert excess.max() <= 0, f"{what}: {excess.max():.3e} beyond the bound"


def check(rows, n, dtype, wdtype, seed, pitch=None, affine=True):
    import bit_nf4_quantized_13_amd as q
    say(f"layernorm rows={rows} n={n} {dtype} {wdtype} pitch={pitch} affine={affine}")
    x, dy, w, b = tensors(rows, n, dtype, wdtype, seed, pitch)
    w, b = (w, b) if affine else (None, None)
    y, mean, rstd = q.qlora_layernorm_fwd(x, w, b, eps=1e-5)
    dx, dw, db = q.qlora_layernorm_bwd(x, dy, mean, rstd, w)
    dx2, none_w, none_b = q.qlora_layernorm_bwd(x, dy, mean, rstd, w, need_dw=False, need_db=False)
    torch.cuda.synchronize()
    assert none_w is None and none_b is None
    xh, dyh = host(x), host(dy)
    wh, bh = (host(w), host(b)) if affine else (None, None)
    y_ref, mean_ref, rstd_ref = step.layernorm(xh, wh, bh)
    store = 2.0 ** -8 if dtype == torch.bfloat16 else 2 * U
    wa = np.abs(wh) if affine else 1.0
    ba = np.abs(bh) if affine else 0.0
    scale = np.abs(xh).max(1, keepdims=True)
    within(host(mean)[:, None], mean_ref[:, None], 64 * U * scale, "mean")
    # the deviations carry the mean's error, their squares twice that, the root half
    within(host(rstd)[:, None] / rstd_ref[:, None], 1.0, 160 * U * (1 + scale * rstd_ref[:, None]), "rstd")
    unit = scale * rstd_ref[:, None] * (1 + scale * rstd_ref[:, None])
    within(host(y), y_ref, store * np.abs(y_ref) + 256 * U * (unit * wa + ba), "y")
    # the backward against the same statistics that the kernel was given
    dx_ref, dw_ref, db_ref = step.layernorm_backward(xh, dyh, host(mean), host(rstd), wh)
    hat = np.abs(xh - host(mean)[:, None]) * host(rstd)[:, None] + np.abs(scale) * host(rstd)[:, None] * U
    g = np.abs(dyh) * wa
    size = host(rstd)[:, None] * (g + g.mean(1, keepdims=True) + hat * (g * hat).mean(1, keepdims=True))
    for got in (dx, dx2):
        within(host(got), dx_ref, store * np.abs(dx_ref) + 80 * U * size, "dx")
    rows_deep = 96 + rows / 64
    within(host(dw), dw_ref, rows_deep * U * (np.abs(dyh) * hat).sum(0), "dw")
    within(host(db), db_ref, rows_deep * U * np.abs(dyh).sum(0), "db")
    # the same bits again, and alone
    again = q.qlora_layernorm_bwd(x, dy, mean, rstd, w)
    assert all(torch.equal(s, t) for s, t in zip((dx, dw, db), again))
    only_b = q.qlora_layernorm_bwd(x, dy, mean, rstd, w, need_dw=False)
    assert only_b[1] is None and torch.equal(only_b[2], db)


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths(n, dtype):
    for rows in (1, 5):
        check(rows, n, dtype, torch.float32 if n % 2 else torch.bfloat16, 11 * n + rows)


@pytest.mark.parametrize("rows,n", [(300, 64), (4200, 130), (1500, 1025), (700, 2750), (600, 4099), (300, 8192),
                                    (270, 9001), (260, 16500), (5000, 8), (333, 17), (9000, 128), (77, 129), (2100, 255),
                                    (700, 256), (41, 257)])
def test_many_rows(rows, n):
    """More rows than the first pass of the workgroups takes, and than the partial rows."""
    check(rows, n, torch.bfloat16, torch.float32, rows + n)


@pytest.mark.parametrize("n,pitch", [(64, 65), (513, 520), (4096, 4097), (4096, 4104), (16400, 16411)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_pitch_and_no_parameters(n, pitch, dtype):
    check(6, n, dtype, torch.float32, n, pitch=pitch)
    check(3, n, dtype, torch.float32, n + 1, affine=False)


def test_views_at_odd_addresses():
    """Arrays that start one element past a 16-byte boundary give the same bits."""
    import bit_nf4_quantized_13_amd as q
    say("layernorm odd addresses")
    x, dy, w, b = tensors(9, 1000, torch.bfloat16, torch.bfloat16, 3)

    def moved(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return s.copy_(t)
    want = q.qlora_layernorm_fwd(x, w, b)
    got = q.qlora_layernorm_fwd(moved(x), moved(w), moved(b), out=moved(x))
    assert all(torch.equal(s, t) for s, t in zip(want, got))
    y, mean, rstd = want
    assert all(torch.equal(s, t) for s, t in zip(q.qlora_layernorm_bwd(x, dy, mean, rstd, w),
                                                 q.qlora_layernorm_bwd(moved(x), moved(dy), moved(mean), moved(rstd), moved(w))))


def test_large_mean_and_constant_rows():
    """A mean far above the spread keeps the variance; a constant row has y = bias and rstd = eps^-1/2."""
    import bit_nf4_quantized_13_amd as q
    say("layernorm large mean")
    x, _, w, b = tensors(4, 3000, torch.float32, torch.float32, 5, offset=4096.0)
    x[3] = 7.25
    y, mean, rstd = q.qlora_layernorm_fwd(x, w, b, eps=1e-5)
    y_ref, mean_ref, rstd_ref = step.layernorm(host(x), host(w), host(b))
    # the mean is off by at most 64 u 4100, 0.016 of a spread of 1: the variance by its square
    within(host(rstd)[:3] / rstd_ref[:3], 1.0, 64 * U * 8 + (64 * U * 4200) ** 2, "rstd")
    within(host(y)[:3], y_ref[:3], 64 * U * 4200 * (np.abs(host(w)) * 1.01) + 1e-4, "y")
    assert torch.equal(y[3], b) and abs(float(rstd[3]) - 1e-5 ** -0.5) <= 1e-4


def test_gradient_against_differences():
    """dx, dw, db in fp32 against central differences of sum(dy y) in fp64."""
    import bit_nf4_quantized_13_amd as q
    say("layernorm differences")
    x, dy, w, b = tensors(3, 13, torch.float32, torch.float32, 8)
    _, mean, rstd = q.qlora_layernorm_fwd(x, w, b)
    got = [host(t) for t in q.qlora_layernorm_bwd(x, dy, mean, rstd, w)]
    args = [host(x), host(w), host(b)]
    step_size = 1e-5
    for k, index in ((0, 0), (1, 1), (2, 2)):
        diff = np.zeros_like(args[k])
        for i in np.ndindex(*args[k].shape):
            both = []
            for sign in (1, -1):
                moved = [a.copy() for a in args]
                moved[k][i] += sign * step_size
                both.append((host(dy) * step.layernorm(*moved)[0]).sum())
            diff[i] = (both[0] - both[1]) / (2 * step_size)
        # the differences' own error is of the order of step^2 = 1e-10; the kernel's about 100 u
        assert np.abs(got[index] - diff).max() <= 1e-5 * max(1.0, np.abs(diff).max())


def test_other_stream():
    import bit_nf4_quantized_13_amd as q
    x, dy, w, b = tensors(64, 2000, torch.bfloat16, torch.float32, 21)
    want = q.qlora_layernorm_fwd(x, w, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = q.qlora_layernorm_fwd(x, w, b)
        grads = q.qlora_layernorm_bwd(x, dy, got[1], got[2], w)
    side.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(want, got))
    assert all(torch.equal(s, t) for s, t in zip(grads, q.qlora_layernorm_bwd(x, dy, want[1], want[2], w)))

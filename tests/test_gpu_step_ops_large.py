"""The fine-tuning step's operators beyond 2^31 elements, in captured graphs and
on other streams.  Every one treats rows (sequences, blocks) apart from each other
and gives the same bits for the same row, so the oracle of a large call's last rows
is a small call on those rows, which the other tests hold against fp64."""
import pytest
import torch

from tests.helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def lib():
    import bit_nf4_quantized_13_amd as q
    yield q
    torch.cuda.empty_cache()


def test_layernorm_past_2_31_elements(lib):
    say("layernorm past 2^31 elements")
    m, n = 300_001, 7168
    x = torch.randn(1000, n, device="cuda").bfloat16().repeat(301, 1)[:m].contiguous()
    w, b = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    y, mean, rstd = lib.qlora_layernorm_fwd(x, w, b)
    y1, mean1, rstd1 = lib.qlora_layernorm_fwd(x[:1000], w, b)
    for a in (0, 150_000, 299_000):
        assert torch.equal(y[a:a + 1000], y1) and torch.equal(rstd[a:a + 1000], rstd1)
    dx, dw, db = lib.qlora_layernorm_bwd(x, y, mean, rstd, w)
    dx1, dw1, db1 = lib.qlora_layernorm_bwd(x[:1000], y1, mean1, rstd1, w)
    for a in (0, 150_000, 299_000):
        assert torch.equal(dx[a:a + 1000], dx1)
    last = lib.qlora_layernorm_bwd(x[300_000:], y[300_000:], mean[300_000:], rstd[300_000:], w)
    # 300 times the first thousand rows and one more; fp32 sums in 256 partials of at most
    # 1172 rows and their total of 256: 1428 roundings of 2^-24 of the magnitudes' sum
    for got, one, tail, size in zip((dw, db), (dw1, db1), last[1:],
                                    (lambda: (y1.double() * (x[:1000].double() - mean1[:, None]) * rstd1[:, None]).abs().sum(0),
                                     lambda: y1.double().abs().sum(0))):
        want = 300.0 * one.double() + tail.double()
        assert bool(((got.double() - want).abs() <= 301 * size() * 2.0 ** -24 * 2 * 1428).all())


def test_logprob_past_2_31_elements(lib):
    say("logprob past 2^31 elements")
    m, v = 70_000, 32_000
    x = torch.randn(1000, v, device="cuda").bfloat16().repeat(70, 1)
    t = torch.arange(1000, device="cuda").repeat(70) * 31 % v
    out = lib.qlora_logprob_fwd(x, t, top=3)
    one = lib.qlora_logprob_fwd(x[:1000], t[:1000], top=3)
    for a, b in zip(out, one):
        assert torch.equal(a[-1000:], b) and torch.equal(a[35_000:36_000], b)
    g = torch.randn(1000, device="cuda")
    want = lib.qlora_logprob_bwd(x[:1000], t[:1000], one[2], one[1], g, g)
    got = lib.qlora_logprob_bwd(x, t, out[2], out[1], g.repeat(70), g.repeat(70), out=x)
    assert torch.equal(got[-1000:], want) and torch.equal(got[35_000:36_000], want)


def test_more_rows_than_one_launch_takes(lib):
    """A launch's threads are fewer than 2^32: rows beyond are launched after one another."""
    say("layernorm 2^26 rows")
    m, n = (1 << 26) + 5, 8
    x = torch.randn(1001, n, device="cuda").bfloat16().repeat(m // 1001 + 1, 1)[:m].contiguous()
    y, mean, rstd = lib.qlora_layernorm_fwd(x)
    y1, mean1, rstd1 = lib.qlora_layernorm_fwd(x[:1001])
    dx = lib.qlora_layernorm_bwd(x, y, mean, rstd, need_dw=False, need_db=False)[0]
    dx1 = lib.qlora_layernorm_bwd(x[:1001], y1, mean1, rstd1, need_dw=False, need_db=False)[0]
    for got, one in ((y, y1), (mean, mean1), (rstd, rstd1), (dx, dx1)):
        whole = m // 1001 * 1001
        assert bool((got[:whole].view(-1, *one.shape) == one).all()) and torch.equal(got[whole:], one[:m - whole])
    say("logprob 2^23 rows")
    m, v = (1 << 23) + 9, 9
    x = torch.randn(1001, v, device="cuda").bfloat16().repeat(m // 1001 + 1, 1)[:m].contiguous()
    t = torch.arange(1001, device="cuda").repeat(m // 1001 + 1)[:m] % 10
    out = lib.qlora_logprob_fwd(x, t, top=2)
    one = lib.qlora_logprob_fwd(x[:1001], t[:1001], top=2)
    g = torch.ones(m, device="cuda")
    d = lib.qlora_logprob_bwd(x, t, out[2], out[1], g, g)
    d1 = lib.qlora_logprob_bwd(x[:1001], t[:1001], one[2], one[1], g[:1001], g[:1001])
    for got, want in (*zip(out, one), (d, d1)):
        whole = m // 1001 * 1001
        assert bool((got[:whole].view(-1, *want.shape) == want).all()) and torch.equal(got[whole:], want[:m - whole])


def test_attention_past_2_31_elements(lib):
    """2^31 + elements of q and of each gradient; the sequences are short."""
    say("attention past 2^31 elements")
    h, hk, d, per, copies = 16, 4, 64, 700, 3001
    draw = lambda n: torch.randn(per, n, d, device="cuda").bfloat16()  # noqa: E731
    q1, k1, v1, do1 = draw(h), draw(hk), draw(hk), draw(h)
    starts = torch.tensor([0, 1, 300, 431, 700], dtype=torch.int32, device="cuda")
    q, k, v, do = (t.repeat(copies, 1, 1) for t in (q1, k1, v1, do1))
    cu = torch.cat([starts[:-1] + i * per for i in range(copies)] + [starts[-1:] + (copies - 1) * per])
    assert q.numel() > 1 << 31
    o, lse, res = lib.qlora_attention_fwd(q, k, v, cu, save_residual=True)
    o1, lse1, res1 = lib.qlora_attention_fwd(q1, k1, v1, starts, save_residual=True)
    grads = lib.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res)
    # the whole call adds a group's heads in one workgroup, the small one in partials: fp32 sums
    # of the same products in another order, rounded to bf16 once
    first = lib.qlora_attention_bwd(q1, k1, v1, o1, lse1, do1, starts, residual=res1)
    for a in (0, 1500, copies - 1):
        part = slice(a * per, (a + 1) * per)
        assert torch.equal(o[part], o1) and torch.equal(res[part], res1) and torch.equal(lse[:, part], lse1)
        assert torch.equal(grads[0][part], first[0])
        for got, want in zip(grads[1:], first[1:]):
            scale = want.float().abs().max()
            assert bool(((got[part].float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -12 * scale).all())
            assert torch.equal(got[part], got[:per])


@pytest.mark.parametrize("bits8", [False, True])
def test_adamw_past_2_31_elements(lib, bits8):
    say(f"adamw past 2^31 elements, 8 bits {bits8}")
    n, tail = (1 << 31) + 2048 * 3 + 77, 2048 * 2 + 77
    p = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_()
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_()
    p1, g1 = p[-tail:].clone(), g[-tail:].clone()
    big = lib.AdamWPlan.zeros([p], [g], bits8=bits8)
    small = lib.AdamWPlan.zeros([p1], [g1], bits8=bits8)
    for step in (1, 2):
        lib.qlora_adamw_step(big, lr=0.01, step=step)
        lib.qlora_adamw_step(small, lr=0.01, step=step)
    assert torch.equal(p[-tail:], p1)
    assert all(torch.equal(big.tensors[i][0][-tail:], small.tensors[i][0]) for i in (2, 3))


def operators(lib, seed):
    """The operators on small inputs, as one function that rewrites its outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(65, 520, generator=g, device="cuda").bfloat16()
    w = torch.randn(520, generator=g, device="cuda")
    logits = torch.randn(33, 20_000, generator=g, device="cuda").bfloat16()
    t = torch.arange(33, device="cuda") * 600
    p = torch.randn(5000, generator=g, device="cuda").bfloat16()
    grad = torch.zeros(5000, device="cuda")
    plan = lib.AdamWPlan.zeros([p], [grad], bits8=True, master=True)

    def run():
        y, mean, rstd = lib.qlora_layernorm_fwd(x, w, None)
        norm = lib.qlora_layernorm_bwd(x, y, mean, rstd, w, need_db=True)
        out = lib.qlora_logprob_fwd(logits, t, top=4)
        dl = lib.qlora_logprob_bwd(logits, t, out[2], out[1], out[0], out[1])
        grad.copy_(dl.view(-1)[:5000])
        lib.qlora_adamw_step(plan, lr=0.01, step=1)
        return [y, *norm, *out, dl]

    return run, plan


def states(plan):
    """The tensors that a step changes."""
    return [plan.tensors[i][0] for i in (0, 2, 3, 4, 5, 6)]


def test_streams_and_graphs(lib):
    """On another stream, and captured: every replay, with eager work and waits between, gives the eager bits."""
    say("operators on a stream and in a graph")
    run, plan = operators(lib, 1)
    want = [t.clone() for t in run()]
    state = [t.clone() for t in states(plan)]
    side = torch.cuda.Stream()
    run2, plan2 = operators(lib, 1)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run2()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(states(plan2), state))
    run3, plan3 = operators(lib, 1)
    start = [t.clone() for t in states(plan3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run3()
    for _ in range(4):
        for t in got:
            t.zero_()
        for t, s in zip(states(plan3), start):
            t.copy_(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(states(plan3), state))
        run()  # eager work between the replays
        torch.cuda.synchronize()

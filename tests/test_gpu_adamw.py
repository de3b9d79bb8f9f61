"""AdamW over lists of tensors: states in fp32 and in 8 bits bit for bit against
the oracle's fp32 steps, weights against 64 bits.

Bounds on a weight (u = 2^-24): the update's few operations to 8 u of itself,
the weight's to 3 u; a stored bf16 adds 2^-8 of the value."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RATES = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05)


def f32(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def make(sizes, pdtype, gdtype, bits8, master, seed, shift=0):
    """Plan, with arrays that start `shift` elements past their allocation."""
    import bit_nf4_quantized_13_amd as q
    g = torch.Generator().manual_seed(seed)

    def put(t):
        s = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")[shift:]
        return s.copy_(t)
    ps, gs, ms, vs, mss, vss, ws = [], [], [], [], [], [], []
    for n in sizes:
        p = 0.1 * torch.randn(n, generator=g)
        ps.append(put(p.to(pdtype)))
        gs.append(put((torch.randn(n, generator=g) * torch.exp(2 * torch.randn(n, generator=g)) * 1e-2).to(gdtype)))
        m = (1e-2 * torch.randn(n, generator=g)).numpy()
        v = (1e-2 * torch.randn(n, generator=g)).square().numpy()
        if n > 600:
            m[256:512], v[256:512] = 0, 0        # a block of states at the start
            gs[-1][256:300] = 0                  # and of gradients that are zero
        if bits8:
            (mc, m_s), (vc, v_s) = step.encode_m(m), step.encode_v(v)
            ms.append(put(torch.from_numpy(mc))), vs.append(put(torch.from_numpy(vc)))
            mss.append(put(torch.from_numpy(m_s))), vss.append(put(torch.from_numpy(v_s)))
        else:
            ms.append(put(torch.from_numpy(m))), vs.append(put(torch.from_numpy(v)))
        if master:
            ws.append(put(p))
    return q.AdamWPlan(ps, gs, ms, vs, mss if bits8 else None, vss if bits8 else None, ws if master else None)


def codes(t):
    return t.cpu().numpy().reshape(-1)


def snapshot(plan):
    return [[t.clone() if t is not None else None for t in ts] for ts in plan.tensors]


def check_step(plan, number, grad_scale=1.0):
    import bit_nf4_quantized_13_amd as q
    before = snapshot(plan)
    q.qlora_adamw_step(plan, step=number, grad_scale=grad_scale, **RATES)
    torch.cuda.synchronize()
    for i in range(plan.count):
        p, g, m, v, ms, vs, w = (ts[i] for ts in before)
        p1, g1, m1, v1, ms1, vs1, w1 = (ts[i] for ts in plan.tensors)
        assert torch.equal(g, g1)
        if not p.numel():
            continue
        if plan.bits8:
            m0, v0 = step.decode_m(codes(m), f32(ms)), step.decode_v(codes(v), f32(vs))
        else:
            m0, v0 = f32(m), f32(v)
        mn, vn = step.adamw_states(m0, v0, f32(g), RATES["beta1"], RATES["beta2"], grad_scale)
        if plan.bits8:
            for got, gs, (code, scale) in ((m1, ms1, step.encode_m(mn)), (v1, vs1, step.encode_v(vn))):
                assert np.array_equal(codes(got), code)
                assert np.array_equal(f32(gs).view(np.uint32), scale.view(np.uint32))
        else:
            assert np.array_equal(f32(m1), mn) and np.array_equal(f32(v1), vn)
        start = f32(w if plan.master else p)
        ref = step.adamw_param(start, mn, vn, step=number, **RATES)
        bound = 3 * U * np.abs(start) + 8 * U * np.abs(ref - start) + U * np.abs(ref)
        if plan.master:
            assert np.all(np.abs(f32(w1) - ref) <= bound)
            assert torch.equal(p1.reshape(-1), w1.reshape(-1).bfloat16())
        else:
            stored = 2.0 ** -8 * np.abs(ref) if p.dtype == torch.bfloat16 else 0
            assert np.all(np.abs(f32(p1) - ref) <= bound * (1 + 2.0 ** -8) + stored)


SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 5000, 8 * 4096]


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("pdtype,master", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, False)])
@pytest.mark.parametrize("gdtype", [torch.bfloat16, torch.float32])
def test_steps(bits8, pdtype, master, gdtype):
    say(f"adamw bits8={bits8} {pdtype} master={master} {gdtype}")
    plan = make(SIZES, pdtype, gdtype, bits8, master, 5)
    check_step(plan, 1)
    check_step(plan, 2)
    check_step(plan, 100000, grad_scale=0.37)


@pytest.mark.parametrize("bits8", [False, True])
def test_odd_addresses(bits8):
    say(f"adamw odd addresses bits8={bits8}")
    check_step(make([1, 300, 4099], torch.bfloat16, torch.float32, bits8, True, 6, shift=1), 3)
    check_step(make([1, 300, 4099], torch.bfloat16, torch.bfloat16, bits8, False, 6, shift=3), 3)


def test_more_tensors_than_one_launch_and_empty_ones():
    say("adamw many tensors")
    sizes = [0 if i % 7 == 3 else 1 + 97 * i % 1500 for i in range(131)]
    check_step(make(sizes, torch.bfloat16, torch.float32, True, False, 7), 4)
    check_step(make([0, 0], torch.float32, torch.float32, False, False, 7), 4)


def test_from_zero_states_and_moments():
    """New states are zeros; a few steps; the values that 8-bit states stand for."""
    import bit_nf4_quantized_13_amd as q
    say("adamw zeros")
    g = torch.Generator().manual_seed(1)
    ps = [torch.randn(700, generator=g).bfloat16().cuda(), torch.randn(8, 64, generator=g).bfloat16().cuda()]
    gs = [torch.randn(p.shape, generator=g).cuda() for p in ps]
    plan = q.AdamWPlan.zeros(ps, gs, bits8=True, master=True)
    for i in range(1, 4):
        check_step(plan, i)
    m, v = q.qlora_adamw_moments(plan)
    for i in range(2):
        _, _, mc, vc, ms, vs, _ = (ts[i] for ts in plan.tensors)
        assert np.array_equal(f32(m[i]), step.decode_m(codes(mc), f32(ms)))
        assert np.array_equal(f32(v[i]), step.decode_v(codes(vc), f32(vs)))
        assert m[i].shape == ps[i].shape


def test_states_of_extreme_size():
    """Blocks that are all zero, tiny enough to be stored as zeros, or hold one large value; v > 0 stays so."""
    import bit_nf4_quantized_13_amd as q
    say("adamw extremes")
    n = 256 * 6
    grad = torch.zeros(n)
    grad[256:512] = 1e-22
    grad[512:768] = 1e-6
    grad[600] = 1e4
    grad[768:1024] = 1e18
    grad[1024] = -3.0
    grad[1280:] = torch.logspace(-8, 0, 256)
    plan = q.AdamWPlan.zeros([torch.zeros(n, device="cuda")], [grad.cuda()], bits8=True)
    check_step(plan, 1)
    check_step(plan, 2)
    v = plan.tensors[3][0].cpu().numpy()
    assert np.all(v[512:768] >= 1) and np.all(v[1280:] >= 1) and np.all(v[:256] == 0)


def test_no_eps_and_gradients_below_the_normal_range_of_their_squares():
    """eps = 0: the update is m over the root of v also where v is denormal."""
    import bit_nf4_quantized_13_amd as q
    say("adamw eps 0")
    grad = torch.full((300,), 1e-20)
    grad[::2] = -0.5
    p = torch.zeros(300).cuda()
    q.qlora_adamw_step(q.AdamWPlan.zeros([p], [grad.cuda()], bits8=False), lr=0.25, step=1, eps=0.0)
    # v = 1e-3 g^2 (1e-43 for the small ones, held to 1 in 70 by its spacing), m = 0.1 g: the step is lr
    assert np.all(np.abs(f32(p)[::2] - 0.25) <= 1e-6)
    assert np.all(np.abs(f32(p)[1::2] + 0.25) <= 0.25 / 100)


def test_8bit_states_follow_32bit_ones():
    """A quadratic's descent with 8-bit states ends where fp32 states end."""
    import bit_nf4_quantized_13_amd as q
    say("adamw descent")
    g = torch.Generator().manual_seed(3)
    want, ends = torch.randn(4096, generator=g).cuda(), []
    for bits8 in (False, True):
        p, grad = torch.zeros(4096, device="cuda"), torch.zeros(4096, device="cuda")
        plan = q.AdamWPlan.zeros([p], [grad], bits8=bits8)
        for i in range(1, 301):
            grad.copy_(p - want)
            q.qlora_adamw_step(plan, lr=0.02, step=i)
        ends.append(float((p - want).norm() / want.norm()))
    # 300 steps of 0.02 reach every target of a few units; both end near them
    assert ends[0] < 0.05 and ends[1] < 0.05, ends

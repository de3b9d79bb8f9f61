"""Values that are not finite in the operators around the projections: what they
reach, and what keeps its value beside them."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.helpers import say

pytestmark = pytest.mark.gpu


def test_nan_is_no_alternative():
    """A row with NaN names the other logits in their order, -1 where none are left; short rows, in which every
    element is looked at, as long ones."""
    import bit_nf4_quantized_13_amd as q
    for v, rows in ((5, 4), (40, 4), (300, 4), (9000, 4), (9000, 300), (40000, 4)):
        for dtype in (torch.bfloat16, torch.float32):
            say(f"logprob NaN alternatives V={v} rows={rows} {dtype}")
            x = (3 * torch.randn(rows, v, generator=torch.Generator().manual_seed(v))).to(dtype).cuda()
            x[1, ::2] = float("nan")
            x[2, 1:] = float("nan")
            x[3, 1] = -float("nan")
            top = min(5, v)
            ids = q.qlora_logprob_fwd(x, torch.zeros(rows, dtype=torch.int64, device="cuda"), top=top)[4]
            for i in range(4):
                row = x[i].float().cpu().numpy()
                order = [int(j) for j in np.argsort(-row, kind="stable") if row[j] == row[j]][:top]  # NaN last
                assert ids[i].tolist() == order + [-1] * (top - len(order)), i


def test_8bit_states_keep_damage_to_the_element():
    """Infinite, NaN and huge gradients (whose squares overflow) in blocks of 8-bit states: the blocks' other elements
    have the codes, scales and weights of a block without them; the element's own m and v are NaN from then on."""
    import bit_nf4_quantized_13_amd as q
    say("adamw not finite")
    n, lost = 256 * 5 + 77, [3, 256 + 255, 512, 513, 700, 256 * 5 + 76]
    g = torch.Generator().manual_seed(5)
    grads = [1e-2 * torch.randn(n, generator=g) for _ in range(3)]
    bad = [t.clone() for t in grads]
    bad[1][lost] = torch.tensor([float("inf"), float("nan"), -float("inf"), 1e25, -1e30, float("nan")])
    bad[1][768:1024] = float("inf")  # a block without any other element
    keep = np.ones(n, dtype=bool)
    keep[lost] = keep[768:1024] = False
    start = torch.randn(n, generator=g)
    plans = []
    for series in (grads, bad):
        p, grad = start.clone().cuda(), torch.zeros(n, device="cuda")
        plan = q.AdamWPlan.zeros([p], [grad], bits8=True)
        mn, vn = np.zeros(n, dtype=np.float32), np.zeros(n, dtype=np.float32)
        for i, t in enumerate(series):
            grad.copy_(t)
            q.qlora_adamw_step(plan, lr=1e-2, step=i + 1)
            with np.errstate(over="ignore", invalid="ignore"):
                mn, vn = step.adamw_states(mn, vn, t.numpy(), 0.9, 0.999)
                # the contract on the elements that are finite: the others as zeros
                gone = ~(np.isfinite(mn) & np.isfinite(vn))
            (mc, ms), (vc, vs) = step.encode_m(np.where(gone, 0, mn)), step.encode_v(np.where(gone, 0, vn))
            assert np.array_equal(plan.tensors[2][0].cpu().numpy(), np.where(gone, -128, mc))
            assert np.array_equal(plan.tensors[3][0].cpu().numpy(), np.where(gone, 0, vc))
            assert np.array_equal(plan.tensors[4][0].cpu().numpy(), ms)
            assert np.array_equal(plan.tensors[5][0].cpu().numpy(), vs)
            mn, vn = (np.where(gone, np.float32("nan"), dec) for dec in (step.decode_m(mc, ms), step.decode_v(vc, vs)))
            values = [t[0].cpu().numpy() for t in q.qlora_adamw_moments(plan)]
            assert np.array_equal(values[0], mn, equal_nan=True) and np.array_equal(values[1], vn, equal_nan=True)
        if series is bad:
            assert np.array_equal(gone, ~keep)
        plans.append(plan)
    weights = [plan.tensors[0][0].cpu().numpy() for plan in plans]
    assert np.all(np.isfinite(weights[1][keep])) and np.all(np.isnan(weights[1][~keep]))
    # a block's scales may differ where the lost element had held them: whole blocks without one keep their bits
    whole = np.repeat([not (~keep[a:a + 256]).any() for a in range(0, n, 256)], 256)[:n]
    assert whole.any() and np.array_equal(weights[0][whole], weights[1][whole])

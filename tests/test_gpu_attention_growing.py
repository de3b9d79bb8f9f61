"""Attention's gradients where the running maximum moves from tile to tile."""
import numpy as np
import pytest
import torch

import tests.test_gpu_attention as base
from oracle import step
from tests.helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,h,hk,d", [(150, 2, 1, 64), (150, 1, 1, 128), (400, 1, 1, 64), (400, 1, 1, 128), (420, 80, 40, 64)])
def test_gradients_of_growing_scores(t, h, hk, d, monkeypatch):
    """Maxima that rise tile after tile, to scores of 270: an exponential's argument is off by 2^-24 of that and
    of the sums on its way, 4 times the share that the bounds' fp32 term has for scores below 100."""
    import bit_nf4_quantized_13_amd as q_
    say(f"attention growing scores T={t} heads={h}/{hk} dim={d}")
    monkeypatch.setattr(base, "SMALL", 4 * base.SMALL)
    q, k, v, do, starts, cu = base.make([t], 0, h, hk, d, 12)
    q.fill_(1.0)
    k.copy_((torch.arange(t).view(t, 1, 1) * (0.64 / d)).expand(t, hk, d))
    o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, 1.0, save_residual=True)
    grads = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, 1.0, residual=res)
    exact = [base.host(x) for x in (q, k, v, do)]
    ro, rl, *refs = step.attention(*exact[:3], starts, 1.0, exact[3])
    bo, *bounds = base.bounds(*exact, starts, 1.0, True)
    assert np.all(np.abs(base.host(lse) - rl) <= base.SMALL * (1 + np.abs(rl)))
    assert np.all(np.abs(base.host(o) - ro) <= bo + base.R * np.abs(ro))
    for got, ref, b, name in zip(grads, refs, bounds, ("dq", "dk", "dv")):
        excess = np.abs(base.host(got) - ref) - (b * (1 + base.R) + base.R * np.abs(ref))
        assert excess.max() <= 1e-30, f"{name}: {excess.max():.3e} beyond the bound"

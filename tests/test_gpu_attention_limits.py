"""Attention at the largest row pitch."""
import pytest
import torch

import tests.test_gpu_attention as base
from tests.helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,h,hk,d", [(140, 3, 1, 40), (330, 2, 1, 128), (420, 80, 40, 64)])
def test_largest_pitch(t, h, hk, d):
    """Rows 2^23 elements apart: a tile of 128 spans 2^31 bytes.  The same bits as dense rows."""
    import bit_nf4_quantized_13_amd as q_
    say(f"attention pitch 2^23 T={t} heads={h}/{hk} dim={d}")
    q, k, v, do, _, cu = base.make([t], 0, h, hk, d, t)
    wide = torch.zeros(t * (1 << 23), dtype=torch.bfloat16, device="cuda").view(t, 1 << 23)
    far, at = [], 0
    for x in (q, k, v, q, k, v):
        n = x.shape[1] * d
        far.append(wide[:, at:at + n].view(t, -1, d))
        at += n
    for x, y in zip(far, (q, k, v)):
        x.copy_(y)
    o, lse, res = q_.qlora_attention_fwd(q, k, v, cu, save_residual=True)
    o2, lse2, res2 = q_.qlora_attention_fwd(*far[:3], cu, save_residual=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(res, res2)
    want = q_.qlora_attention_bwd(q, k, v, o, lse, do, cu, residual=res)
    got = q_.qlora_attention_bwd(*far[:3], o, lse, do, cu, residual=res, outs=tuple(far[3:]))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del wide, far, got
    torch.cuda.empty_cache()

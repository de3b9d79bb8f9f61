"""Values that are not finite in the operators around the projections: what they
reach, and what keeps its value beside them."""
import numpy as np
import pytest
import torch

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

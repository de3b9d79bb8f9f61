"""Workspaces that the caller gives: taken as they are, and refused before any launch where
the kernels could not write to them as one piece of device memory."""
import pytest
import torch

from tests.helpers import say

pytestmark = pytest.mark.gpu


def calls():
    import bit_nf4_quantized_13_amd as q
    x = torch.randn(6, 9000, device="cuda")
    y, mean, rstd = q.qlora_layernorm_fwd(x)
    t = torch.arange(6, device="cuda")
    a = torch.randn(40, 2, 64, device="cuda").bfloat16()
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    o, lse, _ = q.qlora_attention_fwd(a, a, a, cu)
    return {"layernorm": lambda ws: q.qlora_layernorm_bwd(x, y, mean, rstd, workspace=ws),
            "logprob": lambda ws: q.qlora_logprob_fwd(x, t, top=3, workspace=ws),
            "attention": lambda ws: q.qlora_attention_bwd(a, a, a, o, lse, a, cu, workspace=ws)}


@pytest.mark.parametrize("name", ["layernorm", "logprob", "attention"])
def test_given_workspaces(name):
    import bit_nf4_quantized_13_amd as q
    say(f"workspace {name}")
    call, size = calls()[name], 1 << 22
    want, got = call(None), call(torch.empty(size, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(ValueError, match="workspace"):
        call(torch.empty(size, dtype=torch.uint8))                            # on the host
    with pytest.raises(ValueError, match="workspace"):
        call(torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2])    # with holes
    with pytest.raises(q.QloraError):
        call(torch.empty(15, dtype=torch.uint8, device="cuda"))                 # fewer than any call needs

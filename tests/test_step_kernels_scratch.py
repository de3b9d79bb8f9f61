"""No kernel of the operators around the projections keeps values in scratch memory:
spilled registers cost time without any wrong result to show it.  No GPU."""
import os
import re
import shutil
import subprocess

import pytest

from bit_nf4_quantized_13_amd import build


@pytest.mark.parametrize("source", ["layernorm", "attention", "logprob", "adamw"])
def test_no_scratch(source, tmp_path):
    if shutil.which(build.HIPCC) is None:
        pytest.skip("no hipcc")
    out = tmp_path / "kernels.s"
    subprocess.run([build.HIPCC, "-x", "hip", "-S", "--cuda-device-only", os.path.join(build.CSRC, source + ".hip"), "-o",
                    str(out)] + build.COMMON_FLAGS, check=True, capture_output=True, timeout=300)
    meta = out.read_text().rpartition(".amdgpu_metadata")[2]
    sizes = dict(re.findall(r"\.name:\s+(\S+)\n\s+\.private_segment_fixed_size:\s+(\d+)", meta))
    assert sizes
    assert not {n: s for n, s in sizes.items() if s != "0"}

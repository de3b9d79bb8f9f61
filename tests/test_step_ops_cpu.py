"""The C ABI of the operators around the linear layer on the host: arguments are
refused with the documented status before anything is launched, structs have the
header's layout, and the oracle's formulas agree with differences.  No GPU."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import bit_nf4_quantized_13_amd as q
from oracle import step
from tests.conftest import ROOT

FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation


def norm_fwd(x=FAKE, xt=0, m=4, n=64, ld=64, w=FAKE, b=FAKE, wt=0, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE):
    return q.library().qlora_layernorm_fwd(x, xt, m, n, ld, w, b, wt, eps, y, mean, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), q.QLORA_EINVAL), (dict(y=None), q.QLORA_EINVAL), (dict(m=0), q.QLORA_EINVAL),
    (dict(n=0), q.QLORA_EINVAL), (dict(ld=63), q.QLORA_EINVAL), (dict(eps=-1.0), q.QLORA_EINVAL),
    (dict(eps=float("nan")), q.QLORA_EINVAL), (dict(eps=float("inf")), q.QLORA_EINVAL),
    (dict(xt=2), q.QLORA_ENOTSUP), (dict(wt=-1), q.QLORA_ENOTSUP), (dict(m=1 << 31), q.QLORA_ENOTSUP),
    (dict(n=1 << 31, ld=1 << 31), q.QLORA_ENOTSUP), (dict(x=FAKE + 1), q.QLORA_EALIGN),
    (dict(xt=1, x=FAKE + 2), q.QLORA_EALIGN), (dict(wt=1, w=FAKE + 2), q.QLORA_EALIGN),
    (dict(b=FAKE + 1), q.QLORA_EALIGN), (dict(y=FAKE + 1), q.QLORA_EALIGN), (dict(mean=FAKE + 2), q.QLORA_EALIGN),
])
def test_layernorm_fwd_refusals(kw, status):
    assert norm_fwd(**kw) == status


def norm_bwd(x=FAKE, dy=FAKE, xt=0, m=4, n=64, ld=64, mean=FAKE, rstd=FAKE, w=FAKE, wt=0, dx=FAKE, dw=FAKE, db=FAKE,
             ws=FAKE, ws_bytes=1 << 30):
    return q.library().qlora_layernorm_bwd(x, dy, xt, m, n, ld, mean, rstd, w, wt, dx, dw, db, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), q.QLORA_EINVAL), (dict(mean=None), q.QLORA_EINVAL), (dict(rstd=None), q.QLORA_EINVAL),
    (dict(dx=None), q.QLORA_EINVAL), (dict(m=-3), q.QLORA_EINVAL), (dict(xt=7), q.QLORA_ENOTSUP),
    (dict(dy=FAKE + 1), q.QLORA_EALIGN), (dict(dw=FAKE + 2), q.QLORA_EALIGN), (dict(ws=None), q.QLORA_EWORKSPACE),
    (dict(ws_bytes=2047), q.QLORA_EWORKSPACE), (dict(ws=FAKE + 8), q.QLORA_EALIGN),
])
def test_layernorm_bwd_refusals(kw, status):
    assert q.layernorm_workspace_bytes(4, 64) == 2048  # 4 partial rows of dw and db
    assert norm_bwd(**kw) == status


def attention(call="fwd", shape=None, no_shape=False, q_=FAKE, k=FAKE, v=FAKE, cu=FAKE, o=FAKE, res=None, lse=FAKE,
              do=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, lddq=512, lddk=128, lddv=128, ws=FAKE, ws_bytes=1 << 30):
    s = dict(T=100, sequences=2, heads=8, kv_heads=2, dim=64, ldq=512, ldk=128, ldv=128, scale=0.125)
    s.update(shape or {})
    p = None if no_shape else ctypes.byref(q._CAttentionShape(**s))
    if call == "fwd":
        return q.library().qlora_attention_fwd(p, q_, k, v, cu, o, res, lse, None)
    return q.library().qlora_attention_bwd(p, q_, k, v, o, res, lse, do, cu, dq, lddq, dk, lddk, dv, lddv, ws, ws_bytes,
                                           None)


@pytest.mark.parametrize("call", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(no_shape=True), q.QLORA_EINVAL), (dict(q_=None), q.QLORA_EINVAL), (dict(k=None), q.QLORA_EINVAL),
    (dict(v=None), q.QLORA_EINVAL), (dict(cu=None), q.QLORA_EINVAL), (dict(o=None), q.QLORA_EINVAL),
    (dict(lse=None), q.QLORA_EINVAL), (dict(shape=dict(T=0)), q.QLORA_EINVAL),
    (dict(shape=dict(sequences=0)), q.QLORA_EINVAL), (dict(shape=dict(heads=7)), q.QLORA_EINVAL),
    (dict(shape=dict(kv_heads=0)), q.QLORA_EINVAL), (dict(shape=dict(dim=-8)), q.QLORA_EINVAL),
    (dict(shape=dict(scale=0.0)), q.QLORA_EINVAL), (dict(shape=dict(scale=float("nan"))), q.QLORA_EINVAL),
    (dict(shape=dict(scale=float("inf"))), q.QLORA_EINVAL), (dict(shape=dict(ldq=504)), q.QLORA_EINVAL),
    (dict(shape=dict(scale=1e-20)), q.QLORA_ENOTSUP),
    (dict(shape=dict(ldk=120)), q.QLORA_EINVAL), (dict(shape=dict(dim=60)), q.QLORA_ENOTSUP),
    (dict(shape=dict(dim=136)), q.QLORA_ENOTSUP), (dict(shape=dict(ldv=132)), q.QLORA_ENOTSUP),
    (dict(shape=dict(ldq=(1 << 23) + 8)), q.QLORA_ENOTSUP), (dict(shape=dict(T=(1 << 30) + 1)), q.QLORA_ENOTSUP),
    (dict(shape=dict(T=1 << 30, heads=512, ldq=512 * 64)), q.QLORA_ENOTSUP),
    (dict(q_=FAKE + 8), q.QLORA_EALIGN), (dict(k=FAKE + 2), q.QLORA_EALIGN), (dict(v=FAKE + 4), q.QLORA_EALIGN),
    (dict(o=FAKE + 8), q.QLORA_EALIGN), (dict(res=FAKE + 8), q.QLORA_EALIGN), (dict(cu=FAKE + 2), q.QLORA_EALIGN),
    (dict(lse=FAKE + 1), q.QLORA_EALIGN),
])
def test_attention_refusals(call, kw, status):
    assert attention(call, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(do=None), q.QLORA_EINVAL), (dict(dq=None), q.QLORA_EINVAL), (dict(dk=None), q.QLORA_EINVAL),
    (dict(dv=None), q.QLORA_EINVAL), (dict(lddq=504), q.QLORA_EINVAL), (dict(lddk=132), q.QLORA_ENOTSUP),
    (dict(do=FAKE + 8), q.QLORA_EALIGN), (dict(dv=FAKE + 8), q.QLORA_EALIGN), (dict(ws=None), q.QLORA_EWORKSPACE),
    (dict(ws_bytes=100 * 8 * 4 - 1), q.QLORA_EWORKSPACE), (dict(ws=FAKE + 8), q.QLORA_EALIGN),
])
def test_attention_bwd_refusals(kw, status):
    assert attention("bwd", **kw) == status


def lp_fwd(x=FAKE, t=0, m=4, v=100, ld=100, tg=FAKE, top=3, lp=FAKE, ent=FAKE, lse=FAKE, tl=FAKE, ti=FAKE, ws=FAKE,
           ws_bytes=1 << 30):
    return q.library().qlora_logprob_fwd(x, t, m, v, ld, tg, top, lp, ent, lse, tl, ti, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), q.QLORA_EINVAL), (dict(m=0), q.QLORA_EINVAL), (dict(v=0), q.QLORA_EINVAL),
    (dict(ld=99), q.QLORA_EINVAL), (dict(top=-1), q.QLORA_EINVAL), (dict(top=3, v=2), q.QLORA_EINVAL),
    (dict(tg=None), q.QLORA_EINVAL), (dict(lp=None), q.QLORA_EINVAL), (dict(tl=None), q.QLORA_EINVAL),
    (dict(ti=None), q.QLORA_EINVAL), (dict(t=5), q.QLORA_ENOTSUP), (dict(top=17), q.QLORA_ENOTSUP),
    (dict(v=(1 << 19) + 1, ld=1 << 20), q.QLORA_ENOTSUP), (dict(m=1 << 26, v=1 << 19, ld=1 << 19), q.QLORA_ENOTSUP),
    (dict(x=FAKE + 1), q.QLORA_EALIGN), (dict(t=1, x=FAKE + 2), q.QLORA_EALIGN), (dict(tg=FAKE + 4), q.QLORA_EALIGN),
    (dict(ti=FAKE + 2), q.QLORA_EALIGN), (dict(ws=None), q.QLORA_EWORKSPACE), (dict(ws_bytes=15), q.QLORA_EWORKSPACE),
    (dict(ws=FAKE + 8), q.QLORA_EALIGN),
])
def test_logprob_fwd_refusals(kw, status):
    assert lp_fwd(**kw) == status


def lp_bwd(x=FAKE, t=0, m=4, v=100, ld=100, tg=FAKE, lse=FAKE, ent=FAKE, dl=FAKE, de=FAKE, dx=FAKE + 1024, ldd=100):
    return q.library().qlora_logprob_bwd(x, t, m, v, ld, tg, lse, ent, dl, de, dx, ldd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(lse=None), q.QLORA_EINVAL), (dict(dx=None), q.QLORA_EINVAL), (dict(ldd=99), q.QLORA_EINVAL),
    (dict(tg=None), q.QLORA_EINVAL), (dict(dl=None), q.QLORA_EINVAL), (dict(ent=None), q.QLORA_EINVAL),
    (dict(tg=None, dl=None, de=None), q.QLORA_EINVAL), (dict(dx=FAKE, ldd=101), q.QLORA_EINVAL),
    (dict(t=2), q.QLORA_ENOTSUP), (dict(lse=FAKE + 1), q.QLORA_EALIGN), (dict(dx=FAKE + 1), q.QLORA_EALIGN),
])
def test_logprob_bwd_refusals(kw, status):
    assert lp_bwd(**kw) == status


def adamw(n=64, param=FAKE, grad=FAKE, m=FAKE, v=FAKE, ms=FAKE, vs=FAKE, master=None, count=1, no_tensors=False, **over):
    c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0, step=1, param_type=0,
             grad_type=1, state_type=1, use_master=0)
    c.update(over)
    table = (q._CAdamWTensor * 1)(q._CAdamWTensor(param, grad, m, v, ms, vs, master, n))
    config = q._CAdamWConfig(**c)
    return q.library().qlora_adamw_step(None if no_tensors else table, count, ctypes.byref(config), None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(no_tensors=True), q.QLORA_EINVAL), (dict(count=-1), q.QLORA_EINVAL), (dict(n=-1), q.QLORA_EINVAL),
    (dict(param=None), q.QLORA_EINVAL), (dict(grad=None), q.QLORA_EINVAL), (dict(m=None), q.QLORA_EINVAL),
    (dict(ms=None), q.QLORA_EINVAL), (dict(vs=None), q.QLORA_EINVAL), (dict(step=0), q.QLORA_EINVAL),
    (dict(beta1=1.0), q.QLORA_EINVAL), (dict(beta2=-0.1), q.QLORA_EINVAL), (dict(beta2=NAN), q.QLORA_EINVAL),
    (dict(eps=-1.0), q.QLORA_EINVAL), (dict(lr=INF), q.QLORA_EINVAL), (dict(weight_decay=NAN), q.QLORA_EINVAL),
    (dict(grad_scale=INF), q.QLORA_EINVAL), (dict(master=FAKE), q.QLORA_EINVAL), (dict(use_master=1), q.QLORA_EINVAL),
    (dict(use_master=1, param_type=1, master=FAKE), q.QLORA_EINVAL), (dict(param_type=2), q.QLORA_ENOTSUP),
    (dict(grad_type=-1), q.QLORA_ENOTSUP), (dict(state_type=2), q.QLORA_ENOTSUP), (dict(n=(1 << 40) + 1), q.QLORA_ENOTSUP),
    (dict(param=FAKE + 1), q.QLORA_EALIGN), (dict(grad=FAKE + 2), q.QLORA_EALIGN), (dict(vs=FAKE + 2), q.QLORA_EALIGN),
    (dict(state_type=0, m=FAKE + 2, ms=None, vs=None), q.QLORA_EALIGN),
    (dict(use_master=1, master=FAKE + 2), q.QLORA_EALIGN),
    (dict(count=0), q.QLORA_OK), (dict(n=0, param=None), q.QLORA_OK),    # nothing to do, nothing launched
])
def test_adamw_refusals(kw, status):
    assert adamw(**kw) == status


def test_adamw_null_config_and_moments():
    lib = q.library()
    table = (q._CAdamWTensor * 1)(q._CAdamWTensor(None, None, FAKE, FAKE, FAKE, FAKE, None, 64))
    outs = (ctypes.c_void_p * 1)(FAKE)
    none = (ctypes.c_void_p * 1)(None)
    odd = (ctypes.c_void_p * 1)(FAKE + 2)
    assert lib.qlora_adamw_step(table, 1, None, None) == q.QLORA_EINVAL
    assert lib.qlora_adamw_moments(None, 1, outs, outs, None) == q.QLORA_EINVAL
    assert lib.qlora_adamw_moments(table, 1, None, outs, None) == q.QLORA_EINVAL
    assert lib.qlora_adamw_moments(table, 1, outs, none, None) == q.QLORA_EINVAL
    assert lib.qlora_adamw_moments(table, 1, odd, outs, None) == q.QLORA_EALIGN


def test_workspace_sizes():
    assert q.layernorm_workspace_bytes(0, 8) == 0 and q.layernorm_workspace_bytes(8, 0) == 0
    assert q.layernorm_workspace_bytes(10000, 8192) == 256 * 8192 * 8
    assert q.logprob_workspace_bytes(4, 0) == 0 and q.logprob_workspace_bytes(4, (1 << 19) + 1) == 0
    assert q.logprob_workspace_bytes(4, 100, 17) == 0 and q.logprob_workspace_bytes(4, 100, 16) > 0


STRUCTS = (("qlora_adamw_tensor", q._CAdamWTensor), ("qlora_adamw_config", q._CAdamWConfig),
           ("qlora_attention_shape", q._CAttentionShape))


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    body = ""
    for name, t in STRUCTS:
        body += f'printf("%zu\\n", sizeof({name}));\n'
        body += "".join(f'printf("%zu\\n", offsetof({name}, {f[0]}));\n' for f in t._fields_)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qlora_nf4.h"\nint main(void){\n' + body + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for _, t in STRUCTS:
        want += [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]
    assert got == want


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        q.qlora_layernorm_fwd(x)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        q.qlora_logprob_fwd(x.half(), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="at least one"):
        q.AdamWPlan([], [], [], [])
    with pytest.raises(ValueError, match="device tensor"):
        q.AdamWPlan([x], [x], [x], [x])
    with pytest.raises(ValueError, match="m_scales and v_scales"):
        q.AdamWPlan([x], [x], [x], [x], m_scales=[x])


def test_oracle_codes_round_trip_and_order():
    """Codes decode and encode to themselves; a value's code error is half a step of the root."""
    rng = np.random.default_rng(0)
    m = (rng.standard_normal(1000) * 1e-3).astype(np.float32)
    v = np.square(m)
    for x, enc, dec, top, power in ((m, step.encode_m, step.decode_m, 127, 2), (v, step.encode_v, step.decode_v, 255, 4)):
        code, scale = enc(x)
        back = dec(code, scale)
        assert np.array_equal(enc(back)[0], code)
        unit = np.repeat(scale.astype(np.float64), 256)[:x.size]
        root = lambda t: (np.abs(t.astype(np.float64)) / unit) ** (1 / power)  # noqa: E731
        err = np.abs(root(x) - root(back))
        small = (code == 1) & (root(x) < 0.5)           # v > 0 is held at code 1
        assert err[~small].max() <= 0.5 + 1e-4 and np.abs(code.astype(int)).max() == top


def test_oracle_gradients_agree_with_differences():
    rng = np.random.default_rng(1)
    x, t = rng.standard_normal((3, 7)), np.array([2, -1, 6])
    dl, de = rng.standard_normal(3), rng.standard_normal(3)
    d = step.logprob_backward(x, t, dl, de)
    h = 1e-6
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        f = [(dl * s[0] + de * s[1]).sum() for s in (step.logprob(a, t), step.logprob(b, t))]
        assert abs((f[0] - f[1]) / (2 * h) - d[i]) <= 1e-7

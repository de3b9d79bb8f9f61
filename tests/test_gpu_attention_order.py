"""NaN and infinity in attention reach what depends on them and nothing else: rows
before a key that is not finite (and keys after a row that is not) keep the bits
that they have without it, inside one tile as well as across tiles."""
import pytest
import torch

from tests.helpers import say

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def run(q, k, v, do, cu, scale=None):
    import bit_nf4_quantized_13_amd as lib
    o, lse, res = lib.qlora_attention_fwd(q, k, v, cu, scale, save_residual=True)
    dq, dk, dv = lib.qlora_attention_bwd(q, k, v, o, lse, do, cu, scale, residual=res)
    torch.cuda.synchronize()
    return dict(o=o, lse=lse.T, dq=dq, dk=dk, dv=dv)


def make(lens, h, hk, d, seed):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    draw = lambda n: torch.randn(t, n, d, generator=g).bfloat16().cuda()  # noqa: E731
    ends = torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda()
    return draw(h), draw(hk), draw(hk), draw(h), ends


def reached(name, row, head, col, shape, group):
    """Which elements of each result depend on element (row, head, col) of the tensor `name`,
    of one sequence: masks of shape [rows, heads(, dim)]."""
    t, h, hk, d = shape
    m = {n: torch.zeros(t, x, d, dtype=torch.bool) for n, x in (("o", h), ("dq", h), ("dk", hk), ("dv", hk))}
    m["lse"] = torch.zeros(t, h, dtype=torch.bool)
    g = head // group if name in ("q", "do") else head
    if name == "q":      # its row's weights
        for n in ("o", "lse", "dq"):
            m[n][row, head] = True
        m["dk"][:row + 1, g] = m["dv"][:row + 1, g] = True
    if name == "k":      # the weights of the rows from its own on, and so all keys
        for n in ("o", "lse", "dq"):
            m[n][row:, g * group:(g + 1) * group] = True
        m["dk"][:, g] = m["dv"][:, g] = True
    if name == "v":      # its column of these rows, and their ds
        m["o"][row:, g * group:(g + 1) * group, col] = True
        m["dq"][row:, g * group:(g + 1) * group] = True
        m["dk"][:, g] = True
    if name == "do":     # its row's ds, and its column of dv
        m["dq"][row, head] = True
        m["dk"][:row + 1, g] = True
        m["dv"][:row + 1, g, col] = True
    return m


# one part, two and four; a head and a group a workgroup of the dk, dv kernel; padded head dimensions
SHAPES = [(150, 4, 2, 64), (100, 2, 1, 128), (140, 3, 1, 40), (190, 4, 2, 128), (330, 160, 80, 64), (420, 160, 80, 128),
          (420, 80, 40, 64), (420, 80, 40, 72), (400, 70, 70, 128), (400, 2, 2, 64), (300, 2, 1, 128), (330, 40, 8, 64),
          (330, 96, 96, 64)]


@pytest.mark.parametrize("t,h,hk,d", SHAPES)
def test_one_element(t, h, hk, d):
    tensors = make([t], h, hk, d, t)
    clean = run(*tensors)
    assert all(bool(x.isfinite().all()) for x in clean.values())
    names = ("q", "k", "v", "do")
    for n, (row, name, value) in enumerate([(0, "v", NAN), (5, "k", NAN), (31, "do", INF), (32, "v", -INF), (63, "q", NAN),
                                            (64, "do", NAN), (70, "v", INF), (99, "v", NAN), (t - 1, "v", INF),
                                            (t - 2, "do", -INF), (40, "q", NAN), (77, "k", NAN), (1, "do", NAN)]):
        say(f"attention order T={t} heads={h}/{hk} dim={d} {name}[{row}] = {value}")
        changed = [x.clone() for x in tensors[:4]]
        x = changed[names.index(name)]
        head, col = (n * 5) % x.shape[1], (n * 17) % d
        x[row, head, col] = value
        got = run(*changed, tensors[4])
        for key, mask in reached(name, row, head, col, (t, h, hk, d), h // hk).items():
            mask = mask.cuda()
            assert torch.equal(got[key][~mask], clean[key][~mask]), key
            assert not bool(got[key][mask].isfinite().any()), key
        if name == "v" and value != value:
            assert bool(got["o"][row:].isnan().any())
        if name == "v" and value == value:  # weights are positive: an infinity stays one, with its sign
            g = h // hk
            assert bool((got["o"][row:, head * g:(head + 1) * g, col] == value).all())


@pytest.mark.parametrize("t,h,hk,d", SHAPES)
def test_infinite_scores_later(t, h, hk, d):
    """Infinite q and k from one row on: the rows before it have finite results.  (Their bits may differ: when
    the running maximum moves is common to the rows of a wave.)"""
    tensors = make([t], h, hk, d, t + 1)
    clean = run(*tensors)
    for row in (1, 33, 90):
        say(f"attention order T={t} heads={h}/{hk} dim={d} infinite from {row}")
        changed = [x.clone() for x in tensors[:4]]
        for x in changed:
            x[row:] = INF
            x[row:, :, ::3] = -INF
        got = run(*changed, tensors[4])
        for key in ("o", "lse", "dq"):
            assert bool(got[key][:row].isfinite().all()), key
        # each of the two is within 2^-8 of a weighted mean of |v| (under 6) and of itself, twice over with its statistics
        assert float((got["o"][:row].float() - clean["o"][:row].float()).abs().max()) <= 4 * 6 * 2.0 ** -8
        assert not bool(got["dk"][:row].isfinite().any()) and not bool(got["dv"][:row].isfinite().any())


def test_infinities_meet():
    """Opposite infinities in one column: each row has the one it takes, then NaN."""
    tensors = make([200], 2, 1, 64, 1)
    say("attention order infinities")
    q, k, v, do, cu = tensors
    v[40, 0, 3], v[50, 0, 3], v[130, 0, 7], v[199, 0, 7] = INF, -INF, -INF, INF
    do[150, 0, 5], do[140, 1, 5] = INF, -INF
    got = run(*tensors)
    o = got["o"][:, :, 3]
    assert bool(o[:40].isfinite().all() and (o[40:50] == INF).all() and o[50:].isnan().all())
    o = got["o"][:, :, 7]
    assert bool(o[:130].isfinite().all() and (o[130:199] == -INF).all() and o[199].isnan().all())
    dv = got["dv"][:, 0, 5]
    assert bool(dv[151:].isfinite().all() and (dv[141:151] == INF).all() and dv[:141].isnan().all())


def test_other_sequences_keep_their_bits():
    """Everything of one sequence NaN and infinite, between two others and rows of none."""
    for lens, h, hk, d in (([70, 90, 60], 4, 2, 64), ([300, 301, 400], 4, 2, 128), ([40] * 30, 16, 4, 64)):
        say(f"attention order sequences {lens[:4]}")
        tensors = make(lens, h, hk, d, 3)
        clean = run(*tensors)
        a, b = lens[0], lens[0] + lens[1]
        for x in tensors[:4]:
            x[a:b] = NAN
            x[a:b, :, 1::2] = INF
        got = run(*tensors)
        keep = torch.ones(sum(lens), dtype=torch.bool)
        keep[a:b] = False
        for key in got:
            assert torch.equal(got[key][keep.cuda()], clean[key][keep.cuda()]), key


@pytest.mark.parametrize("t,h,hk,d", [(200, 2, 1, 64), (190, 2, 2, 128), (400, 2, 1, 64), (420, 80, 40, 72), (330, 160, 80, 64)])
@pytest.mark.parametrize("low,scale", [(-INF, None), (torch.finfo(torch.bfloat16).min, 1.0)])
def test_first_keys_ruled_out(t, h, hk, d, low, scale):
    """Keys whose scores are -inf (or fall there once scaled), more of them than a tile: the later rows attend to
    the other keys as if these were not there."""
    say(f"attention order first keys at {low} T={t} heads={h}/{hk} dim={d}")
    n = 133
    q, k, v, do, cu = make([t], h, hk, d, t + 2)
    q[:, :, 0] = 1.0
    k[:, :, 0] = 0.0
    want = run(q[n:].contiguous(), k[n:].contiguous(), v[n:].contiguous(), do[n:].contiguous(), torch.tensor([0, t - n]).int().cuda(), scale)
    k[:n, :, 0] = low
    got = run(q, k, v, do, cu, scale)
    # o and lse of the two tilings: each within 2^-8 of a weighted mean of |v| (under 6) and of itself; scores below 60
    assert float((got["o"][n:].float() - want["o"].float()).abs().max()) <= 4 * 6 * 2.0 ** -8
    assert float((got["lse"][n:] - want["lse"]).abs().max()) <= 2 * 61 * 2.0 ** -12
    assert bool(got["dv"][n:].isfinite().all())

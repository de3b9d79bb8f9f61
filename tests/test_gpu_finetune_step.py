"""The fine-tuning example: its gradients against torch's autograd in fp64 on the
dequantized weights, the loss over some steps, and the same bits on a second run.

Bound of the gradients: every operator's result is rounded to bf16 (2^-9 of its
size in the mean), and a gradient passes about 40 of them forward and back (12
projections, norms, attention, residuals of 2 layers each way), independent in
sign: sqrt(40) 2^-9 = 1.2 % of a tensor's norm; 5 % is four times that.  The gates of
relu are the step's own: a value within rounding of zero may open on one side
only, and the gradient is that of the branch the step took."""
import pytest
import torch

from tests.helpers import say

pytestmark = pytest.mark.gpu


def reference(model, m, tokens, starts, targets):
    """Loss and the adapters' and norms' gradients, fp64 autograd."""
    q = m.q
    leaves = []

    def leaf(t):
        leaves.append(t.detach().double().requires_grad_(True))
        return leaves[-1]

    def linear(p, x):
        a, b = leaf(p.a), leaf(p.b)
        return x @ q.qlora_nf4_dequantize(p.w).double().T + m.ALPHA / m.RANK * (x @ a.T) @ b.T

    def norm(n, x):
        w, b = leaf(n.weight), leaf(n.bias)
        return torch.nn.functional.layer_norm(x, (m.WIDTH,), w, b, 1e-5)

    def attention(qh, kh, vh):
        out = torch.zeros_like(qh)
        for a, b in zip(starts[:-1].tolist(), starts[1:].tolist()):
            k = kh[a:b].repeat_interleave(m.HEADS // m.KV_HEADS, 1)
            v = vh[a:b].repeat_interleave(m.HEADS // m.KV_HEADS, 1)
            s = torch.einsum("ihd,jhd->hij", qh[a:b], k) * m.DIM ** -0.5
            later = torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1)
            p = torch.softmax(s.masked_fill(later, -float("inf")), -1)
            out = torch.cat([out[:a], torch.einsum("hij,jhd->ihd", p, v), out[b:]])
        return out

    h = model.embedding[tokens].double()
    for la in model.layers:
        x = norm(la.n1, h)
        heads = [linear(p, x).view(len(x), -1, m.DIM) for p in (la.q, la.k, la.v)]
        h = h + linear(la.o, attention(*heads).reshape(len(x), m.WIDTH))
        up = linear(la.up, norm(la.n2, h))
        h = h + linear(la.down, torch.where(la.act > 0, up, 0))
    logits = linear(model.head, norm(model.norm, h))
    keep = targets >= 0
    loss = torch.nn.functional.cross_entropy(logits[keep], targets[keep])
    loss.backward()
    return loss.detach(), [t.grad for t in leaves]


def test_gradients_of_a_step():
    import examples.finetune_step as m
    say("finetune step gradients")
    model = m.Decoder(3)
    g = torch.Generator(device="cuda").manual_seed(5)
    for p in model.projections:  # adapters in use
        p.b.copy_((0.02 * torch.randn(p.b.shape, generator=g, device="cuda")).bfloat16())
    tokens, starts, targets = m.batch(11, total=300)
    loss = model.loss_and_gradients(tokens, starts, targets)
    ref_loss, ref = reference(model, m, tokens, starts, targets)
    assert abs(float(loss) - float(ref_loss)) <= 0.02 * abs(float(ref_loss))
    # the reference's leaves stand in the order in which its expressions are evaluated
    order = []
    for la in model.layers:
        order += [la.n1.dweight, la.n1.dbias] + [t for p in (la.q, la.k, la.v, la.o) for t in (p.da, p.db)]
        order += [la.n2.dweight, la.n2.dbias, la.up.da, la.up.db, la.down.da, la.down.db]
    order += [model.norm.dweight, model.norm.dbias, model.head.da, model.head.db]
    assert len(order) == len(ref)
    for i, (a, b) in enumerate(zip(order, ref)):
        off = float((a.double() - b).norm() / b.norm())
        assert off <= 0.05, (i, tuple(a.shape), off)


def test_loss_falls_and_runs_repeat():
    import examples.finetune_step as m
    say("finetune steps")
    runs = []
    for _ in range(2):
        model = m.Decoder(1)
        runs.append([float(model.step(i, *m.batch(i))) for i in range(1, 41)])
    assert runs[0] == runs[1], "the same steps give the same bits"
    # at the start the loss is that of guessing (log 384 = 5.95, and more for random logits)
    assert sum(runs[0][-5:]) / 5 < 0.6 * runs[0][0], runs[0]
    logp, ids = m.alternatives(model, *m.batch(0, total=200)[:2])
    assert bool((logp[:, 0] >= logp[:, 1]).all()) and int(ids.min()) >= 0 and int(ids.max()) < m.VOCAB

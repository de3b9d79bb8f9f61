"""A fine-tuning step of a small decoder, every operator the library's own.

    python examples/finetune_step.py [steps]

Sequences of different lengths are packed into one row of tokens.  Each layer is
  h += o(attention(q(n1), k(n1), v(n1)))      n1 = layernorm(h)
  h += down(relu(up(n2)))                     n2 = layernorm(h)
with NF4 base weights and trainable adapters in every projection; the head is one
more projection on a last norm.  The loss is the mean negative log-probability of
the next token.  Adapters (bf16, fp32 masters, 8-bit AdamW states) and norm
weights (fp32) are trained; torch supplies memory, the embedding look-up and the
residual additions.  The task is synthetic: sequences that count up from a random
start with one of three step widths.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_nf4_quantized_13_amd as q  # noqa: E402

WIDTH, HEADS, KV_HEADS, FFN, VOCAB, LAYERS, RANK, ALPHA = 256, 4, 2, 512, 384, 2, 8, 16.0
DIM = WIDTH // HEADS


class Projection:
    """One QLoRA projection with the buffers its gradients arrive in."""

    def __init__(self, d: int, k: int, g: torch.Generator):
        self.w = q.qlora_nf4_quantize(torch.randn(d, k, generator=g, device="cuda") * k ** -0.5)
        self.a = (torch.randn(RANK, k, generator=g, device="cuda") * RANK ** -0.5).bfloat16()
        self.b = torch.zeros(d, RANK, device="cuda", dtype=torch.bfloat16)
        self.da = torch.zeros(RANK, k, device="cuda")
        self.db = torch.zeros(d, RANK, device="cuda")

    def forward(self, x):
        self.x = x
        y, self.u = q.qlora_linear_fwd(self.w, x, self.a, self.b, ALPHA)
        return y

    def backward(self, dy):
        dx = torch.empty_like(self.x)
        q.qlora_linear_bwd(self.w, self.x, dy, self.a, self.b, ALPHA, u=self.u, outs=(dx, self.da, self.db))
        return dx


class Norm:
    def __init__(self):
        self.weight, self.bias = torch.ones(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda")
        self.dweight, self.dbias = torch.zeros(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda")

    def forward(self, x):
        self.x = x
        y, self.mean, self.rstd = q.qlora_layernorm_fwd(x, self.weight, self.bias)
        return y

    def backward(self, dy):
        dx = torch.empty_like(dy)
        q.qlora_layernorm_bwd(self.x, dy, self.mean, self.rstd, self.weight, outs=(dx, self.dweight, self.dbias))
        return dx


class Layer:
    def __init__(self, g):
        self.n1, self.n2 = Norm(), Norm()
        self.q, self.o = Projection(WIDTH, WIDTH, g), Projection(WIDTH, WIDTH, g)
        self.k, self.v = Projection(KV_HEADS * DIM, WIDTH, g), Projection(KV_HEADS * DIM, WIDTH, g)
        self.up, self.down = Projection(FFN, WIDTH, g), Projection(WIDTH, FFN, g)

    def forward(self, h, starts):
        x = self.n1.forward(h)
        self.heads = [p.forward(x).view(len(x), -1, DIM) for p in (self.q, self.k, self.v)]
        self.att, self.lse, self.residual = q.qlora_attention_fwd(*self.heads, starts, save_residual=True)
        h = h + self.o.forward(self.att.view(len(x), WIDTH))
        self.act = torch.relu(self.up.forward(self.n2.forward(h)))
        return h + self.down.forward(self.act)

    def backward(self, dh, starts):
        dact = torch.where(self.act > 0, self.down.backward(dh), 0)
        dh = dh + self.n2.backward(self.up.backward(dact))
        datt = self.o.backward(dh).view_as(self.att)
        grads = q.qlora_attention_bwd(*self.heads, self.att, self.lse, datt, starts, residual=self.residual)
        dx = sum(p.backward(t.reshape(len(dh), -1)) for p, t in zip((self.q, self.k, self.v), grads))
        return dh + self.n1.backward(dx)


class Decoder:
    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embedding = torch.randn(VOCAB, WIDTH, generator=g, device="cuda").bfloat16()
        self.layers = [Layer(g) for _ in range(LAYERS)]
        self.norm, self.head = Norm(), Projection(VOCAB, WIDTH, g)
        self.projections = [p for la in self.layers for p in (la.q, la.k, la.v, la.o, la.up, la.down)] + [self.head]
        self.norms = [n for la in self.layers for n in (la.n1, la.n2)] + [self.norm]
        self.adapters = q.AdamWPlan.zeros([t for p in self.projections for t in (p.a, p.b)],
                                          [t for p in self.projections for t in (p.da, p.db)], bits8=True, master=True)
        self.norm_weights = q.AdamWPlan.zeros([t for n in self.norms for t in (n.weight, n.bias)],
                                              [t for n in self.norms for t in (n.dweight, n.dbias)], bits8=False)

    def forward(self, tokens, starts):
        h = self.embedding[tokens]
        for la in self.layers:
            h = la.forward(h, starts)
        return self.head.forward(self.norm.forward(h))

    def loss_and_gradients(self, tokens, starts, targets):
        """The mean loss over the rows with a target (a device scalar); gradients in the buffers."""
        logits = self.forward(tokens, starts)
        logp, entropy, lse, _, _ = q.qlora_logprob_fwd(logits, targets)
        count = (targets >= 0).sum()
        dlogp = (-1.0 / count).expand(len(tokens)).contiguous()
        dlogits = q.qlora_logprob_bwd(logits, targets, lse, None, dlogp, out=logits)
        dh = self.norm.backward(self.head.backward(dlogits))
        for la in reversed(self.layers):
            dh = la.backward(dh, starts)
        return -logp.sum() / count

    def step(self, number, tokens, starts, targets, lr=2e-3):
        loss = self.loss_and_gradients(tokens, starts, targets)
        q.qlora_adamw_step(self.adapters, lr=lr, step=number, weight_decay=0.01)
        q.qlora_adamw_step(self.norm_weights, lr=lr, step=number)
        return loss


def batch(seed: int, total: int = 1024):
    """Packed sequences: tokens, their starts and the next tokens (-100 at the sequences' ends)."""
    g = torch.Generator().manual_seed(seed)
    pieces, starts = [], [0]
    while starts[-1] < total:
        n = min(total - starts[-1], int(torch.randint(1, 200, (1,), generator=g)))
        first, width = int(torch.randint(0, VOCAB, (1,), generator=g)), int(torch.randint(1, 4, (1,), generator=g))
        pieces.append((first + width * torch.arange(n)) % VOCAB)
        starts.append(starts[-1] + n)
    targets = [torch.cat([p[1:], torch.tensor([-100])]) for p in pieces]
    return (torch.cat(pieces).cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), torch.cat(targets).cuda())


def alternatives(model, tokens, starts, top=3):
    """The best next tokens after the last token of each sequence, with their log-probabilities."""
    logits = model.forward(tokens, starts)[(starts[1:] - 1).long()]
    return q.qlora_logprob_fwd(logits, torch.full((len(logits),), -100, device="cuda"), top=top)[3:]


def main(steps: int = 60) -> None:
    model = Decoder()
    for i in range(1, steps + 1):
        loss = model.step(i, *batch(i))
        if i == 1 or i % 10 == 0:
            print(f"step {i}: loss {float(loss):.4f}", flush=True)
    tokens, starts, _ = batch(0, total=300)
    logp, ids = alternatives(model, tokens, starts)
    for s, (i, p) in enumerate(zip(ids.tolist(), logp.tolist())):
        tail = tokens[int(starts[s]):int(starts[s + 1])].tolist()[-3:]
        print(f"after ... {tail}: " + ", ".join(f"{t} ({x:.2f})" for t, x in zip(i, p)))


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)

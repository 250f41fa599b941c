"""One training step of the last layer of a language model whose feed-forward
part is a mixture of experts: a layer norm with the residual's addition, a
router, the tokens' rows sorted and moved to their experts and back with
weights, a second layer norm, the projection to the vocabulary, the log
probabilities of the sampled tokens and the clipped policy loss with a KL term;
then all gradients, back to the layer's input; then one token through the same
layer, as while decoding.

    python examples/expert_step.py [--sequences 8] [--length 64] [--hidden 1024]
                                   [--vocab 32000] [--experts 16] [--top 4]

It prints the loss and how far the gradients are from torch's autograd in 32
bits.  Needs a GPU.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_elementwise_amd as ew  # noqa: E402

EPS, LOW, HIGH, KL, ALIGN = 1e-5, 0.2, 0.25, 0.1, 16
WEIGHTS = ("w1", "b1", "router", "expert", "w2", "b2", "head")


class Layer:
    """The buffers and workspaces of a step, allocated once."""

    def __init__(self, sequences, length, hidden, vocab, experts, top, dev="cuda"):
        def f32(*shape):
            return torch.empty(*shape, device=dev)

        def i32(*shape):
            return torch.empty(*shape, dtype=torch.int32, device=dev)

        def bf16(rows, cols=hidden):
            return torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)

        n = sequences * length
        self.shape, self.experts, self.top = (sequences, length), experts, top
        places = ew.ew_experts_rows(n * top, experts, ALIGN)
        self.total, self.y, self.out, self.y2 = bf16(n), bf16(n), bf16(n), bf16(n)
        self.stats = [f32(n) for _ in range(4)]             # mean and rstd of both norms
        self.slot, self.offsets, self.counts = i32(n, top), i32(experts + 1), i32(experts)
        self.rows, self.z, self.drows = bf16(places), bf16(places), bf16(places)
        self.logp, self.lse, self.dlogp = f32(*self.shape), f32(n), f32(*self.shape)
        self.loss, self.parts, self.weights = f32(1), f32(4), f32(sequences)
        self.dlogits, self.dout, self.dy, self.dx = bf16(n, vocab), bf16(n), bf16(n), bf16(n)
        self.dgates = f32(n, top)
        self.sums = [f32(hidden) for _ in range(4)]
        need = max(ew.ew_layernorm_grad_workspace(n, hidden), ew.ew_logprobs_workspace(n, vocab),
                   ew.ew_experts_sort_workspace(n * top, experts),
                   ew.ew_policy_loss_workspace(sequences, length))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)

    def parts_of(self, m):
        """Each expert's rows of a matrix, its padding among them."""
        return m[:int(self.offsets[-1])].split(self.offsets.diff().tolist())

    def forward(self, x, residual, tokens, m):
        """Logits and the sampled tokens' log probabilities."""
        ew.ew_layernorm_bf16(x, m["w1"], m["b1"], self.y, residual=residual, total=self.total,
                             mean=self.stats[0], rstd=self.stats[1], eps=EPS)
        best = (self.y @ m["router"]).float().topk(self.top, dim=1)
        self.ids, self.gates = best.indices, torch.softmax(best.values, 1)
        ew.ew_experts_sort(self.ids, self.experts, self.slot, self.offsets, counts=self.counts,
                           align=ALIGN, workspace=self.workspace)
        ew.ew_experts_gather_bf16(self.y, self.slot, self.rows, offsets=self.offsets,
                                  counts=self.counts)
        for rows, z, w in zip(self.parts_of(self.rows), self.parts_of(self.z), m["expert"]):
            torch.matmul(rows, w, out=z)
        ew.ew_experts_combine_bf16(self.z, self.slot, self.out, weights=self.gates,
                                   residual=self.total)
        ew.ew_layernorm_bf16(self.out, m["w2"], m["b2"], self.y2, mean=self.stats[2],
                             rstd=self.stats[3], eps=EPS)
        logits = self.y2 @ m["head"]
        ew.ew_logprobs_bf16(logits, tokens, self.logp, lse=self.lse, workspace=self.workspace)
        return logits, self.logp

    def backward(self, logits, tokens, old, ref, advantage, mask, m):
        """The loss, and the gradients of x (and residual) and the weights."""
        ew.ew_policy_loss_f32(self.logp, old, advantage, self.loss, weights=self.weights,
                              ref_logp=ref, mask=mask, stats=self.parts, clip_low=LOW,
                              clip_high=HIGH, kl=KL, mean="sequences", workspace=self.workspace)
        ew.ew_policy_loss_grad_f32(self.logp, old, advantage, self.weights, self.dlogp,
                                   ref_logp=ref, mask=mask, clip_low=LOW, clip_high=HIGH, kl=KL)
        ew.ew_logprobs_grad_bf16(logits, tokens, self.lse, self.dlogp, self.dlogits)
        grads = {"head": self.y2.t() @ self.dlogits}
        dy2 = self.dlogits @ m["head"].t()
        ew.ew_layernorm_grad_bf16(dy2, self.out, m["w2"], self.stats[2], self.stats[3], self.dout,
                                  self.sums[2], self.sums[3], self.workspace)
        # z becomes its gradient
        ew.ew_experts_combine_grad_bf16(self.dout, self.z, self.slot, self.gates, self.z,
                                        self.dgates, offsets=self.offsets, counts=self.counts)
        grads["expert"] = torch.stack([r.t() @ dz for r, dz in zip(self.parts_of(self.rows),
                                                                   self.parts_of(self.z))])
        for dz, drows, w in zip(self.parts_of(self.z), self.parts_of(self.drows), m["expert"]):
            torch.matmul(dz, w.t(), out=drows)
        # the router's softmax over the chosen, then the gather's gradient on top
        g = self.gates * (self.dgates - (self.gates * self.dgates).sum(1, keepdim=True))
        g = g.new_zeros(len(g), self.experts).scatter(1, self.ids, g).bfloat16()
        grads["router"] = self.y.t() @ g
        ew.ew_experts_combine_bf16(self.drows, self.slot, self.dy, residual=g @ m["router"].t())
        ew.ew_layernorm_grad_bf16(self.dy, self.total, m["w1"], self.stats[0], self.stats[1],
                                  self.dx, self.sums[0], self.sums[1], self.workspace,
                                  dtotal=self.dout)
        grads.update(x=self.dx, w1=self.sums[0], b1=self.sums[1], w2=self.sums[2], b2=self.sums[3])
        return self.loss[0], grads


def inputs(sequences, length, hidden, vocab, experts, seed=0, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    n = sequences * length

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g, device=dev)).bfloat16()

    m = {"w1": 1 + randn(hidden, scale=0.1), "b1": randn(hidden, scale=0.1),
         "router": randn(hidden, experts, scale=hidden ** -0.5),
         "expert": randn(experts, hidden, hidden, scale=hidden ** -0.5),
         "w2": 1 + randn(hidden, scale=0.1), "b2": randn(hidden, scale=0.1),
         "head": randn(hidden, vocab, scale=hidden ** -0.5)}
    ends = torch.randint(length // 2, length + 1, (sequences, 1), generator=g, device=dev)
    # how far the policy has moved from that which sampled and from the reference
    moved = torch.tensor([-0.5, -0.05, 0.05, 0.5], device=dev)
    return {"x": randn(n, hidden), "residual": randn(n, hidden),
            "tokens": torch.randint(vocab, (n,), generator=g, device=dev),
            "advantage": torch.randn(sequences, generator=g, device=dev),
            "mask": torch.arange(length, device=dev) < ends,
            "moved": [moved[torch.randint(4, (sequences, length), generator=g, device=dev)]
                      for _ in range(2)]}, m


def reference(x, residual, tokens, advantage, mask, old, ref, ids, m):
    """The same step in 32 bits by torch's autograd, with the router's choices."""
    x = (x.float() + residual.float()).bfloat16().float().requires_grad_()
    m = {k: v.float().requires_grad_() for k, v in m.items()}

    def norm(h, w, b):
        d = h - h.mean(1, keepdim=True)
        return d * torch.rsqrt(d.square().mean(1, keepdim=True) + EPS) * w + b

    y = norm(x, m["w1"], m["b1"])
    gates = torch.softmax((y @ m["router"]).gather(1, ids), 1)
    back = torch.zeros_like(x)
    for e, w in enumerate(m["expert"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        back = back.index_add(0, t, gates[t, j, None] * (y[t] @ w))
    y2 = norm(x + back, m["w2"], m["b2"])
    logp = torch.log_softmax(y2 @ m["head"], 1).gather(1, tokens[:, None]).view(old.shape)
    ratio, a, d = (logp - old).exp(), advantage[:, None], ref - logp
    each = KL * (d.exp() - d - 1) - torch.minimum(ratio * a, ratio.clamp(1 - LOW, 1 + HIGH) * a)
    each = torch.where(mask, each, 0.0).sum(1) / mask.sum(1)
    loss = each.mean()
    loss.backward()
    return loss, {"x": x.grad, **{k: v.grad for k, v in m.items()}}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    for name, value in (("sequences", 8), ("length", 64), ("hidden", 1024), ("vocab", 32000),
                        ("experts", 16), ("top", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    data, m = inputs(a.sequences, a.length, a.hidden, a.vocab, a.experts)
    args = a.hidden, a.vocab, a.experts, a.top
    layer = Layer(a.sequences, a.length, *args)
    logits, logp = layer.forward(data["x"], data["residual"], data["tokens"], m)
    old, ref = (logp - moved for moved in data.pop("moved"))
    loss, grads = layer.backward(logits, data["tokens"], old, ref, data["advantage"], data["mask"], m)
    want_loss, want = reference(**data, old=old, ref=ref, ids=layer.ids, m=m)
    off = {}
    for name in ("x",) + WEIGHTS:
        u, v = grads[name].double(), want[name].double()
        off[name] = float((u - v).norm() / v.norm())
    # (a mean of terms of either sign: against their size)
    off["loss"] = float((loss - want_loss.detach()).abs() / data["advantage"].abs().mean())
    print(f"loss {float(loss):.5f}: policy {float(layer.parts[0]):.5f}, KL {float(layer.parts[1]):.5f}, "
          f"{100 * float(layer.parts[2]):.0f} % of the tokens clipped")
    print("off from autograd in 32 bits: " + ", ".join(f"{k} {v:.1e}" for k, v in off.items()))

    one = Layer(1, 1, *args)
    _, first = one.forward(data["x"][:1], data["residual"][:1], data["tokens"][:1], m)
    print(f"the first token alone: log probability {float(first):.4f}, "
          f"in the batch {float(logp[0, 0]):.4f}, experts {one.ids[0].tolist()}")
    return off, (float(first), float(logp[0, 0]), one.ids[0].tolist(), layer.ids[0].tolist())


if __name__ == "__main__":
    main()

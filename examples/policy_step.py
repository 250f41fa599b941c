"""One training step at the end of a language model, with every row operator of
libew: the last layer's RMS norm with the residual's addition, the projection
to the vocabulary, the log probabilities of the sampled tokens with their
entropy, a policy-gradient loss with an entropy bonus and a distillation term,
and all gradients back to the layer's input; then the same norm in 8 bits and
the best alternatives of one decoding step.

    python examples/policy_step.py [--rows 512] [--hidden 2048] [--vocab 32000]

It prints the losses and how far the gradients are from torch's autograd in
32 bits.  Needs a GPU.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_elementwise_amd as ew  # noqa: E402

EPS, BONUS, DISTILL, TEMPERATURE = 1e-5, 0.01, 0.5, 2.0


class Step:
    """The buffers and workspaces of a step, allocated once."""

    def __init__(self, rows, hidden, vocab, kept, dev="cuda"):
        def f32(*shape):
            return torch.empty(*shape, device=dev)

        def bf16(*shape):
            return torch.empty(*shape, dtype=torch.bfloat16, device=dev)

        self.rows, self.vocab = rows, vocab
        self.total, self.y, self.rstd = bf16(rows, hidden), bf16(rows, hidden), f32(rows)
        self.logp, self.entropy, self.lse = f32(rows), f32(rows), f32(rows)
        self.loss, self.lse_t = f32(rows), f32(rows)
        self.dlogits, self.ddistill = bf16(rows, vocab), bf16(rows, vocab)
        self.dx, self.dweight = bf16(rows, hidden), f32(hidden)
        need = max(ew.ew_logprobs_workspace(rows, vocab), ew.ew_distill_workspace(rows, vocab),
                   ew.ew_rmsnorm_grad_workspace(rows, hidden))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)

    def __call__(self, x, residual, weight, head, tokens, advantage, teacher, ids):
        """Losses (policy, distillation) and gradients of x (and residual),
        the norm's weight and the head; rows without a token count nothing."""
        n = (tokens >= 0).sum()
        ew.ew_rmsnorm_bf16(x, weight, self.y, residual=residual, total=self.total, rstd=self.rstd,
                           eps=EPS)
        logits = self.y @ head
        ew.ew_logprobs_bf16(logits, tokens, self.logp, entropy=self.entropy, lse=self.lse,
                            workspace=self.workspace)
        ew.ew_distill_bf16(logits, teacher, ids, self.loss, lse=self.lse_t, scale=1 / TEMPERATURE,
                           workspace=self.workspace)
        live = (tokens >= 0).float() / n
        policy = -(live * (advantage * self.logp + BONUS * self.entropy)).sum()
        distillation = DISTILL * (live * self.loss).sum()

        ew.ew_logprobs_grad_bf16(logits, tokens, self.lse, -live * advantage, self.dlogits,
                                 entropy=self.entropy, dentropy=-live * BONUS)
        ew.ew_distill_grad_bf16(logits, teacher, ids, self.lse_t, DISTILL * live, self.ddistill,
                                scale=1 / TEMPERATURE)
        ew.ew_add_bf16(self.dlogits, self.ddistill, self.dlogits)
        dhead = self.y.t() @ self.dlogits
        dy = self.dlogits @ head.t()
        ew.ew_rmsnorm_grad_bf16(dy, self.total, weight, self.rstd, self.dx, self.dweight,
                                self.workspace)
        return policy, distillation, self.dx, self.dweight, dhead


def inputs(rows, hidden, vocab, kept, seed=0, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    tokens = torch.randint(vocab, (rows,), generator=g, device=dev)
    tokens[::16] = -100                                     # padding
    ids = torch.stack([torch.randperm(vocab, generator=g, device=dev)[:kept] for _ in range(rows)])
    return {"x": randn(rows, hidden).bfloat16(), "residual": randn(rows, hidden).bfloat16(),
            "weight": (1 + 0.1 * randn(hidden)).bfloat16(),
            "head": (randn(hidden, vocab) / math.sqrt(hidden)).bfloat16(), "tokens": tokens,
            "advantage": randn(rows), "teacher": 3 * randn(rows, kept), "ids": ids}


def reference(x, residual, weight, head, tokens, advantage, teacher, ids):
    """The same step in 32 bits by torch's autograd."""
    total = (x.float() + residual.float()).bfloat16().float().requires_grad_()
    w, hd = weight.float().requires_grad_(), head.float().requires_grad_()
    y = total * torch.rsqrt(total.square().mean(1, keepdim=True) + EPS) * w
    logits = y @ hd
    live = (tokens >= 0).float() / (tokens >= 0).sum()
    logq = torch.log_softmax(logits, 1)
    logp = logq.gather(1, tokens.clamp_min(0)[:, None])[:, 0]
    entropy = -(logq.exp() * logq).sum(1)
    policy = -(live * (advantage * logp + BONUS * entropy)).sum()
    t = torch.softmax(teacher / TEMPERATURE, 1)
    soft = torch.log_softmax(logits / TEMPERATURE, 1).gather(1, ids)
    distillation = DISTILL * (live * (t * (t.log() - soft)).sum(1)).sum()
    (policy + distillation).backward()
    return policy, distillation, total.grad, w.grad, hd.grad


def decode(x, residual, weight, head, top=5):
    """One token: the norm, its 8-bit form, and the best alternatives."""
    rows, hidden = x.shape
    y = torch.empty_like(x)
    q = torch.empty(rows, hidden, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty(rows, -(-hidden // 128), device=x.device)
    ew.ew_rmsnorm_bf16(x, weight, y, residual=residual, eps=EPS)
    ew.ew_rmsnorm_e4m3_bf16(x, weight, q, scales, group=128, residual=residual, eps=EPS)
    logits = y @ head
    logp = torch.empty(rows, device=x.device)
    top_logp = torch.empty(rows, top, device=x.device)
    top_ids = torch.empty(rows, top, dtype=torch.int64, device=x.device)
    space = torch.empty(ew.ew_logprobs_workspace(rows, head.shape[1], top), dtype=torch.uint8,
                        device=x.device)
    ew.ew_logprobs_bf16(logits, logits.argmax(1), logp, top_logp=top_logp, top_ids=top_ids,
                        workspace=space)
    return q, scales, logp, top_logp, top_ids


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--kept", type=int, default=32)
    a = ap.parse_args(argv)
    data = inputs(a.rows, a.hidden, a.vocab, a.kept)
    got = Step(a.rows, a.hidden, a.vocab, a.kept)(**data)
    want = reference(**data)
    off = {}
    for name, u, v in zip(("policy", "distillation", "dx", "dweight", "dhead"), got, want):
        u, v = u.detach().double(), v.detach().double()
        off[name] = float((u - v).norm() / v.norm())
    print(f"policy loss {float(got[0]):.5f}, distillation loss {float(got[1]):.5f}")
    print("off from autograd in 32 bits: " + ", ".join(f"{k} {v:.1e}" for k, v in off.items()))
    q, scales, logp, top_logp, top_ids = decode(data["x"][:1], data["residual"][:1], data["weight"],
                                                data["head"])
    print("best alternatives of the first row: "
          + ", ".join(f"{int(i)} ({float(p):.3f})" for i, p in zip(top_ids[0], top_logp[0])))
    return off, (q, scales, logp, top_logp, top_ids)


if __name__ == "__main__":
    main()

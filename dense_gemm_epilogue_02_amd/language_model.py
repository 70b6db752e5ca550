"""The operators around a language model's products together, as a training
step uses them:

    python -m dense_gemm_epilogue_02_amd.language_model [--tokens 2048] [--vocab 32000] ...

trains one block of mixture-of-experts products between norms, with an
embedding before it and a head after it, on labels and from a teacher's top
logits. Gradients are computed by hand.
"""
from __future__ import annotations

import argparse
import time
from typing import Optional

import torch

from . import (Plan, expert_combine, expert_combine_backward, expert_gather, expert_gather_backward, expert_sort,
               linear_cross_entropy, linear_cross_entropy_backward, linear_distillation, linear_distillation_backward,
               norm_residual, norm_residual_backward)


def _draw(gen, *shape, std):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()


class ExpertBlock:
    """Any number of tokens through their experts: sorted by expert, gate and up
    products, down products, and back with the router's weights. The experts'
    products are grouped GEMMs, whose sizes the host has to know: one wait a
    pass."""

    def __init__(self, hidden: int, inner: int, experts: int, top_k: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.top_k = top_k
        self.router = _draw(gen, experts, hidden, std=hidden ** -0.5)
        self.up = _draw(gen, experts, 2 * inner, hidden, std=hidden ** -0.5)    # the gate's rows first
        self.down = _draw(gen, experts, hidden, inner, std=inner ** -0.5)
        self.plans = {"y": Plan("bf16", la="row", lb="col"), "dx": Plan("bf16", la="row", lb="row"),
                      "dw": Plan("bf16", la="col", lb="row")}

    def _products(self, kind: str, bounds, a, b, out):
        """Per expert and its rows a_e, b_e: y = a_e b[e]^T, dx = a_e b[e], or dw[e] = a_e^T b_e."""
        def problem(e, lo, hi):
            n = hi - lo
            if kind == "dw":
                return a.shape[1], b.shape[1], n, a[lo:hi], b[lo:hi], None, out[e]
            return n, out.shape[1], a.shape[1], a[lo:hi], b[e], None, out[lo:hi]
        problems = [problem(e, lo, hi) for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])) if hi > lo]
        if problems:
            self.plans[kind].run_grouped(problems)
        return out

    def forward(self, x: torch.Tensor):
        """x [T, H] -> (out [T, H], what backward needs)."""
        E, (_, H, I) = self.router.shape[0], self.down.shape
        scores = x.float() @ self.router.float().t()
        top, ids = torch.topk(scores, self.top_k)
        weights = torch.softmax(top, -1)
        order = expert_sort(ids, E)
        rows, bounds = expert_gather(x, order), order.bounds()
        gu = self._products("y", bounds, rows, self.up, rows.new_zeros(rows.shape[0], 2 * I))
        gate, up = gu.float().chunk(2, 1)
        h = (torch.nn.functional.silu(gate) * up).bfloat16()
        y = self._products("y", bounds, h, self.down, rows.new_zeros(rows.shape))
        return expert_combine(y, order, weights), (x, ids, weights, order, bounds, rows, gu, h, y)

    def backward(self, d_out: torch.Tensor, kept):
        """(d_x, gradients of router, up and down)."""
        x, ids, weights, order, bounds, rows, gu, h, y = kept
        d_y, d_weights = expert_combine_backward(d_out, y, order, weights)
        d_down = self._products("dw", bounds, d_y, h, torch.zeros_like(self.down))
        d_h = self._products("dx", bounds, d_y, self.down, torch.zeros_like(h)).float()
        gate, up = gu.float().chunk(2, 1)
        s = torch.sigmoid(gate)
        d_gu = torch.cat([d_h * up * s * (1 + gate * (1 - s)), d_h * gate * s], 1).bfloat16()
        d_up = self._products("dw", bounds, d_gu, rows, torch.zeros_like(self.up))
        d_rows = self._products("dx", bounds, d_gu, self.up, torch.zeros_like(rows))
        d_x = expert_gather_backward(d_rows, order).float()
        # through the weights: a softmax over the chosen scores
        d_top = weights * (d_weights - (weights * d_weights).sum(-1, keepdim=True))
        d_scores = torch.zeros(x.shape[0], self.router.shape[0], device=x.device).scatter_(1, ids, d_top)
        d_router = d_scores.t() @ x.float()
        return (d_x + d_scores @ self.router.float()).bfloat16(), {"router": d_router, "up": d_up, "down": d_down}


class LanguageModel:
    """Embedding -> norm -> experts -> norm with the residual -> head."""

    def __init__(self, vocab: int, hidden: int, inner: int, experts: int, top_k: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.embed, self.head = _draw(gen, vocab, hidden, std=1.0), _draw(gen, vocab, hidden, std=hidden ** -0.5)
        one = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.w_first, self.w_post, self.w_last = one.clone(), one.clone(), one.clone()
        self.block = ExpertBlock(hidden, inner, experts, top_k, seed)

    def forward(self, tokens: torch.Tensor):
        """tokens [T] -> (the head's input [T, H], what backward needs)."""
        residual = self.embed[tokens]
        _, x, saved_first = norm_residual(None, residual, w_next=self.w_first)
        y, kept = self.block.forward(x)
        out, last, saved = norm_residual(y, residual, w_post=self.w_post, w_next=self.w_last)
        return last, (tokens, residual, saved_first, y, kept, out, saved)

    def backward(self, d_last: torch.Tensor, state) -> dict:
        """The gradients of every parameter but the head's from that of its input."""
        tokens, residual, saved_first, y, kept, out, saved = state
        d = norm_residual_backward(None, d_last, y, out, saved, w_post=self.w_post, w_next=self.w_last)
        d_x, grads = self.block.backward(d["d_block"], kept)
        first = norm_residual_backward(d["d_residual"], d_x, None, residual, saved_first, w_next=self.w_first)
        d_embed = torch.zeros(self.embed.shape, device="cuda").index_add_(0, tokens, first["d_residual"].float())
        return {**grads, "w_post": d["d_w_post"], "w_last": d["d_w_next"], "w_first": first["d_w_next"], "embed": d_embed}

    def gradients(self, tokens: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100):
        """(mean loss of the labelled tokens, gradients of every parameter)."""
        last, state = self.forward(tokens)
        labelled = targets != ignore_index
        count = labelled.sum().clamp(min=1)
        loss, saved = linear_cross_entropy(last, self.head, targets, ignore_index=ignore_index)
        d_last, d_head = linear_cross_entropy_backward(labelled.float() / count, last, self.head, targets, saved,
                                                       ignore_index=ignore_index)
        return loss.sum() / count, {"head": d_head, **self.backward(d_last, state)}

    def distilled(self, tokens: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                  temperature: float = 2.0):
        """The same from a teacher's top logits of each token."""
        last, state = self.forward(tokens)
        loss, saved = linear_distillation(last, self.head, teacher_ids, teacher_logits, temperature=temperature)
        d_loss = torch.full_like(loss, 1.0 / loss.numel())
        d_last, d_head = linear_distillation_backward(d_loss, last, self.head, saved, temperature=temperature)
        return loss.mean(), {"head": d_head, **self.backward(d_last, state)}

    def top_logits(self, tokens: torch.Tensor, k: int):
        """What a teacher leaves for a student: its k largest logits of each token and where they are."""
        last, _ = self.forward(tokens)
        plan, T, V = Plan("bf16", la="row", lb="col"), tokens.numel(), self.head.shape[0]
        logits = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
        plan.run(last, self.head, None, logits, T, V, last.shape[1])
        top, ids = torch.topk(logits, k)
        return ids.int(), top

    def update(self, grads: dict, rate: float) -> None:
        for name, d in grads.items():
            owner = self.block if name in ("router", "up", "down") else self
            getattr(owner, name).sub_(rate * d.to(torch.bfloat16))


def main(argv: Optional[list] = None) -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 2048), ("vocab", 32000), ("hidden", 1024), ("inner", 512), ("experts", 16), ("top-k", 2),
                          ("entries", 16), ("steps", 5)):
        p.add_argument(f"--{name}", type=int, default=default)
    p.add_argument("--rate", type=float, default=1.0)
    a = p.parse_args(argv)
    sizes = (a.vocab, a.hidden, a.inner, a.experts, a.top_k)
    model, teacher = LanguageModel(*sizes, seed=0), LanguageModel(*sizes, seed=7)
    gen = torch.Generator(device="cuda").manual_seed(0)
    text = torch.randint(0, a.vocab, (a.tokens + 1,), generator=gen, device="cuda")
    tokens, targets = text[:-1], text[1:].clone()
    targets[: a.tokens // 4] = -100   # a prompt
    ids, logits = teacher.top_logits(tokens, a.entries)
    for name, step in (("labels", lambda: model.gradients(tokens, targets)),
                       ("teacher", lambda: model.distilled(tokens, ids, logits))):
        losses = []
        for _ in range(a.steps):
            torch.cuda.synchronize()
            start = time.perf_counter()
            loss, grads = step()
            model.update(grads, a.rate)
            torch.cuda.synchronize()
            losses.append(f"{float(loss):.4f} ({(time.perf_counter() - start) * 1e3:.1f} ms)")
        print(f"loss on {name}:", " ".join(losses))


if __name__ == "__main__":
    main()

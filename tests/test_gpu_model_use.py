"""The operators around a model's products together, as language_model.py's
training step uses them, against autograd of the same model in 64 bits."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
from dense_gemm_epilogue_02_amd import language_model as lm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


def unit(v):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def reference(m, tokens, loss_of):
    """Loss and gradients of the model in float64; the experts are those that
    the model itself chooses (a choice between close scores is not compared)."""
    p = {n: getattr(m, n).double().requires_grad_() for n in ("embed", "head", "w_first", "w_post", "w_last")}
    p.update({n: getattr(m.block, n).double().requires_grad_() for n in ("router", "up", "down")})
    _, state = m.forward(tokens)
    ids = state[4][1]
    r = p["embed"][tokens]
    x = unit(r) * p["w_first"]
    weights = torch.softmax((x @ p["router"].t()).gather(1, ids), -1)
    y = torch.zeros_like(x)
    for e in range(p["up"].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[t] @ p["up"][e].t()).chunk(2, 1)
        y = y.index_add(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ p["down"][e].t()))
    last = unit(r + unit(y) * p["w_post"]) * p["w_last"]
    loss = loss_of(last @ p["head"].t())
    loss.backward()
    return loss.detach(), {n: t.grad for n, t in p.items()}


# Activations and their gradients are bf16: about a dozen roundings of 2^-9 (rms
# 2^-9 / sqrt 3 of a value each) lie between the loss and a gradient, so 2^-9 *
# sqrt 12 / sqrt 3, times eight, of a gradient's norm.
BOUND = 8 * 2.0 ** -9 * 2


def compare(got, want):
    loss, grads = got
    want_loss, want_grads = want
    assert abs(float(loss - want_loss)) < BOUND * float(want_loss)
    assert set(grads) == set(want_grads)
    for n, r in want_grads.items():
        off = float((grads[n].double() - r).norm() / r.norm())
        assert off < BOUND, f"{n}: {off:.3g} of its norm off, bound {BOUND:.3g}"


def make(T=300, V=1000):
    m = lm.LanguageModel(V, 256, 136, 8, 2, seed=4)
    gen = torch.Generator(device=DEV).manual_seed(0)
    return m, torch.randint(0, V, (T,), generator=gen, device=DEV), torch.randint(0, V, (T,), generator=gen, device=DEV)


def test_gradients_from_labels():
    m, tokens, targets = make()
    targets[:70] = -100
    def loss_of(logits):
        return torch.nn.functional.cross_entropy(logits, targets)
    compare(m.gradients(tokens, targets), reference(m, tokens, loss_of))


def test_gradients_from_a_teacher():
    m, tokens, _ = make(200)
    ids, z = lm.LanguageModel(1000, 256, 136, 8, 2, seed=9).top_logits(tokens, 10)
    def loss_of(logits):
        q = torch.softmax(z.double() / 3.0, -1)
        logp = torch.log_softmax(logits / 3.0, -1).gather(1, ids.long())
        return 9.0 * (q * (torch.log(q) - logp)).sum(-1).mean()
    compare(m.distilled(tokens, ids, z, temperature=3.0), reference(m, tokens, loss_of))


def test_an_expert_without_tokens():
    m, tokens, targets = make(40)
    m.block.router[3] = 0
    m.block.router[3, 0] = -1e4
    x = torch.randn(40, 256, device=DEV).bfloat16().abs()
    out, kept = m.block.forward(x)
    counts = torch.tensor(kept[4]).diff()
    assert int(counts[3]) == 0 and int(counts.sum()) == 80
    d_x, grads = m.block.backward(torch.ones_like(out), kept)
    assert bool((grads["up"][3] == 0).all()) and bool((grads["down"][3] == 0).all())
    assert bool(torch.isfinite(d_x).all()) and all(bool(torch.isfinite(v).all()) for v in grads.values())


def test_many_tokens_are_the_layer_for_few():
    """The experts' products on sorted rows against the layer for up to 64 tokens."""
    m, _, _ = make()
    x = torch.randn(64, 256, device=DEV).bfloat16()
    layer = g.MoeLayer(m.block.router, m.block.up, m.block.down, top_k=2)
    few, ids, p = layer(x, return_routing=True)
    many, kept = m.block.forward(x)
    same = (ids.long() == kept[1]).all(1)
    assert int(same.sum()) >= 60        # close scores may be chosen differently
    # h is rounded on its way here and not there: two roundings of 2^-8 between them
    off = (few[same].float() - many[same].float()).norm() / few[same].float().norm()
    assert float(off) < 4 * 2.0 ** -8


def test_command_runs(capsys):
    lm.main(["--tokens", "200", "--vocab", "700", "--hidden", "128", "--inner", "64", "--experts", "4", "--entries", "5",
             "--steps", "2"])
    out = capsys.readouterr().out
    assert "loss on labels:" in out and "loss on teacher:" in out and "nan" not in out

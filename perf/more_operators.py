"""What a language model's steps need around their products, as cases with
their plain forms.

Operators: the cross entropy of a projection onto the vocabulary without its
logits being kept, and the divergence from a teacher's top logits on the same
projection, both with the gradients of the activations and of the weight; and
tokens sorted by the experts that a router chose and brought back with its
weights, with the gradients. ``run`` computes each from elementary torch
operations where ``own`` is false, and by the package's entry points where it
is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
IGNORED = -100


def listed():
    return [
        # the head of a training step: 4096 tokens, every one with a label
        dict(name="loss_train", op="loss", T=4096, H=4096, V=128000, dtype="bf16", mode="train", ignored=0.0,
             scale=1.0, z_loss=0.0, pad=0),
        # tuning on answers alone: 60 % of the tokens are a prompt without labels; a vocabulary that divides nothing
        dict(name="loss_answers", op="loss", T=4096, H=2048, V=50257, dtype="bf16", mode="train", ignored=0.6,
             scale=1.0, z_loss=1e-4, pad=0),
        # a small head in fp16, a width whose rows are not 16-byte aligned, tokens cut from a wider buffer
        dict(name="loss_ragged", op="loss", T=777, H=1001, V=10007, dtype="f16", mode="train", ignored=0.1,
             scale=0.25, z_loss=0.0, pad=3),
        # scoring a passage: the losses alone
        dict(name="loss_score", op="loss", T=512, H=8192, V=32000, dtype="f16", mode="forward", ignored=0.0,
             scale=1.0, z_loss=0.0, pad=0),
        # the surprise of one decoded token
        dict(name="loss_token", op="loss", T=1, H=4096, V=32000, dtype="bf16", mode="forward", ignored=0.0,
             scale=1.0, z_loss=0.0, pad=0),
        # a student's step on the 64 largest logits that a teacher left
        dict(name="distil_train", op="distil", T=2048, H=4096, V=128000, k=64, dtype="bf16", mode="train", short=0.0,
             temperature=2.0, pad=0),
        # fewer entries for some tokens, none for others
        dict(name="distil_ragged", op="distil", T=500, H=1536, V=32003, k=20, dtype="f16", mode="train", short=0.3,
             temperature=1.0, pad=8),
        # how far a batch of decoded tokens is from the teacher
        dict(name="distil_few", op="distil", T=24, H=2048, V=32000, k=8, dtype="bf16", mode="forward", short=0.0,
             temperature=1.0, pad=0),
        # a training step's tokens to their experts and back
        dict(name="experts_train", op="experts", T=8192, H=4096, E=64, k=6, dtype="bf16", mode="train", dropped=0.0, pad=0),
        # an odd width in fp32, some choices dropped
        dict(name="experts_ragged", op="experts", T=1447, H=1001, E=100, k=3, dtype="f32", mode="train", dropped=0.1, pad=5),
        # a decode batch
        dict(name="experts_few", op="experts", T=64, H=4096, E=64, k=4, dtype="bf16", mode="forward", dropped=0.0, pad=0),
        # many short rows on many experts: a long list to sort
        dict(name="experts_long", op="experts", T=65536, H=512, E=256, k=8, dtype="f16", mode="train", dropped=0.02, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "distil", "experts", "experts"])
    pad = rng.choice([0, 0, 8, 3])
    mode = rng.choice(["train", "train", "forward"])
    if op == "experts":
        E = rng.choice([4, 8, 16, 60, 64, 128, 256])
        T, k = _log(rng, 1, 65536), min(E, rng.choice([1, 2, 4, 6, 8]))
        H = _log(rng, 64, min(8192, max(128, (1 << 27) // (T * k)))) // 8 * 8 + rng.choice([0, 0, 0, 1])
        return dict(op=op, T=T, H=H, E=E, k=k, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), mode=mode,
                    dropped=rng.choice([0.0, 0.0, 0.1]), pad=pad)
    H, V = 8 * _log(rng, 8, 512) + rng.choice([0, 0, 0, 4]), _log(rng, 1000, 128000)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "loss":
        return dict(op=op, T=_log(rng, 1, 4096), H=H, V=V, dtype=dtype, mode=mode, ignored=rng.choice([0.0, 0.0, 0.3, 0.7]),
                    scale=rng.choice([1.0, 1.0, 0.5]), z_loss=rng.choice([0.0, 0.0, 1e-4]), pad=pad)
    return dict(op=op, T=_log(rng, 1, 2048), H=H, V=V, k=rng.choice([1, 8, 20, 64, 100]), dtype=dtype, mode=mode,
                short=rng.choice([0.0, 0.0, 0.3]), temperature=rng.choice([1.0, 2.0, 4.0]), pad=pad)


# ---- inputs ---------------------------------------------------------------


def _rows(gen, rows, cols, dtype, pad, std=1.0):
    """N(0, std^2) rows, cut from a buffer of cols + pad columns."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(std).to(DTYPES[dtype])[:, :cols]


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    T, H, dtype = case["T"], case["H"], case["dtype"]
    if own:
        import dense_gemm_epilogue_02_amd as g
        s["g"] = g
    if case["op"] == "experts":
        E, k = case["E"], case["k"]
        # a router's scores: some experts are asked for more than others
        liked = torch.randn(E, generator=gen, device="cuda")
        scores, ids = torch.topk(torch.randn(T, E, generator=gen, device="cuda") + liked, k)
        s["weights"] = torch.softmax(scores, -1)
        s["ids"] = torch.where(_uniform(gen, T, k) < case["dropped"], -1, ids).int()
        s["x"] = _rows(gen, T, H, dtype, case["pad"])
        s["y"] = _rows(gen, T * k, H, dtype, 0, 0.5)
        if case["mode"] == "train":
            s["d_out"] = _rows(gen, T, H, dtype, case["pad"], 1e-2)
            s["d_rows"] = _rows(gen, T * k, H, dtype, 0, 1e-2)
        return s
    V = case["V"]
    s["x"] = _rows(gen, T, H, dtype, case["pad"])
    s["w"] = _rows(gen, V, H, dtype, 0, 2.0 / math.sqrt(H))
    if case["op"] == "loss":
        # a frequent word is a label more often than a rare one
        labels = (V * _uniform(gen, T) ** 3).long().clamp(max=V - 1)
        s["targets"] = torch.where(_uniform(gen, T) < case["ignored"], IGNORED, labels)
        count = (s["targets"] != IGNORED).sum().clamp(min=1)
        s["d_loss"] = (s["targets"] != IGNORED).float() / count
    else:
        k = case["k"]
        gaps = (_uniform(gen, T, k) * max(1, V // k)).long()
        s["ids"] = (torch.arange(k, device="cuda") * (V // k) + gaps).clamp(max=V - 1).int()
        s["ids"] = s["ids"].gather(1, torch.argsort(_uniform(gen, T, k), dim=1))
        s["logits"] = torch.sort(_rows(gen, T, k, "f32", 0, 2.0), dim=1, descending=True).values + 4
        # a token keeps its first entries
        keep = torch.where(_uniform(gen, T, 1) < case["short"], (_uniform(gen, T, 1) * k).long(), k)
        s["ids"] = torch.where(torch.arange(k, device="cuda") < keep, s["ids"], -1)
        s["d_loss"] = torch.full((T,), 1.0 / T, device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------


def _log_sum(l):
    m = l.amax(1, keepdim=True)
    return (m + torch.log(torch.exp(l - m).sum(1, keepdim=True)))[:, 0]


def _gradients(s, d_logits):
    dt = s["x"].dtype
    return (d_logits @ s["w"].float()).to(dt), (d_logits.t() @ s["x"].float()).to(dt)


def _plain_loss(s):
    scale, z = s["scale"], s["z_loss"]
    logits = scale * (s["x"].float() @ s["w"].float().t())
    lse = _log_sum(logits)
    valid = s["targets"] != IGNORED
    target = torch.where(valid, s["targets"], 0).unsqueeze(1)
    loss = torch.where(valid, lse - logits.gather(1, target)[:, 0] + z * lse * lse, 0.0)
    if s["mode"] == "forward":
        return {"loss": loss}
    d = torch.where(valid, s["d_loss"], 0.0).unsqueeze(1)
    g = torch.exp(logits - lse.unsqueeze(1)) * (1 + 2 * z * lse.unsqueeze(1))
    g.scatter_add_(1, target, -torch.ones_like(target, dtype=torch.float32))
    dx, dw = _gradients(s, g * (d * scale))
    return {"loss": loss, "dx": dx, "dw": dw}


def _plain_distil(s):
    tau = s["temperature"]
    logits = (s["x"].float() @ s["w"].float().t()) / tau
    lse = _log_sum(logits)
    there = s["ids"] >= 0
    at = torch.where(there, s["ids"], 0).long()
    z = torch.where(there, s["logits"].float() / tau, -1e30)
    z = z - z.amax(1, keepdim=True)
    e = torch.where(there, torch.exp(z), 0.0)
    total = e.sum(1, keepdim=True).clamp(min=1e-30)
    q = e / total
    mass = there.any(1).float()
    terms = torch.where(there, q * (z - torch.log(total) - logits.gather(1, at) + lse.unsqueeze(1)), 0.0)
    loss = tau * tau * terms.sum(1)
    if s["mode"] == "forward":
        return {"loss": loss}
    g = torch.exp(logits - lse.unsqueeze(1)) * mass.unsqueeze(1)
    g.scatter_add_(1, at, -q)
    dx, dw = _gradients(s, g * (s["d_loss"] * tau).unsqueeze(1))
    return {"loss": loss, "dx": dx, "dw": dw}


def _plain_experts(s):
    T, H, E, k, dt = s["T"], s["H"], s["E"], s["k"], s["x"].dtype
    ids = s["ids"].flatten().long()
    n = T * k
    chosen = ids >= 0
    by_expert = torch.sort(torch.where(chosen, ids, E), stable=True)
    ends = torch.searchsorted(by_expert.values, torch.arange(E + 1, device=ids.device))
    slot = by_expert.indices                      # the slot of each sorted row
    used = by_expert.values < E
    at = torch.empty_like(slot).scatter_(0, slot, torch.arange(n, device=ids.device))
    row_of = torch.where(chosen, at, -1).view(T, k)
    token = slot // k
    safe, there = at.view(T, k), chosen.view(T, k, 1)
    w = s["weights"].unsqueeze(-1)
    zero = torch.zeros((), device=ids.device)
    y = torch.where(there, s["y"].float()[safe], zero)
    out = {"offsets": ends.int(), "row_of": row_of.int(),
           "rows": torch.where(used.unsqueeze(1), s["x"][token], 0),
           "out": (y * w).sum(1).to(dt)}
    if s["mode"] == "train":
        out["d_x"] = torch.where(there, s["d_rows"].float()[safe], zero).sum(1).to(dt)
        d = s["d_out"].float()
        out["d_y"] = torch.where(used.unsqueeze(1), d[token] * s["weights"].flatten()[slot].unsqueeze(1), zero).to(dt)
        out["d_weights"] = (y * d.unsqueeze(1)).sum(-1)
    return out


# ---- one pass -----------------------------------------------------------------


def run(s):
    op = s["op"]
    if not own:
        return {"loss": _plain_loss, "distil": _plain_distil, "experts": _plain_experts}[op](s)
    g, train = s["g"], s["mode"] == "train"
    if op == "loss":
        how = dict(ignore_index=IGNORED, scale=s["scale"], z_loss=s["z_loss"])
        loss, saved = g.linear_cross_entropy(s["x"], s["w"], s["targets"], **how)
        out = {"loss": loss}
        if train:
            out["dx"], out["dw"] = g.linear_cross_entropy_backward(s["d_loss"], s["x"], s["w"], s["targets"], saved, **how)
        return out
    if op == "distil":
        how = dict(temperature=s["temperature"])
        loss, saved = g.linear_distillation(s["x"], s["w"], s["ids"], s["logits"], **how)
        out = {"loss": loss}
        if train:
            out["dx"], out["dw"] = g.linear_distillation_backward(s["d_loss"], s["x"], s["w"], saved, **how)
        return out
    order = g.expert_sort(s["ids"], s["E"])
    out = {"offsets": order.offsets, "row_of": order.row_of, "rows": g.expert_gather(s["x"], order),
           "out": g.expert_combine(s["y"], order, s["weights"])}
    if train:
        out["d_x"] = g.expert_gather_backward(s["d_rows"], order)
        out["d_y"], out["d_weights"] = g.expert_combine_backward(s["d_out"], s["y"], order, s["weights"])
    return out


def work(case):
    T, H, es = case["T"], case["H"], BYTES[case["dtype"]]
    train = case["mode"] == "train"
    if case["op"] == "experts":
        # x to its rows, and rows to out; in training both again, with the combined rows and their gradient
        n = T * case["k"]
        rows = (2 * n + 2 * T) * H * es
        return {"bytes": rows + (n + T) * H * es + (2 * n + T) * H * es if train else rows,
                "flops": (10 if train else 2) * n * H}
    V = case["V"]
    # rows without a label ask for nothing
    rows = T * (1 - case["ignored"]) if case["op"] == "loss" else T
    product = 2 * rows * H * V
    matrices = (rows + V) * H * es
    # the gradients need two products more
    return {"bytes": 2 * matrices if train else matrices, "flops": product * (3 if train else 1)}


# ---- the definitions in 64 bits -----------------------------------------------


def _exact_head(s, weights_of, train):
    """The losses, and the gradients by rows: weights_of(rows, logits, log of
    their sum) gives the losses of some rows and the gradient of their logits."""
    x, w = s["x"].double(), s["w"].double()
    T, step = x.shape[0], 512
    loss, dx = [], []
    dw = torch.zeros_like(w) if train else None
    for at in range(0, T, step):
        rows = slice(at, min(at + step, T))
        logits = torch.mm(x[rows], w.t())
        value, d = weights_of(rows, logits)
        loss.append(value)
        if train:
            dx.append(torch.mm(d, w))
            dw.addmm_(d.t(), x[rows])
    out = {"loss": torch.cat(loss)}
    if train:
        out["dx"], out["dw"] = torch.cat(dx), dw
    return out


def _exact_loss(s):
    def of(rows, raw):
        t = s["targets"][rows]
        logp = torch.log_softmax(raw * s["scale"], 1)
        lse = (raw[:, 0] * s["scale"]) - logp[:, 0]
        named = (torch.arange(raw.shape[1], device=raw.device) == t.unsqueeze(1)).double()
        use = (t != IGNORED).double()
        value = use * (-(logp * named).sum(1) + s["z_loss"] * lse.square())
        d = (1 + 2 * s["z_loss"] * lse).unsqueeze(1) * torch.exp(logp) - named
        return value, d * (use * s["d_loss"][rows].double() * s["scale"]).unsqueeze(1)
    return _exact_head(s, of, s["mode"] == "train")


def _exact_distil(s):
    tau = s["temperature"]

    def of(rows, raw):
        ids, z = s["ids"][rows], s["logits"][rows].double() / tau
        logp = torch.log_softmax(raw / tau, 1)
        # the teacher's distribution over the vocabulary, entry by entry
        q = torch.zeros_like(logp)
        share = torch.softmax(torch.where(ids >= 0, z, -math.inf), 1).nan_to_num(0.0)
        at = torch.arange(raw.shape[0], device=raw.device)
        for j in range(ids.shape[1]):
            q[at, ids[:, j].clamp(min=0).long()] += torch.where(ids[:, j] >= 0, share[:, j], 0.0)
        value = (torch.special.xlogy(q, q) - q * logp).sum(1) * tau ** 2
        d = torch.exp(logp) * q.sum(1, keepdim=True) - q
        return value, d * (s["d_loss"][rows].double() * tau).unsqueeze(1)
    return _exact_head(s, of, s["mode"] == "train")


def _exact_experts(s):
    T, H, E, k = (s[n] for n in ("T", "H", "E", "k"))
    ids = s["ids"].long()
    n = T * k
    slots = torch.arange(n, device=ids.device).view(T, k)
    # place of a slot: by expert, then by its own number; dropped ones behind all
    key = torch.where(ids < 0, E, ids) * n + slots
    place = torch.empty(n, dtype=torch.long, device=ids.device)
    place[torch.argsort(key.flatten())] = torch.arange(n, device=ids.device)
    counts = torch.bincount(ids[ids >= 0], minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    row_of = torch.where(ids < 0, -1, place.view(T, k))
    t, j = torch.nonzero(ids >= 0, as_tuple=True)
    p = row_of[t, j]
    rows = torch.zeros(n, H, dtype=torch.float64, device=ids.device)
    rows[p] = s["x"][t].double()
    weight = s["weights"].double()
    result = torch.zeros(T, H, dtype=torch.float64, device=ids.device)
    for c in range(k):
        u = t[j == c]
        result[u] += weight[u, c].unsqueeze(1) * s["y"][row_of[u, c]].double()
    out = {"offsets": offsets.int(), "row_of": row_of.int(), "rows": rows, "out": result}
    if s["mode"] == "train":
        d_x, d_y = torch.zeros_like(result), torch.zeros_like(rows)
        d_weights = torch.zeros(T, k, dtype=torch.float64, device=ids.device)
        for c in range(k):
            u = t[j == c]
            at = row_of[u, c]
            d_x[u] += s["d_rows"][at].double()
            d_y[at] = weight[u, c].unsqueeze(1) * s["d_out"][u].double()
            d_weights[u, c] = torch.linalg.vecdot(s["d_out"][u].double(), s["y"][at].double())
        out["d_x"], out["d_y"], out["d_weights"] = d_x, d_y, d_weights
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"loss": _exact_loss, "distil": _exact_distil, "experts": _exact_experts}[case["op"]](s)

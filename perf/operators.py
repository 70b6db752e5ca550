"""The feed-forward block's operators, as cases with their plain forms.

Operators: MXFP4 quantisation (one E8M0 scale per 32 elements, e2m1 elements
packed two per byte, rows padded to a multiple of 256 elements), the linear
layer on MXFP4 operands with its backward pass, a mixture-of-experts layer for
a few tokens, and the norms before and after a block fused with its gate and
residual scale. ``run`` computes each from elementary torch operations where
``own`` is false, and by the package's entry points where it is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "mx4": 0.5 + 1 / 32}
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a projection's master weight quantised for all three products of a training step
        dict(name="quantise_weight", op="quantise", rows=4096, cols=8192, dtype="bf16", axis="both", pad=0),
        # a ragged fp32 activation quantised along the tokens, as a weight gradient needs it
        dict(name="quantise_ragged", op="quantise", rows=333, cols=1447, dtype="f32", axis="0", pad=5),
        # one decoded token through a square projection
        dict(name="linear_token", op="linear", M=1, N=8192, K=8192, dtype="bf16", bias=False, pad=0),
        # the fused QKV projection of a 4096-token prefill
        dict(name="linear_prefill", op="linear", M=4096, N=10240, K=8192, dtype="bf16", bias=True, pad=0),
        # both gradients of a square projection over 4096 tokens
        dict(name="backward_layer", op="backward", M=4096, N=8192, K=8192, dtype="bf16", pad=0),
        # both gradients of a small layer with sizes that divide nothing, tokens cut from a wider buffer
        dict(name="backward_ragged", op="backward", M=777, N=1000, K=2057, dtype="f16", pad=3),
        # one decoded token, 16-bit experts
        dict(name="moe_token", op="moe", T=1, H=4096, I=1024, E=64, k=4, weights="bf16", renorm=True),
        # a decode batch of 16 on MXFP4 experts: nearly every expert is read
        dict(name="moe_mx4", op="moe", T=16, H=4096, I=2048, E=32, k=4, weights="mx4", renorm=True),
        # a full decode batch on many small experts of an odd width
        dict(name="moe_batch", op="moe", T=64, H=2048, I=1000, E=64, k=6, weights="f16", renorm=False),
        # between two blocks of one decoded token
        dict(name="norm_token", op="norm", T=1, H=8192, dtype="bf16", mode="forward", post=True,
             gate="none", scale=True, pad=0),
        # a training step's 4096 tokens of four sequences, the gate a vector of each sequence
        dict(name="norm_train", op="norm", T=4096, H=8192, dtype="bf16", mode="train", post=True,
             gate="group", scale=True, pad=0),
        # an odd width in fp32, every token with a gate of its own, rows cut from a wider buffer
        dict(name="norm_train_ragged", op="norm", T=511, H=2001, dtype="f32", mode="train", post=True,
             gate="row", scale=True, pad=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "linear", "linear", "backward", "moe", "moe", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    pad = rng.choice([0, 0, 8, 3])
    if op == "quantise":
        return dict(op=op, rows=_log(rng, 1, 4096), cols=_log(rng, 32, 8192), dtype=dtype,
                    axis=rng.choice(["0", "1", "both"]), pad=pad)
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 2048), N=8 * _log(rng, 8, 1280) + rng.choice([0, 0, 1]),
                    K=32 * _log(rng, 2, 256) + rng.choice([0, 0, 8, 5]), dtype=dtype,
                    bias=rng.random() < 0.5, pad=pad)
    if op == "backward":
        return dict(op=op, M=_log(rng, 16, 4096), N=8 * _log(rng, 8, 1024) + rng.choice([0, 0, 1]),
                    K=8 * _log(rng, 8, 1024) + rng.choice([0, 0, 3]), dtype=dtype, pad=pad)
    if op == "moe":
        E = rng.choice([4, 8, 16, 32, 64, 100])
        k = rng.choice([1, 2, 4, 4, 6, 8])
        H = 8 * _log(rng, 32, 512)
        most = max(128, (1 << 27) // (E * H))   # weights no larger than the largest listed layer's
        return dict(op=op, T=_log(rng, 1, 64), H=H, I=min(most, 8 * _log(rng, 16, 256)) // 8 * 8 + rng.choice([0, 0, 3]),
                    E=E, k=min(k, E), weights=rng.choice(["bf16", "bf16", "f16", "mx4", "mx4"]), renorm=rng.random() < 0.7)
    return dict(op=op, T=_log(rng, 1, 4096), H=_log(rng, 64, 8192), dtype=dtype,
                mode=rng.choice(["forward", "train"]), post=rng.random() < 0.7,
                gate=rng.choice(["none", "row", "group", "shared"]), scale=rng.random() < 0.6, pad=pad)


# ---- inputs ---------------------------------------------------------------


def _rows(gen, rows, cols, dtype, pad, std=1.0):
    """N(0, std^2) rows, cut from a buffer of cols + pad columns."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(std).to(DTYPES[dtype])[:, :cols]


def _pack(w):
    """The MXFP4 storage of w along its last dimension: packed codes and scale
    bytes of rows padded to a multiple of 256 elements."""
    k = w.shape[-1]
    kp = -(-k // 256) * 256
    v = torch.nn.functional.pad(w.float(), (0, kp - k)).unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, 0)
    q = _on_grid(torch.ldexp(v, -e)).flatten(-2)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) + 8 * (q < 0)
    return ((code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8).contiguous(),
            (e + 127).squeeze(-1).to(torch.uint8).contiguous())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if own:
        import dense_gemm_epilogue_02_amd as g
        s["g"] = g
    if op == "quantise":
        s["x"] = _rows(gen, case["rows"], case["cols"], case["dtype"], case["pad"])
        # a few outlier columns, as activations have them
        s["x"][:, :: 61] *= 16
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _rows(gen, M, K, case["dtype"], case["pad"])
        s["codes"], s["scales"] = _pack(_rows(gen, N, K, "bf16", 0, 0.02))
        s["bias"] = _rows(gen, 1, N, "bf16", 0)[0] if case["bias"] else None
        if own:
            s["layer"] = g.Mx4Linear(g.Mx4(s["codes"], s["scales"], K))
    elif op == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _rows(gen, M, K, case["dtype"], case["pad"])
        s["dy"] = _rows(gen, M, N, case["dtype"], case["pad"], 1e-3)
        # the weight as the input gradient reads it: rows of K, blocks along N
        s["codes"], s["scales"] = _pack(_rows(gen, N, K, "bf16", 0, 0.02).t())
        if own:
            s["layer"] = g.Mx4Linear(None, g.Mx4(s["codes"], s["scales"], N))
    elif op == "moe":
        T, H, I, E, kind = case["T"], case["H"], case["I"], case["E"], case["weights"]
        dt = "bf16" if kind == "mx4" else kind
        s["x"] = _rows(gen, T, H, dt, 0)
        s["router"] = _rows(gen, E, H, dt, 0, 2.0 / math.sqrt(H))
        up = [_rows(gen, 2 * I, H, dt, 0, 1 / math.sqrt(H)) for _ in range(E)]
        down = [_rows(gen, H, I, dt, 0, 1 / math.sqrt(I)) for _ in range(E)]
        if kind == "mx4":
            up, down = [_pack(w) for w in up], [_pack(w) for w in down]
            for name, w in (("up", up), ("down", down)):
                s[name], s[name + "_scales"] = (torch.stack(t) for t in zip(*w))
            ups = (s["up"], s["up_scales"], H)
            downs = (s["down"], s["down_scales"], I)
        else:
            s["up"], s["down"] = torch.stack(up), torch.stack(down)
        if own:
            w13, w2 = (g.Mx4(*ups), g.Mx4(*downs)) if kind == "mx4" else (s["up"], s["down"])
            s["layer"] = g.MoeLayer(s["router"], w13, w2, top_k=case["k"], renormalize=case["renorm"])
    else:
        T, H, dt, pad = case["T"], case["H"], case["dtype"], case["pad"]
        s["block"] = _rows(gen, T, H, dt, pad, 0.5)
        s["residual"] = _rows(gen, T, H, dt, pad, 2.0)
        s["w_post"] = _rows(gen, 1, H, dt, 0, 0.2)[0] + 1 if case["post"] else None
        s["w_next"] = _rows(gen, 1, H, dt, 0, 0.2)[0] + 1
        s["scale"] = _rows(gen, 1, H, dt, 0, 0.1)[0] + 0.5 if case["scale"] else None
        groups = {"none": 0, "row": T, "shared": 1, "group": 4 if T % 4 == 0 else 1}[case["gate"]]
        s["gate"] = _rows(gen, groups, H, dt, 0) if groups else None
        if case["mode"] == "train":
            s["d_out"] = _rows(gen, T, H, dt, pad, 1e-2)
            s["d_next"] = _rows(gen, T, H, dt, pad, 1e-2)
    return s


# ---- plain forms ------------------------------------------------------------


def _on_grid(v):
    """Round to nearest even onto the e2m1 values, saturating at 6."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _quantised(x):
    """The values that x's MXFP4 form along its last dimension stands for, in fp32."""
    k = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -k % 32)).unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, 0)
    return torch.ldexp(_on_grid(torch.ldexp(v, -e)), e).flatten(-2)[..., :k]


def _values(codes, scales, k):
    """What packed codes and scale bytes stand for, in fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, 32))
    return torch.ldexp(table[c.int()], scales.int().unsqueeze(-1) - 127).flatten(-2)[..., :k]


def _route(s):
    logits = s["x"].double() @ s["router"].double().t()
    top, ids = (t[:, :s["k"]] for t in torch.sort(logits, dim=-1, descending=True, stable=True))
    p = torch.softmax(top, -1) if s["renorm"] else torch.exp(top - torch.logsumexp(logits, -1, keepdim=True))
    return ids, p.float()


def _plain_moe(s):
    T, H, I, E, k = (s[n] for n in ("T", "H", "I", "E", "k"))
    ids, p = _route(s)
    x = s["x"].float()
    if T * k < E:     # the chosen experts' weights, gathered
        pick = ids.reshape(-1)
        up, down = s["up"][pick], s["down"][pick]
        rows = x.repeat_interleave(k, 0).unsqueeze(1)
    else:             # every expert on every token
        pick = slice(None)
        up, down = s["up"], s["down"]
        rows = x.expand(E, T, H)
    if s["weights"] == "mx4":
        up, down = _values(up, s["up_scales"][pick], H), _values(down, s["down_scales"][pick], I)
    gu = torch.bmm(rows, up.float().transpose(1, 2).contiguous())
    h = gu[..., :I] * torch.sigmoid(gu[..., :I]) * gu[..., I:]
    y = torch.bmm(h, down.float().transpose(1, 2).contiguous())
    if T * k < E:
        y = y.reshape(T, k, H)
    else:
        y = y[ids, torch.arange(T, device=ids.device).unsqueeze(1)]
    return (y * p.unsqueeze(-1)).sum(1).to(s["x"].dtype), ids.int(), p


def _plain_norm(s):
    dt = s["block"].dtype
    f = {n: s[n].float() if s.get(n) is not None else None
         for n in ("block", "residual", "w_post", "w_next", "scale", "gate", "d_out", "d_next")}
    T, H = f["block"].shape
    one = torch.ones((), device=f["block"].device)
    b, w_post, w_next = f["block"], f["w_post"], f["w_next"]
    groups = 0 if f["gate"] is None else f["gate"].shape[0]
    gate = one if not groups else f["gate"].repeat_interleave(T // groups, 0)
    scale = one if f["scale"] is None else f["scale"]
    if w_post is None:
        y = b
    else:
        rb = torch.rsqrt(b.square().mean(-1, keepdim=True) + EPS)
        y = b * rb * w_post
    r = (f["residual"] + scale * gate * y).to(dt)
    rf = r.float()
    rr = torch.rsqrt(rf.square().mean(-1, keepdim=True) + EPS)
    out = {"out": r, "next": (rf * rr * w_next).to(dt)}
    if s["mode"] == "forward":
        return out
    xn = rf * rr
    g = f["d_next"] * w_next
    d = f["d_out"] + rr * (g - xn * (g * xn).mean(-1, keepdim=True))
    out["d_residual"] = d.to(dt)
    out["d_w_next"] = (f["d_next"] * xn).sum(0).to(dt)
    if f["scale"] is not None:
        out["d_scale"] = (d * gate * y).sum(0).to(dt)
    if groups:
        out["d_gate"] = (d * scale * y).reshape(groups, T // groups, H).sum(1).to(dt)
    dy = d * scale * gate
    if w_post is None:
        out["d_block"] = dy.to(dt)
    else:
        xb = b * rb
        out["d_w_post"] = (dy * xb).sum(0).to(dt)
        g = dy * w_post
        out["d_block"] = (rb * (g - xb * (g * xb).mean(-1, keepdim=True))).to(dt)
    return out


# ---- one pass -----------------------------------------------------------------


def run(s):
    op = s["op"]
    if op == "quantise":
        x = s["x"]
        if own:
            q = s["g"].mx4_quantize(x, axis=s["axis"] if s["axis"] == "both" else int(s["axis"]))
            return [s["g"].mx4_dequantize(t, x.dtype) for t in (q if s["axis"] == "both" else [q])]
        views = {"1": [x], "0": [x.t()], "both": [x, x.t()]}[s["axis"]]
        return [_quantised(v).to(x.dtype) for v in views]
    if op == "linear":
        if own:
            return s["layer"].forward(s["x"], s["bias"])
        y = _quantised(s["x"]) @ _values(s["codes"], s["scales"], s["K"]).t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)
    if op == "backward":
        if own:
            return s["layer"].backward(s["dy"], s["x"])
        dx = _quantised(s["dy"]) @ _values(s["codes"], s["scales"], s["N"]).t()
        dw = _quantised(s["dy"].t()) @ _quantised(s["x"].t()).t()
        return dx.to(torch.bfloat16), dw.to(torch.bfloat16)
    if op == "moe":
        return s["layer"](s["x"], return_routing=True) if own else _plain_moe(s)
    if not own:
        return _plain_norm(s)
    g = s["g"]
    r, h, saved = g.norm_residual(s["block"], s["residual"], w_post=s["w_post"], gate=s["gate"],
                                  scale=s["scale"], w_next=s["w_next"], eps=EPS)
    out = {"out": r, "next": h}
    if s["mode"] == "train":
        d = g.norm_residual_backward(s["d_out"], s["d_next"], s["block"], r, saved, w_post=s["w_post"],
                                     gate=s["gate"], scale=s["scale"], w_next=s["w_next"])
        out.update({n: v for n, v in d.items() if v is not None})
    return out


def work(case):
    op = case["op"]
    if op == "quantise":
        n, es = case["rows"] * case["cols"], BYTES[case["dtype"]]
        return {"bytes": n * es * (3 if case["axis"] == "both" else 2), "flops": 0}
    if op in ("linear", "backward"):
        M, N, K, es = case["M"], case["N"], case["K"], BYTES[case["dtype"]]
        if op == "linear":
            return {"bytes": M * K * es + N * K * BYTES["mx4"] + 2 * M * N, "flops": 2 * M * N * K}
        return {"bytes": M * (K + N) * es + N * K * BYTES["mx4"] + 2 * (M + N) * K, "flops": 4 * M * N * K}
    if op == "moe":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        # distinct experts that T tokens of k choices each reach, were the choices even
        reached = E * (1 - (1 - k / E) ** T)
        return {"bytes": reached * 3 * H * I * BYTES[case["weights"]] + 2 * E * H + 4 * T * H,
                "flops": 2 * T * H * (E + 3 * I * k)}
    n, es = case["T"] * case["H"], BYTES[case["dtype"]]
    passes = 4 + (case["gate"] == "row")
    if case["mode"] == "train":
        # block, the new residual, two gradients in; two out (and the gate's in and out)
        passes += 6 + 2 * (case["gate"] == "row")
    return {"bytes": passes * n * es, "flops": 12 * n}


# ---- the definitions in 64 bits -----------------------------------------------


def _exact_values(codes, scales, k):
    lo, hi = (codes % 16).long(), (codes // 16).long()
    c = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.long, device=codes.device)
    c[..., 0::2], c[..., 1::2] = lo, hi
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)[c % 8]
    v = torch.where(c >= 8, -mag, mag)
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1))[..., :k]


def _exact_quantised(x):
    """Nearest e2m1 value of each element at its block's scale, by the borders between neighbours."""
    rows, k = x.shape
    v = torch.zeros(rows, -(-k // 32) * 32, dtype=torch.float64, device=x.device)
    v[:, :k] = x.double()
    v = v.reshape(rows, -1, 32)
    amax = v.abs().max(-1, keepdim=True).values
    s = torch.exp2(torch.floor(torch.log2(amax.clamp(min=1e-300))) - 2)
    s = torch.where(amax > 0, s, torch.ones_like(s))
    a = v.abs() / s
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    # a border belongs to the neighbour with the even code
    below, above = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    i = torch.where(below == above, below, torch.where(below % 2 == 0, below, above))
    return (torch.sign(v) * grid[i] * s).reshape(rows, -1)[:, :k]


def _exact_expert(s, e, x, share):
    """What expert e adds to the tokens that chose it, each by its share."""
    y, I = torch.zeros_like(x), s["I"]
    t = torch.nonzero(share).flatten()
    if s["weights"] == "mx4":
        up = _exact_values(s["up"][e], s["up_scales"][e], s["H"])
        down = _exact_values(s["down"][e], s["down_scales"][e], I)
    else:
        up, down = s["up"][e].double(), s["down"][e].double()
    a, b = x[t] @ up[:I].t(), x[t] @ up[I:].t()
    y[t] = share[t, None] * ((a / (1 + torch.exp(-a)) * b) @ down.t())
    return y


def _exact_moe(s):
    k, x = s["k"], s["x"].double()
    logits = torch.stack([x @ w for w in s["router"].double()], 1)
    # rank of an expert: how many come before it, larger or equal with a lower index
    index = torch.arange(s["E"], device=x.device)
    before = (logits.unsqueeze(1) > logits.unsqueeze(2)) | (
        (logits.unsqueeze(1) == logits.unsqueeze(2)) & (index < index.unsqueeze(1)))
    rank = before.sum(2)
    ids = torch.argsort(rank, dim=1)[:, :k]
    chosen = rank < k
    share = torch.exp(logits - logits.max(1, keepdim=True).values)
    share = share / (torch.where(chosen, share, 0.0) if s["renorm"] else share).sum(1, keepdim=True)
    y = sum(_exact_expert(s, e, x, share[:, e] * chosen[:, e]) for e in range(s["E"]))
    return y, ids.int(), torch.gather(share, 1, ids)


def _exact_norm(s):
    d = {n: s[n].double() for n in ("block", "residual", "w_post", "w_next", "scale", "gate", "d_out", "d_next")
         if s.get(n) is not None}
    T, H = d["block"].shape
    groups = d["gate"].shape[0] if "gate" in d else 0
    of_row = torch.arange(T, device="cuda") // (T // groups) if groups else None
    gate = d["gate"][of_row] if groups else torch.ones(T, H, dtype=torch.float64, device="cuda")
    scale = d.get("scale", torch.ones(H, dtype=torch.float64, device="cuda"))
    unit = lambda v: v / torch.sqrt((v * v).sum(1, keepdim=True) / H + EPS)  # noqa: E731

    def through(v, dn):
        """The gradient of v from that of unit(v)."""
        n = torch.sqrt((v * v).sum(1, keepdim=True) / H + EPS)
        return dn / n - v * (dn * v).sum(1, keepdim=True) / (H * n ** 3)

    y = unit(d["block"]) * d["w_post"] if "w_post" in d else d["block"]
    # the stored residual is what the next norm and the backward pass read
    r = (d["residual"] + scale * gate * y).to(s["block"].dtype).double()
    out = {"out": d["residual"] + scale * gate * y, "next": unit(r) * d["w_next"]}
    if s["mode"] == "train":
        g = d["d_out"] + through(r, d["d_next"] * d["w_next"])
        out["d_residual"] = g
        out["d_w_next"] = torch.einsum("th,th->h", d["d_next"], unit(r))
        if "scale" in d:
            out["d_scale"] = torch.einsum("th,th,th->h", g, gate, y)
        if groups:
            out["d_gate"] = torch.zeros_like(d["gate"]).index_add_(0, of_row, g * scale * y)
        dy = g * scale * gate
        if "w_post" in d:
            out["d_w_post"] = torch.einsum("th,th->h", dy, unit(d["block"]))
            dy = through(d["block"], dy * d["w_post"])
        out["d_block"] = dy
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        views = {"1": [s["x"]], "0": [s["x"].t()], "both": [s["x"], s["x"].t()]}[case["axis"]]
        return [_exact_quantised(v) for v in views]
    if op == "linear":
        y = _exact_quantised(s["x"]) @ _exact_values(s["codes"], s["scales"], case["K"]).t()
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "backward":
        dx = _exact_quantised(s["dy"]) @ _exact_values(s["codes"], s["scales"], case["N"]).t()
        dw = _exact_quantised(s["dy"].t()) @ _exact_quantised(s["x"].t()).t()
        return dx, dw
    return _exact_moe(s) if op == "moe" else _exact_norm(s)

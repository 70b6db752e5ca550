"""Plain 64-bit forms of the feed-forward block's operators (CPU, torch
float64 / numpy), with the error bounds that the tests use. Written from the
definitions in include/gemm_block.h; no code of the package is used."""
from __future__ import annotations

import math

import numpy as np
import torch

# half a rounding step of a value, relative to it
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F32 = 2.0 ** -24


def least(half):
    """Half the smallest step of a type: what a value below its normal range
    is rounded by at most (fp16; the others' is below anything drawn here)."""
    return 2.0 ** -25 if half == HALF[torch.float16] else 1e-37


GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def padded(k):
    return -(-k // 256) * 256


# ---- MXFP4 ---------------------------------------------------------------------


def quantize(x: torch.Tensor):
    """(values [R, k] float64, scale bytes [R, ceil(k / 32)]) of x's MXFP4 form along its rows."""
    a = x.double().numpy()
    R, k = a.shape
    nb = -(-k // 32)
    v = np.zeros((R, nb * 32))
    v[:, :k] = a
    v = v.reshape(R, nb, 32)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(-1)
    _, e = np.frexp(amax)                       # amax = m 2^e, m in [1/2, 1)
    byte = np.clip(e - 1 - 2 + 127, 0, 254)
    byte = np.where(amax == 0, 127, byte)
    s = np.ldexp(1.0, byte - 127)[..., None]
    q = np.abs(v) / s
    d = np.abs(q[..., None] - GRID)             # nearest, ties to the even code
    near = d.min(-1, keepdims=True)
    cand = d == near
    even = cand & (np.arange(8) % 2 == 0)
    i = np.where(even.any(-1), even.argmax(-1), cand.argmax(-1))
    val = np.sign(v) * GRID[i] * s
    val = np.where(bad[..., None], np.nan, val)
    byte = np.where(bad, 255, byte)
    return torch.from_numpy(val.reshape(R, -1)[:, :k].copy()), torch.from_numpy(byte.astype(np.uint8))


def unpack(codes: torch.Tensor, scales: torch.Tensor, k: int):
    """The values of packed codes and scale bytes (2-D), in float64."""
    c = codes.cpu().numpy()
    n = np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    v = np.where(n >= 8, -1.0, 1.0) * GRID[n & 7]
    b = scales.cpu().numpy().astype(np.int64)
    s = np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return torch.from_numpy((v.reshape(c.shape[0], -1, 32) * s[..., None]).reshape(c.shape[0], -1)[:, :k].copy())


def pack(w: torch.Tensor):
    """w [R, k] as (codes, scales, values): numpy packing of quantize()."""
    v, byte = quantize(w)
    R, k = w.shape
    kp = padded(k)
    s = np.ldexp(1.0, byte.numpy().astype(np.int64) - 127).repeat(32, -1)[:, :k]
    q = v.numpy() / s
    code = np.abs(np.abs(q)[..., None] - GRID).argmin(-1) + 8 * (q < 0)
    full = np.zeros((R, kp), np.uint8)
    full[:, :k] = code
    sc = np.full((R, kp // 32), 127, np.uint8)
    sc[:, :byte.shape[1]] = byte.numpy()
    return torch.from_numpy(full[:, 0::2] | full[:, 1::2] << 4), torch.from_numpy(sc), v


def matmul_bound(a, b, half):
    """|error| of a @ b.T in fp32 sums of exact products, rounded once: every
    one of k additions off by at most a step of fp32 of the running sum, plus
    half a step of the result."""
    ref = a @ b.t()
    return ref, a.shape[1] * 2 * F32 * (a.abs() @ b.abs().t()) + half * ref.abs() + 1e-37


# ---- mixture of experts ------------------------------------------------------------


def route(x, router, k, renorm, mask=None):
    """(ids, probs): stable descending order, NaN after every number."""
    l = x.double() @ router.double().t()
    T, E = l.shape
    key = torch.where(torch.isnan(l), -math.inf, l)
    ids = torch.empty(T, k, dtype=torch.int64)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (bool(torch.isnan(l[t, e])), -float(key[t, e]), e))
        ids[t] = torch.tensor(order[:k])
    top = torch.gather(l, 1, ids)
    p = torch.exp(top - top[:, :1])
    p = p / (p.sum(1, keepdim=True) if renorm else torch.exp(l - top[:, :1]).sum(1, keepdim=True))
    if mask is not None:
        ids[~mask] = -1
        p[~mask] = 0
    return ids, p


def moe(x, up, down, ids, p, half):
    """(out, bound) from weights in float64: the products' fp32 sums (each
    addition a step), the activation's few steps, h's and the output's
    rounding to the type."""
    x = x.double()
    T, H = x.shape
    out, err = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    inner = down.shape[2]
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0:
                continue
            gu, mag = up[e] @ x[t], up[e].abs() @ x[t].abs()
            dgu = H * 2 * F32 * mag
            g, u = gu[:inner], gu[inner:]
            s = g / (1 + torch.exp(-g))
            h = s * u
            # |silu'| <= 1.1; exp, division and product: 16 steps
            dh = (1.1 * u.abs() * dgu[:inner] + s.abs() * dgu[inner:] + 1.1 * dgu[:inner] * dgu[inner:]
                  + (half + 16 * F32) * h.abs())
            dh = dh + least(half)
            d, dm = down[e] @ h, down[e].abs() @ h.abs()
            pt = p[t, j]
            out[t] += pt * d
            err[t] += pt * (down[e].abs() @ dh + (inner + ids.shape[1] + 4) * 2 * F32 * (dm + down[e].abs() @ dh))
    return out, err + half * out.abs() + least(half)


# ---- norms --------------------------------------------------------------------------


def _gate(gate, act, T):
    if gate is None:
        return 1.0, 1.0
    g = gate.double().repeat_interleave(T // gate.shape[0], 0)
    if act == "sigmoid":
        s = 1 / (1 + torch.exp(-g))
        return s, s * (1 - s)
    return g, torch.ones_like(g)


def norm_out(block, residual, w_post, gate, scale, eps, act, half):
    """(out before its rounding, bound after it)."""
    b, r = block.double(), residual.double()
    T, H = b.shape
    y = b
    if w_post is not None:
        y = b / torch.sqrt((b * b).mean(1, keepdim=True) + eps) * w_post.double()
    a, _ = _gate(gate, act, T)
    term = y * a * (1.0 if scale is None else scale.double())
    out = r + term
    # the mean of squares: H steps, halved by the root; 8 products; sigmoid's exp 32 steps
    return out, ((H / 2 + 48) * F32) * term.abs() + (half + F32) * out.abs() + least(half)


def norm_next(out, w_next, eps, half):
    o = out.double()
    n = o / torch.sqrt((o * o).mean(1, keepdim=True) + eps) * w_next.double()
    return n, (half + (o.shape[1] / 2 + 16) * F32) * n.abs() + least(half)


def norm_grads(d_out, d_next, block, out, w_post, gate, scale, w_next, eps, act, half):
    """{name: (gradient, bound)}. The bounds follow each fp32 sum of H (or T)
    terms through the formula with one step per addition and 64 for the rest."""
    o = out.double()
    T, H = o.shape
    c = (H + 64) * F32
    d = d_out.double() if d_out is not None else torch.zeros(T, H, dtype=torch.float64)
    mag = d.abs()
    res = {}
    if w_next is not None:
        rr = 1 / torch.sqrt((o * o).mean(1, keepdim=True) + eps)
        xn, dn = o * rr, d_next.double()
        g = dn * w_next.double()
        d = d + rr * (g - xn * (g * xn).mean(1, keepdim=True))
        mag = mag + rr * (g.abs() + xn.abs() * (g * xn).abs().mean(1, keepdim=True))
        t = dn * xn
        ref = t.sum(0)
        res["d_w_next"] = (ref, (c + T * F32) * t.abs().sum(0) + half * ref.abs())
    dd = c * mag
    res["d_residual"] = (d, dd + half * d.abs())
    if block is None:
        return res
    b = block.double()
    rb = 1 / torch.sqrt((b * b).mean(1, keepdim=True) + eps) if w_post is not None else torch.ones(T, 1, dtype=torch.float64)
    xb = b * rb
    wp = w_post.double() if w_post is not None else 1.0
    a, slope = _gate(gate, act, T)
    s = scale.double() if scale is not None else 1.0
    y = xb * wp

    def column(factor, name, groups=None):
        t, e = d * factor, (dd * factor.abs() + c * (mag * factor.abs()))
        n = T
        if groups:
            n = T // groups
            t, e, m = (v.reshape(groups, n, H).sum(1) for v in (t, e, (t.abs())))
        else:
            t, e, m = t.sum(0), e.sum(0), t.abs().sum(0)
        res[name] = (t, e + n * F32 * (m + e) + half * t.abs())

    ones = torch.ones(T, H, dtype=torch.float64)
    if scale is not None:
        column(a * y * ones, "d_scale")
    if gate is not None:
        column(s * y * slope * ones, "d_gate", gate.shape[0])
    if w_post is not None:
        column(s * a * xb * ones, "d_w_post")
    G = d * s * a * wp
    mG = (mag * (s * a * wp * ones).abs())
    dG = dd * (s * a * wp * ones).abs() + 64 * F32 * mG
    if w_post is not None:
        db = rb * (G - xb * (G * xb).mean(1, keepdim=True))
        e = rb * (dG + xb.abs() * (dG * xb.abs()).mean(1, keepdim=True)) + c * rb * (
            mG + xb.abs() * (mG * xb.abs()).mean(1, keepdim=True))
    else:
        db, e = G, dG
    res["d_block"] = (db, e + half * db.abs())
    return res


def check(got, ref, bound, what):
    """|got - ref| <= bound; NaN in the same places; a value past the type's
    range, by more than its bound, is the infinity that it rounds to."""
    top = torch.finfo(got.dtype).max
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    over = ~nan & (ref.abs() - bound > top * (1 + 2.0 ** -7))
    assert torch.equal(got[over], torch.copysign(torch.full_like(ref[over], math.inf), ref[over])), \
        f"{what}: no infinity past the type's range"
    skip = nan | over
    d = torch.where(skip, 0.0, (got - ref).abs())
    bound = torch.where(skip, 1.0, bound)
    worst = (d / bound.clamp_min(1e-300)).max() if d.numel() else torch.tensor(0.0)
    assert bool((d <= bound).all()), \
        f"{what}: error {float(d.max()):.3g}, {float(worst):.3g} times its bound"

"""Plain 64-bit forms of the operators around a model's products, with the
error bounds that the tests use. Written from the definitions in
include/gemm_model.h; no code of the package is used. They run where their
inputs lie."""
from __future__ import annotations

import math

import torch

from block_ref import F32, HALF, least

HW = 2.0 ** -22   # of an exponential or logarithm of the hardware, relative


def logits(x, w, scale):
    """(scale x W^T, a bound on the error of its sums in fp32). A sum of H
    products of 16-bit values, each rounding at most 2^-24 of a partial sum,
    which is at most |x| |w| (2-norms): the roundings are independent, sqrt(H) of
    them have a standard deviation below sqrt(H) 2^-24 |x| |w|; eight of those."""
    l = scale * (x.double() @ w.double().t())
    size = x.double().norm(dim=1, keepdim=True) * w.double().norm(dim=1)
    return l, 8 * math.sqrt(x.shape[1] + 16) * F32 * scale * size


def _lse(l, e):
    """(log sum exp, its error) of logits with errors e: that of the largest
    logit's neighbourhood, of the exponentials' arguments (rounded at up to
    2^-24 of |l|) and of the sum."""
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse.unsqueeze(1))
    err = (p * (e + HW * (2 + l.abs() + lse.abs().unsqueeze(1)))).sum(1) + HW * (1 + lse.abs())
    return lse, err


def cross_entropy(x, w, targets, ignore, scale, z):
    """(loss, error, what the gradient takes)"""
    l, e = logits(x, w, scale)
    lse, e_lse = _lse(l, e)
    use = targets != ignore
    t = torch.where(use, targets, 0).long().unsqueeze(1)
    picked, e_picked = l.gather(1, t)[:, 0], e.gather(1, t)[:, 0]
    loss = lse - picked + z * lse ** 2
    err = e_lse * (1 + 2 * abs(z) * lse.abs()) + e_picked + 4 * F32 * (lse.abs() + picked.abs() + abs(z) * lse ** 2)
    loss, err = (torch.where(use, v, 0.0) for v in (loss, err))
    q = torch.zeros_like(l).scatter_(1, t, 1.0)
    return loss, err, dict(l=l, e=e, lse=lse, e_lse=e_lse, q=q, use=use, mass=torch.ones_like(lse) + 2 * z * lse, by=scale,
                           most=1 + 2 * abs(z) * lse.abs())


def distribution(ids, z, tau, V):
    """The teacher's distribution over the vocabulary, [T, V]."""
    T, k = ids.shape
    z = torch.where(ids >= 0, z.double() / tau, -math.inf)
    top = z.amax(1, keepdim=True)
    e = torch.where(z == -math.inf, 0.0, torch.exp(z - torch.where(top == -math.inf, 0.0, top)))
    total = e.sum(1, keepdim=True)
    e = torch.where(total > 0, e / total, 0.0)
    q = torch.zeros(T, V, dtype=torch.float64, device=ids.device)
    rows = torch.arange(T, device=ids.device)
    for j in range(k):
        q[rows, ids[:, j].clamp(min=0).long()] += e[:, j]
    return q


def distillation(x, w, ids, z, tau, scale=1.0):
    l, e = logits(x, w, scale / tau)
    lse, e_lse = _lse(l, e)
    q = distribution(ids, z, tau, w.shape[0])
    use = q.sum(1) > 0
    logq = torch.where(q > 0, torch.log(torch.where(q > 0, q, 1.0)), 0.0)
    loss = tau ** 2 * (q * (logq - l + lse.unsqueeze(1))).sum(1)
    # q's own error: an exponential and a quotient
    real = torch.where((ids >= 0) & torch.isfinite(z), z.double().abs(), 0.0)
    e_q = HW * (4 + 2 * real.amax(1) / tau)
    terms = q * (logq.abs() + l.abs() + lse.abs().unsqueeze(1))
    err = tau ** 2 * ((terms * (e_q.unsqueeze(1) + 4 * HW)).sum(1) + (q * (e + e_lse.unsqueeze(1))).sum(1)
                      + use * e_q * (1 + ids.shape[1] * F32))
    return loss, err, dict(l=l, e=e, lse=lse, e_lse=e_lse, q=q, use=use, mass=use.double(), by=scale * tau,
                           most=torch.ones_like(lse), e_q=e_q)


def gradients(d_loss, x, w, kept, half):
    """((dx, error), (dw, error)): a gradient of the logits is rounded to the
    type once (fp16: 2^-39 of the largest possible one where it is below the
    normal range), the products sum in fp32, the results are rounded once."""
    l, lse, q, use = (kept[n] for n in ("l", "lse", "q", "use"))
    d = torch.where(use, d_loss.double(), 0.0) * kept["by"]
    use = use & (d != 0)
    rows = use.nonzero()[:, 0]
    l, lse, q, d, mass = l[rows], lse[rows], q[rows], d[rows], kept["mass"][rows]
    p = torch.exp(l - lse.unsqueeze(1))
    g = d.unsqueeze(1) * (mass.unsqueeze(1) * p - q)
    e_l = kept["e"][rows] + kept["e_lse"][rows].unsqueeze(1) + HW * (2 + l.abs() + lse.abs().unsqueeze(1))
    e_q = kept["e_q"][rows].unsqueeze(1) if "e_q" in kept else 0.0
    # beyond the first order, exp(e) - 1 <= 2 e
    e_g = half * g.abs() + d.abs().unsqueeze(1) * (2 * e_l * mass.abs().unsqueeze(1) * p + q * (e_q + 4 * F32)
                                                   + 4 * F32 * mass.abs().unsqueeze(1) * p)
    if half == HALF[torch.float16] and d.numel():
        e_g = e_g + 2.0 ** -38 * (d.abs() * kept["most"][rows]).max()
    xs, ws = x.double()[rows], w.double()

    def product(a, e_a, b):
        r = a @ b
        size = a.abs() @ b.abs()
        err = e_a @ b.abs() + 8 * math.sqrt(a.shape[1] + 16) * F32 * size
        return r, (1 + half) * err + half * r.abs() + least(half)

    dx, e_dx = product(g, e_g, ws)
    full = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    e_full = torch.zeros_like(full)
    full[rows], e_full[rows] = dx, e_dx
    return (full, e_full), product(g.t(), e_g.t(), xs)


# ---- tokens by expert ----------------------------------------------------------


def order(ids, experts):
    """(offsets, row_of) by counting, slot by slot."""
    flat = ids.flatten().tolist()
    lists = [[] for _ in range(experts)]
    for s, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(s)
    offsets, row_of = [0], [-1] * len(flat)
    for group in lists:
        for i, s in enumerate(group):
            row_of[s] = offsets[-1] + i
        offsets.append(offsets[-1] + len(group))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(row_of, dtype=torch.int32).view(ids.shape))


def gather(x, row_of):
    T, k = row_of.shape
    rows = torch.zeros(T * k, x.shape[1], dtype=x.dtype)
    for j in range(k):
        on = row_of[:, j] >= 0
        rows[row_of[on, j].long()] = x[on]
    return rows


def combine(rows, row_of, weights, half):
    T, k = row_of.shape
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for j in range(k):
        on = row_of[:, j] >= 0
        y = rows[row_of[on, j].long()].double()
        c = torch.ones(y.shape[0], 1, dtype=torch.float64) if weights is None else weights[on, j, None].double()
        out[on] += c * y
        size[on] += (c * y).abs()
    return out, (k + 1) * F32 * size + half * out.abs() + least(half)


def combine_backward(d_out, rows, row_of, weights, half):
    T, k = row_of.shape
    H = rows.shape[1]
    d_rows = torch.zeros(rows.shape, dtype=torch.float64)
    d_weights, size = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for j in range(k):
        on = row_of[:, j] >= 0
        p = row_of[on, j].long()
        c = 1.0 if weights is None else weights[on, j, None].double()
        d_rows[p] = c * d_out[on].double()
        terms = d_out[on].double() * rows[p].double()
        d_weights[on, j] = terms.sum(1)
        size[on, j] = terms.abs().sum(1)
    # a lane's sum of up to H / 64 products, rounded for each, then the lanes'
    e_w = (H / 64 + 18) * F32 * size
    return (d_rows, (F32 + half) * d_rows.abs() + least(half)), (d_weights, e_w)

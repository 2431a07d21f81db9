"""Scoring and distillation on the LM head in fp64, from their definitions, on
the inputs' device; and inputs whose logits are exact in fp32."""
import math

import torch

BF, F64 = torch.bfloat16, torch.float64


def grid_inputs(M, d, V, device="cuda", seed=0, sure=6.0, w_step=2.0 ** -8):
    """H [M, d], Wt [V, d] bf16 and the token y [M] that each hidden state
    leans to, on grids of powers of two: products are multiples of 2^-11 and
    their sums stay far below 2^13, so every fp32 sum of them is exact in any
    order.  Equal logits occur."""
    g = torch.Generator().manual_seed(seed)

    def grid(x, step):
        return torch.round(x / step) * step

    W = grid(torch.randn(V, d, generator=g) * 0.05, w_step)
    y = torch.randint(0, V, (M,), generator=g)
    lean = torch.rand(M, 1, generator=g) * (2 * sure / (0.0025 * d))
    H = grid(torch.randn(M, d, generator=g) * 0.5 + lean * W[y], 2.0 ** -3).clamp(-15, 15)
    return H.to(BF).to(device), W.to(BF).to(device), y.to(torch.int32).to(device)


def logits(H, W):
    return H.to(F64) @ W.to(F64).t()


def score(H, W, y=None, T=1.0, k=0):
    """{"logp", "entropy", "ids", "top"} of every row.  The largest logit's own
    exponential, 1, is left out of the sum: log(1 + s) loses an s below 2^-53
    even here, log1p(s) does not."""
    L = logits(H, W)
    x = (L - L.amax(1, keepdim=True)) / T
    s = x.exp().scatter(1, x.argmax(1, keepdim=True), 0.0).sum(1, keepdim=True)
    lq = x - torch.log1p(s)
    out = {"entropy": (torch.log1p(s) - (x.exp() * x).sum(1, keepdim=True) / (1 + s))[:, 0]}
    if y is not None:
        inside = (y >= 0) & (y < W.shape[0])
        got = lq.gather(1, torch.where(inside, y, 0).long()[:, None])[:, 0]
        out["logp"] = torch.where(inside, got, torch.zeros_like(got))
    if k:
        order = torch.sort(L, dim=1, descending=True, stable=True).indices[:, :k]
        out["ids"], out["top"] = order.to(torch.int32), lq.gather(1, order)
    return out


LISTED, NORMALIZED, TAIL = 0, 1, 2


def distill(H, W, ids, val, w, mode, T=1.0):
    """{"loss" [M], "stats" [4], "dL", "dH", "dW"}.  Per row: targets t_v = sum
    of p over the list's entries for v, p = exp(val) or (NORMALIZED) the
    softmax of val / T over the used entries; mass P = sum t; r = max(0, 1 - P)
    for TAIL, else 0; q = softmax(L / T), R = the q mass off the list.
      cross = - sum_v t_v log q_v - r log R
      loss  = cross + sum_v t_v log t_v + r log r
    An entry is used where its token lies in [0, V)."""
    M, V = H.shape[0], W.shape[0]
    lq = torch.log_softmax(logits(H, W) / T, 1)
    used = (ids >= 0) & (ids < V)
    v = torch.where(used, val.to(F64), torch.full_like(val, -math.inf, dtype=F64))
    if mode == NORMALIZED:
        p = torch.softmax(v / T, 1)
        p = torch.where(used.any(1, keepdim=True), p, torch.zeros_like(p))
    else:
        p = v.exp()
    at = torch.where(used, ids, 0).long()
    t = torch.zeros_like(lq).scatter_add_(1, at, torch.where(used, p, torch.zeros_like(p)))
    on = torch.zeros_like(lq).scatter_add_(1, at, used.to(F64)) > 0
    P = t.sum(1)
    r = (1 - P).clamp(min=0) if mode == TAIL else torch.zeros_like(P)
    q = lq.exp()
    lR = torch.logsumexp(lq.masked_fill(on, -math.inf), 1)
    zero = torch.zeros((), dtype=F64, device=H.device)
    cross = -torch.where(t > 0, t * lq, zero).sum(1) - torch.where(r > 0, r * lR, zero)
    loss = cross + torch.special.entr(t).sum(1).neg() + torch.special.entr(r).neg()
    weight = torch.full((M,), 1.0 / M, dtype=F64, device=H.device) if w is None else w.to(F64)
    live = weight != 0
    loss = torch.where(live, loss, zero)
    Q = torch.where(on, q, zero).sum(1)
    stats = torch.stack([(weight * torch.where(live, x, zero)).sum() for x in (loss, cross, P, Q)])
    spread = torch.where(on, zero, (lq - lR[:, None]).exp() * r[:, None])
    spread = torch.where(r[:, None] > 0, spread, zero)
    dL = ((P + r)[:, None] * q - t - spread) * (weight / T)[:, None]
    dL = torch.where(live[:, None], dL, zero)
    return {"loss": loss, "stats": stats, "dL": dL, "dH": dL @ W.to(F64), "dW": dL.t() @ H.to(F64)}

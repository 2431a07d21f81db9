"""Operators of scoring and of distillation on the LM head, as cases that can be
timed and compared: log-probabilities of given tokens with the entropy of their
distribution and the most probable alternatives (one new token to a teacher's
pass over a training batch), and the loss of a student against a teacher's most
probable tokens, with the gradients of the hidden states and of the head.

`run` computes each operator with elementary torch operations where `own` is
false, and through the public entry points of this repository's binding where
it is true.  `exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

BF = torch.bfloat16


def _lib():
    import gemm_epilogue_transformer_tma_gb300 as C
    return C


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # serving: one new token at the 7B width, its log-probability and 20 alternatives
        {"name": "score_token", "op": "score", "M": 1, "d": 4096, "V": 32000, "k": 20, "labels": True,
         "temperature": 1.0},
        # serving: the next tokens of 48 sequences, a 128256-token vocabulary, before any is sampled
        {"name": "score_batch", "op": "score", "M": 48, "d": 4096, "V": 128256, "k": 8, "labels": False,
         "temperature": 0.8},
        # the perplexity of a ragged prompt, with each position's entropy; a vocabulary that ends inside a tile
        {"name": "score_prompt", "op": "score", "M": 1111, "d": 2048, "V": 50280, "k": 0, "labels": True,
         "temperature": 1.0},
        # a teacher's pass over a training batch: 64 alternatives for every token
        {"name": "score_teacher", "op": "score", "M": 4096, "d": 2048, "V": 128256, "k": 64, "labels": True,
         "temperature": 1.0},
        # a student's validation loss on a few sequences (no gradient)
        {"name": "distill_eval", "op": "distill", "M": 333, "d": 1024, "V": 32000, "k": 16, "mode": "tail",
         "temperature": 1.0},
        # a small micro-batch of the update, softened distributions
        {"name": "distill_train_small", "op": "distill_train", "M": 136, "d": 1024, "V": 32000, "k": 32,
         "mode": "tail", "temperature": 2.0},
        # a packed ragged batch against raw teacher logits, normalised over the list
        {"name": "distill_train_ragged", "op": "distill_train", "M": 1777, "d": 2048, "V": 50280, "k": 20,
         "mode": "normalized", "temperature": 1.3},
        # the update at the 1B width and a 128256-token vocabulary
        {"name": "distill_train_1b", "op": "distill_train", "M": 4096, "d": 2048, "V": 128256, "k": 64,
         "mode": "tail", "temperature": 1.0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log_uniform(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["score", "score", "distill", "distill_train"])
    T = rng.choice([0.7, 1.0, 1.0, 1.5, 2.0])
    M, d, V = _log_uniform(rng, 1, 4096), _mult(rng, 256, 4096, 8), _mult(rng, 1000, 128256, 8)
    M = max(1, min(M, 4096 * 2048 * 128256 // (d * V)))
    if op == "score":
        k = rng.choice([0, 1, _log_uniform(rng, 2, 128)])
        return {"op": op, "M": M, "d": d, "V": V, "k": k, "labels": k == 0 or rng.random() < 0.7, "temperature": T}
    return {"op": op, "M": M, "d": d, "V": V, "k": _log_uniform(rng, 1, 128),
            "mode": rng.choice(["listed", "normalized", "tail", "tail"]), "temperature": T}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _grid(x, step):
    return torch.round(x / step) * step


def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)


def _head(gen, M, d, V):
    """Hidden states, the head and the tokens that follow.  Each hidden state
    leans towards its token's row of the head by an amount of its own, so rows
    run from flat to nearly certain.  Both lie on a grid of powers of two (as
    values restored from 8-bit storage do): their products sum without
    rounding in 32 bits, so which of two tokens ranks first does not depend on
    the order of a sum, and equal logits occur."""
    W = _grid(_normal(gen, (V, d), 0.02), 2.0 ** -8)
    y = torch.randint(0, V, (M,), generator=gen, device="cuda", dtype=torch.int64)
    lean = torch.rand((M, 1), generator=gen, device="cuda") * (12.0 / (0.0004 * d))
    H = _grid(_normal(gen, (M, d)) + lean * W[y], 2.0 ** -3).clamp_(-15.0, 15.0)
    return H.to(BF), W.to(BF), y


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, d, V, T = case["M"], case["d"], case["V"], case["temperature"]
    H, W, y = _head(gen, M, d, V)
    s = {"case": case, "H": H, "W": W}
    if case["op"] == "score":
        # what was sampled is the likely token in three rows of four
        other = torch.randint(0, V, (M,), generator=gen, device="cuda", dtype=torch.int64)
        rare = torch.rand(M, generator=gen, device="cuda") < 0.25
        s["y"] = torch.where(rare, other, y).to(torch.int32) if case["labels"] else None
        return s
    # the teacher: the same head on hidden states of its own near the student's, surer of the token or less so
    k, mode = case["k"], case["mode"]
    more = (torch.rand((M, 1), generator=gen, device="cuda") - 0.4) * (6.0 / (0.0004 * d))
    Ht = _grid(H.float() + _normal(gen, (M, d), 0.3) + more * W[y].float(), 2.0 ** -3)
    L = Ht @ W.float().t()
    top, ids = torch.topk(L, k, dim=1)
    if mode == "normalized":
        val = top.clone()
    else:
        val = top / T - torch.logsumexp(L.div_(T), 1, keepdim=True)
        # some rows mix the token that followed in as an entry of its own,
        # beside the teacher's entry for it
        if k >= 4:
            mixed = (torch.rand(M, generator=gen, device="cuda") < 0.25)[:, None]
            val = torch.where(mixed, val + math.log(0.9), val)
            last = torch.arange(k, device="cuda")[None] == k - 1
            ids = torch.where(mixed & last, y[:, None], ids)
            val = torch.where(mixed & last, torch.full_like(val, math.log(0.1)), val)
    del L
    # a quarter of the rows have a shorter list: entries that are not used
    short = (torch.rand(M, generator=gen, device="cuda") < 0.25)[:, None]
    length = torch.randint(1, k + 1, (M, 1), generator=gen, device="cuda")
    unused = short & (torch.arange(k, device="cuda")[None] >= length)
    s["ids"] = torch.where(unused, torch.full_like(ids, -1), ids).to(torch.int32)
    s["val"] = val.contiguous()
    # prompt and padding tokens carry no weight; the rest share a mean
    keep = torch.rand(M, generator=gen, device="cuda") >= 0.125
    s["w"] = keep.float() / keep.sum().clamp(min=1).float()
    return s


def prepare(case, seed):
    """The inputs, and with the framework's operators the output buffers and
    workspaces that a program keeps beside them."""
    s = _inputs(case, seed)
    if not own:
        return s
    C = _lib()
    M, d, V = case["M"], case["d"], case["V"]

    def f32(*shape):
        return torch.empty(*shape, device="cuda")

    if case["op"] == "score":
        k = case["k"]
        s["ws"] = torch.empty(C.coda_lmhead_score_workspace_bytes(M, d, V, k), dtype=torch.uint8, device="cuda")
        s["logp"] = f32(M) if case["labels"] else None
        s["entropy"] = f32(M)
        s["top"] = (torch.empty(M, k, dtype=torch.int32, device="cuda"), f32(M, k)) if k else (None, None)
    else:
        grads = case["op"] == "distill_train"
        s["ws"] = torch.empty(C.coda_lmhead_distill_workspace_bytes(M, d, V, case["k"], grads), dtype=torch.uint8,
                              device="cuda")
        s["stats"], s["row_loss"] = f32(4), f32(M)
        s["dH"] = torch.empty(M, d, dtype=BF, device="cuda") if grads else None
        s["dW"] = torch.empty(V, d, dtype=BF, device="cuda") if grads else None
    return s


# ---------------------------------------------------------------------------
# the framework's own operators
# ---------------------------------------------------------------------------

def _run_own(s):
    C = _lib()
    case = s["case"]
    if case["op"] == "score":
        ids, top = s["top"]
        C.coda_lmhead_score(s["H"], s["W"], s["y"], case["temperature"], s["logp"], s["entropy"], ids, top, s["ws"])
        out = {"entropy": s["entropy"]}
        if case["labels"]:
            out["logp"] = s["logp"]
        if case["k"]:
            out.update(top_ids=ids, top_logp=top)
        return out
    mode = {"listed": C.CODA_DISTILL_LISTED, "normalized": C.CODA_DISTILL_NORMALIZED, "tail": C.CODA_DISTILL_TAIL}
    C.coda_lmhead_distill(s["H"], s["W"], s["ids"], s["val"], s["w"], mode[case["mode"]], case["temperature"],
                          s["stats"], s["row_loss"], s["dH"], s["dW"], s["ws"])
    out = {"stats": s["stats"], "row_loss": s["row_loss"]}
    if case["op"] == "distill_train":
        out.update(dH=s["dH"], dW=s["dW"])
    return out


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_score(s):
    case = s["case"]
    T, k = case["temperature"], case["k"]
    L = s["H"].float() @ s["W"].float().t()
    V = L.shape[1]
    out = {}
    if k:
        # value and token as one whole number each: larger logits first, then lower tokens
        b = L.view(torch.int32)
        key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
        key = (key << 32) | torch.arange(V - 1, -1, -1, device="cuda")
        best = torch.topk(key, k, dim=1).values
        ids = V - 1 - (best & 0xFFFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        del b, key
    # relative to the row's largest logit, so the sum's digits below one stay
    # where a row is nearly certain
    mx = L.amax(1, keepdim=True)
    x = L.sub_(mx).div_(T)
    e = torch.exp(x)
    S = e.sum(1, keepdim=True, dtype=torch.float64)
    log_s = torch.log(S)
    out["entropy"] = (log_s - e.mul_(x).sum(1, keepdim=True, dtype=torch.float64) / S)[:, 0].float()
    if case["labels"]:
        out["logp"] = (x.gather(1, s["y"].long()[:, None]) - log_s)[:, 0].float()
    if k:
        out["top_logp"] = (x.gather(1, ids) - log_s).float()
    return out


def _plain_distill(s, grads):
    case = s["case"]
    T, mode, w = case["temperature"], case["mode"], s["w"]
    H, W = s["H"].float(), s["W"].float()
    x = H @ W.t()
    x = x.sub_(x.amax(1, keepdim=True)).div_(T)
    used = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    # the list, in 64 bits: what the loss of a row near its teacher is a small difference of
    val = torch.where(used, s["val"], torch.full_like(s["val"], -math.inf)).double()
    if mode == "normalized":
        p = torch.exp((val - val.amax(1, keepdim=True)) / T)
        p = p / p.sum(1, keepdim=True)
    else:
        p = torch.exp(val)
    P = p.sum(1)
    r = (1 - P).clamp(min=0) if mode == "tail" else torch.zeros_like(P)
    # entries for one token add up
    same = (ids[:, :, None] == ids[:, None, :]) & used[:, :, None] & used[:, None, :]
    merged = (same * p[:, None, :]).sum(2)
    first = used / same.sum(2).clamp(min=1)
    on = torch.zeros_like(x).scatter_add_(1, ids, used.float()) > 0
    x_list = x.gather(1, ids).double()
    e = torch.exp(x)
    rest = torch.where(on, torch.zeros_like(e), e).sum(1, dtype=torch.float64)
    S = rest + (torch.exp(x_list) * first).sum(1)
    lq = x_list - torch.log(S)[:, None]
    has = p > 0
    ent = torch.where(has, p * torch.log(torch.where(has, merged, torch.ones_like(p))), torch.zeros_like(p)).sum(1)
    ce = -torch.where(has, p * lq, torch.zeros_like(p)).sum(1)
    some = (r > 0) & (rest > 0)
    ent = ent + torch.where(r > 0, r * torch.log(r), torch.zeros_like(r))
    ce = ce - torch.where(some, r * torch.log(rest / S), torch.zeros_like(r))
    listed_q = 1 - rest / S
    zero = torch.zeros_like(ce)
    loss = torch.where(w != 0, ent + ce, zero)
    stats = torch.stack([(w * loss).sum(), (w * torch.where(w != 0, ce, zero)).sum(), (w * P).sum(),
                         (w * listed_q).sum()])
    out = {"stats": stats.float(), "row_loss": loss.float()}
    if grads:
        # d loss / d logits = w ((P + r) q - t - r q / (q off the list) off the list) / T
        f = ((P + r) / S).float()[:, None]
        f_rest = (f[:, 0] - torch.where(some, r / rest, torch.zeros_like(r)).float())[:, None]
        g = e * torch.where(on, f, f_rest)
        g.scatter_add_(1, ids, -p.float())
        g *= (w / T)[:, None]
        out.update(dH=(g @ W).to(BF), dW=(g.t() @ H).to(BF))
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _plain_score(state) if op == "score" else _plain_distill(state, op == "distill_train")


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    M, d, V, k = case["M"], case["d"], case["V"], case["k"]
    n = 2 * (M * d + V * d)
    if case["op"] == "score":
        return {"bytes": n + M * (4 + (8 if case["labels"] else 0) + 8 * k), "flops": 2 * M * d * V}
    if case["op"] == "distill":
        return {"bytes": n + M * (8 + 8 * k), "flops": 2 * M * d * V}
    return {"bytes": 2 * n + M * (8 + 8 * k), "flops": 6 * M * d * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    M, T, k = case["M"], case["temperature"], case["k"]
    H, W = s["H"].double(), s["W"].double()
    dev = H.device
    if case["op"] == "score":
        lp = torch.empty(M, dtype=torch.float64, device=dev)
        ent = torch.empty(M, dtype=torch.float64, device=dev)
        ids = torch.empty(M, k, dtype=torch.int32, device=dev)
        top = torch.empty(M, k, dtype=torch.float64, device=dev)
        for r in range(0, M, 256):
            sl = slice(r, min(M, r + 256))
            raw = H[sl] @ W.t()
            logq = torch.log_softmax(raw / T, 1)
            ent[sl] = -(logq.exp() * logq).sum(1)
            if case["labels"]:
                lp[sl] = logq.gather(1, s["y"][sl, None].long())[:, 0]
            if k:
                order = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :k]
                ids[sl] = order.to(torch.int32)
                top[sl] = logq.gather(1, order)
        out = {"entropy": ent}
        if case["labels"]:
            out["logp"] = lp
        if k:
            out.update(top_ids=ids, top_logp=top)
        return out
    grads = case["op"] == "distill_train"
    dH = torch.empty_like(H) if grads else None
    dW = torch.zeros_like(W) if grads else None
    loss = torch.zeros(M, dtype=torch.float64, device=dev)
    tot = torch.zeros(4, dtype=torch.float64, device=dev)
    for r in range(0, M, 512):
        sl = slice(r, min(M, r + 512))
        w = s["w"][sl].double()
        i, v = s["ids"][sl].long(), s["val"][sl].double()
        v = v.masked_fill(i < 0, -math.inf)
        logq = torch.log_softmax(H[sl] @ W.t() / T, 1)
        p = torch.softmax(v / T, 1) if case["mode"] == "normalized" else v.exp()
        i = i.clamp(min=0)
        target = torch.zeros_like(logq).scatter_add_(1, i, p)
        member = torch.zeros_like(logq).scatter_add_(1, i, (s["ids"][sl] >= 0).double()) > 0
        mass = p.sum(1)
        log_rest = torch.logsumexp(logq.masked_fill(member, -math.inf), 1)
        extra = (1 - mass).clamp(min=0) if case["mode"] == "tail" else torch.zeros_like(mass)
        cross = -(target * logq).sum(1) - torch.where(extra > 0, extra * log_rest, torch.zeros_like(extra))
        own_ent = torch.special.entr(target).sum(1) + torch.special.entr(extra)
        q = logq.exp()
        loss[sl] = torch.where(w != 0, cross - own_ent, torch.zeros_like(cross))
        tot += torch.stack([(w * (cross - own_ent)).sum(), (w * cross).sum(), (w * mass).sum(),
                            (w * (q * member).sum(1)).sum()])
        if grads:
            # the target spreads the rest's mass over the rest as the student does
            spread = torch.exp(logq - log_rest[:, None]) * extra[:, None]
            dl = (mass + extra)[:, None] * q - target - spread.masked_fill(member, 0.0)
            dl *= (w / T)[:, None]
            dH[sl] = dl @ W
            dW.addmm_(dl.t(), H[sl])
    out = {"stats": tot, "row_loss": loss}
    if grads:
        out.update(dH=dH, dW=dW)
    return out

"""The operators of a fine-grained FP8 post-training step and of serving it, as
cases that can be timed and compared: storage of a tensor as 8-bit codes with a
scale for each block of 128 values, linear layers on such codes (one token to
a training batch, forward and backward), the norm of the query and key heads
with the rotary embedding (forward, backward), and the clipped policy loss on
the LM head with its KL term and gradients.

`run` computes each operator with elementary torch operations where `own` is
false, and through the public entry points of this repository's binding where
it is true.  `exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

BF = torch.bfloat16
BLOCK = 128
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}


def _lib():
    import gemm_epilogue_transformer_tma_gb300 as C
    return C


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a layer's input kept for the backward in 8 bits: the token count and
        # width of the 7B block, both block directions
        {"name": "store8_7b", "op": "store8", "rows": 8192, "cols": 4096, "fmt": "e4m3"},
        # a ragged micro-batch's gradient: odd token count, width not a multiple of 128
        {"name": "store8_ragged", "op": "store8", "rows": 333, "cols": 2064, "fmt": "e5m2"},
        # serving: one new token through the QKV projection of the 7B width
        # (32 query and 8 key/value heads of 128)
        {"name": "linear8_token", "op": "linear8", "M": 1, "K": 4096, "N": 6144},
        # serving: a small batch of tokens through the down projection of the 7B block
        {"name": "linear8_batch", "op": "linear8", "M": 48, "K": 14336, "N": 4096},
        # serving: a ragged chunk of a prompt
        {"name": "linear8_chunk", "op": "linear8", "M": 1111, "K": 4096, "N": 6144},
        # training, forward and backward: the 1B output projection
        {"name": "linear8_train_1b", "op": "linear8_train", "M": 8192, "K": 2048, "N": 2048},
        # training, forward and backward: the 7B gate/up projection, the largest product
        {"name": "linear8_train_7b", "op": "linear8_train", "M": 8192, "K": 4096, "N": 28672},
        # serving: the new tokens of 64 sequences, each at its own far position
        {"name": "qknorm_rope_tokens", "op": "qknorm_rope", "M": 64, "n_q": 32, "n_kv": 8, "hd": 128, "S": 32768,
         "scattered": True},
        # training, forward and backward, 4 sequences of 2048 at the 7B width
        {"name": "qknorm_rope_train_7b", "op": "qknorm_rope_train", "M": 8192, "n_q": 32, "n_kv": 8, "hd": 128,
         "S": 2048, "scattered": False},
        # training on a packed ragged batch with narrow heads (80 is no power of two)
        {"name": "qknorm_rope_train_ragged", "op": "qknorm_rope_train", "M": 1777, "n_q": 6, "n_kv": 3, "hd": 80,
         "S": 1000, "scattered": True},
        # scoring a small batch of sampled tokens (no gradient): loss and log-probabilities
        {"name": "policy_score", "op": "policy", "M": 136, "d": 1024, "V": 32000, "temperature": 0.8},
        # the policy update at the 1B width and a 128256-token vocabulary, with gradients
        {"name": "policy_train_1b", "op": "policy_train", "M": 4096, "d": 2048, "V": 128256, "temperature": 1.0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log_uniform(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["store8", "linear8", "linear8_train", "qknorm_rope", "qknorm_rope_train", "policy",
                     "policy_train"])
    if op == "store8":
        return {"op": op, "rows": _log_uniform(rng, 1, 8192), "cols": _mult(rng, 64, 8192, 16),
                "fmt": rng.choice(["e4m3", "e5m2"])}
    if op == "linear8":
        return {"op": op, "M": _log_uniform(rng, 1, 4096), "K": _mult(rng, 512, 14336, 16),
                "N": _mult(rng, 512, 14336, 16)}
    if op == "linear8_train":
        return {"op": op, "M": _log_uniform(rng, 100, 8192), "K": _mult(rng, 256, 4096, 16),
                "N": _mult(rng, 256, 16384, 16)}
    if op in ("qknorm_rope", "qknorm_rope_train"):
        n_kv = rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "M": _log_uniform(rng, 1, 8192), "n_q": n_kv * rng.choice([1, 2, 4]), "n_kv": n_kv,
                "hd": rng.choice([64, 80, 96, 128, 192, 256]), "S": _log_uniform(rng, 256, 32768),
                "scattered": rng.random() < 0.5}
    return {"op": op, "M": _log_uniform(rng, 100, 4096), "d": _mult(rng, 256, 2048, 8),
            "V": _mult(rng, 1000, 64000, 8), "temperature": rng.choice([0.7, 1.0, 1.3])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)


def _activations(gen, rows, cols):
    """Activations of a trained layer: unit scale with one channel in 64
    twenty times larger, the reason for scales finer than one per tensor."""
    x = _normal(gen, (rows, cols))
    x[:, (torch.arange(cols, device="cuda") % 64) == 7] *= 20.0
    return x.to(BF)


def _gradient(gen, rows, cols):
    """Upstream gradients: small, with token norms spread over a few binades."""
    x = _normal(gen, (rows, cols), 1e-3)
    x *= torch.exp(_normal(gen, (rows, 1)))
    return x.to(BF)


def _rope_tables(S, hd, base=10000.0):
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    ang = torch.arange(S, device="cuda", dtype=torch.float64)[:, None] * base ** (-2.0 * i / hd)
    return torch.cos(ang).to(torch.float32), torch.sin(ang).to(torch.float32)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "store8":
        r, c = case["rows"], case["cols"]
        s["x"] = _activations(gen, r, c) if case["fmt"] == "e4m3" else _gradient(gen, r, c)
    elif op in ("linear8", "linear8_train"):
        M, K, N = case["M"], case["K"], case["N"]
        s["X"] = _activations(gen, M, K)
        s["W"] = _normal(gen, (N, K), 0.02).to(BF)
        if op == "linear8_train":
            s["dY"] = _gradient(gen, M, N)
    elif op in ("qknorm_rope", "qknorm_rope_train"):
        M, hd, S = case["M"], case["hd"], case["S"]
        width = (case["n_q"] + 2 * case["n_kv"]) * hd
        s["qkv"] = _normal(gen, (M, width), 1.5).to(BF)
        s["gq"] = (torch.rand(hd, generator=gen, device="cuda") + 0.5).to(BF)
        s["gk"] = (torch.rand(hd, generator=gen, device="cuda") + 0.5).to(BF)
        s["cos"], s["sin"] = _rope_tables(S, hd)
        s["pos"] = None
        if case["scattered"]:
            s["pos"] = torch.randint(0, S, (M,), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
        if op == "qknorm_rope_train":
            s["dout"] = _gradient(gen, M, width)
    else:
        M, d, V = case["M"], case["d"], case["V"]
        s["H"] = _normal(gen, (M, d)).to(BF)
        s["W"] = _normal(gen, (V, d), 0.02).to(BF)
        s["y"] = torch.randint(0, V, (M,), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
        # group-normalised advantages; one token in eight is a prompt or
        # padding token and carries no weight; the rest share a mean
        s["adv"] = _normal(gen, (M,))
        keep = torch.rand(M, generator=gen, device="cuda") >= 0.125
        s["w"] = keep.float() / keep.sum().clamp(min=1).float()
        # the sampling policy and the reference lie near the current one
        lp = torch.empty(M, device="cuda")
        for r in range(0, M, 512):
            lg = (s["H"][r:r + 512] @ s["W"].t()).float() / case["temperature"]
            lp[r:r + 512] = lg.gather(1, s["y"][r:r + 512, None].long())[:, 0] - torch.logsumexp(lg, 1)
        s["old"] = lp + _normal(gen, (M,), 0.2)
        s["ref"] = lp + _normal(gen, (M,), 0.4)
    return s


def prepare(case, seed):
    """The inputs, and what a program keeps beside them: a served layer's
    weight codes, and with the framework's operators the output buffers and
    workspaces."""
    s = _inputs(case, seed)
    op = case["op"]
    if not own:
        if op == "linear8":
            s["W"] = _tile_codes(s["W"].float(), "e4m3")
        return s
    C = _lib()

    def u8(*shape):
        return torch.empty(*shape, dtype=torch.uint8, device="cuda")

    def bf(*shape):
        return torch.empty(*shape, dtype=BF, device="cuda")

    if op == "store8":
        r, c = case["rows"], case["cols"]
        s["q"] = [u8(r, c), u8(r, c)]
        s["s"] = [u8(C.coda_fp8_block_scale_bytes(r, c)), u8(C.coda_fp8_block_scale_bytes(c, r))]
        s["out"] = [bf(r, c), bf(r, c)]
    elif op in ("linear8", "linear8_train"):
        M, K, N = case["M"], case["K"], case["N"]
        b = C.coda_fp8_block_scale_bytes
        t = s["lin"] = {"Xq": u8(M, K), "sX": u8(b(M, K)), "Wq": u8(N, K), "sW": u8(b(N, K)), "sWt": u8(b(K, N)),
                        "Y": bf(M, N)}
        if op == "linear8":
            C.coda_fp8_block_quantize_weight(s.pop("W"), t["Wq"], t["sW"], t["sWt"], C.E4M3)
        else:
            t.update(Xc=u8(M, K), sXc=u8(b(K, M)), Gq=u8(M, N), sG=u8(b(M, N)), Gc=u8(M, N), sGc=u8(b(N, M)),
                     dX=bf(M, K), dW=bf(N, K))
    elif op in ("qknorm_rope", "qknorm_rope_train"):
        M, hd = case["M"], case["hd"]
        s["out"] = torch.empty_like(s["qkv"])
        if op == "qknorm_rope_train":
            s["dqkv"] = torch.empty_like(s["qkv"])
            s["dgq"], s["dgk"] = torch.empty(hd, device="cuda"), torch.empty(hd, device="cuda")
            s["ws"] = u8(C.coda_qknorm_rope_bwd_workspace_bytes(M, hd))
    else:
        M, d, V = case["M"], case["d"], case["V"]
        grads = op == "policy_train"
        s["ws"] = u8(C.coda_lmhead_policy_workspace_bytes(M, d, V, grads))
        s["stats"], s["logp"] = torch.empty(4, device="cuda"), torch.empty(M, device="cuda")
        s["dH"], s["dW"] = (bf(M, d), bf(V, d)) if grads else (None, None)
    return s


# ---------------------------------------------------------------------------
# the framework's own operators
# ---------------------------------------------------------------------------

def _run_own(s):
    C = _lib()
    case = s["case"]
    op = case["op"]
    if op == "store8":
        fmt = C.E4M3 if case["fmt"] == "e4m3" else C.E5M2
        (q0, q1), (s0, s1), (o0, o1) = s["q"], s["s"], s["out"]
        C.coda_fp8_block_quantize(s["x"], q0, s0, q1, s1, fmt)
        C.coda_fp8_block_dequantize(q0, s0, False, o0, fmt)
        C.coda_fp8_block_dequantize(q1, s1, True, o1, fmt)
        return {"row": o0, "col": o1}
    if op == "linear8":
        M, K, N, t = case["M"], case["K"], case["N"], s["lin"]
        C.coda_fp8_block_quantize(s["X"], t["Xq"], t["sX"], None, None, C.E4M3)
        C.coda_gemm_fp8_block(t["Xq"], False, C.E4M3, t["sX"], t["Wq"], False, C.E4M3, t["sW"], t["Y"], M, N, K)
        return {"Y": t["Y"]}
    if op == "linear8_train":
        M, K, N, t = case["M"], case["K"], case["N"], s["lin"]
        C.coda_fp8_block_quantize_weight(s["W"], t["Wq"], t["sW"], t["sWt"], C.E4M3)
        C.coda_fp8_block_quantize(s["X"], t["Xq"], t["sX"], t["Xc"], t["sXc"], C.E4M3)
        C.coda_gemm_fp8_block(t["Xq"], False, C.E4M3, t["sX"], t["Wq"], False, C.E4M3, t["sW"], t["Y"], M, N, K)
        C.coda_fp8_block_quantize(s["dY"], t["Gq"], t["sG"], t["Gc"], t["sGc"], C.E5M2)
        C.coda_gemm_fp8_block(t["Gq"], False, C.E5M2, t["sG"], t["Wq"], True, C.E4M3, t["sWt"], t["dX"], M, K, N)
        C.coda_gemm_fp8_block(t["Gc"], True, C.E5M2, t["sGc"], t["Xc"], True, C.E4M3, t["sXc"], t["dW"], N, K, M)
        return {"Y": t["Y"], "dX": t["dX"], "dW": t["dW"]}
    if op in ("qknorm_rope", "qknorm_rope_train"):
        nq, nkv, hd = case["n_q"], case["n_kv"], case["hd"]
        C.coda_qknorm_rope(s["qkv"], s["gq"], s["gk"], s["cos"], s["sin"], s["out"], nq, nkv, hd, 1e-6, s["pos"])
        if op == "qknorm_rope":
            return {"out": s["out"]}
        C.coda_qknorm_rope_bwd(s["dout"], s["qkv"], s["gq"], s["gk"], s["cos"], s["sin"], s["dqkv"], s["dgq"],
                               s["dgk"], s["ws"], nq, nkv, hd, 1e-6, s["pos"])
        return {"out": s["out"], "dqkv": s["dqkv"], "dgq": s["dgq"], "dgk": s["dgk"]}
    C.coda_lmhead_policy(s["H"], s["W"], s["y"], s["adv"], s["w"], s["old"], s["ref"], 0.2, 0.28, 0.05,
                         case["temperature"], s["stats"], s["logp"], s["dH"], s["dW"], s["ws"])
    out = {"stats": s["stats"], "logp": s["logp"]}
    if op == "policy_train":
        out.update(dH=s["dH"], dW=s["dW"])
    return out


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _scale_of(amax, fmt):
    """The smallest power of two 2^k, k >= -126, with amax / 2^k <= the
    format's largest value; 1 for amax = 0.  Both largest values are
    0.875 * 2^e."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - (9 if fmt == "e4m3" else 16), e - (8 if fmt == "e4m3" else 15))
    k = torch.where(amax > 0, k.clamp(min=-126), torch.zeros_like(k))
    return ((k + 127) << 23).view(torch.float32)


def _blocks(x, rb, cb):
    """x [R][C] zero-padded to whole rb x cb blocks, as [R/rb][rb][C/cb][cb]."""
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, -C % cb, 0, -R % rb))
    return x.view(x.shape[0] // rb, rb, x.shape[1] // cb, cb)


def _quantized(x, fmt, rb, cb):
    """x rounded to codes times block scales, as fp32 values."""
    R, C = x.shape
    b = _blocks(x, rb, cb)
    s = _scale_of(b.abs().amax(dim=(1, 3), keepdim=True), fmt)
    v = (b / s).to(F8[fmt]).float() * s
    return v.reshape(v.shape[0] * rb, -1)[:R, :C]


def _tile_codes(W, fmt):
    """Weight codes [N][K] with one scale for each 128 x 128 tile."""
    N, K = W.shape
    b = _blocks(W, BLOCK, BLOCK)
    s = _scale_of(b.abs().amax(dim=(1, 3), keepdim=True), fmt)
    q = (b / s).to(F8[fmt])
    return q.reshape(q.shape[0] * BLOCK, -1)[:N, :K].contiguous(), s[:, 0, :, 0]


def _tile_values(q, s):
    N, K = q.shape
    return q.float() * s.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _heads(s):
    c = s["case"]
    nq, nk, hd = c["n_q"], c["n_kv"], c["hd"]
    return nq, nk, hd, (nq + nk) * hd


def _plain_rows(s):
    """cos and sin of every token, [M][1][hd / 2]."""
    M, S = s["qkv"].shape[0], s["cos"].shape[0]
    pos = s["pos"].long() if s["pos"] is not None else torch.arange(M, device="cuda") % S
    return s["cos"][pos][:, None], s["sin"][pos][:, None]


def _plain_norm(s):
    """(x, rstd, g) of the q and k heads, fp32 [M][heads][hd]."""
    nq, nk, hd, rot = _heads(s)
    x = s["qkv"][:, :rot].float().reshape(-1, nq + nk, hd)
    g = torch.cat([s["gq"].float().expand(nq, hd), s["gk"].float().expand(nk, hd)])
    rstd = 1.0 / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6)
    return x, rstd, g


def _plain_qknorm_rope(s):
    nq, nk, hd, rot = _heads(s)
    x, rstd, g = _plain_norm(s)
    n = x * rstd * g
    c, sn = _plain_rows(s)
    a, b = n[..., :hd // 2], n[..., hd // 2:]
    y = torch.cat([a * c - b * sn, b * c + a * sn], 2).reshape(-1, rot)
    return torch.cat([y, s["qkv"][:, rot:].float()], 1).to(BF)


def _plain_qknorm_rope_bwd(s):
    nq, nk, hd, rot = _heads(s)
    x, rstd, g = _plain_norm(s)
    dy = s["dout"][:, :rot].float().reshape(-1, nq + nk, hd)
    c, sn = _plain_rows(s)
    a, b = dy[..., :hd // 2], dy[..., hd // 2:]
    dn = torch.cat([a * c + b * sn, b * c - a * sn], 2)
    xh = x * rstd
    prod = dn * xh
    dgq, dgk = prod[:, :nq].sum((0, 1)), prod[:, nq:].sum((0, 1))
    dh = dn * g
    dx = rstd * (dh - xh * (dh * xh).mean(2, keepdim=True))
    dqkv = torch.cat([dx.reshape(-1, rot), s["dout"][:, rot:].float()], 1).to(BF)
    return dqkv, dgq, dgk


def _plain_policy(s, grads):
    T = s["case"]["temperature"]
    y = s["y"].long()[:, None]
    H, W = s["H"].float(), s["W"].float()
    L = H @ W.t() / T
    mx = L.amax(1, keepdim=True)
    lse = mx + torch.log(torch.exp(L - mx).sum(1, keepdim=True))
    lp = (L.gather(1, y) - lse)[:, 0]
    w, A = s["w"], s["adv"]
    r = torch.exp(lp - s["old"])
    cl = r.clamp(1 - 0.2, 1 + 0.28)
    free = r * A <= cl * A
    surr = torch.where(free, r * A, cl * A)
    x = (s["ref"] - lp).double()
    kl = (torch.exp(x) - x - 1).float()
    stats = torch.stack([(w * (0.05 * kl - surr)).sum(), (w * -surr).sum(), (w * kl).sum(),
                         (w * (~free).float()).sum()])
    out = {"stats": stats, "logp": lp}
    if grads:
        g = w * (0.05 * (1 - torch.exp(s["ref"] - lp)) - torch.where(free, A * r, torch.zeros_like(r)))
        # d loss / d logits = g (onehot - softmax) / T
        L.sub_(lse).exp_().mul_(-1.0)
        L.scatter_add_(1, y, torch.ones_like(y, dtype=torch.float32))
        L.mul_((g / T)[:, None])
        out.update(dH=(L @ W).to(BF), dW=(L.t() @ H).to(BF))
    return out


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "store8":
        x = s["x"].float()
        return {"row": _quantized(x, case["fmt"], 1, BLOCK).to(BF), "col": _quantized(x, case["fmt"], BLOCK, 1).to(BF)}
    if op == "linear8":
        return {"Y": (_quantized(s["X"].float(), "e4m3", 1, BLOCK) @ _tile_values(*s["W"]).t()).to(BF)}
    if op == "linear8_train":
        X, G = s["X"].float(), s["dY"].float()
        W = _quantized(s["W"].float(), "e4m3", BLOCK, BLOCK)
        Y = _quantized(X, "e4m3", 1, BLOCK) @ W.t()
        dX = _quantized(G, "e5m2", 1, BLOCK) @ W
        dW = _quantized(G, "e5m2", BLOCK, 1).t() @ _quantized(X, "e4m3", BLOCK, 1)
        return {"Y": Y.to(BF), "dX": dX.to(BF), "dW": dW.to(BF)}
    if op == "qknorm_rope":
        return {"out": _plain_qknorm_rope(s)}
    if op == "qknorm_rope_train":
        out = _plain_qknorm_rope(s)
        dqkv, dgq, dgk = _plain_qknorm_rope_bwd(s)
        return {"out": out, "dqkv": dqkv, "dgq": dgq, "dgk": dgk}
    return _plain_policy(s, op == "policy_train")


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "store8":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n + 2 * 2 * n, "flops": 6 * n}
    if op == "linear8":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + N * K + 2 * M * N, "flops": 2 * M * N * K}
    if op == "linear8_train":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * (2 * M * K + 2 * N * K + 2 * M * N), "flops": 6 * M * N * K}
    if op in ("qknorm_rope", "qknorm_rope_train"):
        n = case["M"] * (case["n_q"] + 2 * case["n_kv"]) * case["hd"]
        rot = case["M"] * (case["n_q"] + case["n_kv"]) * case["hd"]
        tab = min(case["M"], case["S"]) * case["hd"] * 4
        if op == "qknorm_rope":
            return {"bytes": 4 * n + tab, "flops": 8 * rot}
        return {"bytes": 8 * n + tab, "flops": 26 * rot}
    M, d, V = case["M"], case["d"], case["V"]
    n = 2 * (M * d + V * d)
    if op == "policy":
        return {"bytes": n + 24 * M, "flops": 2 * M * d * V}
    return {"bytes": 2 * n + 24 * M, "flops": 6 * M * d * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _pow2(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_round(v, fmt):
    """Round to nearest, ties to even, onto the 8-bit format's grid: spacing
    2^(e - m) in the binade [2^e, 2^(e+1)), no finer than at the least
    normal exponent."""
    mant, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    step = _pow2((torch.frexp(v)[1] - 1).clamp(min=emin) - mant)
    return torch.round(v / step) * step


def _exact_quantized(x, fmt, rb, cb):
    x = x.double()
    R, C = x.shape
    p = torch.zeros(-(-R // rb) * rb, -(-C // cb) * cb, dtype=torch.float64, device=x.device)
    p[:R, :C] = x
    t = p.view(p.shape[0] // rb, rb, p.shape[1] // cb, cb)
    amax = t.abs().amax((1, 3), keepdim=True)
    k = torch.ceil(torch.log2((amax / F8_MAX[fmt]).clamp(min=2.0 ** -126)))
    # the least k with amax <= max * 2^k, whatever log2 rounded to
    k = torch.where(amax > F8_MAX[fmt] * _pow2(k), k + 1, k)
    k = torch.where((amax <= F8_MAX[fmt] * _pow2(k - 1)) & (k > -126), k - 1, k)
    k = torch.where(amax > 0, k, torch.zeros_like(k))
    t.copy_(_exact_round(t / _pow2(k), fmt) * _pow2(k))
    return p[:R, :C]


def _exact_qknorm(s, grads):
    c = s["case"]
    nq, nk, hd = c["n_q"], c["n_kv"], c["hd"]
    h, M = hd // 2, c["M"]
    pos = s["pos"].long() if s["pos"] is not None else torch.arange(M, device="cuda") % c["S"]
    rot = torch.complex(s["cos"].double()[pos], s["sin"].double()[pos])[:, None, :]
    out = s["qkv"].double()
    dq = s["dout"].double() if grads else None
    dg = []
    for lo, n, g in ((0, nq, s["gq"].double()), (nq, nk, s["gk"].double())):
        sl = slice(lo * hd, (lo + n) * hd)
        x = s["qkv"].double()[:, sl].reshape(M, n, hd)
        inv = (x.pow(2).sum(2, keepdim=True) / hd + 1e-6).rsqrt()
        z = x * inv
        y = torch.complex(*(z * g).split(h, 2)) * rot
        out[:, sl] = torch.cat([y.real, y.imag], 2).reshape(M, -1)
        if grads:
            u = torch.complex(*s["dout"].double()[:, sl].reshape(M, n, hd).split(h, 2)) * rot.conj()
            u = torch.cat([u.real, u.imag], 2)
            dg.append(torch.einsum("mnh,mnh->h", u, z))
            u = u * g
            dq[:, sl] = (inv * (u - z * (u * z).sum(2, keepdim=True) / hd)).reshape(M, -1)
    if not grads:
        return {"out": out}
    return {"out": out, "dqkv": dq, "dgq": dg[0], "dgk": dg[1]}


def _exact_policy(s, grads):
    c = s["case"]
    M, T = c["M"], c["temperature"]
    H, W = s["H"].double(), s["W"].double()
    lp = torch.empty(M, dtype=torch.float64, device="cuda")
    dH = torch.empty_like(H) if grads else None
    dW = torch.zeros_like(W) if grads else None
    tot = torch.zeros(4, dtype=torch.float64, device="cuda")
    for r in range(0, M, 1024):
        sl = slice(r, min(M, r + 1024))
        y = s["y"][sl].long()
        idx = torch.arange(y.numel(), device="cuda")
        logp = torch.log_softmax(H[sl] @ W.t() / T, 1)
        p = logp[idx, y]
        lp[sl] = p
        A, w = s["adv"][sl].double(), s["w"][sl].double()
        ratio = torch.exp(p - s["old"][sl].double())
        held = torch.minimum(torch.maximum(ratio, torch.full_like(p, 0.8)), torch.full_like(p, 1.28))
        active = ratio * A <= held * A
        gain = torch.minimum(ratio * A, held * A)
        q = s["ref"][sl].double() - p
        kl = torch.expm1(q) - q
        tot += torch.stack([(w * (0.05 * kl - gain)).sum(), -(w * gain).sum(), (w * kl).sum(),
                            (w * ~active).sum()])
        if grads:
            g = -w * torch.where(active, ratio * A, torch.zeros_like(p)) - 0.05 * w * torch.expm1(q)
            dl = logp.exp_()
            dl[idx, y] -= 1
            dl *= (-g / T)[:, None]
            dH[sl] = dl @ W
            dW.addmm_(dl.t(), H[sl])
    out = {"stats": tot, "logp": lp}
    if grads:
        out.update(dH=dH, dW=dW)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "store8":
        return {"row": _exact_quantized(s["x"], case["fmt"], 1, BLOCK),
                "col": _exact_quantized(s["x"], case["fmt"], BLOCK, 1)}
    if op == "linear8":
        return {"Y": _exact_quantized(s["X"], "e4m3", 1, BLOCK) @ _exact_quantized(s["W"], "e4m3", BLOCK, BLOCK).t()}
    if op == "linear8_train":
        Wq = _exact_quantized(s["W"], "e4m3", BLOCK, BLOCK)
        return {"Y": _exact_quantized(s["X"], "e4m3", 1, BLOCK) @ Wq.t(),
                "dX": _exact_quantized(s["dY"], "e5m2", 1, BLOCK) @ Wq,
                "dW": _exact_quantized(s["dY"], "e5m2", BLOCK, 1).t() @ _exact_quantized(s["X"], "e4m3", BLOCK, 1)}
    if op in ("qknorm_rope", "qknorm_rope_train"):
        return _exact_qknorm(s, op.endswith("train"))
    return _exact_policy(s, op.endswith("train"))

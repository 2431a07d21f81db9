"""Plain fp64 definitions of the post-training step's operators: block scales
of 8-bit codes, the norm of the query and key heads with the rotary embedding,
and the clipped policy loss on the LM head, each with its gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring): nothing in the product
imports this file.
"""
from __future__ import annotations

import numpy as np

from .coda_oracle import fp8_decode, fp8_quantize, fp8_scale, lse_rows, rope_angles

BLOCK = 128
NAN_BYTE = 255


def _scale_byte(block, fmt):
    """k + 127 of the block's scale 2^k, or NAN_BYTE."""
    if not np.all(np.isfinite(block)):
        return NAN_BYTE
    return int(np.log2(float(fp8_scale(block, fmt)))) + 127


def block_quantize(x, rb, cb, fmt="e4m3"):
    """(codes [R][C], scale bytes [ceil(R/rb)][ceil(C/cb)]) of x with one
    power-of-two scale for each rb x cb block; NaN codes 0x7f and the byte 255
    for a block that holds an infinity or a NaN."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    q = np.zeros((R, C), np.uint8)
    s = np.zeros((-(-R // rb), -(-C // cb)), np.uint8)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            sl = np.s_[i * rb:(i + 1) * rb, j * cb:(j + 1) * cb]
            b = _scale_byte(x[sl], fmt)
            s[i, j] = b
            q[sl] = 0x7F if b == NAN_BYTE else fp8_quantize(x[sl], 2.0 ** (b - 127), fmt)
    return q, s


def block_dequantize(q, s, rb, cb, fmt="e4m3"):
    """code * 2^(byte - 127) per element; NaN in poisoned blocks."""
    e = np.repeat(np.repeat(s.astype(np.float64), rb, 0), cb, 1)[:q.shape[0], :q.shape[1]]
    v = fp8_decode(q, fmt) * np.exp2(e - 127.0)
    return np.where(e == NAN_BYTE, np.nan, v)


def packed_bytes(rows, K):
    return -(-rows // 128) * -(-K // 512) * 512


def pack_scales(rowwise, rows, K):
    """rowwise[r][b], one byte per row and block of 128 along K, in the packed
    order: 128 rows x 4 blocks per 512 bytes, row r at 16 (r mod 32) +
    4 ((r mod 128) / 32); 127 where there is no row or block."""
    kq = -(-K // 512)
    out = np.full(packed_bytes(rows, K), 127, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(-(-K // 128)), indexing="ij")
    out[((r // 128) * kq + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4] = rowwise
    return out


def qknorm_rope(x, gq, gk, positions, n_q, n_kv, D, eps, base=10000.0):
    """x[M][(n_q + 2 n_kv) D]: every q and k head divided by its rms (mean of
    squares plus eps), times its weight, rotated (rotate-half) at its row's
    position; v heads as they are."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    ang = rope_angles(np.asarray(positions), D, base)
    c, s = np.cos(ang), np.sin(ang)
    for h in range(n_q + n_kv):
        sl = np.s_[:, h * D:(h + 1) * D]
        v = x[sl]
        n = v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * (gq if h < n_q else gk)
        a, b = n[:, :D // 2], n[:, D // 2:]
        out[sl] = np.concatenate([a * c - b * s, b * c + a * s], 1)
    return out


def qknorm_rope_backward(x, dout, gq, gk, positions, n_q, n_kv, D, eps, base=10000.0):
    """(dx, dgq, dgk) of qknorm_rope, by the chain rule one step at a time:
    rotation, weight, division by the rms."""
    x, dout = np.asarray(x, np.float64), np.asarray(dout, np.float64)
    dx = dout.copy()
    dg = [np.zeros(D), np.zeros(D)]
    ang = rope_angles(np.asarray(positions), D, base)
    c, s = np.cos(ang), np.sin(ang)
    for h in range(n_q + n_kv):
        sl = np.s_[:, h * D:(h + 1) * D]
        v, d = x[sl], dout[sl]
        a, b = d[:, :D // 2], d[:, D // 2:]
        dn = np.concatenate([a * c + b * s, b * c - a * s], 1)
        rms = np.sqrt((v * v).mean(1, keepdims=True) + eps)
        dg[h >= n_q] += (dn * v / rms).sum(0)
        u = dn * (gq if h < n_q else gk)
        dx[sl] = u / rms - v * (u * v).mean(1, keepdims=True) / rms ** 3
    return dx, dg[0], dg[1]


def policy_terms(lp, adv, w, old, ref, lo, hi, beta):
    """Per token: loss share, -w s, w kl, clipped weight, and d loss / d lp."""
    r = np.exp(lp - old) if old is not None else np.ones_like(lp)
    clipped = np.clip(r, lo, hi)
    free = r * adv <= clipped * adv
    s = np.minimum(r * adv, clipped * adv)
    x = ref - lp if ref is not None else np.zeros_like(lp)
    kl = np.expm1(x) - x
    g = w * (-beta * np.expm1(x) - np.where(free, r * adv, 0.0))
    return w * (beta * kl - s), -w * s, w * kl, w * ~free, g


def policy_loss(H, Wt, labels, adv, w, old, ref, clip_low, clip_high, beta, temperature):
    """The clipped policy loss with its KL term on logits H Wt^T / T, and its
    gradients.  Rows of weight 0 are left out before anything of theirs is
    read."""
    H, Wt = np.asarray(H, np.float64), np.asarray(Wt, np.float64)
    M = H.shape[0]
    V = Wt.shape[0]
    w = np.full(M, 1.0 / M) if w is None else np.asarray(w, np.float64)
    y = np.asarray(labels, np.int64)
    good = (y >= 0) & (y < V)
    L = H @ Wt.T / temperature
    lse = lse_rows(L)
    lp = np.where(good, L[np.arange(M), np.where(good, y, 0)] - lse, 0.0)
    k = good & (w != 0)

    def of(v):
        return None if v is None else np.asarray(v, np.float64)[k]

    terms = policy_terms(lp[k], of(adv), w[k], of(old), of(ref), 1.0 - clip_low, 1.0 + clip_high, beta)
    g = np.zeros(M)
    g[k] = terms[4]
    dL = -np.exp(L - lse[:, None])
    dL[np.arange(M)[good], y[good]] += 1.0
    dL *= (g / temperature)[:, None]
    return {"stats": np.array([t.sum() for t in terms[:4]]), "logp": lp, "dH": dL @ Wt, "dWt": dL.T @ H, "g": g}

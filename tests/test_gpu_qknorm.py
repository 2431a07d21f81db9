"""Norm of the q and k heads with RoPE, and its backward, against the fp64
oracle.

Bounds, elementwise.  Forward: one rounding to bf16 (2^-8 relative) of an fp32
value whose error is at most a few fp32 roundings of |n1| + |n2|, taken as
2^-20 of them.  Backward: the same with the magnitudes of the two terms of dx.
dgq, dgk: fp32 sums, rows * heads * 2^-24 times the sum of magnitudes, and
2^-20 of it for the rounding of each term."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import step_oracle as S
from tests._guard import Guards
from tests._parity import assert_device_ok, f64

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

BF, F32 = torch.bfloat16, torch.float32


def _bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(BF).cuda()


class Problem:
    def __init__(self, M, nq, nk, D, S_, scattered, seed=0):
        rng = np.random.default_rng(seed)
        self.dims = (nq, nk, D)
        self.M, self.S = M, S_
        width = (nq + 2 * nk) * D
        self.qkv = _bf(rng.standard_normal((M, width)) * np.exp2(rng.integers(-6, 6, (M, 1))))
        self.dout = _bf(rng.standard_normal((M, width)) * 1e-2)
        self.gq, self.gk = _bf(rng.uniform(-1.5, 1.5, D)), _bf(rng.uniform(0.5, 1.5, D))
        self.cos, self.sin = torch.empty(S_, D // 2, device="cuda"), torch.empty(S_, D // 2, device="cuda")
        C.coda_rope_table(self.cos, self.sin)
        self.pos = torch.from_numpy(rng.integers(0, S_, M).astype(np.int32)).cuda() if scattered else None
        self.positions = self.pos.cpu().numpy() if scattered else np.arange(M) % S_
        self.gd = Guards()

    def forward(self, out=None, eps=1e-6, **kw):
        out = self.gd.like(self.qkv) if out is None else out
        nq, nk, D = self.dims
        C.coda_qknorm_rope(self.qkv if "x" not in kw else kw["x"], self.gq, self.gk, self.cos, self.sin, out, nq, nk,
                           D, eps, self.pos)
        return out

    def backward(self, dqkv=None, eps=1e-6, dout=None, qkv=None):
        nq, nk, D = self.dims
        dqkv = self.gd.like(self.qkv) if dqkv is None else dqkv
        dgq, dgk = self.gd.new((D,), F32), self.gd.new((D,), F32)
        ws = self.gd.new((C.coda_qknorm_rope_bwd_workspace_bytes(self.M, D),), torch.uint8)
        C.coda_qknorm_rope_bwd(self.dout if dout is None else dout, self.qkv if qkv is None else qkv, self.gq,
                               self.gk, self.cos, self.sin, dqkv, dgq, dgk, ws, nq, nk, D, eps, self.pos)
        return dqkv, dgq, dgk


# the table is fp32: its rounding, 2^-24 of each of the two products, is inside 2^-20
SLACK = 2.0 ** -20


def _pair_mag(v, nq, nk, D):
    """|v_i| + |v_{i + D/2}| of every element of the rotated heads."""
    a = np.abs(v).reshape(v.shape[0], nq + 2 * nk, 2, D // 2)
    return np.broadcast_to(a.sum(2, keepdims=True), a.shape).reshape(v.shape)


CASES = [(1, 1, 1, 16, 4), (3, 4, 2, 64, 2), (64, 32, 8, 128, 4096), (257, 6, 3, 80, 100), (130, 5, 1, 96, 999),
         (77, 3, 3, 112, 50), (40, 2, 1, 256, 64), (33, 2, 2, 512, 40), (19, 7, 5, 32, 8), (2000, 8, 2, 128, 512),
         (5, 40, 40, 48, 7), (1500, 3, 1, 208, 300)]


@pytest.mark.parametrize("scattered", [False, True], ids=["in_order", "scattered"])
@pytest.mark.parametrize("M,nq,nk,D,S_", CASES)
def test_forward_and_backward(M, nq, nk, D, S_, scattered):
    pb = Problem(M, nq, nk, D, S_, scattered, seed=M + D)
    x, d, gq, gk = (f64(t) for t in (pb.qkv, pb.dout, pb.gq, pb.gk))
    eps = 1e-6
    y = pb.forward()
    dx, dgq, dgk = pb.backward()
    pb.gd.check("qknorm_rope")
    assert_device_ok()
    ref = S.qknorm_rope(x, gq, gk, pb.positions, nq, nk, D, eps)
    n = S.qknorm_rope(x, gq, gk, np.zeros(M, int), nq, nk, D, eps)  # position 0: the norm alone
    assert (np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + SLACK * _pair_mag(n, nq, nk, D)).all()
    rot = (nq + nk) * D
    assert torch.equal(y[:, rot:], pb.qkv[:, rot:]) and torch.equal(dx[:, rot:], pb.dout[:, rot:])
    rx, rq, rk = S.qknorm_rope_backward(x, d, gq, gk, pb.positions, nq, nk, D, eps)
    # magnitudes of dx's two terms, r |dn g| and r^3 |x| mean |dn g x|
    h = x[:, :rot].reshape(M, nq + nk, D)
    g = np.where((np.arange(nq + nk) < nq)[:, None], gq, gk)
    dn = _pair_mag(d, nq, nk, D)[:, :rot].reshape(M, nq + nk, D)
    r = 1.0 / np.sqrt((h * h).mean(2, keepdims=True) + eps)
    t = np.abs(dn * g)
    mag = r * t + r ** 3 * np.abs(h) * (t * np.abs(h)).mean(2, keepdims=True)
    err = np.abs(f64(dx) - rx)[:, :rot].reshape(mag.shape)
    # the mean is a sum of D fp32 terms: D 2^-24 of it
    assert (err <= 2.0 ** -8 * np.abs(rx[:, :rot].reshape(mag.shape)) + (SLACK + D * 2.0 ** -24) * mag).all()
    terms = dn * np.abs(h) * r
    for got, want, part in ((dgq, rq, terms[:, :nq]), (dgk, rk, terms[:, nq:])):
        m = part.sum((0, 1))
        assert (np.abs(f64(got) - want) <= (SLACK + part.shape[0] * part.shape[1] * 2.0 ** -24) * m).all()


def test_in_place_and_repeatable():
    pb = Problem(300, 8, 2, 128, 64, True)
    y = pb.forward()
    a = pb.backward()
    b = pb.backward()
    assert all(torch.equal(u, v) for u, v in zip(a, b))     # a fixed order of sums
    z = pb.qkv.clone()
    pb.forward(out=z, x=z)
    assert torch.equal(y, z)
    d = pb.dout.clone()
    in_dout = pb.backward(dqkv=d, dout=d)
    q = pb.qkv.clone()
    in_qkv = pb.backward(dqkv=q, qkv=q)
    for c in (in_dout, in_qkv):
        # the grid differs when v stays in place, hence the order of dg's sums
        assert torch.equal(c[0], a[0])
        for u, v in zip(c[1:], a[1:]):
            assert torch.allclose(u, v, rtol=1e-4, atol=1e-5)
    assert_device_ok()


def test_zero_rows_and_no_kv_heads():
    """A zero head: rstd = 1 / sqrt(eps), its output 0, its gradient that of
    a linear map; and a qkv with query heads alone."""
    nq, D, M = 3, 64, 6
    x = np.random.default_rng(3).standard_normal((M, nq * D))
    x[2] = 0.0
    qkv, dout = _bf(x), _bf(np.ones((M, nq * D)))
    gq = _bf(np.ones(D))
    cos, sin = torch.empty(M, D // 2, device="cuda"), torch.empty(M, D // 2, device="cuda")
    C.coda_rope_table(cos, sin)
    out, dx, dgq = torch.empty_like(qkv), torch.empty_like(qkv), torch.empty(D, device="cuda")
    ws = torch.empty(C.coda_qknorm_rope_bwd_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")
    C.coda_qknorm_rope(qkv, gq, None, cos, sin, out, nq, 0, D, 1e-4)
    C.coda_qknorm_rope_bwd(dout, qkv, gq, None, cos, sin, dx, dgq, None, ws, nq, 0, D, 1e-4)
    assert_device_ok()
    assert (out[2] == 0).all()
    rx, rq, _ = S.qknorm_rope_backward(f64(qkv), f64(dout), np.ones(D), np.ones(D), np.arange(M), nq, 0, D, 1e-4)
    assert np.abs(f64(dx)[2] - rx[2]).max() <= 2.0 ** -8 * np.abs(rx[2]).max() * 1.01
    assert np.abs(rx[2]).max() > 50            # 1 / sqrt(1e-4) = 100 times a rotation of ones
    assert np.allclose(f64(dgq), rq, rtol=1e-5, atol=1e-5)


def test_eps_zero_with_heads_that_fill_no_chunk():
    pb = Problem(37, 3, 1, 64, 16, False)
    dx, dgq, dgk = pb.backward(eps=0.0)
    rx, rq, rk = S.qknorm_rope_backward(f64(pb.qkv), f64(pb.dout), f64(pb.gq), f64(pb.gk), pb.positions, 3, 1, 64,
                                        0.0)
    assert np.allclose(f64(dgq), rq, rtol=1e-4, atol=1e-5) and np.allclose(f64(dgk), rk, rtol=1e-4, atol=1e-5)
    assert np.linalg.norm(f64(dx) - rx) <= 2.0 ** -8 * np.linalg.norm(rx)
    assert_device_ok()


def test_nan_row_stays_in_its_head():
    pb = Problem(8, 2, 1, 64, 16, False)
    pb.qkv[3, 70] = float("nan")       # head 1 of row 3
    y = pb.forward()
    nan = torch.isnan(y)
    assert nan[3, 64:128].all() and int(nan.sum()) == 64
    assert_device_ok()


def test_positions_outside_the_table_are_reported():
    pb = Problem(4, 2, 1, 64, 16, True)
    pb.pos.copy_(torch.tensor([0, 16, -1, 15], dtype=torch.int32))
    y = pb.forward()
    st, bits = C.coda_sync_status()
    assert st == 8 and bits == 1 << 9 and C.STATUS_NAMES[st] == "CODA_ERR_POSITION_RANGE"
    n = S.qknorm_rope(f64(pb.qkv), f64(pb.gq), f64(pb.gk), np.array([0, 0, 0, 15]), 2, 1, 64, 1e-6)
    assert np.abs(f64(y) - n).max() <= 2.0 ** -8 * np.abs(n).max() * 1.01
    assert_device_ok()                 # read and cleared


def test_refusals_and_empty_batches():
    lib, h = C.load_library(), C.handle()
    st = torch.cuda.current_stream().cuda_stream
    b = torch.zeros(1 << 16, device="cuda")
    p, odd = ctypes.c_void_p(b.data_ptr()), ctypes.c_void_p(b.data_ptr() + 8)

    def fwd(q=p, gq=p, gk=p, c=p, s=p, pos=None, out=p, M=2, nq=2, nk=1, D=64, S_=4, eps=1e-6):
        return lib.coda_qknorm_rope(h, q, gq, gk, c, s, pos, out, M, nq, nk, D, S_, eps, st)

    assert fwd(q=None) == 1 and fwd(gq=None) == 1 and fwd(gk=None) == 1 and fwd(c=None) == 1 and fwd(out=None) == 1
    assert fwd(nq=0) == 1 and fwd(S_=0) == 1 and fwd(M=-1) == 1 and fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1
    assert fwd(q=odd) == 2 and fwd(out=odd) == 2 and fwd(D=24) == 2 and fwd(D=528) == 3
    assert fwd(q=None, out=None, M=0) == 0

    def bwd(dout=p, dgq=p, dgk=p, ws=p, n=1 << 18, M=2, nq=2, D=64):
        return lib.coda_qknorm_rope_bwd(h, dout, p, p, p, p, p, None, p, dgq, dgk, ws, n, M, nq, 1, D, 4, 1e-6, st)

    assert bwd(n=1000) == 4 and bwd(ws=None) == 1 and bwd(dgk=None) == 1 and bwd(dgq=odd) == 2 and bwd(D=528) == 3
    assert bwd(nq=1023) == 3
    dgq, dgk = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    assert lib.coda_qknorm_rope_bwd(h, None, None, p, p, p, p, None, None, ctypes.c_void_p(dgq.data_ptr()),
                                    ctypes.c_void_p(dgk.data_ptr()), None, 0, 0, 2, 1, 64, 4, 1e-6, st) == 0
    assert (dgq == 0).all() and (dgk == 0).all()
    with pytest.raises(ValueError):
        C.coda_qknorm_rope(torch.zeros(2, 100, dtype=BF, device="cuda"), None, None, b.view(-1, 32), b.view(-1, 32),
                           None, 2, 1, 64)
    assert_device_ok()

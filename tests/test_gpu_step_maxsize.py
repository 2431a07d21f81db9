"""The post-training operators past 2^31 elements, where every offset needs 64
bits.  The inputs repeat a small batch that is graded against the fp64 oracle,
so every repetition has to give the same rows."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as S
from tests._parity import assert_device_ok, assert_frob, f64
from tests.test_gpu_policy import Problem as PolicyProblem
from tests.test_gpu_qknorm import SLACK, Problem as HeadProblem, _pair_mag

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

BF, U8 = torch.bfloat16, torch.uint8


def _u8(*shape):
    return torch.zeros(*shape, dtype=U8, device="cuda")


def test_quantize_and_back():
    R, C_, k = 512, 28672, 160                 # 2.35e9 elements
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    base = (torch.randn(R, C_, generator=g, device="cuda")
            * torch.exp2(torch.randint(-9, 9, (R, C_), generator=g, device="cuda").float())).to(BF)
    src = base.repeat(k, 1)
    M = R * k
    assert M * C_ > 2 ** 31

    def run(x):
        m = x.shape[0]
        o = (_u8(m, C_), _u8(C.coda_fp8_block_scale_bytes(m, C_)), _u8(m, C_), _u8(C.coda_fp8_block_scale_bytes(C_, m)))
        C.coda_fp8_block_quantize(x, *o)
        return o

    small, big = run(base), run(src)
    q, s = S.block_quantize(f64(base), 1, 128)
    assert (small[0].cpu().numpy() == q).all()
    assert (small[1].cpu().numpy() == S.pack_scales(s, R, C_)).all()
    for i in (0, 2):
        assert (big[i].view(k, R, C_) == small[i]).all()
    assert (big[1].view(k, -1) == small[1]).all()
    # column blocks: a repetition's 512 rows are one chunk of every 128 columns
    assert (big[3].view(C_ // 128, k, 512) == small[3].view(C_ // 128, 1, 512)).all()
    del src
    for col in (False, True):
        a, b = torch.empty_like(base), torch.empty(M, C_, dtype=BF, device="cuda")
        C.coda_fp8_block_dequantize(small[2 * col], small[2 * col + 1], col, a)
        C.coda_fp8_block_dequantize(big[2 * col], big[2 * col + 1], col, b)
        assert (b.view(k, R, C_) == a).all()
    assert_device_ok()


def test_gemm_output():
    R, N, K, k = 256, 28672, 144, 300          # 2.2e9 outputs
    g = torch.Generator(device="cuda")
    g.manual_seed(4)

    def ints(*shape):                          # exact in e4m3, and so are the fp32 sums
        return torch.randint(-4, 5, shape, generator=g, device="cuda").to(BF)

    A, W = ints(R, K), ints(N, K)
    M = R * k
    assert M * N > 2 ** 31
    Aq, sA, Wq, sW = _u8(M, K), _u8(C.coda_fp8_block_scale_bytes(M, K)), _u8(N, K), _u8(C.coda_fp8_block_scale_bytes(N, K))
    sWt = _u8(C.coda_fp8_block_scale_bytes(K, N))
    C.coda_fp8_block_quantize(A.repeat(k, 1), Aq, sA, None, None)
    C.coda_fp8_block_quantize_weight(W, Wq, sW, sWt)
    out = torch.full((M, N), float("nan"), dtype=BF, device="cuda")
    C.coda_gemm_fp8_block(Aq, False, C.E4M3, sA, Wq, False, C.E4M3, sW, out, M, N, K)
    want = (A.float() @ W.float().T).to(BF)    # integers below 2^24: exact in any order
    assert (out.view(k, R, N) == want).all()
    assert_device_ok()


def test_head_norm_and_backward():
    R, nq, nk, D, k = 512, 32, 8, 128, 700     # 2.2e9 elements
    pb = HeadProblem(R, nq, nk, D, R, scattered=False, seed=5)
    width = (nq + 2 * nk) * D
    M = R * k
    assert M * width > 2 ** 31
    y, (dx, dgq, dgk) = pb.forward(), pb.backward()
    x, dout = pb.qkv.repeat(k, 1), pb.dout.repeat(k, 1)
    out = torch.full_like(x, float("nan"))
    C.coda_qknorm_rope(x, pb.gq, pb.gk, pb.cos, pb.sin, out, nq, nk, D)
    assert (out.view(k, R, width) == y).all()
    bq, bk = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = _u8(C.coda_qknorm_rope_bwd_workspace_bytes(M, D))
    out.fill_(float("nan"))
    C.coda_qknorm_rope_bwd(dout, x, pb.gq, pb.gk, pb.cos, pb.sin, out, bq, bk, ws, nq, nk, D)
    assert (out.view(k, R, width) == dx).all()
    # dg: a thread's chain of fp32 sums (2 heads of each of its rows, fewer
    # than 4096) and the joins of the partial sums, relative to the magnitudes
    xs, ds = f64(pb.qkv), f64(pb.dout)
    _, rq, rk = S.qknorm_rope_backward(xs, ds, f64(pb.gq), f64(pb.gk), np.arange(R), nq, nk, D, 1e-6)
    h = xs.reshape(R, nq + 2 * nk, D)
    terms = _pair_mag(ds, nq, nk, D).reshape(h.shape) * np.abs(h) / np.sqrt((h * h).mean(2, keepdims=True) + 1e-6)
    for got, want, part in ((bq, rq, terms[:, :nq]), (bk, rk, terms[:, nq:nq + nk])):
        assert (np.abs(f64(got) - k * want) <= (4096 * 2.0 ** -24 + SLACK) * k * part.sum((0, 1))).all()
    assert_device_ok()


@pytest.mark.parametrize("k,form", [(30, 1), (115, 1), (115, 2)],
                         ids=["one_narrow_chunk_kept", "narrow_chunks_kept", "computed_twice"])
def test_policy_rows(k, form):
    """115 repetitions: a chunk of dL holds 2.26e9 elements.  Kept are 29696
    and 7680 of the columns."""
    R, d, V = 600, 64, 33000
    M = R * k
    assert M * min(V, 32768) > 2 ** (31 if k == 115 else 29)
    pb = PolicyProblem(R, d, V, seed=6)
    r = pb.run()
    pb.grade(r)
    small = (pb.stats.clone(), pb.logp.clone(), pb.dH.clone())
    a = list(pb.args)
    a[0] = a[0].repeat(k, 1)
    for i in range(2, 7):
        a[i] = a[i].repeat(k)
    logp, dH, dW, stats = (torch.empty(M, device="cuda"), torch.empty(M, d, dtype=BF, device="cuda"),
                           torch.empty_like(pb.W), torch.empty(4, device="cuda"))
    a[11:16] = [stats, logp, dH, dW, _u8(C.coda_lmhead_policy_workspace_bytes(M, d, V, form))]
    C.coda_lmhead_policy(*a)
    assert (logp.view(k, R) == small[1]).all()
    # the statistics: one fp32 rounding each of a sum carried in two words
    assert (np.abs(f64(stats) - k * f64(small[0])) <= k * 2.0 ** -22 * np.abs(f64(small[0]))).all()
    ref = torch.from_numpy(r["dH"]).cuda()
    for rows in dH.view(k, R, d).double():
        assert (rows - ref).norm() <= 5e-3 * ref.norm()
    assert_frob(dW, k * r["dWt"], "dW")
    assert_device_ok()

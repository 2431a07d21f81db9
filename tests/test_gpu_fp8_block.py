"""Block-scaled 8-bit codes and the GEMM on them, against the fp64 oracle.

Codes and scales are compared bit for bit.  GEMMs on small integers with
power-of-two scales have exact fp32 sums, so their outputs equal the oracle's
rounded once to bf16.  On general codes the bound is that rounding (2^-8
relative) plus fp32 accumulation, K 2^-23 times the sum of the products'
magnitudes."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import coda_oracle as O
from oracle import step_oracle as S
from tests._guard import Guards
from tests._parity import assert_device_ok, f64

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

BF, U8 = torch.bfloat16, torch.uint8
FMT = {"e4m3": C.E4M3, "e5m2": C.E5M2}


def _bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(BF).cuda()


def _u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _spread(rng, rows, cols):
    """Values over many binades, with a zero block and bf16 extremes."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, cols)))
    x[:, :16][rng.random((rows, 16)) < 0.5] = 0.0
    x[0, 0], x[-1, -1] = 3.0e38, 1e-40
    if rows > 2:
        x[1] = 0.0
    return f64(_bf(x))


def _scales(rows, K):
    return torch.empty(C.coda_fp8_block_scale_bytes(rows, K), dtype=U8, device="cuda")


SHAPES = [(1, 16), (3, 128), (127, 144), (128, 512), (129, 528), (333, 2064), (640, 1040)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_bit_exact(rows, cols, fmt):
    x = _spread(np.random.default_rng(rows * 7 + cols), rows, cols)
    src = _bf(x)
    gd = Guards()
    qr, qc = gd.new((rows, cols), U8), gd.new((rows, cols), U8)
    sr = gd.new((C.coda_fp8_block_scale_bytes(rows, cols),), U8)
    sc = gd.new((C.coda_fp8_block_scale_bytes(cols, rows),), U8)
    C.coda_fp8_block_quantize(src, qr, sr, qc, sc, FMT[fmt])
    gd.check("quantize")
    assert_device_ok()
    rq, rs = S.block_quantize(x, 1, 128, fmt)
    cq, cs = S.block_quantize(x, 128, 1, fmt)
    assert (qr.cpu().numpy() == rq).all() and (qc.cpu().numpy() == cq).all()
    assert (sr.cpu().numpy() == S.pack_scales(rs, rows, cols)).all()
    assert (sc.cpu().numpy() == S.pack_scales(cs.T, cols, rows)).all()
    # one direction alone gives the same bytes
    q1, s1 = torch.zeros_like(qr), torch.zeros_like(sr)
    C.coda_fp8_block_quantize(src, q1, s1, None, None, FMT[fmt])
    q2, s2 = torch.zeros_like(qc), torch.zeros_like(sc)
    C.coda_fp8_block_quantize(src, None, None, q2, s2, FMT[fmt])
    for a, b in ((q1, qr), (s1, sr), (q2, qc), (s2, sc)):
        assert torch.equal(a, b)
    # and the way back
    d = torch.empty(rows, cols, dtype=BF, device="cuda")
    for q, s, col, want in ((qr, sr, False, S.block_dequantize(rq, rs, 1, 128, fmt)),
                            (qc, sc, True, S.block_dequantize(cq, cs, 128, 1, fmt))):
        C.coda_fp8_block_dequantize(q, s, col, d, FMT[fmt])
        assert torch.equal(d, _bf(want))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("N,K", [(1, 16), (130, 144), (256, 640), (999, 528)])
def test_weight_tiles_bit_exact(N, K, fmt):
    x = _spread(np.random.default_rng(N + K), N, K)
    gd = Guards()
    q = gd.new((N, K), U8)
    s = gd.new((C.coda_fp8_block_scale_bytes(N, K),), U8)
    st = gd.new((C.coda_fp8_block_scale_bytes(K, N),), U8)
    C.coda_fp8_block_quantize_weight(_bf(x), q, s, st, FMT[fmt])
    gd.check("quantize_weight")
    rq, rs = S.block_quantize(x, 128, 128, fmt)
    assert (q.cpu().numpy() == rq).all()
    # rows past the weight carry their tile's scale or 1: compare the rows that exist
    ref = S.pack_scales(np.repeat(rs, 128, 0)[:N], N, K)
    real = S.pack_scales(np.zeros((N, rs.shape[1]), np.uint8), N, K) == 0
    assert (s.cpu().numpy()[real] == ref[real]).all()
    ref = S.pack_scales(np.repeat(rs.T, 128, 0)[:K], K, N)
    real = S.pack_scales(np.zeros((K, rs.shape[0]), np.uint8), K, N) == 0
    assert (st.cpu().numpy()[real] == ref[real]).all()


def test_poisoned_blocks_stay_in_their_blocks():
    x = np.random.default_rng(0).standard_normal((256, 256)).astype(np.float32)
    x[5, 130], x[200, 7], x[201, 8] = np.nan, np.inf, -np.inf
    q, s, qc, sc = (torch.empty(256, 256, dtype=U8, device="cuda"), _scales(256, 256),
                    torch.empty(256, 256, dtype=U8, device="cuda"), _scales(256, 256))
    C.coda_fp8_block_quantize(_bf(x), q, s, qc, sc)
    x = np.where(np.isfinite(x), f64(_bf(x)), x)
    rq, rs = S.block_quantize(x, 1, 128)
    cq, cs = S.block_quantize(x, 128, 1)
    assert (q.cpu().numpy() == rq).all() and (qc.cpu().numpy() == cq).all()
    assert (s.cpu().numpy() == S.pack_scales(rs, 256, 256)).all()
    assert (sc.cpu().numpy() == S.pack_scales(cs.T, 256, 256)).all()
    # through the GEMM: the rows with a poisoned block are NaN, the others are not
    W = np.random.default_rng(1).standard_normal((64, 256))
    wq, ws, wt = torch.empty(64, 256, dtype=U8, device="cuda"), _scales(64, 256), _scales(256, 64)
    C.coda_fp8_block_quantize_weight(_bf(W), wq, ws, wt)
    Y = torch.empty(256, 64, dtype=BF, device="cuda")
    C.coda_gemm_fp8_block(q, False, 0, s, wq, False, 0, ws, Y, 256, 64, 256)
    assert_device_ok()
    nan = torch.isnan(Y).cpu().numpy()
    assert sorted(set(np.nonzero(nan)[0].tolist())) == [5, 200, 201] and nan[[5, 200, 201]].all()


def _int_codes(rng, rows, K, fmt):
    v = rng.integers(-4, 5, (rows, K)).astype(np.float64)
    return v, O.FP8_FORMATS[fmt][2](v)


def _int_gemm(rng, M, N, K, a_mn, b_mn, fa, fb):
    a, qa = _int_codes(rng, M, K, fa)
    b, qb = _int_codes(rng, N, K, fb)
    kb = -(-K // 128)
    # products of at most 16 2^3 in units of 2^-3: K 2^10 units, exact in fp32
    ea, eb = rng.integers(-2, 3, (M, kb)), rng.integers(-1, 2, (N, kb))
    sa, sb = _u8(S.pack_scales((ea + 127).astype(np.uint8), M, K)), _u8(S.pack_scales((eb + 127).astype(np.uint8), N, K))
    av = a * np.exp2(np.repeat(ea, 128, 1)[:, :K])
    bv = b * np.exp2(np.repeat(eb, 128, 1)[:, :K])
    A = _u8(qa.T if a_mn else qa)
    B = _u8(qb.T if b_mn else qb)
    gd = Guards()
    out = gd.new((M, N), BF)
    C.coda_gemm_fp8_block(A, a_mn, FMT[fa], sa, B, b_mn, FMT[fb], sb, out, M, N, K)
    gd.check("gemm_fp8_block")
    assert_device_ok()
    return out, av, bv


LAYOUTS = [(False, False), (False, True), (True, True)]
GEMMS = [(1, 8, 16), (5, 72, 144), (16, 128, 128), (33, 264, 272), (64, 1000, 640), (100, 256, 2064),
         (129, 136, 528), (257, 520, 400), (300, 1288, 1040)]


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kk", "km", "mm"])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_known_answer(M, N, K, layout):
    a_mn, b_mn = layout
    if a_mn:
        M = -(-M // 16) * 16
        K -= 3                     # a token count: any
    if b_mn:
        N = -(-N // 16) * 16
    rng = np.random.default_rng(M + N + K)
    for fa, fb in (("e4m3", "e4m3"), ("e5m2", "e4m3")):
        out, a, b = _int_gemm(rng, M, N, K, a_mn, b_mn, fa, fb)
        assert torch.equal(out, _bf(a @ b.T)), (fa, fb)


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kk", "km", "mm"])
@pytest.mark.parametrize("M,N,K", [(5008, 272, 2080), (272, 528, 9008), (3008, 2064, 2576), (272, 5200, 4112),
                                   (1040, 1296, 4112), (2000, 1040, 8704)])
def test_gemm_long_contractions(M, N, K, layout):
    """Few output tiles and a long K: ranges of K on their own SMs."""
    a_mn, b_mn = layout
    if a_mn:
        K -= 5
    out, a, b = _int_gemm(np.random.default_rng(K), M, N, K, a_mn, b_mn, "e4m3", "e4m3")
    assert torch.equal(out, _bf((torch.from_numpy(a).cuda() @ torch.from_numpy(b).cuda().t()).cpu().numpy()))


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kk", "km", "mm"])
def test_gemm_many_tiles_per_pair(layout):
    """Several tiles per SM pair: the accumulators that share columns, ragged
    edges in both extents, a K of several scale chunks and a tail."""
    out, a, b = _int_gemm(np.random.default_rng(9), 4000, 5008, 1168, *layout, "e4m3", "e5m2")
    assert torch.equal(out, _bf((torch.from_numpy(a).cuda() @ torch.from_numpy(b).cuda().t()).cpu().numpy()))


@pytest.mark.parametrize("M", [1, 7, 60, 200, 700])
def test_linear_layer_forward_backward(M):
    """Y, dX and dW of a linear layer from bf16 tensors, each against the
    product of the oracle's dequantised operands."""
    N, K = 336, 784
    rng = np.random.default_rng(M)
    x, w, dy = (f64(_bf(v)) for v in (rng.standard_normal((M, K)), rng.standard_normal((N, K)) * 0.02,
                                      rng.standard_normal((M, N)) * 1e-3))
    u = dict(dtype=U8, device="cuda")
    Xq, Xc, Wq, Gq, Gc = (torch.empty(s, **u) for s in ((M, K), (M, K), (N, K), (M, N), (M, N)))
    sX, sXc, sW, sWt, sG, sGc = (_scales(*s) for s in ((M, K), (K, M), (N, K), (K, N), (M, N), (N, M)))
    C.coda_fp8_block_quantize(_bf(x), Xq, sX, Xc, sXc, C.E4M3)
    C.coda_fp8_block_quantize_weight(_bf(w), Wq, sW, sWt, C.E4M3)
    C.coda_fp8_block_quantize(_bf(dy), Gq, sG, Gc, sGc, C.E5M2)
    Y, dX, dW = (torch.empty(s, dtype=BF, device="cuda") for s in ((M, N), (M, K), (N, K)))
    C.coda_gemm_fp8_block(Xq, False, C.E4M3, sX, Wq, False, C.E4M3, sW, Y, M, N, K)
    C.coda_gemm_fp8_block(Gq, False, C.E5M2, sG, Wq, True, C.E4M3, sWt, dX, M, K, N)
    C.coda_gemm_fp8_block(Gc, True, C.E5M2, sGc, Xc, True, C.E4M3, sXc, dW, N, K, M)
    assert_device_ok()

    def deq(v, rb, cb, fmt="e4m3"):
        return S.block_dequantize(*S.block_quantize(v, rb, cb, fmt), rb, cb, fmt)

    wd = deq(w, 128, 128)
    for got, a, b in ((Y, deq(x, 1, 128), wd.T), (dX, deq(dy, 1, 128, "e5m2"), wd),
                      (dW, deq(dy, 128, 1, "e5m2").T, deq(x, 128, 1))):
        ref, mag = a @ b, np.abs(a) @ np.abs(b)
        assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + a.shape[1] * 2.0 ** -23 * mag + 1e-38).all()


def test_empty_problems_and_refusals():
    lib, h = C.load_library(), C.handle()
    st = torch.cuda.current_stream().cuda_stream
    buf = torch.zeros(1 << 16, dtype=U8, device="cuda")
    p = ctypes.c_void_p(buf.data_ptr())
    odd = ctypes.c_void_p(buf.data_ptr() + 8)
    OK, INVALID, ALIGN, UNSUPPORTED = 0, 1, 2, 3

    def gemm(A=p, amn=0, fa=0, sA=p, B=p, bmn=0, fb=0, sB=p, Cc=p, M=16, N=16, K=128):
        return lib.coda_gemm_fp8_block(h, A, amn, fa, sA, B, bmn, fb, sB, Cc, M, N, K, st)

    assert gemm(sA=None) == INVALID and gemm(sB=None) == INVALID and gemm(Cc=None) == INVALID
    assert gemm(fa=2) == INVALID and gemm(fb=-1) == INVALID and gemm(K=0) == INVALID and gemm(M=-1) == INVALID
    assert gemm(amn=1) == UNSUPPORTED
    assert gemm(K=120) == ALIGN and gemm(N=12) == ALIGN and gemm(bmn=1, N=24) == ALIGN
    assert gemm(amn=1, bmn=1, M=8) == ALIGN and gemm(sA=odd) == ALIGN and gemm(A=odd) == ALIGN
    assert gemm(M=0, A=None, sA=None, Cc=None) == OK
    one = torch.ones(16, 16, dtype=BF, device="cuda")
    assert gemm(A=None, amn=1, sA=None, B=None, bmn=1, sB=None, Cc=ctypes.c_void_p(one.data_ptr()), K=0) == OK
    assert (one == 0).all()

    def quant(src=p, fmt=0, q=p, s=p, qc=None, sc=None, rows=1, cols=128):
        return lib.coda_fp8_block_quantize(h, src, fmt, q, s, qc, sc, rows, cols, st)

    assert quant(src=None) == INVALID and quant(fmt=3) == INVALID and quant(q=None) == INVALID
    assert quant(q=None, s=None) == INVALID and quant(qc=p, sc=p) == INVALID and quant(qc=odd, sc=p) == ALIGN
    assert quant(cols=120) == ALIGN and quant(rows=-1) == INVALID and quant(rows=0, src=None) == OK
    assert lib.coda_fp8_block_quantize_weight(h, p, 0, p, p, None, 16, 128, st) == INVALID
    assert lib.coda_fp8_block_quantize_weight(h, p, 0, p, p, p, 0, 128, st) == INVALID
    assert lib.coda_fp8_block_quantize_weight(h, p, 0, p, p, p, 16, 24, st) == ALIGN
    assert lib.coda_fp8_block_dequantize(h, p, None, 0, 0, p, 1, 128, st) == INVALID
    assert lib.coda_fp8_block_dequantize(h, p, p, 0, 2, p, 1, 128, st) == INVALID
    assert lib.coda_fp8_block_dequantize(h, None, None, 0, 0, None, 0, 128, st) == OK
    # the binding's shapes
    q, x = torch.empty(4, 128, dtype=U8, device="cuda"), torch.zeros(4, 128, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        C.coda_fp8_block_quantize(x, q, torch.empty(16, dtype=U8, device="cuda"), None, None)
    with pytest.raises(ValueError):
        C.coda_fp8_block_quantize(x, q, None, None, None)
    with pytest.raises(ValueError):
        C.coda_fp8_block_quantize(x.to_sparse(), q, _scales(4, 128), None, None)
    with pytest.raises(ValueError):
        C.coda_fp8_block_quantize(x.cpu(), q, _scales(4, 128), None, None)
    with pytest.raises(ValueError):
        C.coda_fp8_block_quantize(x[:, ::2], q, _scales(4, 128), None, None)
    with pytest.raises(TypeError):
        C.coda_fp8_block_quantize(None, q, _scales(4, 128), None, None)
    with pytest.raises(TypeError):
        C.coda_fp8_block_quantize(x.float(), q, _scales(4, 128), None, None)
    assert_device_ok()


def test_captured_graph_and_second_stream():
    """A captured quantise + GEMM replays on new inputs with the eager bits,
    and so does the same pair on another stream."""
    M, N, K = 40, 272, 1040
    w = torch.randn(N, K, device="cuda").to(BF)
    Wq, sW, sWt = torch.empty(N, K, dtype=U8, device="cuda"), _scales(N, K), _scales(K, N)
    C.coda_fp8_block_quantize_weight(w, Wq, sW, sWt)
    x = torch.randn(M, K, device="cuda").to(BF)
    Xq, sX, Y = torch.empty(M, K, dtype=U8, device="cuda"), _scales(M, K), torch.empty(M, N, dtype=BF, device="cuda")

    def step(stream=None):
        C.coda_fp8_block_quantize(x, Xq, sX, None, None, stream=stream)
        C.coda_gemm_fp8_block(Xq, False, 0, sX, Wq, False, 0, sW, Y, M, N, K, stream=stream)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        x.copy_(torch.randn(M, K, device="cuda"))
        step()
        want = Y.clone()
        Y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
        Y.zero_()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        step(s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(Y, want)
    assert_device_ok()

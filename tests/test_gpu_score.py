"""Scoring on the LM head against its definition in fp64.

The inputs lie on grids that make every logit exact in fp32 (tests/_lmhead.py),
so the ranks have to be those of fp64, ties by token.  What is left are the
roundings behind the logits.  With s = sum exp(x / T) over all but the largest:
an exponential is off by 2^-22 (the instruction) and its argument's rounding,
|x / T| 2^-23 with |x / T| < 90 below the cut-off, 2^-16.5 at the farthest; a
sum of 128 in four chains adds 34 roundings of 2^-24, its merging at most 2 (T /
128 + 7) of 2^-23: below 2^-18 in all for T <= 1002 blocks.  logp = x / T -
log1p(s) and the entropy log1p(s) - (u / T) / (1 + s) are sums of terms of one
sign, so that all of this is relative to the result: 2^-16 covers exponentials
at the cut-off, whose share of s is nil, and everything else."""
import ctypes

import pytest
import torch

from tests import _lmhead as R
from tests._guard import Guards
from tests._parity import assert_device_ok

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

F32, I32 = torch.float32, torch.int32
REL = 2.0 ** -16


class Call:
    def __init__(self, H, W, y=None, T=1.0, k=0, entropy=True):
        M, V = H.shape[0], W.shape[0]
        self.H, self.W, self.y, self.T, self.k = H, W, y, T, k
        self.gd = Guards()
        self.logp = self.gd.new((M,), F32) if y is not None else None
        self.entropy = self.gd.new((M,), F32) if entropy else None
        self.ids = self.gd.new((M, k), I32) if k else None
        self.top = self.gd.new((M, k), F32) if k else None
        self.ws = self.gd.new((C.coda_lmhead_score_workspace_bytes(M, H.shape[1], V, k),), torch.uint8)
        self.args = (H, W, y, T, self.logp, self.entropy, self.ids, self.top, self.ws)

    def run(self):
        C.coda_lmhead_score(*self.args)
        self.gd.check("lmhead_score")
        return self

    def outputs(self):
        return [t for t in (self.logp, self.entropy, self.ids, self.top) if t is not None]

    def grade(self, rows=slice(None)):
        r = R.score(self.H[rows], self.W, None if self.y is None else self.y[rows], self.T, self.k)
        if self.k:
            assert torch.equal(self.ids[rows], r["ids"])
            assert near(self.top[rows], r["top"])
        if self.y is not None:
            assert near(self.logp[rows], r["logp"])
        if self.entropy is not None:
            assert near(self.entropy[rows], r["entropy"])
        assert_device_ok()


def near(got, ref):
    return bool(((got.double() - ref).abs() <= REL * ref.abs() + 1e-30).all())


@pytest.mark.parametrize("M,d,V,k", [
    (1, 8, 8, 8), (1, 64, 1000, 1), (2, 256, 4096, 20), (5, 64, 136, 136), (16, 64, 1000, 5), (17, 72, 2048, 256),
    (48, 512, 5000, 8), (64, 200, 3000, 64), (65, 64, 3000, 64), (128, 64, 1048, 20), (136, 72, 1000, 20),
    (300, 128, 520, 256), (129, 256, 33000, 64), (700, 64, 20008, 128), (1, 4096, 32000, 20), (3, 1024, 128256, 100)])
@pytest.mark.parametrize("T", [1.0, 0.7, 3.0])
def test_every_output(M, d, V, k, T):
    H, W, y = R.grid_inputs(M, d, V, seed=M + k)
    Call(H, W, y, T, k).run().grade()


@pytest.mark.parametrize("M,d,V", [(1, 64, 1000), (40, 136, 2056), (300, 64, 1000), (1111, 64, 5000)])
def test_without_alternatives(M, d, V):
    H, W, y = R.grid_inputs(M, d, V, seed=M)
    a, b, c = Call(H, W, y).run(), Call(H, W).run(), Call(H, W, y, entropy=False).run()
    a.grade()
    b.grade()
    assert torch.equal(a.entropy, b.entropy) and torch.equal(a.logp, c.logp)
    k = Call(H, W, k=3, entropy=False).run()
    k.grade()


@pytest.mark.parametrize("M", [1, 30, 200])
@pytest.mark.parametrize("V,k", [(264, 256), (4096, 64), (50280, 100)])
def test_equal_logits_rank_by_token(M, V, k):
    """A row of zeros, one with a single logit that differs, one with two
    values only, and a row whose largest are the same."""
    H, W, y = R.grid_inputs(M + 3, 64, V, seed=5)
    W[:, 0] = 0
    W[V // 2, 0] = 1.0
    W[:, 1] = (torch.arange(V, device="cuda") % 3 == 1).to(W.dtype)
    H[0] = 0
    for i, (a, b) in enumerate(((1.0, 0.0), (0.0, 2.0), (0.0, -4.0))):
        H[M + i] = 0
        H[M + i, 0], H[M + i, 1] = a, b
    Call(H, W, y, 1.0, k).run().grade()


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("offset", [0.0, 512.0])
def test_many_logits_near_the_kth(M, offset):
    """Thousands of candidates in one row: logits that differ only in their
    last digits (steps of 2^-11 at 512 need all of fp32's), and descending and
    ascending ones."""
    V, k = 40000, 200
    H, W, y = R.grid_inputs(M + 2, 64, V, seed=6)
    W[:, :4] = 0
    W[:, 0] = 1.0
    r = torch.arange(V, device="cuda")
    W[:, 1] = (r % 256).to(W.dtype)
    W[:, 2] = (r // 256).to(W.dtype)
    H[0] = 0
    H[0, 0], H[0, 1], H[0, 2] = offset, 2.0 ** -11, 0.0
    H[M] = 0
    H[M, 0], H[M, 1], H[M, 2] = offset, 2.0 ** -11, 2.0 ** -3
    H[M + 1] = -H[M]
    c = Call(H, W, y, 1.0, k).run()
    c.grade()


def test_rows_from_flat_to_certain():
    """Entropy and log-probability of rows up to 1 - 1e-30 certain keep their
    relative precision; the one token's logit decides."""
    V = 3000
    W = torch.zeros(V, 64, dtype=torch.bfloat16, device="cuda")
    W[:, 0] = (torch.arange(V, device="cuda") % 5).to(W.dtype) / 8
    W[1234, 1] = 1.0
    H = torch.zeros(80, 64, dtype=torch.bfloat16, device="cuda")
    H[:, 0] = 1.0
    H[:, 1] = torch.arange(80, device="cuda").to(H.dtype)
    y = torch.full((80,), 1234, dtype=I32, device="cuda")
    for rows in (slice(0, 80), slice(3, 60)):
        c = Call(H[rows], W, y[rows], 1.0, 2).run()
        c.grade()
        assert c.entropy[-1].item() > 0 and c.logp[-1].item() < 0


@pytest.mark.parametrize("M", [40, 200])
def test_labels_outside_the_vocabulary(M):
    H, W, y = R.grid_inputs(M, 64, 1000)
    y[3], y[M - 1] = -100, -2 ** 31
    Call(H, W, y).run().grade()
    y[5] = 1000
    c = Call(H, W, y, k=3).run()
    assert C.coda_sync_status()[0] == 7
    c.grade()
    assert c.logp[5].item() == 0


@pytest.mark.parametrize("M", [9, 140])
@pytest.mark.parametrize("k", [5, 200])
def test_nan_rows_leave_the_others(M, k):
    H, W, y = R.grid_inputs(M, 64, 9000)
    a = Call(H, W, y, k=k).run()
    H2 = H.clone()
    H2[4] = float("nan")
    b = Call(H2, W, y, k=k).run()
    keep = torch.arange(M, device="cuda") != 4
    for p, q in zip(a.outputs(), b.outputs()):
        assert torch.equal(p[keep], q[keep])
    assert torch.isnan(b.logp[4]) and torch.isnan(b.entropy[4]) and torch.isnan(b.top[4]).all()
    assert torch.equal(b.ids[4], torch.arange(k, dtype=I32, device="cuda"))
    # one NaN logit: the others keep their ranks
    W2 = W.clone()
    W2[int(a.ids[0, 0])] = float("nan")
    c = Call(H, W2, y, k=k).run()
    assert torch.equal(c.ids[0, :k - 1], a.ids[0, 1:]) and torch.isnan(c.top).all()
    assert_device_ok()


def test_tokens_without_rows():
    H, W, y = R.grid_inputs(1, 64, 1000)
    C.coda_lmhead_score(H[:0], W, y[:0], 1.0, torch.empty(0, device="cuda"), None, None, None,
                        torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert_device_ok()


def test_a_workspace_serves_smaller_batches_and_other_streams():
    H, W, y = R.grid_inputs(150, 64, 3000)
    big = Call(H, W, y, 1.0, 7)
    for m in (150, 64, 1, 100):
        c = Call(H[:m], W, y[:m], 1.0, 7)
        c.args = c.args[:-1] + (big.ws,)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            C.coda_lmhead_score(*c.args)
        torch.cuda.current_stream().wait_stream(s)
        c.grade()


@pytest.mark.parametrize("M,k", [(1, 20), (33, 0), (150, 7)])
def test_captured_graph(M, k):
    H, W, y = R.grid_inputs(M, 64, 3000)
    c = Call(H, W, y, 1.0, k).run()
    want = [t.clone() for t in c.outputs()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        C.coda_lmhead_score(*c.args)
    for t in c.outputs():
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, c.outputs()))
    H.copy_(R.grid_inputs(M, 64, 3000, seed=9)[0])
    g.replay()
    torch.cuda.synchronize()
    c.grade()


@pytest.mark.parametrize("M,V", [(2, 3000), (200, 3000), (2100, 20000)])
def test_a_workspace_aligned_to_16_bytes(M, V):
    """As the entry points ask for, and other outputs to 4."""
    H, W, y = R.grid_inputs(M, 64, V)
    k = 5
    n = C.coda_lmhead_score_workspace_bytes(M, 64, V, k)
    f = torch.empty(M * (2 + 2 * k) + 8, device="cuda")
    logp, entropy, top = f[1:1 + M], f[1 + M:1 + 2 * M], f[3 + 2 * M:3 + (2 + k) * M].view(M, k)
    ids = f[5 + (2 + k) * M:5 + (2 + 2 * k) * M].view(torch.int32).view(M, k)
    r = R.score(H, W, y, 1.0, k)
    for off in (16, 48, 240):
        ws = torch.empty(n + off, dtype=torch.uint8, device="cuda")[off:]
        C.coda_lmhead_score(H, W, y, 1.0, logp, entropy, ids, top, ws)
        assert torch.equal(ids, r["ids"]) and near(logp, r["logp"]) and near(top, r["top"])
        assert_device_ok()


def test_rows_in_turn():
    """More logits than a workspace holds at a time: 4096 rows of this
    vocabulary, then the others."""
    V = 131072
    H, W, y = R.grid_inputs(4100, 16, V)
    c = Call(H, W, y, 1.0, 3).run()
    for rows in (slice(0, 40), slice(4090, 4100)):
        c.grade(rows)


def test_scoring_head():
    from gemm_epilogue_transformer_tma_gb300.path import ScoringHead
    H, W, y = R.grid_inputs(90, 64, 3000)
    head = ScoringHead(W, 128, k=4, temperature=0.9)
    logp, entropy, ids, top = head.score(H, y)
    r = R.score(H, W, y, 0.9, 4)
    assert torch.equal(ids, r["ids"]) and near(logp, r["logp"]) and near(entropy, r["entropy"]) and near(top, r["top"])
    logp, entropy, ids, top = head.score(H[:3])
    assert logp is None and torch.equal(ids, r["ids"][:3])
    assert ScoringHead(W, 8).score(H[:5], y[:5])[2:] == (None, None)


def test_refusals():
    lib, h = C.load_library(), C.handle()
    st = torch.cuda.current_stream().cuda_stream
    M, d, V, k = 16, 64, 136, 4
    n = C.coda_lmhead_score_workspace_bytes(M, d, V, k)
    b = torch.zeros(max(n, 1 << 16), dtype=torch.uint8, device="cuda")
    p = ctypes.c_void_p(b.data_ptr())
    odd = ctypes.c_void_p(b.data_ptr() + 2)

    def call(**kw):
        a = dict(H=p, W=p, y=p, T=1.0, logp=p, ent=p, ids=p, top=p, k=k, ws=p, n=n, M=M, d=d, V=V)
        a.update(kw)
        return lib.coda_lmhead_score(h, a["H"], a["W"], a["y"], a["T"], a["logp"], a["ent"], a["ids"], a["top"], a["k"],
                                     a["ws"], a["n"], a["M"], a["d"], a["V"], st)

    for kw, want in [(dict(H=None), 1), (dict(W=None), 1), (dict(ws=None), 1), (dict(y=None), 1), (dict(logp=None), 1),
                     (dict(ids=None), 1), (dict(top=None), 1), (dict(k=0), 1), (dict(ids=None, top=None), 1),
                     (dict(k=-1), 1), (dict(k=257), 1), (dict(k=137), 1), (dict(M=-1), 1), (dict(V=0), 1),
                     (dict(T=0.0), 1), (dict(T=-1.0), 1), (dict(T=float("nan")), 1), (dict(T=float("inf")), 1),
                     (dict(T=1e-39), 1), (dict(d=60), 2), (dict(V=140), 2), (dict(H=odd), 2), (dict(y=odd), 2),
                     (dict(ent=odd), 2), (dict(n=n - 1), 4), (dict(M=0, H=None, ws=None, n=0), 0),
                     (dict(y=None, logp=None, ent=None, ids=None, top=None, k=0), 1)]:
        assert call(**kw) == want, kw
    assert C.coda_lmhead_score_workspace_bytes(0, d, V, 0) == 0
    assert C.coda_lmhead_score_workspace_bytes(M, d, V, 137) == 0
    H, W, y = R.grid_inputs(M, d, V)
    f = torch.empty(M, device="cuda")
    for bad in (dict(H=H.float()), dict(y=y.long()), dict(W=W[:, ::2]), dict(logp=f[:3]), dict(ent=f.double()),
                dict(top=None), dict(ws=b.cpu())):
        a = dict(H=H, W=W, y=y, T=1.0, logp=f, ent=f.clone(), ids=torch.empty(M, k, dtype=I32, device="cuda"),
                 top=torch.empty(M, k, device="cuda"), ws=b)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            C.coda_lmhead_score(*a.values())
    with pytest.raises(C.CodaError):
        C.coda_lmhead_score(H, W, y, 0.0, f, None, None, None, b)
    assert_device_ok()


@pytest.mark.parametrize("V,k", [(20000, 8), (50280, 64), (40008, 256)])
def test_only_some_logits_kept(V, k):
    """Many rows and columns: the first columns bound what of the others is
    kept.  Among the rows: zeros, one value but for the last columns, logits that
    rise and fall with the token, NaN, and all but a few equal."""
    M = 4100
    H, W, y = R.grid_inputs(M, 64, V, seed=7)
    v = torch.arange(V, device="cuda")
    W[:, :3] = 0
    W[:, 0] = (v // 256).to(W.dtype)
    W[:, 1] = (v >= V - 40).to(W.dtype)
    W[:, 2] = (v % 7 == 0).to(W.dtype)
    H[:, :3] = 0
    for i, (a, b, c) in enumerate(((0, 0, 0), (0, 2, 0), (0.125, 0, 0), (-0.125, 0, 0), (0, 0, 1), (0, 0, -1),
                                   (0.125, -3, 0.5))):
        H[64 * i] = 0
        H[64 * i, :3] = torch.tensor([a, b, c], dtype=torch.float32).to(H.dtype)
    c = Call(H, W, y, 1.0, k).run()
    for m in (0, 1000, 4000):
        c.grade(slice(m, m + 100))
    c.grade(torch.arange(0, 448, 64, device="cuda"))
    want = [t.clone() for t in c.outputs()]
    H[70] = float("nan")
    c.run()
    keep = torch.arange(M, device="cuda") != 70
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(want, c.outputs()))
    assert torch.equal(c.ids[70], torch.arange(k, dtype=I32, device="cuda")) and torch.isnan(c.logp[70])
    assert_device_ok()


def test_a_temperature_without_its_power_of_two_is_refused():
    """1 / 4e-39 is an fp32 number, log2(e) / 4e-39 is not.  At 5e-39 a row is its
    largest logits' alone."""
    H, W, y = R.grid_inputs(16, 64, 136)
    f, e = torch.empty(16, device="cuda"), torch.empty(16, device="cuda")
    ws = torch.empty(C.coda_lmhead_score_workspace_bytes(16, 64, 136, 0), dtype=torch.uint8, device="cuda")
    with pytest.raises(C.CodaError):
        C.coda_lmhead_score(H, W, y, 4e-39, f, e, None, None, ws)
    C.coda_lmhead_score(H, W, y, 5e-39, f, e, None, None, ws)
    L = R.logits(H, W)
    equal = (L == L.amax(1, keepdim=True)).sum(1).double()
    assert ((e.double() - equal.log()).abs() <= 2.0 ** -20).all()
    assert_device_ok()

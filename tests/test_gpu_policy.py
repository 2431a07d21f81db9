"""The clipped policy loss on the LM head against the fp64 oracle.

logp: fp32 logits of bf16 products (d 2^-23 of the sum of magnitudes bounds
them) and a few fp32 roundings of lse.  dHs, dWt: dL is rounded to bf16 once
and the result once, relative Frobenius at most 2 * 2^-8 / sqrt(3) with room
for the accumulation: the bars of the cross-entropy, 5e-3."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import step_oracle as S
from tests._guard import Guards
from tests._parity import assert_device_ok, assert_frob, f64

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

BF, F32 = torch.bfloat16, torch.float32


class Problem:
    least = False   # the gradients' least workspace: the logits computed twice

    def __init__(self, M, d, V, T=1.0, seed=0, weighted=True):
        rng = np.random.default_rng(seed)
        self.M, self.d, self.V, self.T = M, d, V, T
        self.H = torch.from_numpy(rng.standard_normal((M, d)).astype(np.float32)).to(BF).cuda()
        self.W = torch.from_numpy((rng.standard_normal((V, d)) * 0.05).astype(np.float32)).to(BF).cuda()
        self.y = rng.integers(0, V, M).astype(np.int32)
        self.adv = rng.standard_normal(M).astype(np.float32)
        self.w = (rng.uniform(0.5, 1.5, M) / M).astype(np.float32) if weighted else None
        lp = S.policy_loss(f64(self.H), f64(self.W), self.y, self.adv, None, None, None, 0.2, 0.2, 0.0, T)["logp"]
        self.old = (lp + rng.normal(0, 0.3, M)).astype(np.float32)
        self.ref = (lp + rng.normal(0, 0.5, M)).astype(np.float32)

    def run(self, grads=True, old=True, ref=True, lo=0.2, hi=0.28, beta=0.05, stream=None):
        def dev(a):
            return None if a is None else torch.from_numpy(a).cuda()

        gd = Guards()
        self.stats, self.logp = gd.new((4,), F32), gd.new((self.M,), F32)
        self.dH = gd.like(self.H) if grads else None
        self.dW = gd.like(self.W) if grads else None
        form = 2 if grads and self.least else int(grads)
        ws = gd.new((C.coda_lmhead_policy_workspace_bytes(self.M, self.d, self.V, form),), torch.uint8)
        self.args = (self.H, self.W, dev(self.y), dev(self.adv), dev(self.w), dev(self.old) if old else None,
                     dev(self.ref) if ref else None, lo, hi, beta, self.T, self.stats, self.logp, self.dH, self.dW, ws)
        C.coda_lmhead_policy(*self.args, stream=stream)
        gd.check("lmhead_policy")
        return S.policy_loss(f64(self.H), f64(self.W), self.y, self.adv, self.w, self.old if old else None,
                             self.ref if ref else None, lo, hi, beta, self.T)

    def grade(self, r, grads=True):
        mag = (np.abs(f64(self.H)) @ np.abs(f64(self.W)).T).max(1) / self.T
        tol = self.d * 2.0 ** -23 * mag + 2.0 ** -20
        assert (np.abs(f64(self.logp) - r["logp"]) <= tol).all()
        # the shares of the statistics move by at most |g| (and the clipped
        # weight by a token that sits on the border, of which there is none)
        g = np.abs(r["g"]).sum() + np.abs(self.w if self.w is not None else 1.0 / self.M).sum()
        assert (np.abs(f64(self.stats) - r["stats"]) <= 4 * tol.max() * g + 2.0 ** -20).all()
        if grads:
            assert_frob(self.dH, r["dH"], "dH")
            assert_frob(self.dW, r["dWt"], "dWt")
        assert_device_ok()


@pytest.mark.parametrize("M,d,V,T", [(1, 8, 8, 1.0), (5, 64, 136, 0.7), (136, 72, 1000, 1.3), (300, 128, 520, 1.0),
                                     (129, 256, 33000, 1.0)])
@pytest.mark.parametrize("old,ref", [(True, True), (False, True), (True, False), (False, False)])
def test_loss_and_gradients(M, d, V, T, old, ref):
    pb = Problem(M, d, V, T, seed=M)
    pb.grade(pb.run(old=old, ref=ref))


def test_forward_only_equals_the_full_call():
    pb = Problem(77, 64, 640, 0.9)
    pb.run(grads=False)
    a = (pb.stats.clone(), pb.logp.clone())
    pb.grade(pb.run())
    assert torch.equal(a[0], pb.stats) and torch.equal(a[1], pb.logp)
    dW = pb.dW.clone()
    pb.run()
    assert torch.equal(dW, pb.dW)              # repeatable


def test_uniform_weights_and_open_clip():
    pb = Problem(50, 64, 264, weighted=False)
    pb.grade(pb.run(lo=1.0, hi=float("inf")))
    assert pb.stats[3].item() == 0.0           # nothing is clipped
    pb.grade(pb.run(lo=0.0, hi=0.0))


def test_padding_rows_add_nothing_whatever_they_hold():
    """A padded batch: rows of weight 0 with labels of -100 and rubbish in
    every per-token input leave the other rows' results as they are."""
    pb = Problem(60, 64, 264)
    pad = np.zeros(60, bool)
    pad[[0, 7, 31, 32, 59]] = True
    pb.w[pad] = 0.0
    clean = pb.run()
    pb.grade(clean)
    got = [t.clone() for t in (pb.stats, pb.dH, pb.dW)]
    pb.y[pad] = [-100, 264, 2 ** 31 - 1, -1, 3]
    pb.adv[pad] = np.nan
    pb.old[pad], pb.ref[pad] = -np.inf, np.inf
    r = pb.run()
    pb.grade(r)
    assert all(torch.equal(a, b) for a, b in zip(got, (pb.stats, pb.dH, pb.dW)))
    assert (pb.dH[torch.from_numpy(pad).cuda()] == 0).all()


def test_all_rows_masked():
    pb = Problem(9, 64, 264)
    pb.w[:] = 0.0
    pb.run()
    assert (pb.stats == 0).all() and (pb.dH == 0).all() and (pb.dW == 0).all()
    assert_device_ok()


def test_a_bad_label_with_weight_is_reported():
    pb = Problem(40, 64, 264)
    pb.y[[3, 39]] = [264, -1]
    r = pb.run()
    st, _ = C.coda_sync_status()
    assert st == 7
    pb.grade(r)
    assert (pb.dH[3] == 0).all() and pb.logp[3].item() == 0.0


def test_narrow_chunks_give_the_same_gradients():
    pb = Problem(100, 64, 1000)
    pb.run()
    dW = pb.dW.clone()
    C.coda_set_lmhead_chunk(256)
    try:
        pb.grade(pb.run())
    finally:
        C.coda_set_lmhead_chunk(0)
    assert torch.equal(dW, pb.dW)


def test_a_workspace_serves_smaller_batches():
    """The bytes grow with the tokens, also where the number of K ranges of
    the data gradient falls."""
    for d, V in ((64, 4096), (512, 8000), (4096, 4096), (2048, 128256)):
        for grads in (False, True):
            n = [C.coda_lmhead_policy_workspace_bytes(m, d, V, grads) for m in range(1, 12000, 85)]
            assert n == sorted(n)


@pytest.mark.parametrize("M,d,V", [(700, 512, 4096), (300, 264, 2056), (40, 2048, 2048), (2600, 1024, 264)])
def test_data_gradient_in_ranges_of_the_vocabulary(M, d, V):
    pb = Problem(M, d, V)
    pb.grade(pb.run())


def _one_rounding(got, ref, what):
    """Relative Frobenius error against that of the reference itself rounded
    to bf16: the label entries of dL, the bulk of both gradients, are kept in
    fp32, so the rounding of the results is nearly all there is (a factor 1.1
    leaves room for the bf16 of the other entries and fp32 accumulation)."""
    r = torch.from_numpy(ref)
    own = (r.to(BF).double() - r).norm()
    assert (got.cpu().double() - r).norm() <= 1.1 * own, what


@pytest.mark.parametrize("M,d,V", [(60, 256, 1000), (2600, 1024, 520)])
@pytest.mark.parametrize("pairing", [True, False], ids=["sm_pair", "single_sm"])
def test_gradients_carry_one_rounding(M, d, V, pairing):
    """Advantages whose gradient factors sit just above a power of two, where
    bf16 is coarsest; V = 520 makes labels repeat (the sums per label), M =
    2600 takes the grouped launch."""
    pb = Problem(M, d, V, seed=11)
    pb.w[:] = 1.0 / 64
    pb.adv = np.where(pb.adv > 0, 1.01, -1.01).astype(np.float32)
    C.coda_set_sm_pairing(pairing)
    try:
        r = pb.run(old=False, ref=False)
    finally:
        C.coda_set_sm_pairing(True)
    assert_device_ok()
    _one_rounding(pb.dH, r["dH"], "dH")
    _one_rounding(pb.dW, r["dWt"], "dWt")


def test_every_token_has_the_same_label():
    pb = Problem(700, 64, 264)
    pb.y[:] = 77
    r = pb.run()
    pb.grade(r)
    a = pb.dW.clone()
    pb.run()
    assert torch.equal(a, pb.dW)               # the sum per label has a fixed order


def test_captured_graph():
    pb = Problem(48, 64, 520)
    pb.run()
    want = [t.clone() for t in (pb.stats, pb.logp, pb.dH, pb.dW)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        C.coda_lmhead_policy(*pb.args)
    for t in (pb.stats, pb.logp, pb.dH, pb.dW):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (pb.stats, pb.logp, pb.dH, pb.dW)))
    assert_device_ok()


def test_refusals():
    lib, h = C.load_library(), C.handle()
    st = torch.cuda.current_stream().cuda_stream
    M, d, V = 16, 64, 136
    n = C.coda_lmhead_policy_workspace_bytes(M, d, V, True)
    b = torch.zeros(max(n, 1 << 16), dtype=torch.uint8, device="cuda")
    p = ctypes.c_void_p(b.data_ptr())
    odd = ctypes.c_void_p(b.data_ptr() + 2)

    def call(H=p, y=p, adv=p, w=p, old=p, ref=p, lo=0.2, hi=0.2, beta=0.1, T=1.0, stats=p, logp=p, dH=p, dW=p, ws=p,
             n=n, M=M, d=d, V=V):
        return lib.coda_lmhead_policy(h, H, p, y, adv, w, old, ref, lo, hi, beta, T, stats, logp, dH, dW, ws, n, M, d,
                                      V, st)

    nan, inf = float("nan"), float("inf")
    assert call(H=None) == 1 and call(y=None) == 1 and call(adv=None) == 1 and call(stats=None) == 1
    assert call(logp=None) == 1 and call(dH=None) == 1 and call(dW=None) == 1 and call(ws=None) == 1
    assert call(lo=-0.1) == 1 and call(lo=1.1) == 1 and call(lo=nan) == 1 and call(hi=-0.1) == 1 and call(hi=nan) == 1
    assert call(beta=-1.0) == 1 and call(beta=nan) == 1 and call(beta=inf) == 1
    assert call(T=0.0) == 1 and call(T=inf) == 1 and call(T=nan) == 1
    least = C.coda_lmhead_policy_workspace_bytes(M, d, V, 2)
    assert call(M=0) == 1 and call(V=0) == 1 and call(d=12) == 2 and call(adv=odd) == 2 and call(n=least - 1) == 4
    assert C.coda_lmhead_policy_workspace_bytes(M, d, V, 3) == 0
    assert_device_ok()


@pytest.mark.parametrize("M", [40, 700])
def test_exponentials_past_fp32(M):
    """A ratio or a KL term that overflows fp32 stays out of what it is
    multiplied by zero in: tokens without advantage, kl_coef = 0.  The KL
    statistic itself is then an infinity, not a NaN."""
    pb = Problem(M, 64, 264)
    pb.adv[::3] = 0.0
    pb.old[::3] -= 200.0                       # r = inf at A = 0
    pb.ref[1::4] += 100.0                      # kl = e^100
    r = pb.run(beta=0.0)
    assert pb.stats[2].item() == np.inf
    pb.stats[2], r["stats"][2] = 0.0, 0.0
    pb.grade(r)
    pb = Problem(M, 64, 264)
    pb.old[5], pb.adv[5] = pb.old[5] - 200.0, -1.0   # unclipped: the loss itself overflows
    pb.run()
    assert pb.stats[0].item() == np.inf and pb.stats[1].item() == np.inf and np.isfinite(pb.stats[2].item())
    assert_device_ok()


def test_a_temperature_without_a_reciprocal_is_refused():
    pb = Problem(4, 64, 136)
    pb.T = 1e-39
    with pytest.raises(C.CodaError):
        C.coda_lmhead_policy(*pb_args(pb))
    assert_device_ok()


def pb_args(pb):
    def e(*s):
        return torch.zeros(*s, device="cuda")

    n = C.coda_lmhead_policy_workspace_bytes(pb.M, pb.d, pb.V, False)
    return (pb.H, pb.W, torch.from_numpy(pb.y).cuda(), e(pb.M), None, None, None, 0.2, 0.2, 0.0, pb.T, e(4), e(pb.M),
            None, None, torch.empty(n, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("M,d,V,T", [(1, 8, 8, 1.0), (136, 72, 1000, 1.3), (300, 128, 520, 1.0), (129, 256, 33000, 1.0),
                                     (2600, 1024, 264, 1.0)])
def test_least_workspace(M, d, V, T):
    """The logits computed a second time: the same statistics, and gradients
    within the same bounds."""
    pb = Problem(M, d, V, T, seed=M)
    pb.run()
    a = (pb.stats.clone(), pb.logp.clone())
    pb.least = True
    need = [C.coda_lmhead_policy_workspace_bytes(M, d, V, k) for k in (0, 2, 1)]
    assert need == sorted(need)
    pb.grade(pb.run())
    assert torch.equal(a[0], pb.stats) and torch.equal(a[1], pb.logp)
    C.coda_set_lmhead_chunk(256)
    try:
        pb.grade(pb.run())
    finally:
        C.coda_set_lmhead_chunk(0)


@pytest.mark.parametrize("pairing", [True, False], ids=["sm_pair", "single_sm"])
def test_least_workspace_carries_one_rounding(pairing):
    pb = Problem(60, 256, 1000, seed=11)
    pb.least = True
    pb.w[:] = 1.0 / 64
    pb.adv = np.where(pb.adv > 0, 1.01, -1.01).astype(np.float32)
    C.coda_set_sm_pairing(pairing)
    try:
        r = pb.run(old=False, ref=False)
    finally:
        C.coda_set_sm_pairing(True)
    assert_device_ok()
    _one_rounding(pb.dH, r["dH"], "dH")
    _one_rounding(pb.dW, r["dWt"], "dWt")


def test_confident_policy():
    """Probabilities near one half on the label and on another token: the
    entries beside the label's count as much as it, and are rounded twice when
    they are kept (3 2^-8 with the result's rounding bounds each element's
    terms; a third of it in the mean square)."""
    pb = Problem(96, 64, 520, seed=8)
    pb.W.zero_()
    rows = torch.randn(520, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    pb.W.copy_(rows)
    a, b = torch.from_numpy(pb.y.astype(np.int64)).cuda(), (torch.from_numpy(pb.y.astype(np.int64)).cuda() + 7) % 520
    pb.H.copy_((rows[a].float() + rows[b].float()).to(BF) * 0.5)
    for least in (False, True):
        pb.least = least
        r = pb.run(old=False, ref=False)
        assert_device_ok()
        assert_frob(pb.dH, r["dH"], "dH")
        assert_frob(pb.dW, r["dWt"], "dWt")


def test_narrow_kept_chunks():
    """Whole chunks and a last one of 232 columns, tokens not a multiple of 32."""
    pb = Problem(77, 64, 1000)
    C.coda_set_lmhead_chunk(256)
    try:
        pb.grade(pb.run())
    finally:
        C.coda_set_lmhead_chunk(0)
    dW = pb.dW.clone()
    pb.grade(pb.run())
    assert torch.equal(dW, pb.dW)
    pb = Problem(64, 64, 512)
    C.coda_set_lmhead_chunk(512)
    try:
        pb.grade(pb.run())
    finally:
        C.coda_set_lmhead_chunk(0)


def test_a_head_takes_any_number_of_tokens_up_to_its_own():
    from gemm_epilogue_transformer_tma_gb300.path import PolicyHead
    pb = Problem(700, 128, 1000, T=0.9)
    big = PolicyHead(pb.W, 700, clip=(0.2, 0.28), kl_coef=0.05, temperature=0.9)
    least = PolicyHead(pb.W, 700, clip=(0.2, 0.28), kl_coef=0.05, temperature=0.9, least_memory=True)
    assert least.ws.numel() < big.ws.numel()

    def cut(a, m):
        return torch.from_numpy(a[:m].copy()).cuda()

    for m in (40, 700, 1, 333):
        w = (pb.w[:m] * 700 / m).astype(np.float32)
        args = (pb.H[:m].contiguous(), cut(pb.y, m), cut(pb.adv, m), cut(w, m), cut(pb.old, m), cut(pb.ref, m))
        own = PolicyHead(pb.W, m, clip=(0.2, 0.28), kl_coef=0.05, temperature=0.9)
        for u, v in zip(big.step(*args), own.step(*args)):
            assert torch.equal(u, v)
        ref = S.policy_loss(f64(args[0]), f64(pb.W), pb.y[:m], pb.adv[:m], w, pb.old[:m], pb.ref[:m], 0.2, 0.28, 0.05,
                            0.9)
        _, _, dH, dW = least.step(*args)
        assert_frob(dH, ref["dH"], "dH")
        assert_frob(dW, ref["dWt"], "dWt")
    assert_device_ok()

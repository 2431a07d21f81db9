"""Distillation from a teacher's list on the LM head against its definition in
fp64, on inputs whose logits are exact in fp32 (tests/_lmhead.py).

row_loss: log q carries the rounding of an exponential's argument (relative to
|y| = |L log2(e) / T| < 64 bits: 2^-18 absolute at the farthest, and as much again
for the row's sum), weighted by |t - q| where the terms are summed as they are
here, and by at most t in the worst case: 2^-17 (P + r + 1) bounds it, and 2^-19 of the
loss its own summation.  stats: those shares times |weight|, cross-entropy with
|log q| 2^-22 more.

Gradients: dL is rounded to bf16, relative 2^-8 / sqrt(3) rms at most, dWt's
contraction meets Hs scaled and rounded once more, and both results are rounded:
sqrt(3) 2^-8 / sqrt(3) = 3.9e-3 of the norm where the terms do not cancel; the bar
of the LM head's other gradients, 5e-3."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _lmhead as R
from tests._guard import Guards
from tests._parity import assert_device_ok, assert_frob

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
MODES = [R.LISTED, R.NORMALIZED, R.TAIL]


def teacher(H, W, y, k, mode, T, seed=0, noise=0.5):
    """A list for every row: the top tokens of a teacher near the student;
    some rows end with an entry of their own for the token y, some are short,
    one is empty, and orders are mixed."""
    g = torch.Generator().manual_seed(seed)
    M, V = H.shape[0], W.shape[0]
    Lt = R.logits(H, W) + noise * torch.randn(M, V, generator=g, dtype=torch.float64).to(H.device)
    top, ids = torch.topk(Lt, k, 1)
    val = top if mode == R.NORMALIZED else top / T - torch.logsumexp(Lt / T, 1, keepdim=True)
    if k >= 3 and mode != R.NORMALIZED:
        val[::4] += np.log(0.9)
        ids[::4, -1], val[::4, -1] = y[::4].long(), np.log(0.1)
    perm = torch.randperm(k, generator=g).to(H.device)
    ids[1::3], val[1::3] = ids[1::3][:, perm], val[1::3][:, perm]
    if k >= 2:
        ids[2::5, 1:] = -1
        ids[3::7, 0] = -100
    if M > 4:
        ids[4] = -1
    w = torch.rand(M, generator=g) + 0.5
    w[torch.rand(M, generator=g) < 0.15] = 0.0
    return ids.to(I32).contiguous(), val.float().contiguous(), (w / M).to(H.device)


class Call:
    def __init__(self, H, W, ids, val, w, mode, T=1.0, grads=True):
        (M, d), V, k = H.shape, W.shape[0], ids.shape[1]
        self.H, self.W, self.ids, self.val, self.w, self.mode, self.T = H, W, ids, val, w, mode, T
        self.gd = Guards()
        self.stats, self.loss = self.gd.new((4,), F32), self.gd.new((M,), F32)
        self.dH, self.dW = (self.gd.like(H), self.gd.like(W)) if grads else (None, None)
        self.ws = self.gd.new((C.coda_lmhead_distill_workspace_bytes(M, d, V, k, grads),), torch.uint8)
        self.args = (H, W, ids, val, w, mode, T, self.stats, self.loss, self.dH, self.dW, self.ws)

    def run(self):
        C.coda_lmhead_distill(*self.args)
        self.gd.check("lmhead_distill")
        return self

    def outputs(self):
        return [t for t in (self.stats, self.loss, self.dH, self.dW) if t is not None]

    def grade(self, grads=True):
        r = R.distill(self.H, self.W, self.ids, self.val, self.w, self.mode, self.T)
        one = torch.ones_like(self.loss).double()
        used = (self.ids >= 0) & (self.ids < self.W.shape[0])
        mass = one * 2 if self.mode != R.LISTED else torch.where(used, self.val.double().exp(), 0.0).sum(1) + 1
        tol = 2.0 ** -17 * (mass + 1) + 2.0 ** -19 * r["loss"].abs()
        assert ((self.loss.double() - r["loss"]).abs() <= tol).all()
        weight = one / len(one) if self.w is None else self.w.double().abs()
        lim = (weight * tol).sum() + 2.0 ** -20 * r["stats"].abs()
        lim[1] += 2.0 ** -18 * r["stats"][1].abs()
        assert ((self.stats.double() - r["stats"]).abs() <= lim).all()
        if self.dH is not None and grads:
            assert_frob(self.dH, r["dH"].cpu().numpy(), "dH")
            assert_frob(self.dW, r["dW"].cpu().numpy(), "dWt")
        assert_device_ok()
        return r


def make(M, d, V, k, mode, T=1.0, seed=0, noise=0.5, grads=True):
    H, W, y = R.grid_inputs(M, d, V, seed=seed)
    return Call(H, W, *teacher(H, W, y, k, mode, T, seed, noise), mode, T, grads)


@pytest.mark.parametrize("M,d,V,k", [
    (1, 8, 264, 1), (5, 64, 136, 7), (33, 64, 1000, 128), (136, 72, 1000, 20), (300, 128, 520, 256),
    (129, 256, 33000, 64), (700, 512, 4096, 16), (40, 2048, 2048, 5), (2600, 1024, 264, 9), (1100, 2560, 1048, 33)])
@pytest.mark.parametrize("mode", MODES)
def test_loss_and_gradients(M, d, V, k, mode):
    make(M, d, V, k, mode, T=1.3 if k % 2 else 1.0, seed=M).run().grade()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [50, 200])
def test_forward_only_equals_the_full_call(mode, M):
    c = make(M, 64, 3000, 20, mode).run()
    f = Call(c.H, c.W, c.ids, c.val, c.w, mode, grads=False).run()
    f.grade()
    assert torch.equal(c.stats, f.stats) and torch.equal(c.loss, f.loss)
    C.coda_lmhead_distill(*f.args[:8], None, *f.args[9:])      # without row losses
    assert torch.equal(c.stats, f.stats)
    again = [t.clone() for t in c.outputs()]
    c.run()
    assert all(torch.equal(a, b) for a, b in zip(again, c.outputs()))


@pytest.mark.parametrize("M,d,V,k", [(1, 256, 9000, 1), (1, 256, 520, 40), (7, 256, 9000, 3), (40, 1024, 1000, 20),
                                     (64, 512, 9000, 64), (65, 512, 9000, 20), (700, 512, 4096, 16),
                                     (1100, 2560, 1048, 33)])
@pytest.mark.parametrize("mode", MODES)
def test_a_largest_entry_that_outweighs_its_row_is_not_rounded(M, d, V, k, mode):
    """dH carries one rounding, and dW up to 64 rows; of more, dW also that of
    the scaled Hs, half a step (2^-8) of each of its products: a bound, as rows that
    are few and values of Hs that repeat do not average.  The other entries of dL
    are rounded once or twice: half a step each, of independent signs."""
    c = make(M, d, V, k, mode, seed=M + k).run()
    r = c.grade()
    dL, H, W = r["dL"], c.H.double(), c.W.double()
    rest = dL.scatter(1, dL.abs().argmax(1, keepdim=True), 0.0).abs()
    for got, ref, others, scaled in ((c.dH, r["dH"], rest ** 2 @ W ** 2, None),
                                     (c.dW, r["dW"], (rest ** 2).t() @ H ** 2, dL.abs().t() @ H.abs())):
        one = (ref.to(BF).double() - ref).norm()
        bar = ((1.02 * one) ** 2 + 2 * 2.0 ** -16 * others.sum()).sqrt()
        if scaled is not None and M > 64:
            bar += 2.0 ** -8 * scaled.norm()
        assert (got.double() - ref).norm() <= bar


@pytest.mark.parametrize("M", [6, 200])
@pytest.mark.parametrize("mode", MODES)
def test_small_masses_keep_their_digits(mode, M):
    """Teachers and students whose lists hold a thousandth of the probability:
    the loss, far below the logarithms it is made of, and the cross-entropy of a
    tail that is nearly everything.  Terms of one sign, or taken as they are:
    relative 2^-18 of each."""
    V, k = 20000, 4
    H, W, y = R.grid_inputs(M, 64, V, sure=0.5, seed=M)
    H = (H.float() / 4).to(BF)
    ids = torch.randint(0, V, (M, k), generator=torch.Generator().manual_seed(2)).to(I32).cuda()
    lq = torch.log_softmax(R.logits(H, W), 1).gather(1, ids.long())
    val = (lq + 0.7 * torch.randn(M, k, generator=torch.Generator().manual_seed(3)).cuda()).float()
    c = Call(H, W, ids, val, torch.full((M,), 1 / M, device="cuda"), mode, grads=False).run()
    r = R.distill(H, W, ids, val, c.w, mode)
    t = (torch.softmax(val.double(), 1) if mode == R.NORMALIZED else val.double().exp())
    size = (t * (val.double() - lq).abs()).sum(1) + (t - lq.exp()).abs().sum(1)
    assert ((c.loss.double() - r["loss"]).abs() <= 2.0 ** -18 * size + 2.0 ** -22 * r["loss"].abs() + 1e-12).all()
    assert ((c.stats.double() - r["stats"]).abs() <= 2.0 ** -18 * r["stats"].abs() + 2.0 ** -18 * size.mean()).all()


def test_single_sm_gemms():
    c = make(1100, 2560, 1048, 33, R.TAIL)
    C.coda_set_sm_pairing(False)
    try:
        c.run().grade()
    finally:
        C.coda_set_sm_pairing(True)


def test_uniform_weight():
    c = make(70, 64, 1000, 6, R.TAIL)
    c.w = None
    c.args = c.args[:4] + (None,) + c.args[5:]
    c.run().grade()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [60, 1200])
def test_padding_rows_add_nothing_whatever_they_hold(mode, M):
    c = make(M, 64 if M < 1000 else 2560, 264, 7, mode).run()
    c.grade()
    want = [t.clone() for t in c.outputs()]
    pad = c.w == 0
    assert pad.any()
    c.ids[pad], c.val[pad] = 2 ** 31 - 1, float("nan")
    c.H[pad] = float("nan")
    c.run()
    assert_device_ok()
    assert all(torch.equal(a, b) for a, b in zip(want, c.outputs()))
    assert (c.dH[pad] == 0).all() and (c.loss[pad] == 0).all()
    c.w.zero_()
    c.run()
    assert all((t == 0).all() for t in c.outputs())
    assert_device_ok()


@pytest.mark.parametrize("mode", MODES)
def test_rows_without_entries(mode):
    c = make(20, 64, 264, 4, mode)
    c.ids.fill_(-1)
    c.run()
    if mode == R.TAIL:   # all tokens are the tail: r = R = 1
        assert c.loss.abs().max() <= 2.0 ** -22 and c.dH.float().abs().max() <= 2.0 ** -20
    else:
        assert (c.loss == 0).all() and (c.dH == 0).all() and (c.dW == 0).all()
    assert_device_ok()


@pytest.mark.parametrize("mode", [R.LISTED, R.TAIL])
@pytest.mark.parametrize("M", [24, 200])
def test_targets_of_zero(mode, M):
    """Entries with a probability of 0, or one that fp32 does not hold, in all of
    a row's list: with LISTED nothing is asked of the row, with TAIL all of it off
    the list."""
    c = make(M, 64, 264, 4, mode)
    c.ids.copy_((torch.arange(M, device="cuda")[:, None] + 50 * torch.arange(4, device="cuda")[None]).to(I32))
    for i, v in enumerate([-float("inf"), torch.finfo(F32).min, -200.0]):
        c.val[i::4] = v
    c.run()
    # tokens up to M - 1 + 150: of 200 rows some lie outside the vocabulary
    assert C.coda_sync_status()[0] == (7 if M == 200 else 0)
    r = c.grade()
    assert torch.isfinite(c.dH.float()).all() and torch.isfinite(c.dW.float()).all()
    if mode == R.LISTED:
        none = torch.arange(M, device="cuda") % 4 < 3
        assert (c.loss[none] == 0).all() and (c.dH[none] == 0).all()
        assert r["dL"][none].abs().max() < 1e-80


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [24, 200])
def test_a_student_beyond_doubt_of_its_label(mode, M):
    """All of the target on one token, which the student has at 1 - e^-200: what
    is left of the gradient is below fp32, and is 0."""
    H = torch.zeros(M, 64, device="cuda")
    W = torch.zeros(1000, 64, device="cuda")
    H[:, 0], H[:, 1] = 1.0, torch.arange(M, device="cuda") % 16 / 8.0
    W[7, 0], W[:, 1] = 200.0, torch.arange(1000, device="cuda") % 8 / 8.0
    ids = torch.tensor([[3, 7]], dtype=I32, device="cuda").repeat(M, 1)
    val = torch.tensor([[-float("inf"), 0.0]], device="cuda").repeat(M, 1)
    c = Call(H.to(BF), W.to(BF), ids, val, None, mode).run()
    assert (c.loss.abs() <= 2.0 ** -20).all()
    assert (c.dH == 0).all() and (c.dW == 0).all()
    assert_device_ok()


def test_a_token_outside_the_vocabulary_is_reported():
    c = make(40, 64, 264, 4, R.TAIL)
    live = int(torch.nonzero(c.w != 0)[5])
    c.ids[live, 2] = 264
    c.run()
    assert C.coda_sync_status()[0] == 7
    c.grade()


@pytest.mark.parametrize("mode", [R.LISTED, R.TAIL])
def test_the_whole_vocabulary_listed(mode):
    """No token off the list: the tail's term is left out."""
    c = make(12, 64, 136, 136, mode)
    c.run()
    r = R.distill(c.H, c.W, c.ids, c.val, c.w, R.LISTED)
    full = ((c.ids >= 0) & (c.ids < 136)).all(1) & (torch.sort(c.ids, 1).values.diff(dim=1) > 0).all(1)
    assert full.any()
    assert ((c.loss.double() - r["loss"]).abs() <= 2.0 ** -15)[full].all()
    assert_frob(c.dH[full], r["dH"][full].cpu().numpy(), "dH")
    if mode == R.LISTED:
        c.grade()
    assert_device_ok()


@pytest.mark.parametrize("noise", [0.0, 2.0 ** -10])
def test_a_student_near_its_teacher(noise):
    """The loss is a square of the difference: it keeps its relative precision
    down to losses of 1e-7, and gradients stay near the formula's."""
    M, V, k = 64, 3000, 30
    H, W, y = R.grid_inputs(M, 64, V, seed=3)
    w = teacher(H, W, y, k, R.TAIL, 1.0, 3)[2]
    L = R.logits(H, W)
    g = torch.Generator().manual_seed(1)
    Lt = L + noise * torch.randn(M, V, generator=g, dtype=torch.float64).cuda()
    top, t = torch.topk(Lt, k, 1)
    ids, val = t.to(I32), (top - torch.logsumexp(Lt, 1, keepdim=True)).float()
    c = Call(H, W, ids, val, w, R.TAIL).run()
    r = R.distill(H, W, ids, val, w, R.TAIL)
    live = w != 0
    # a difference |t - q| of noise t, off by 2^-19 t: relative 2 2^-19 / noise of the square
    bar = 2.0 ** -40 + (2.0 ** -18 / noise * r["loss"] if noise else 0.0)
    assert ((c.loss.double() - r["loss"]).abs() <= bar)[live].all()
    if noise:
        # dL is a difference of t and q: 2^-19 of them, 2^-9 of noise, beside its own rounding
        assert_frob(c.dH, r["dH"].cpu().numpy(), "dH")
    assert_device_ok()


@pytest.mark.parametrize("T", [1.0, 1.3])
@pytest.mark.parametrize("M", [40, 300])
def test_a_difference_within_the_list_keeps_its_digits(M, T):
    """Two tokens' targets moved by 2^-8 of the smaller one, against each other, so
    that the list's mass stays: the loss, 2^-17 of that target and more, is made of the
    differences alone.  The exponentials off the list may be off by 2^-21 together,
    which the loss meets times R - r; the list's and their quotients by 2^-34, times
    the 2^-8 of their logarithms' ratio; sums and logarithms by 2^-20 of the loss."""
    H, W, _ = R.grid_inputs(M, 64, 2000, seed=9)
    q = torch.softmax(R.logits(H, W) / T, 1)
    top, ids = torch.topk(q, 2, 1)
    step = top[:, 1] * 2.0 ** -8
    val = torch.stack([top[:, 0] + step, top[:, 1] - step], 1).log().float()
    c = Call(H, W, ids.to(I32), val, None, R.TAIL, T).run()
    r = R.distill(H, W, c.ids, val, None, R.TAIL, float(np.float32(T)))  # the temperature of the call
    apart = (top.sum(1) - val.double().exp().sum(1)).abs()
    bar = 2.0 ** -20 * r["loss"] + 2.0 ** -21 * apart + 2.0 ** -41
    assert ((c.loss.double() - r["loss"]).abs() <= bar).all()
    assert_device_ok()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("gap", [50.0, 200.0])
def test_logits_far_from_the_listed_ones(mode, gap):
    """Rows whose unlisted logits lie far above or below those of the list, in
    part or all of the vocabulary: blocks at a scale of their own."""
    M, V, k = 24, 1000, 5
    H = torch.zeros(M, 64, device="cuda")
    W = torch.zeros(V, 64, device="cuda")
    v = torch.arange(V, device="cuda")
    W[:, 0] = (v % 7) / 8.0
    W[:, 1] = (v >= 500).float()
    W[:, 2] = (v < k).float()
    W[:, 3] = torch.randint(-8, 8, (V,), generator=torch.Generator().manual_seed(0)).cuda() / 8.0
    H[:, 0], H[:, 3] = 1.0, 0.5
    H[0::4, 1] = gap      # the upper half above the list
    H[1::4, 1] = -gap     # below it
    H[2::4, 2] = gap      # the list above all others
    H[3::4, 2] = -gap     # below
    H[:, 4] = torch.arange(M, device="cuda") / 8.0
    H, W = H.to(BF), W.to(BF)
    ids = torch.arange(k, dtype=I32, device="cuda").expand(M, k).contiguous()
    val = torch.log(torch.tensor([0.4, 0.2, 0.1, 0.05, 0.05], device="cuda")).expand(M, k).contiguous()
    c = Call(H, W, ids, val, torch.full((M,), 1 / M, device="cuda"), mode).run()
    r = R.distill(H, W, ids, val, c.w, mode)
    # |log q| up to gap: relative 2^-18 of each term
    assert ((c.loss.double() - r["loss"]).abs() <= 2.0 ** -17 * (r["loss"].abs() + 2)).all()
    for i in range(4):
        assert_frob(c.dH[i::4], r["dH"][i::4].cpu().numpy(), f"dH {i}")
    assert_frob(c.dW, r["dW"].cpu().numpy(), "dWt")
    assert_device_ok()


@pytest.mark.parametrize("M", [40, 1100])
def test_nan_of_a_weighted_row(M):
    d = 64 if M < 1000 else 2560
    c = make(M, d, 264, 4, R.TAIL).run()
    dH, loss = c.dH.clone(), c.loss.clone()
    t = int(torch.nonzero(c.w != 0)[9])
    keep = torch.arange(M, device="cuda") != t
    for what in ("H", "val"):
        H, val = c.H.clone(), c.val.clone()
        if what == "H":
            H[t] = float("nan")
        else:
            val[t] = float("nan")
            if not (c.ids[t] >= 0).any():
                continue
        x = Call(H, c.W, c.ids, val, c.w, R.TAIL).run()
        assert torch.equal(x.dH[keep], dH[keep]) and torch.equal(x.loss[keep], loss[keep])
        assert torch.isnan(x.loss[t]) and torch.isnan(x.stats[0]) and torch.isnan(x.dH[t]).all()
        assert torch.isnan(x.dW).any()
    assert_device_ok()


@pytest.mark.parametrize("V", [1816, 1864], ids=["one_block", "three_blocks"])
def test_tiles_behind_a_ragged_vocabulary(V):
    """17 x 8 tiles on fewer SM pairs: pairs that take the last vocabulary
    tile, with an odd number of 32 wide stores, go on to tiles of the next rows."""
    c = make(4128, 64, V, 5, R.TAIL).run()
    r = R.distill(c.H, c.W, c.ids, c.val, c.w, R.TAIL)
    got, ref = c.dH.double().reshape(-1, 32, 64), r["dH"].reshape(-1, 32, 64)
    assert ((got - ref).norm(dim=(1, 2)) <= 5e-3 * ref.norm(dim=(1, 2))).all()
    assert_frob(c.dW, r["dW"].cpu().numpy(), "dWt")
    assert_device_ok()


@pytest.mark.parametrize("M,d", [(48, 64), (1100, 2560)])
def test_captured_graph_and_other_stream(M, d):
    c = make(M, d, 520, 6, R.TAIL).run()
    want = [t.clone() for t in c.outputs()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        C.coda_lmhead_distill(*c.args)
    for t in c.outputs():
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, c.outputs()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in c.outputs():
        t.zero_()
    with torch.cuda.stream(s):
        C.coda_lmhead_distill(*c.args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, c.outputs()))
    assert_device_ok()


@pytest.mark.parametrize("M,d", [(100, 64), (1100, 2560)])
def test_a_workspace_aligned_to_16_bytes_serves_smaller_batches(M, d):
    c = make(M, d, 520, 6, R.TAIL).run()
    big = torch.empty(C.coda_lmhead_distill_workspace_bytes(M + 300, d, 520, 6, True) + 16, dtype=torch.uint8,
                      device="cuda")[16:]
    want = [t.clone() for t in c.outputs()]
    C.coda_lmhead_distill(*c.args[:-1], big)
    assert all(torch.equal(a, b) for a, b in zip(want, c.outputs()))
    assert_device_ok()


def test_two_streams_with_workspaces_of_their_own():
    """Calls that overlap on the GPU."""
    calls = [make(136, 1024, 4096, 9, R.TAIL, seed=s) for s in range(3)] + [make(1100, 2560, 1048, 5, R.TAIL)]
    want = [[t.clone() for t in c.run().outputs()] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for c in calls:
        for t in c.outputs():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                C.coda_lmhead_distill(*c.args)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(w, c.outputs()))
    assert_device_ok()


def test_from_a_teachers_scores_to_a_students_gradients():
    """A ScoringHead's lists go into a DistillHead as they are."""
    from gemm_epilogue_transformer_tma_gb300.path import DistillHead, ScoringHead
    Ht, Wt, y = R.grid_inputs(150, 128, 2000, seed=1)
    Hs, Ws, _ = R.grid_inputs(150, 64, 2000, seed=2)
    _, _, ids, top = ScoringHead(Wt, 256, k=20).score(Ht, y)
    head = DistillHead(Ws, 256, 20)
    w = torch.full((150,), 1 / 150, device="cuda")
    stats, loss, dH, dW = head.step(Hs, ids, top, w)
    r = R.distill(Hs, Ws, ids, top, w, R.TAIL)
    assert ((loss.double() - r["loss"]).abs() <= 2.0 ** -15 * (1 + r["loss"])).all()
    assert_frob(dH, r["dH"].cpu().numpy(), "dH")
    assert_frob(dW, r["dW"].cpu().numpy(), "dWt")
    f = DistillHead(Ws, 150, 20, backward=False).step(Hs, ids, top, w)
    assert torch.equal(f[1], loss) and f[2] is None and f[3] is None
    assert_device_ok()


def test_gradients_against_differences():
    """The step along dH lowers the loss by |dH|^2."""
    c = make(30, 64, 520, 8, R.TAIL, seed=4).run()
    r = R.distill(c.H, c.W, c.ids, c.val, c.w, R.TAIL)
    H = c.H.double()
    step = 1e-4 / c.dH.double().norm()

    def loss(x):
        keep = R.logits
        try:
            R.logits = lambda a, b: x @ c.W.double().t()
            return R.distill(c.H, c.W, c.ids, c.val, c.w, R.TAIL)["stats"][0].item()
        finally:
            R.logits = keep

    slope = (loss(H + step * c.dH.double()) - loss(H - step * c.dH.double())) / (2 * step.item())
    assert abs(slope / (c.dH.double() * r["dH"]).sum().item() - 1) < 1e-3


def test_refusals():
    lib, h = C.load_library(), C.handle()
    st = torch.cuda.current_stream().cuda_stream
    M, d, V, k = 16, 64, 136, 4
    n = C.coda_lmhead_distill_workspace_bytes(M, d, V, k, True)
    f = C.coda_lmhead_distill_workspace_bytes(M, d, V, k, False)
    b = torch.zeros(max(n, 1 << 16), dtype=torch.uint8, device="cuda")
    p = ctypes.c_void_p(b.data_ptr())
    odd = ctypes.c_void_p(b.data_ptr() + 2)

    def call(**kw):
        a = dict(H=p, W=p, ids=p, val=p, w=p, mode=2, T=1.0, stats=p, loss=p, dH=p, dW=p, k=k, ws=p, n=n, M=M, d=d, V=V)
        a.update(kw)
        return lib.coda_lmhead_distill(h, *(a[x] for x in ("H", "W", "ids", "val", "w", "mode", "T", "stats", "loss",
                                                           "dH", "dW", "k", "ws", "n", "M", "d", "V")), st)

    for kw, want in [(dict(H=None), 1), (dict(W=None), 1), (dict(ids=None), 1), (dict(val=None), 1),
                     (dict(stats=None), 1), (dict(ws=None), 1), (dict(dH=None), 1), (dict(dW=None), 1),
                     (dict(k=0), 1), (dict(k=257), 1), (dict(mode=3), 1), (dict(mode=-1), 1), (dict(M=0), 1),
                     (dict(M=-1), 1), (dict(T=0.0), 1), (dict(T=float("inf")), 1), (dict(T=1e-39), 1),
                     (dict(T=float("nan")), 1), (dict(d=60), 2), (dict(V=140), 2), (dict(H=odd), 2), (dict(ids=odd), 2),
                     (dict(loss=odd), 2), (dict(n=n - 1), 4), (dict(n=f - 1, dH=None, dW=None), 4)]:
        assert call(**kw) == want, kw
    c = make(M, d, V, k, R.TAIL)
    for i, bad in ((0, c.H.float()), (2, c.ids.long()), (3, c.val[:, :2]), (4, c.w[:3]), (5, 2 ** 40), (9, None),
                   (11, c.ws.cpu())):
        a = list(c.args)
        a[i] = bad
        with pytest.raises((ValueError, TypeError, C.CodaError)):
            C.coda_lmhead_distill(*a)
    assert_device_ok()


def test_a_temperature_without_its_power_of_two_is_refused():
    """1 / 4e-39 is an fp32 number, log2(e) / 4e-39 is not."""
    c = make(16, 64, 136, 4, R.TAIL)
    for T, fine in ((4e-39, False), (5e-39, True)):
        a = list(c.args)
        a[6] = T
        if fine:
            C.coda_lmhead_distill(*a)
        else:
            with pytest.raises(C.CodaError):
                C.coda_lmhead_distill(*a)
    assert_device_ok()

"""The post-training step's operators as they are used together: a QKV
projection on block-scaled codes, the head norm with RoPE, the policy loss on
the LM head over the rotated queries, and the gradients back to the input and
every weight.  Each stage is graded on its own inputs as the GPU left them;
the chain end to end against fp64 without any 8-bit rounding, by the error its
codes bring."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as S
from tests._parity import assert_device_ok, f64, frob_err

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")
from gemm_epilogue_transformer_tma_gb300.path import BlockScaledLinear, PolicyHead, QKVProjection  # noqa: E402

BF = torch.bfloat16
NQ, NK, D, d, V, SEQ = 4, 2, 64, 320, 1000, 96


def _bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(BF).cuda()


class Step:
    def __init__(self, M, seed=0):
        rng = np.random.default_rng(seed)
        self.X = _bf(rng.standard_normal((M, d)))
        self.W = _bf(rng.standard_normal(((NQ + 2 * NK) * D, d)) * 0.05)
        self.gq, self.gk = _bf(rng.uniform(0.5, 1.5, D)), _bf(rng.uniform(0.5, 1.5, D))
        self.Wt = _bf(rng.standard_normal((V, NQ * D)) * 0.05)
        self.pos = rng.integers(0, SEQ, M).astype(np.int32)
        self.y = rng.integers(0, V, M).astype(np.int32)
        self.adv = rng.standard_normal(M).astype(np.float32)
        w = (rng.random(M) < 0.8).astype(np.float32)
        self.w = w / max(w.sum(), 1.0)
        self.old = (-np.log(V) + rng.normal(0, 0.5, M)).astype(np.float32)
        self.dev = [torch.from_numpy(a).cuda() for a in (self.pos, self.y, self.adv, self.w, self.old)]
        self.proj = QKVProjection(self.W, self.gq, self.gk, NQ, NK, M, SEQ)
        self.head = PolicyHead(self.Wt, M, clip=(0.2, 0.28), temperature=0.9)
        self.H = torch.empty(M, NQ * D, dtype=BF, device="cuda")
        self.dout = torch.zeros(M, (NQ + 2 * NK) * D, dtype=BF, device="cuda")

    def run(self):
        pos, y, adv, w, old = self.dev
        self.out = self.proj.forward(self.X, pos)
        self.H.copy_(self.out[:, :NQ * D])           # stands in for the attention between them
        self.stats, self.logp, dH, self.dWt = self.head.step(self.H, y, adv, w, old)
        self.dout[:, :NQ * D] = dH
        self.dX, self.dW, self.dgq, self.dgk = self.proj.backward(self.dout)
        return [self.out, self.stats, self.logp, self.dWt, self.dX, self.dW, self.dgq, self.dgk]


@pytest.mark.parametrize("M", [1, 63, 300, 777])
def test_a_step_stage_by_stage_and_end_to_end(M):
    s = Step(M, seed=M)
    s.run()
    assert_device_ok()
    gq, gk = f64(s.gq), f64(s.gk)
    x, w, y = f64(s.X), f64(s.W), f64(s.proj.linear.Y)

    def deq(v, rb, cb, fmt="e4m3"):
        return S.block_dequantize(*S.block_quantize(v, rb, cb, fmt), rb, cb, fmt)

    def near(got, ref, mag, k):     # one bf16 rounding, k fp32 accumulations
        assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -23 * mag + 1e-30).all()

    xd, wd = deq(x, 1, 128), deq(w, 128, 128)
    near(s.proj.linear.Y, xd @ wd.T, np.abs(xd) @ np.abs(wd).T, d)
    r = S.qknorm_rope(y, gq, gk, s.pos, NQ, NK, D, 1e-6)
    assert np.abs(f64(s.out) - r).max() <= 2.0 ** -8 * np.abs(r).max()
    ref = S.policy_loss(f64(s.H), f64(s.Wt), s.y, s.adv, s.w, s.old, None, 0.2, 0.28, 0.0, 0.9)
    assert np.abs(f64(s.logp) - ref["logp"]).max() < 1e-4
    assert np.abs(f64(s.stats) - ref["stats"]).max() < 1e-3
    dx, rq, rk = S.qknorm_rope_backward(y, f64(s.dout), gq, gk, s.pos, NQ, NK, D, 1e-6)
    dq = f64(s.proj.dqkv[:M])
    assert np.linalg.norm(dq - dx) <= 2.0 ** -8 * np.linalg.norm(dx) + 1e-12
    assert np.allclose(f64(s.dgq), rq, rtol=1e-3, atol=1e-6) and (f64(s.dgk) == 0).all() and (rk == 0).all()
    gd, gc, xc = deq(dq, 1, 128, "e5m2"), deq(dq, 128, 1, "e5m2"), deq(x, 128, 1)
    near(s.dX, gd @ wd, np.abs(gd) @ np.abs(wd), s.W.shape[0])
    near(s.dW, gc.T @ xc, np.abs(gc).T @ np.abs(xc), M)

    # without codes: e4m3 rounds to 2^-4 / sqrt(3) = 3.6 % rms at most, e5m2
    # to 7.2 %; two e4m3 operands give qkv 5.1 %, which the norm and the head
    # pass on to dout (twice: through H and through r), and the gradient's own
    # codes and the other operand add in quadrature: below 20 %
    e = x @ w.T
    eo = S.qknorm_rope(e, gq, gk, s.pos, NQ, NK, D, 1e-6)
    assert frob_err(s.out, eo) < 0.06
    er = S.policy_loss(eo[:, :NQ * D], f64(s.Wt), s.y, s.adv, s.w, s.old, None, 0.2, 0.28, 0.0, 0.9)
    if M >= 63:     # a token near a clip border decides between a gradient and none
        same = (er["g"] != 0) == (ref["g"] != 0)
        assert same.mean() > 0.9
        if same.all():
            ed = np.concatenate([er["dH"], np.zeros((M, 2 * NK * D))], 1)
            eg, _, _ = S.qknorm_rope_backward(e, ed, gq, gk, s.pos, NQ, NK, D, 1e-6)
            assert frob_err(s.dX, eg @ w) < 0.2 and frob_err(s.dW, eg.T @ x) < 0.2


def test_a_step_repeats_and_replays_bit_for_bit():
    s = Step(200)
    want = [t.clone() for t in s.run()]
    again = s.run()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = s.run()
    for t in outs:
        t.zero_()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    assert_device_ok()


def test_two_steps_on_two_streams():
    """Two steps with their own buffers, interleaved on two streams, give the
    bits each gives alone."""
    a, b = Step(150, 1), Step(260, 2)
    want = [[t.clone() for t in s.run()] for s in (a, b)]
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            ra = a.run()
        with torch.cuda.stream(sb):
            rb = b.run()
    torch.cuda.synchronize()
    for w, r in zip(want, (ra, rb)):
        assert all(torch.equal(x, y) for x, y in zip(w, r))
    assert_device_ok()


def test_linear_layer_takes_any_number_of_tokens_up_to_its_own():
    """A layer sized for 300 tokens fed 5, 300 and none in turn: the results
    of layers sized for each, and an empty weight gradient."""
    W = _bf(np.random.default_rng(0).standard_normal((144, 272)) * 0.05)
    big = BlockScaledLinear(W, 300)
    for m in (5, 300, 1, 128):
        x, dy = torch.randn(m, 272, device="cuda").to(BF), torch.randn(m, 144, device="cuda").to(BF)
        own = BlockScaledLinear(W, m)
        for u, v in zip((big.forward(x), *big.backward(dy)), (own.forward(x), *own.backward(dy))):
            assert torch.equal(u, v)
    x = torch.empty(0, 272, dtype=BF, device="cuda")
    assert big.forward(x).shape == (0, 144)
    dX, dW = big.backward(torch.empty(0, 144, dtype=BF, device="cuda"))
    assert dX.shape == (0, 272) and (dW == 0).all()
    assert_device_ok()

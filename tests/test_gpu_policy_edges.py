"""The policy loss where its epilogues, row kernels and roundings meet their
limits: ragged vocabularies behind many tiles."""
import numpy as np
import pytest
import torch

from tests._parity import assert_device_ok, assert_frob, f64
from tests.test_gpu_policy import Problem

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")


@pytest.mark.parametrize("V", [1816, 1864], ids=["one_block", "three_blocks"])
def test_tiles_behind_a_ragged_vocabulary(V):
    """17 x 8 tiles on fewer SM pairs: the pairs that take the last, ragged
    vocabulary tile (24 or 72 columns of a block of 128: an odd number of 32
    wide stores) go on to tiles of the next rows.  Nearly all probability lies
    in those columns, so that a stored block which another one replaced shows
    in the 32 rows it belongs to.  Bar per 32 rows: three roundings to bf16
    (kept exponential, dL, result) of 2^-8 / sqrt(3) rms each, 3.9e-3."""
    pb = Problem(4128, 64, V, seed=V)
    pb.W[1792:] *= 8
    r = pb.run(old=False, ref=False)
    assert_device_ok()
    got = f64(pb.dH).reshape(-1, 32, 64)
    ref = r["dH"].reshape(-1, 32, 64)
    err = np.linalg.norm(got - ref, axis=(1, 2)) / np.linalg.norm(ref, axis=(1, 2))
    assert err.max() <= 5e-3, err.argmax()
    assert_frob(pb.dW, r["dWt"], "dWt")
    want = (pb.dH.clone(), pb.dW.clone())
    pb.run(old=False, ref=False)
    assert torch.equal(want[0], pb.dH) and torch.equal(want[1], pb.dW)

"""Workspace sizes of scoring and distillation and the refusals that need no
device."""
import ctypes

import pytest

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

SHAPES = [(64, 8), (64, 1000), (4096, 4096), (2048, 128256), (1024, 32000), (64, 1048576)]


@pytest.mark.parametrize("d,V", SHAPES)
def test_score_workspace(d, V):
    """It grows with the rows, so one serves fewer rows too, up to the rows that
    2 GB of logits hold (256 at least); no alternatives need the least."""
    need = C.coda_lmhead_score_workspace_bytes
    rows = sorted(set(range(1, 400)) | set(range(400, 40000, 377)))
    for k in (0, 1, min(V, 256)):
        sizes = [need(m, d, V, k) for m in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0
        if k:
            held = max(256, 2 ** 29 // V)
            assert need(40000, d, V, k) <= 4 * held * V + 40 * held * (V // 128 + 153) + 4096
            assert sizes[-1] > need(rows[-1], d, V, 0) or held < rows[-1]
    assert need(0, d, V, 0) == need(8, 0, V, 0) == need(8, d, 0, 0) == need(-1, d, V, 0) == 0
    assert need(8, d, V, -1) == need(8, d, V, 257) == need(8, d, V, V + 1) == 0


@pytest.mark.parametrize("d,V", SHAPES)
def test_distill_workspace(d, V):
    need = C.coda_lmhead_distill_workspace_bytes
    for k in (1, 33, 256):
        for grads in (False, True):
            sizes = [need(m, d, V, k, grads) for m in range(1, 20000, 61)]
            assert sizes == sorted(sizes) and sizes[0] > 0
        assert need(100, d, V, k, True) >= need(100, d, V, k, False) + 200 * (V + d)
    for bad in ((0, d, V, 1), (1, 0, V, 1), (1, d, 0, 1), (1, d, V, 0), (1, d, V, 257), (-5, d, V, 1)):
        assert need(*bad, False) == 0


def test_a_null_handle_is_refused():
    lib = C.load_library()
    p = ctypes.c_void_p(256)
    assert lib.coda_lmhead_score(None, p, p, p, 1.0, p, p, p, p, 1, p, 1 << 20, 2, 8, 8, None) == 1
    assert lib.coda_lmhead_distill(None, p, p, p, p, p, 2, 1.0, p, p, p, p, 1, p, 1 << 20, 2, 8, 8, None) == 1

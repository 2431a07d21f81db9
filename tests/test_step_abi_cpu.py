"""Workspace sizes of the post-training operators and the refusals that need no
device (the library loads and answers these without one)."""
import ctypes

import pytest

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

SHAPES = [(64, 4096), (4096, 4096), (2048, 128256), (1024, 32000), (64, 33000)]


@pytest.mark.parametrize("d,V", SHAPES)
def test_policy_workspace(d, V):
    """Every form grows with the tokens, so a workspace serves fewer tokens
    too; the forms are ordered; what is kept stays within 1 GB of 2-byte
    values."""
    need = C.coda_lmhead_policy_workspace_bytes
    sizes = {k: [need(m, d, V, k) for m in range(1, 40000, 37)] for k in (0, 1, 2)}
    for k in (0, 1, 2):
        assert sizes[k] == sorted(sizes[k]) and sizes[k][0] > 0
    assert all(a < b <= c for a, b, c in zip(sizes[0], sizes[2], sizes[1]))
    assert max(c - b for b, c in zip(sizes[2], sizes[1])) <= 2 ** 30 + 256
    assert need(0, d, V, 1) == 0 and need(8, 0, V, 1) == 0 and need(8, d, 0, 1) == 0
    assert need(8, d, V, 3) == 0 and need(8, d, V, -1) == 0
    assert need(8, d, V, True) == need(8, d, V, 1)


def test_scale_bytes_and_head_workspace():
    b = C.coda_fp8_block_scale_bytes
    assert b(1, 1) == 512 and b(128, 512) == 512 and b(129, 512) == 1024 and b(128, 513) == 1024
    assert b(0, 128) == 0 and b(128, 0) == 0 and b(-1, 8) == 0
    w = C.coda_qknorm_rope_bwd_workspace_bytes
    assert w(0, 128) == 0 and w(8, 0) == 0 and w(8, 528) == 0 and w(1, 128) == w(10 ** 6, 128) > 0


def test_a_null_handle_is_refused():
    lib = C.load_library()
    p = ctypes.c_void_p(256)
    assert lib.coda_qknorm_rope(None, p, p, p, p, p, None, p, 2, 2, 1, 64, 4, 1e-6, None) == 1
    assert lib.coda_fp8_block_quantize(None, p, 0, p, p, None, None, 2, 16, None) == 1
    assert lib.coda_gemm_fp8_block(None, p, 0, 0, p, p, 0, 0, p, p, 2, 16, 16, None) == 1
    assert lib.coda_lmhead_policy(None, p, p, p, p, p, p, p, 0.2, 0.2, 0.0, 1.0, p, p, None, None, p, 1 << 20, 2, 8, 8,
                                  None) == 1

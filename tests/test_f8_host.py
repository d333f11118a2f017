"""The 8-bit entry points without a GPU: bad arguments are rejected on the host
before anything is enqueued (these calls never reach a launch)."""
import pytest

A32 = 0x7F0000000000          # a fake device address, 32-byte aligned, never read


@pytest.fixture(scope="module")
def L():
    from microscaling_fp4_quantization_block_b200 import build
    build.build()
    import microscaling_fp4_quantization_block_b200 as m
    return m.lib()


def test_f8_quantize_rejects_bad_arguments(L):
    q = L.fp4q_f8_quantize
    assert q(A32, -1, 64, 0, A32, A32, None) == -2
    assert q(A32, 4, 24, 0, A32, A32, None) == -2                    # cols % 16
    assert q(A32, 4, 64, 2, A32, A32, None) == -4                    # no such grain
    assert q(A32, 1 << 60, 1 << 10, 0, A32, A32, None) == -2         # rows * cols overflows
    assert q(A32, 1 << 50, 16, 0, A32, A32, None) == -2              # more groups than a grid holds
    assert q(A32, 1 << 50, 16, 1, A32, A32, None) == -2
    for bad in ((None, A32, A32), (A32, None, A32), (A32, A32, None)):
        assert q(bad[0], 4, 64, 0, bad[1], bad[2], None) == -1
    assert q(A32 + 16, 4, 64, 0, A32, A32, None) == -3
    assert q(A32, 4, 64, 0, A32 + 8, A32, None) == -3
    assert q(A32, 4, 64, 0, A32, A32 + 2, None) == -3
    assert q(None, 0, 64, 0, None, None, None) == 0
    assert q(None, 7, 0, 1, None, None, None) == 0


def test_f8_gemm_rejects_bad_arguments(L):
    g = L.fp4q_f8_gemm
    assert g(A32, A32, -1, A32, A32, 8, 64, 0, A32, None) == -2
    assert g(A32, A32, 4, A32, A32, 8, 24, 0, A32, None) == -2       # k % 16
    assert g(A32, A32, 1 << 31, A32, A32, 8, 64, 0, A32, None) == -2
    assert g(A32, A32, 4, A32, A32, 1 << 31, 64, 0, A32, None) == -2
    assert g(A32, A32, 4, A32, A32, 8, 1 << 31, 0, A32, None) == -2
    assert g(A32, A32, 4, A32, A32, 8, 64, 2, A32, None) == -4       # no such output type
    assert g(A32, A32, 4, A32, A32, 8, 64, 0, None, None) == -1
    assert g(None, A32, 4, A32, A32, 8, 64, 0, A32, None) == -1
    assert g(A32, None, 4, A32, A32, 8, 64, 0, A32, None) == -1
    assert g(A32, A32, 4, None, A32, 8, 64, 0, A32, None) == -1
    assert g(A32, A32, 4, A32, None, 8, 64, 0, A32, None) == -1
    assert g(A32 + 8, A32, 4, A32, A32, 8, 64, 0, A32, None) == -3
    assert g(A32, A32, 4, A32 + 8, A32, 8, 64, 0, A32, None) == -3
    assert g(A32, A32 + 2, 4, A32, A32, 8, 64, 0, A32, None) == -3
    assert g(A32, A32, 4, A32, A32 + 1, 8, 64, 0, A32, None) == -3
    assert g(A32, A32, 4, A32, A32, 8, 64, 0, A32 + 1, None) == -3
    assert g(A32, A32, 4, A32, A32, 8, 64, 1, A32 + 2, None) == -3
    assert g(None, None, 0, None, None, 8, 64, 0, None, None) == 0
    assert g(None, None, 4, None, None, 0, 64, 0, None, None) == 0

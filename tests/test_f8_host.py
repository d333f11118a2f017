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


def test_moe_rejects_bad_arguments(L):
    import ctypes

    import microscaling_fp4_quantization_block_b200 as m
    mat = lambda **k: m.Fp4qMoeMatrix(**{**dict(codes=A32, scales=A32, gscale=None, gscale_stride=0), **k})
    good = dict(x=A32, tokens=2, hidden=128, inter=128, experts=8, top_k=2, router=A32, norm=1, fmt=0, up=mat(),
                down=mat(), ids=A32, w=A32, y=A32, ws=A32, ws_bytes=1 << 30)

    def call(**k):
        c = {**good, **k}
        ref = lambda v: None if v is None else ctypes.addressof(v)
        return L.fp4q_moe(c["x"], c["tokens"], c["hidden"], c["inter"], c["experts"], c["top_k"], c["router"],
                          c["norm"], c["fmt"], ref(c["up"]), ref(c["down"]), c["ids"], c["w"], c["y"], c["ws"],
                          c["ws_bytes"], None)

    assert call(tokens=0) == 0 and call(tokens=0, x=None, ids=None, w=None, y=None, ws=None) == 0
    for k in (dict(tokens=-1), dict(hidden=0), dict(inter=-32), dict(experts=0), dict(top_k=0), dict(hidden=48),
              dict(inter=16), dict(fmt=3, hidden=160), dict(fmt=3, inter=64)):
        assert call(**k) == -2, k
    for k in (dict(tokens=65), dict(top_k=9), dict(experts=513), dict(experts=64, top_k=17), dict(hidden=65568),
              dict(fmt=2), dict(fmt=4), dict(fmt=0, up=mat(gscale=A32)), dict(fmt=3, down=mat(gscale=A32)),
              dict(fmt=1, up=mat(gscale=A32, gscale_stride=2))):
        assert call(**k) == -4, k
    for k in (dict(x=None), dict(up=None), dict(down=None), dict(ids=None), dict(w=None), dict(y=None), dict(ws=None),
              dict(up=mat(codes=None)), dict(down=mat(scales=None))):
        assert call(**k) == -1, k
    for k in (dict(x=A32 + 8), dict(router=A32 + 8), dict(ids=A32 + 2), dict(w=A32 + 1), dict(y=A32 + 8),
              dict(ws=A32 + 8), dict(up=mat(codes=A32 + 8)), dict(down=mat(scales=A32 + 4)),
              dict(fmt=1, up=mat(gscale=A32 + 2))):
        assert call(**k) == -3, k
    need = L.fp4q_moe_workspace_size(2, 128, 128, 8, 2)
    assert need > 0 and call(ws_bytes=need - 1) == -6
    assert L.fp4q_moe_workspace_size(65, 128, 128, 8, 2) == 0


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes(L):
    """Checked before the library or a device is asked."""
    import torch

    import microscaling_fp4_quantization_block_b200 as m
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    codes, scales = torch.zeros((4, 128), dtype=torch.uint8), torch.ones((4, 1))
    with pytest.raises(ValueError):
        m.fp4q_f8_quantize(x)
    with pytest.raises(ValueError):
        m.fp4q_f8_quantize(x.float())
    with pytest.raises(ValueError):
        m.fp4q_f8_gemm(codes, scales, codes, scales[:1])
    with pytest.raises(ValueError):
        m.fp4q_moe(x, x, 2, (codes, scales, None), (codes, scales, None), "mxfp4")
    with pytest.raises(ValueError):
        m.fp4q_moe(x, x, 2, (codes, scales, None), (codes, scales, None), "e8m0")

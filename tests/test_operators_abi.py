"""The operators on caller buffers answer bad arguments on the host, before any CUDA call."""

import pytest
import torch

import sparse_moe_layer_fp32_b200 as bm

BAD, UNSUPPORTED, OK = bm.ERR_INVALID_ARG, bm.ERR_UNSUPPORTED, bm.OK
P = 1 << 20  # an aligned address that nothing reads: every call below is refused


def _grouped(name, rows=4, groups=2, n=16, k=32, t=bm.TYPE_BF16, out_type=bm.TYPE_BF16, a=P, b=P, c=P, off=P,
             lda=None, ldb=None, ldc=None):
    lib = bm.lib()
    if name == "beam_moe_grouped_gemm_wgrad":
        return lib.beam_moe_grouped_gemm_wgrad(a, n if lda is None else lda, b, k if ldb is None else ldb, off, rows,
                                               groups, n, k, t, c, out_type, None)
    cols, out = (k, n) if name == "beam_moe_grouped_gemm" else (n, k)
    return getattr(lib, name)(a, cols if lda is None else lda, b, off, rows, groups, n, k, t, c,
                              out if ldc is None else ldc, out_type, None)


@pytest.mark.parametrize("name", ["beam_moe_grouped_gemm", "beam_moe_grouped_gemm_dgrad",
                                  "beam_moe_grouped_gemm_wgrad"])
def test_grouped_products(name):
    assert _grouped(name, rows=-1) == BAD
    assert _grouped(name, groups=0) == BAD
    assert _grouped(name, n=0) == BAD
    assert _grouped(name, k=0) == BAD
    assert _grouped(name, t=bm.TYPE_FP32, out_type=bm.TYPE_FP32) == BAD
    assert _grouped(name, t=3) == BAD
    assert _grouped(name, out_type=bm.TYPE_FP16) == BAD     # the operands' type or FP32
    assert _grouped(name, n=20) == UNSUPPORTED
    assert _grouped(name, k=36) == UNSUPPORTED
    assert _grouped(name, groups=1025) == UNSUPPORTED
    assert _grouped(name, rows=2**31 - 1) == UNSUPPORTED
    assert _grouped(name, a=None) == BAD
    assert _grouped(name, b=None) == BAD
    assert _grouped(name, c=None) == BAD
    assert _grouped(name, off=None) == BAD
    assert _grouped(name, a=P + 8) == BAD
    assert _grouped(name, b=P + 2) == BAD
    assert _grouped(name, c=P + 4) == BAD
    assert _grouped(name, off=P + 2) == BAD
    assert _grouped(name, lda=8) == BAD                     # shorter than a row
    assert _grouped(name, lda=36) == BAD                    # rows off 16-byte boundaries
    if name == "beam_moe_grouped_gemm_wgrad":
        assert _grouped(name, ldb=24) == BAD
        assert _grouped(name, ldb=36) == BAD
    else:
        assert _grouped(name, ldc=8) == BAD
        assert _grouped(name, ldc=36) == BAD
        assert _grouped(name, rows=0, a=None, c=None) == OK  # nothing to do
        # more output tiles than the kernel numbers
        assert _grouped(name, rows=2**31 - 2**17, n=2**30, k=2**30) == UNSUPPORTED


def test_tensors_have_to_be_on_a_gpu():
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        bm.beam_moe_grouped_gemm(x, w, off)
    with pytest.raises(ValueError):
        bm.beam_moe_grouped_gemm_wgrad(x, x, off)

"""The operators on caller buffers answer bad arguments on the host, before any CUDA call."""

import warnings

import pytest
import torch

import sparse_moe_layer_fp32_b200 as bm

BAD, UNSUPPORTED, OK = bm.ERR_INVALID_ARG, bm.ERR_UNSUPPORTED, bm.OK
P = 1 << 20  # an aligned address that nothing reads: every call below is refused


def _grouped(name, rows=4, groups=2, n=16, k=32, t=bm.TYPE_BF16, out_type=bm.TYPE_BF16, a=P, b=P, c=2 * P, off=P,
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
    assert _grouped(name, a=P, b=3 * P, c=P) == BAD         # the output is an operand
    assert _grouped(name, a=3 * P, b=P, c=P) == BAD
    assert _grouped(name, a=P + 8) == BAD
    assert _grouped(name, b=P + 2) == BAD
    assert _grouped(name, c=2 * P + 4) == BAD
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
        assert _grouped(name, n=2**30 + 8) == UNSUPPORTED
        assert _grouped(name, k=2**30 + 8) == UNSUPPORTED


def _quantize(form=0, src=P, t=bm.TYPE_BF16, ld=64, rows=4, cols=64, alpha=1.0, codes=P, ldc=32, sf=P, ldsf=16,
              alpha_out=None):
    return bm.lib().beam_moe_quantize_fp4(form, src, t, ld, rows, cols, alpha, codes, ldc, sf, ldsf, alpha_out, None)


def _dequantize(form=0, codes=P, ldc=32, sf=P, ldsf=16, alpha=None, rows=4, cols=64, out=P, t=bm.TYPE_BF16, ldo=64):
    return bm.lib().beam_moe_dequantize_fp4(form, codes, ldc, sf, ldsf, alpha, rows, cols, out, t, ldo, None)


def _gemm(form=0, a=P, lda=32, asf=P, ldasf=16, alpha_a=None, b=P, ldb=32, bsf=P, ldbsf=16, alpha_b=None, m=4, n=8,
          k=64, out=P, t=bm.TYPE_BF16, ldo=8):
    return bm.lib().beam_moe_gemm_fp4(form, a, lda, asf, ldasf, alpha_a, b, ldb, bsf, ldbsf, alpha_b, m, n, k, out, t,
                                      ldo, None)


def test_fp4_quantiser():
    for form in (bm.FP4_MX, bm.FP4_NV):
        for call in (_quantize, _dequantize):
            assert call(form=form, rows=-1) == BAD
            assert call(form=form, cols=-32) == BAD
            assert call(form=2) == BAD
            assert call(form=form, t=3) == BAD
            assert call(form=form, cols=48) == UNSUPPORTED
            assert call(form=form, rows=2**60) == UNSUPPORTED
            assert call(form=form, rows=0) == OK
            assert call(form=form, cols=0) == OK
            assert call(form=form, codes=None) == BAD
            assert call(form=form, codes=P + 8) == BAD
            assert call(form=form, sf=None) == BAD
            assert call(form=form, ldc=16) == BAD
            assert call(form=form, ldc=40) == BAD
            assert call(form=form, ldsf=1) == BAD
        assert _quantize(form=form, src=None) == BAD
        assert _quantize(form=form, src=P + 2) == BAD
        assert _quantize(form=form, ld=32) == BAD
        assert _quantize(form=form, ld=68) == BAD
        assert _quantize(form=form, sf=P + 4) == BAD
        assert _quantize(form=form, ldsf=24) == BAD
        assert _dequantize(form=form, out=None) == BAD
        assert _dequantize(form=form, out=P + 2) == BAD
        assert _dequantize(form=form, ldo=68) == BAD
        assert _dequantize(form=form, alpha=P + 2) == BAD
    assert _quantize(form=bm.FP4_NV, alpha=0.0) == BAD             # nowhere to put the scale found
    assert _quantize(form=bm.FP4_NV, alpha=float("inf")) == BAD
    assert _quantize(form=bm.FP4_NV, alpha_out=P + 2) == BAD
    assert _quantize(form=bm.FP4_NV, alpha=float("nan"), codes=2 * P, sf=3 * P, alpha_out=4 * P) == BAD


def test_fp4_product():
    for form in (bm.FP4_MX, bm.FP4_NV):
        assert _gemm(form=form, m=-1) == BAD
        assert _gemm(form=form, n=-1) == BAD
        assert _gemm(form=form, k=0) == BAD
        assert _gemm(form=form, k=48) == UNSUPPORTED
        assert _gemm(form=form, m=2**31 - 1) == UNSUPPORTED
        assert _gemm(form=form, k=2**31 - 32) == UNSUPPORTED
        assert _gemm(form=form, m=2**30, n=2**30, ldo=2**30) == UNSUPPORTED
        assert _gemm(form=form, t=5) == BAD
        assert _gemm(form=form, m=0) == OK
        assert _gemm(form=form, n=0) == OK
        for name in ("a", "asf", "b", "bsf", "out"):
            assert _gemm(form=form, **{name: None}) == BAD
        for name in ("a", "asf", "b", "bsf"):
            assert _gemm(form=form, **{name: P + 8}) == BAD
        for name in ("lda", "ldb"):
            assert _gemm(form=form, **{name: 16}) == BAD
            assert _gemm(form=form, **{name: 40}) == BAD
        for name in ("ldasf", "ldbsf"):
            assert _gemm(form=form, **{name: 1}) == BAD
            assert _gemm(form=form, **{name: 24}) == BAD
        assert _gemm(form=form, ldo=7) == BAD
        assert _gemm(form=form, out=P + 1) == BAD
        assert _gemm(form=form, alpha_a=P + 1) == BAD
        assert _gemm(form=form, alpha_b=P + 2) == BAD
    assert _gemm(form=2) == BAD


def test_tensors_have_to_be_on_a_gpu():
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        bm.beam_moe_grouped_gemm(x, w, off)
    with pytest.raises(ValueError):
        bm.beam_moe_grouped_gemm_wgrad(x, x, off)


def test_debug_timeout():
    call = bm.lib().beam_moe_debug_operators_timeout
    assert call(0, P, None) == BAD
    assert call(5 * 10**8 + 1, P, None) == BAD
    assert call(10**6, None, None) == BAD
    assert call(10**6, P + 2, None) == BAD


def test_tensor_scales_that_single_precision_does_not_hold():
    # they would reach the library as 0 ("find the scale") or infinity
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for alpha in (1e-46, 7e-46, 5e-324, 3.5e38, 1e39):
        with pytest.raises(ValueError, match="alpha"):
            bm.beam_moe_quantize_fp4(x, "nvfp4", alpha=alpha)
    for alpha in (8e-46, 1e-45, 3.4e38):  # the smallest and the largest pass to the next check
        with pytest.raises(ValueError, match="device"):
            bm.beam_moe_quantize_fp4(x, "nvfp4", alpha=alpha)


def test_an_input_that_requires_a_gradient_is_warned_about():
    # the results carry no gradient (every call ends at the check of the device)
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    dy, off = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    calls = [(lambda x, w: bm.beam_moe_grouped_gemm(x, w, off), (x, w), (xg, w), (x, wg)),
             (lambda w: bm.beam_moe_grouped_gemm_dgrad(dy, w, off), (w,), (wg,)),
             (lambda x: bm.beam_moe_grouped_gemm_wgrad(dy, x, off), (x,), (xg,)),
             (lambda x: bm.beam_moe_quantize_fp4(x, "mxfp4"), (x,), (xg,))]
    for call, plain, *traced in calls:
        for args in traced:
            with pytest.warns(UserWarning, match="gradient") as seen, pytest.raises(ValueError, match="device"):
                call(*args)
            assert seen[0].filename == __file__  # the caller's line
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with pytest.raises(ValueError, match="device"):
                call(*plain)
            with torch.no_grad(), pytest.raises(ValueError, match="device"):
                call(*traced[0])


def test_types_that_are_none_of_the_operators():
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    dy, off = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    codes, sf = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8)[:, :4]
    for kind in (torch.float64, torch.int32, torch.float8_e4m3fn):
        for call in (lambda: bm.beam_moe_grouped_gemm(x, w, off, out_dtype=kind),
                     lambda: bm.beam_moe_grouped_gemm_dgrad(dy, w, off, out_dtype=kind),
                     lambda: bm.beam_moe_grouped_gemm_wgrad(dy, x, off, out_dtype=kind),
                     lambda: bm.beam_moe_gemm_fp4(codes, sf, codes, sf, "nvfp4", out_dtype=kind),
                     lambda: bm.beam_moe_dequantize_fp4(codes, sf, "nvfp4", out_dtype=kind)):
            with pytest.raises(ValueError, match="BF16, FP16 or FP32"):
                call()
    for alpha in (0.5, torch.ones(1, dtype=torch.float64), torch.ones(2)):  # one FP32 value on the device
        with pytest.raises(ValueError, match="alpha"):
            bm.beam_moe_gemm_fp4(codes, sf, codes, sf, "nvfp4", alpha_a=alpha)
        with pytest.raises(ValueError, match="alpha"):
            bm.beam_moe_dequantize_fp4(codes, sf, "nvfp4", alpha=alpha)

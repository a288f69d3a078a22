"""The operators in a row, as a program uses them: a BF16 mixture-of-experts layer trained through
the routing and the grouped products, and 4-bit projections one after another."""

import os

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bm():
    import sparse_moe_layer_fp32_b200 as m
    yield m
    m.beam_moe_check_operators()


def _draw(shape, kind, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(kind)


@pytest.mark.parametrize("tokens", [1, 7, 300])
def test_a_layers_training_step(bm, tokens):
    hidden, experts, top_k, inter = 256, 16, 2, 128
    x, w_r = _draw((tokens, hidden), BF16, 1), _draw((experts, hidden), FP32, 2, hidden ** -0.5)
    w_gu, w_d = _draw((experts, 2 * inter, hidden), BF16, 3, 0.06), _draw((experts, hidden, inter), BF16, 4, 0.09)
    dout = _draw((tokens, hidden), BF16, 5)

    ids, weight = bm.beam_moe_route(x, w_r, top_k)
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)  # slots sorted by expert
    offsets = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=experts).cumsum(0)]).int()
    token, slot_w = order // top_k, weight.flatten()[order][:, None]

    # forward
    rows = x[token]
    gu = bm.beam_moe_grouped_gemm(rows, w_gu, offsets)
    g, u = gu.float().chunk(2, 1)
    h = (torch.nn.functional.silu(g) * u).to(BF16)
    y = bm.beam_moe_grouped_gemm(h, w_d, offsets)
    out = torch.zeros(tokens, hidden, device="cuda").index_add_(0, token, y.float() * slot_w)
    # backward
    dy = (dout[token].float() * slot_w).to(BF16)
    dw_d = bm.beam_moe_grouped_gemm_wgrad(dy, h, offsets, out_dtype=FP32)
    dh = bm.beam_moe_grouped_gemm_dgrad(dy, w_d, offsets).float()
    s = torch.sigmoid(g)
    dgu = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1).to(BF16)
    dw_gu = bm.beam_moe_grouped_gemm_wgrad(dgu, rows, offsets, out_dtype=FP32)
    drows = bm.beam_moe_grouped_gemm_dgrad(dgu, w_gu, offsets)
    dx = torch.zeros(tokens, hidden, device="cuda").index_add_(0, token, drows.float())

    # the same in 64 bits by automatic differentiation, every expert over every row
    xd, gud, dd = (t.double().requires_grad_() for t in (x, w_gu, w_d))
    mask = torch.nn.functional.one_hot(flat[order], experts).double()
    a = torch.einsum("rk,enk,re->rn", xd[token], gud, mask)
    gd, ud = a.chunk(2, 1)
    yd = torch.einsum("rk,enk,re->rn", torch.nn.functional.silu(gd) * ud, dd, mask)
    ref = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda").index_add(0, token, yd * slot_w.double())
    gx, ggu, gd_ = torch.autograd.grad((ref * dout.double()).sum(), (xd, gud, dd))
    # Between the inputs and any of these results lie at most five roundings to BF16, each at most
    # 2^-8 of the value; carried through products of random rows a relative error keeps its size.
    for got, want in ((out, ref), (dx, gx), (dw_gu, ggu), (dw_d, gd_)):
        assert bool(((got.double() - want).norm() <= 5 * 2.0 ** -8 * want.norm()))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("tokens", [1, 200])
def test_projections_in_4_bits_one_after_another(bm, fmt, tokens):
    # x -> w1 -> w2, activations quantised on the way: every stage against 64 bits on the operands
    # that the stage read
    x = _draw((tokens, 512), BF16, 6)
    quantised = [bm.beam_moe_quantize_fp4(_draw(s, FP32, 7 + i, 0.05), fmt) for i, s in enumerate(((320, 512), (96, 320)))]
    v = x
    for w in quantised:
        q = bm.beam_moe_quantize_fp4(v, fmt)
        nxt = bm.beam_moe_gemm_fp4(q[0], q[1], w[0], w[1], fmt, alpha_a=q[2], alpha_b=w[2], out_dtype=BF16)
        a, b = (bm.beam_moe_dequantize_fp4(t[0], t[1], fmt, alpha=t[2], out_dtype=FP32).double() for t in (q, w))
        ref, k = a @ b.t(), a.shape[1]
        # the values read back are rounded to FP32 by alpha (2^-24 each), the sum as in the product's
        # own tests, one rounding to BF16
        acc = ((k + 15) // 16 * 2.0 ** -22 + 2.0 ** -21) * (a.abs() @ b.abs().t())
        assert bool(((nxt.double() - ref).abs() <= acc + 2.0 ** -8 * (ref.abs() + acc)).all())
        v = nxt


@pytest.mark.parametrize("tokens", [4, 64])
def test_a_layer_right_behind_the_operators(bm, tokens):
    # x and the residual come out of the operators' last kernels, which let the layer's first one
    # start early: the same bits as with the GPU waited for in between
    import dataclasses

    import moe_inputs as mi
    from sparse_moe_layer_fp32_b200 import synthetic
    shape = dataclasses.replace(mi.SHAPES["tiny"], tokens=tokens)
    layer = synthetic.make_layer(shape, synthetic.make_weights(shape, 0, threads=2))
    hidden = shape.hidden
    w = bm.beam_moe_quantize_fp4(_draw((hidden, hidden), FP32, 20, 0.06), "mxfp4")
    dense = _draw((1, hidden, hidden), BF16, 21, 0.06)
    off = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")

    def step(v, wait):
        residual = bm.beam_moe_grouped_gemm(v, dense, off)
        q = bm.beam_moe_quantize_fp4(v, "mxfp4")
        x = bm.beam_moe_gemm_fp4(q[0], q[1], w[0], w[1], "mxfp4")
        if wait:
            torch.cuda.synchronize()
        out = layer.forward(x, residual)
        q = bm.beam_moe_quantize_fp4(out, "mxfp4")  # and an operator right behind the layer
        return out, bm.beam_moe_dequantize_fp4(q[0], q[1], "mxfp4")

    inputs = [_draw((tokens, hidden), BF16, 30 + i) for i in range(40)]
    want = [step(v, True) for v in inputs]
    torch.cuda.synchronize()
    got = [step(v, False) for v in inputs]
    layer.check()
    assert all(torch.equal(a, b) for g, r in zip(got, want) for a, b in zip(g, r))
    layer.close()


@pytest.mark.parametrize("tokens,hidden,experts", [(9, 256, 16), (200, 5120, 256)])
def test_routing_right_behind_the_operators(bm, tokens, hidden, experts):
    # x comes out of an operator's kernel, which lets the router's first one (more than 8 tokens:
    # the tiled product) start early: the same bits as with the GPU waited for in between
    wr = _draw((experts, hidden), FP32, 50, hidden ** -0.5)
    w = bm.beam_moe_quantize_fp4(_draw((hidden, 256), FP32, 51, 0.06), "nvfp4")
    dense = _draw((1, hidden, 256), BF16, 52, 0.06)
    off = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    inputs = [_draw((tokens, 256), BF16, 60 + i) for i in range(20)]

    def step(v, wait):
        out = []
        for behind in ("4 bits", "grouped", "read back"):
            q = bm.beam_moe_quantize_fp4(v, "nvfp4")
            if behind == "4 bits":
                x = bm.beam_moe_gemm_fp4(q[0], q[1], w[0], w[1], "nvfp4", alpha_a=q[2], alpha_b=w[2])
            elif behind == "grouped":
                x = bm.beam_moe_grouped_gemm(v, dense, off)
            else:
                q = bm.beam_moe_quantize_fp4(x, "nvfp4")
                x = bm.beam_moe_dequantize_fp4(q[0], q[1], "nvfp4", alpha=q[2])
            if wait:
                torch.cuda.synchronize()
            out += bm.beam_moe_route(x, wr, 2)
        return out

    want = [step(v, True) for v in inputs]
    torch.cuda.synchronize()
    got = [step(v, False) for v in inputs]
    assert all(torch.equal(a, b) for g, r in zip(got, want) for a, b in zip(g, r))


def test_columns_of_one_buffer(bm):
    # operands and outputs that are columns of the same matrix do not share memory, and are taken
    rows, n, k = 70, 40, 96
    buf = _draw((rows, 256), BF16, 70)
    w, off = _draw((2, n, k), BF16, 71, 0.1), torch.tensor([0, 30, rows], dtype=torch.int32, device="cuda")
    want = bm.beam_moe_grouped_gemm(buf[:, :k].contiguous(), w, off)
    got = bm.beam_moe_grouped_gemm(buf[:, :k], w, off, out=buf[:, k:k + n])
    assert torch.equal(got, want) and got.data_ptr() == buf[:, k:].data_ptr()
    dwant = bm.beam_moe_grouped_gemm_dgrad(want, w, off)
    assert torch.equal(bm.beam_moe_grouped_gemm_dgrad(buf[:, k:k + n], w, off, out=buf[:, 144:144 + k]), dwant)
    with pytest.raises(bm.BeamMoeError) as err:
        bm.beam_moe_grouped_gemm(buf[:, :k], w, off, out=buf[:, k - 8:k - 8 + n])
    assert err.value.status == bm.ERR_INVALID_ARG
    # codes and scales of one buffer's rows; the product's result behind them
    for fmt, block in (("mxfp4", 32), ("nvfp4", 16)):
        q = bm.beam_moe_quantize_fp4(dwant, fmt)
        whole = torch.zeros((rows, 256), dtype=torch.uint8, device="cuda")
        codes, sf = whole[:, :k // 2], whole[:, 48:48 + k // block]
        codes.copy_(q[0])
        sf.copy_(q[1])
        out = torch.as_strided(whole.view(BF16), (rows, 60), (128, 1), 32)
        other = [t[:60] for t in q[:2]]
        ref = bm.beam_moe_gemm_fp4(q[0], q[1], other[0], other[1], fmt, alpha_a=q[2], alpha_b=q[2])
        assert torch.equal(bm.beam_moe_gemm_fp4(codes, sf, other[0], other[1], fmt, alpha_a=q[2], alpha_b=q[2],
                                                out=out), ref)
        assert torch.equal(codes, q[0]) and torch.equal(sf, q[1])


def test_the_readme_example(bm, repo_root):
    with open(os.path.join(repo_root, "README.md")) as f:
        code = [part for part in f.read().split("```") if part.startswith("python") and "grouped_gemm(" in part]
    assert len(code) == 1
    tokens, hidden, inter, experts, top_k = 40, 256, 128, 16, 2
    names = dict(bm=bm, torch=torch, E=experts, top_k=top_k, x=_draw((tokens, hidden), BF16, 80),
                 router_w=_draw((experts, hidden), FP32, 81), proj=_draw((96, hidden), FP32, 82, 0.05),
                 w_gate_up=_draw((experts, 2 * inter, hidden), BF16, 83, 0.06),
                 dy=_draw((tokens * top_k, 2 * inter), BF16, 84))
    exec(code[0].removeprefix("python"), names)
    assert names["y"].shape == (tokens * top_k, 2 * inter) and names["dx"].shape == (tokens * top_k, hidden)
    assert names["dw"].shape == (experts, 2 * inter, hidden) and names["out"].shape == (tokens, 96)
    for slot in range(tokens * top_k):
        e = int(names["ids"].flatten()[names["order"][slot]])
        row = names["x"][int(names["order"][slot]) // top_k].double()
        ref = names["w_gate_up"][e].double() @ row
        size = names["w_gate_up"][e].double().abs() @ row.abs()
        # 16 additions into FP32 of at most 2^-22 of the absolute sum, one rounding to BF16
        assert bool(((names["y"][slot].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -17 * size).all())

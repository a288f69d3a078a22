"""The bounded waits of the operators on caller buffers, made to run out with a short limit."""

import pytest
import torch

pytestmark = pytest.mark.gpu

LIMIT = 20_000_000  # 20 ms


@pytest.fixture(scope="module")
def bm():
    import sparse_moe_layer_fp32_b200 as m
    return m


def test_a_wait_that_gives_up_is_reported_once(bm):
    bm.beam_moe_check_operators()
    result = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.randn(8, 64, device="cuda").bfloat16()
    for _ in range(2):
        result.zero_()
        bm.beam_moe_debug_operators_timeout(LIMIT, result)
        with pytest.raises(bm.BeamMoeError) as err:
            bm.beam_moe_check_operators()
        assert err.value.status == bm.ERR_TIMEOUT
        assert result[0].item() == 1
        bm.beam_moe_check_operators()  # cleared by the check that reported it
        # and the operators go on
        q = bm.beam_moe_quantize_fp4(x, "mxfp4")
        assert torch.isfinite(bm.beam_moe_gemm_fp4(q[0], q[1], q[0], q[1], "mxfp4")).all()
        bm.beam_moe_check_operators()


def test_a_shared_tiles_sums_where_a_side_gives_up(bm):
    result = torch.zeros(4, dtype=torch.int32, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    bm.beam_moe_debug_operators_timeout(LIMIT, result)
    end.record()
    torch.cuda.synchronize()
    assert result[:3].tolist() == [1, 1, 1]
    # waits of a few limits each: none ran into the 2 s limit
    assert start.elapsed_time(end) < 1000
    with pytest.raises(bm.BeamMoeError):
        bm.beam_moe_check_operators()
    bm.beam_moe_check_operators()


def test_the_limit_counts_from_the_last_progress(bm):
    result = torch.zeros(4, dtype=torch.int32, device="cuda")
    bm.beam_moe_debug_operators_timeout(LIMIT, result)
    assert result[3].item() == 1
    with pytest.raises(bm.BeamMoeError):
        bm.beam_moe_check_operators()


def test_a_sum_longer_than_the_limit(bm):
    # one tile's sum over 2^30 - 1 rows takes longer than the waits' 2 s.  Rows of +-1, each times the
    # row behind it: the sums walk within +-2^20 and are exact in FP32
    rows = 2 ** 30
    buf = torch.empty((rows, 8), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    step = 1 << 22
    for i in range(0, rows, step):
        buf[i:i + step] = torch.randint(0, 2, (step, 8), generator=g, device="cuda") * 2 - 1
    dy, x = buf[:-1], buf[1:]
    off = torch.tensor([0, rows - 1], dtype=torch.int32, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    dw = bm.beam_moe_grouped_gemm_wgrad(dy, x, off, out_dtype=torch.float32)
    end.record()
    bm.beam_moe_check_operators()
    print(f"sum over {rows - 1} rows: {start.elapsed_time(end):.0f} ms")
    ref = torch.zeros((8, 8), dtype=torch.float64, device="cuda")
    for i in range(0, rows - 1, step):
        ref += (dy[i:i + step].float().t() @ x[i:i + step].float()).double()  # whole numbers below 2^24
    assert torch.equal(dw[0].double(), ref)


@pytest.mark.parametrize("k", [2 ** 29 + 96, 2 ** 30 + 2 ** 20 + 32])
def test_a_product_of_long_rows(bm, k):
    # few tiles and long sums: as long as pairs that share a tile wait for, and longer.  Codes of +-1:
    # the sums walk within +-2^20 and are exact in FP32
    n = 3
    g = torch.Generator(device="cuda")
    g.manual_seed(2)

    def matrix(rows):
        codes = torch.empty((rows, (k // 2 + 15) // 16 * 16), dtype=torch.uint8, device="cuda")
        for r in range(rows):
            codes[r] = torch.randint(0, 256, (codes.shape[1],), generator=g, device="cuda", dtype=torch.uint8)
        codes.bitwise_and_(0x88).bitwise_or_(0x22)
        sf = torch.full((rows, (k // 32 + 15) // 16 * 16), 127, dtype=torch.uint8, device="cuda")
        return codes[:, :k // 2], sf[:, :k // 32]

    a, b = matrix(1), matrix(n)
    out = bm.beam_moe_gemm_fp4(a[0], a[1], b[0], b[1], "mxfp4", out_dtype=torch.float32)
    bm.beam_moe_check_operators()
    for j in range(n):
        signs = a[0][0] ^ b[0][j]
        minus = sum(int(((part >> bit) & 1).sum()) for part in signs.split(1 << 26) for bit in (3, 7))
        assert out[0, j].item() == k - 2 * minus


def test_a_check_on_another_stream_takes_what_is_there(bm):
    # every report is given by one check and no report is lost, whichever streams ask
    streams = [torch.cuda.Stream() for _ in range(2)]
    result = torch.zeros(4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    bm.beam_moe_debug_operators_timeout(LIMIT, result, stream=streams[0])
    streams[0].synchronize()
    with pytest.raises(bm.BeamMoeError):
        bm.beam_moe_check_operators(stream=streams[1])
    for s in streams:
        bm.beam_moe_check_operators(stream=s)

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
    assert result.tolist() == [1, 1, 1, 0]
    # three waits of one or two limits each: none ran into the 2 s limit
    assert start.elapsed_time(end) < 1000
    with pytest.raises(bm.BeamMoeError):
        bm.beam_moe_check_operators()
    bm.beam_moe_check_operators()


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

"""Offsets that the host holds, as the Python functions of the experts' MXFP8
operators check them. Runs only without a GPU: the tensors live on the CPU and
the launches are recorded instead of made."""
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq

if torch.cuda.is_available():
    pytest.skip("host-validation tests with CPU tensors run without a GPU only", allow_module_level=True)


@pytest.fixture
def launches(monkeypatch):
    made = []
    monkeypatch.setattr(mxq, "_same_device", lambda *ts: 0)
    monkeypatch.setattr(mxq, "_byte_tensors", lambda *ts: 0)
    monkeypatch.setattr(mxq, "_launch", lambda fn, index, *args: made.append((fn, args)))
    return made


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def product(offsets):
    return mxq.mxfp8_gemm_grouped(u8(200, 64), u8(4096), u8(2, 32, 64), u8(1024), offsets)


def transposes(offsets):
    return mxq.mxfp8_quantize_columnwise_grouped(torch.zeros(200, 32), row_offsets=offsets)


def gradients(offsets):
    P = (200 + 127 * 2) // 128 * 128
    return mxq.mxfp8_gemm_grouped_wgrad(u8(16, P), u8(2048), u8(16, P), u8(2048), offsets)


@pytest.mark.parametrize("call", [product, transposes, gradients])
@pytest.mark.parametrize("kind", [list, tuple, torch.tensor])
def test_offsets_start_at_zero(call, kind, launches):
    """The kernels take the first offset as 0: [50, 100, 200] would count rows 0 to 49 as expert 0's."""
    for good in ([0, 0, 0], [0, 100, 200], [0, 50, 120]):
        call(kind(good))
    assert len(launches) == 3
    for bad in ([50, 100, 200], [1, 1, 1], [200, 200, 200], [-1, 0, 200]):
        with pytest.raises(ValueError, match="row_offsets must"):
            call(kind(bad))
    assert len(launches) == 3


@pytest.mark.parametrize("call", [product, transposes, gradients])
def test_offsets_rise_within_the_rows(call, launches):
    for bad in ([0, 100, 500], [0, 100, 99], [0, -1, 200]):
        with pytest.raises(ValueError, match="row_offsets must"):
            call(bad)
    assert not launches


def test_weight_gradients_of_offsets_that_the_columns_do_not_hold(launches):
    """An expert whose columns lie behind P would silently get zeros, or a part of its sum."""
    two = lambda P, off: mxq.mxfp8_gemm_grouped_wgrad(u8(16, P), u8(2048), u8(16, P), u8(2048), off)
    two(256, [0, 1, 2]), two(384, [0, 129, 200]), two(128, [0, 0, 128]), two(0, [0, 0, 0])
    assert len(launches) == 4
    for P, off in ((128, [0, 1, 2]), (256, [0, 129, 200]), (256, torch.tensor([0, 1, 130]))):
        with pytest.raises(ValueError, match="columns"):
            two(P, off)
    assert len(launches) == 4


def test_scales_of_the_experts_rows_are_enough(launches):
    """Rows behind the last offset belong to no expert: scales that hold the experts' tiles are not refused, and the
    library is given the rows that they can hold (it wants scales for every row)."""
    K, N, M = 320, 32, 1000
    w, sw = u8(2, N, K), u8(2 * mxq._tile_bytes(N, K // 32))
    tile = mxq._tile_bytes(128, K // 32)
    for tiles, offsets, rows in ((8, [0, 500, 1000], 1000), (8, [0, 0, 800], 1000), (7, [0, 0, 800], 896), (7, [0, 128, 896], 896),
                                 (2, [0, 1, 2], 256), (1, [0, 0, 100], 128), (0, [0, 0, 0], 0), (9, [0, 500, 1000], 1000)):
        y = mxq.mxfp8_gemm_grouped(u8(M, K), u8(tiles * tile), w, sw, offsets)
        fn, args = launches.pop()
        assert fn == "mxfp8_gemm_grouped" and args[2] == tiles * tile and args[7] == rows and y.shape == (M, N)
        assert args[2] >= mxq._tile_bytes(rows, K // 32)
    for tiles, offsets in ((7, [0, 500, 1000]), (6, [0, 0, 800]), (1, [0, 1, 2]), (0, [0, 0, 1])):
        with pytest.raises(ValueError, match="scales"):
            mxq.mxfp8_gemm_grouped(u8(M, K), u8(tiles * tile), w, sw, offsets)
    assert not launches

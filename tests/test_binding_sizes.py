"""CPU checks that the binding refuses sizes past 32 bits, which ctypes would cut down to their low
half: 2^32 + 8 tokens would be 8 tokens, and the rest of the outputs whatever memory held."""
import pytest
import torch

FAR = 1 << 32


@pytest.fixture()
def fg(monkeypatch):
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_routing(fg):
    i32 = torch.int32
    few = meta(5, 3, dtype=i32)
    for call in (lambda: fg.route_contiguous(meta(FAR + 8, dtype=i32), 4), lambda: fg.route_contiguous(few, FAR + 4),
                 lambda: fg.route_contiguous(few, 4, align=FAR + 128), lambda: fg.route_contiguous(few, 4, align=128 - FAR),
                 lambda: fg.route_contiguous(few, 4, M=FAR + 512), lambda: fg.route_masked(meta(3, FAR + 2, dtype=torch.int64), 4, 8),
                 lambda: fg.route_masked(few, FAR + 1, 8), lambda: fg.route_masked(few, 4, FAR + 8), lambda: fg.route_rows(FAR + 1, 8, 32),
                 lambda: fg.route_rows(1, 8, 32, FAR + 128), lambda: fg.route_rows(1, 8 - FAR, 32)):
        with pytest.raises(ValueError, match="past 32 bits"):
            call()
    assert fg.route_rows(1, 8, 32) == 1024 and fg.route_rows(-1, 8, 32) == -1


def test_rows_of_any_other_size(fg):
    """Routings of other lengths than route_* makes, and rows of other sizes."""
    route = fg.Route(meta(5, 1, dtype=torch.int32), meta(640, dtype=torch.int32), meta(640, dtype=torch.int32), None, None, 128)
    long_route = route._replace(rows=meta(FAR + 5, 1, dtype=torch.int32))
    tall = route._replace(src=meta(FAR + 640, dtype=torch.int32))
    f32 = torch.float32
    wide = FAR + 128
    for call in (lambda: fg.dispatch_f16(meta(5, wide), route), lambda: fg.dispatch_f16(meta(FAR + 5, 64), long_route),
                 lambda: fg.dispatch_f16(meta(5, 64), tall), lambda: fg.dispatch_fp8(meta(5, wide), route, 0),
                 lambda: fg.combine_f16(meta(640, wide), None, route), lambda: fg.combine_f16(meta(640, 64), None, long_route),
                 lambda: fg.combine_f16_backward(meta(5, wide), meta(640, wide), meta(5, 1, dtype=f32), route),
                 lambda: fg.dispatch_f16_backward(meta(640, wide), route),
                 lambda: fg.lora_f16(meta(5, wide), meta(2, 16, wide), meta(2, 64, 16), route)):
        with pytest.raises(ValueError, match="past 32 bits"):
            call()
    # row distances are 64-bit numbers
    x = torch.empty_strided((5, 64), (FAR, 1), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="CUDA"):
        fg.lora_f16(x, meta(2, 16, 64), meta(2, 64, 16), route)

"""The 64-bit reference of the 4-bit formats, on the CPU, against tables, torch's own E4M3
conversion and neighbours, and the binding's scale layout and refusals."""
import pytest
import torch

import block_wise_w8a8_b200 as w8
import fp4_ref as ref


def test_e2m1_nearest_with_ties_to_even():
    a = torch.tensor([0, 0.25, 0.2501, 0.5, 0.75, 0.7499, 1.25, 1.2501, 1.75, 2.5, 2.5001, 3.5, 3.4999, 5, 5.0001, 6, 9],
                     dtype=torch.float64)
    want = [0, 0, 1, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 6, 7, 7, 7]
    assert ref.e2m1(a).tolist() == want
    levels = torch.tensor(ref.LEVELS, dtype=torch.float64)
    v = torch.rand(4096, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 7
    near = (v[:, None] - levels).abs().argmin(1)
    assert torch.equal(ref.e2m1(v).long(), near)


def test_e4m3_is_torchs():
    every = torch.arange(127, dtype=torch.uint8)
    v = every.view(torch.float8_e4m3fn).double()
    assert torch.equal(ref.e4m3_value(every), v)
    assert torch.equal(ref.e4m3(v), every)
    mid = (v[1:] + v[:-1]) / 2
    a = torch.cat((mid, mid * (1 + 1e-6), mid * (1 - 1e-6)))
    assert torch.equal(ref.e4m3(a), a.float().to(torch.float8_e4m3fn).view(torch.uint8))


def test_quantize_pins():
    """Blocks worked out by hand."""
    x = torch.zeros((1, 64), dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 6.0, -1.25, 7.5, 0.25      # amax 7.5: e = 2 - 2 = 0
    x[0, 32] = 2.0 ** -130                                          # below what a scale reaches
    code, s, f = ref.quantize(x, "mxfp4")
    assert code[0, :4].tolist() == [7, 8 + 2, 7, 0] and s.tolist() == [[127, 0]] and f is None
    assert int(code[0, 32]) == 0
    x = torch.zeros((1, 32), dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 6.0, 0.5
    x[0, 16], x[0, 17] = -3.0, 1.25
    code, s, f = ref.quantize(x, "nvfp4")
    # A = 6: factor 1 / 448, scales 448 and 224 (bytes 0x7E, 0x76), units 1 and 0.5
    assert s.tolist() == [[0x7E, 0x76]] and f.tolist() == [torch.tensor(6.0 / 2688).item()]
    assert code[0, [0, 1, 16, 17]].tolist() == [7, 1, 15, 4]


@pytest.mark.parametrize("rows,blocks", [(1, 1), (3, 2), (128, 4), (130, 9), (300, 128)])
def test_scale_tiles_follow_the_formula(rows, blocks):
    s = torch.randint(0, 256, (rows, blocks), dtype=torch.uint8, generator=torch.Generator().manual_seed(rows))
    t = w8.fp4_tile_scales(s)
    assert t.shape == (-(-rows // 128), -(-blocks // 4), 512)
    for r, b in [(0, 0), (rows - 1, blocks - 1), (rows // 2, blocks // 2)]:
        assert t[r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] == s[r, b]
    assert torch.equal(w8.fp4_untile_scales(t, rows, blocks), s)
    assert int(t.count_nonzero()) == int(s.count_nonzero())         # zeros past the end
    assert torch.equal(w8.fp4_tile_scales(s.view(torch.float8_e4m3fn)), t)
    with pytest.raises(ValueError):
        w8.fp4_untile_scales(t, rows + 128, blocks)


def test_binding_refuses_before_the_library(monkeypatch):
    def boom():
        raise AssertionError("the library must not be reached")
    monkeypatch.setattr(w8, "lib", boom)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w8.fp4_quantize(x)                                           # host memory
    with pytest.raises(ValueError):
        w8.fp4_quantize(x, "fp4")                                    # no such format
    with pytest.raises(ValueError):
        w8.FP4Tensor(x.view(torch.uint8), None, None, "mxfp4")
    with pytest.raises(ValueError):
        w8.block_norm(x, x)
    with pytest.raises(TypeError):
        w8.fp4_dequantize(x)
    with pytest.raises(TypeError):
        w8.fp4_linear_prequant(x, None)
    with pytest.raises(ValueError):
        w8.FP4Weight(x)
    with pytest.raises(ValueError):
        w8.fp4_tile_scales(x)


def test_size_queries():
    L = w8.lib()
    assert L.w8a8_fp4_scale_bytes(1, 32, 0) == 512
    assert L.w8a8_fp4_scale_bytes(129, 160, 0) == 2 * 2 * 512
    assert L.w8a8_fp4_scale_bytes(128, 160, 1) == 3 * 512
    assert L.w8a8_fp4_scale_bytes(128, 40, 1) == 0 and L.w8a8_fp4_scale_bytes(128, 64, 2) == 0
    assert w8.fp4_linear_workspace_bytes(5, 96, "nvfp4") == 256 + 2 * 512 + 5 * 4
    assert w8.fp4_linear_workspace_bytes(5, 96, "mxfp4") == 256 + 512
    assert w8.fp4_linear_workspace_bytes(5, 100) == 0 and w8.fp4_linear_workspace_bytes(0, 96) == 0

"""Weights that no FP4 product can stand for are refused where they are packed, and products
without channels before anything is computed."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, math.nan, math.inf, -math.inf, 1e-60, 1e60])
def test_scales_that_float32_does_not_hold(scale):
    from latent_kv_decode_b200 import ops
    with pytest.raises(ops.MlaError):
        ops.pack_fp4_weight(torch.ones((2, 512), device="cuda"), scale=scale)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_weights_without_a_largest_magnitude(bad):
    from latent_kv_decode_b200 import ops
    w = torch.ones((2, 512), device="cuda")
    w[1, 3] = bad
    with pytest.raises(ops.MlaError):
        ops.pack_fp4_weight(w)


@pytest.mark.parametrize("size", [0.0, 2.0 ** -149, 2.0 ** -130, 1e-30, 1.0, 3e38])
def test_weights_of_any_size(size):
    # group maxima are the format's end, 448 * 6, or as near to it as a normal scale allows
    from latent_kv_decode_b200 import ops
    w = torch.full((3, 512), size, device="cuda")
    w[1] = -w[1]
    e, scale = ops.pack_fp4_weight(w)
    x = torch.zeros((1, 512), dtype=torch.bfloat16, device="cuda")
    x[0, 7] = 1.0
    y = ops.mla_fp4_linear(x, e, scale).double()
    # E4M3's and E2M1's half steps of such a maximum (2^-4, and 2^-10 below its normal range, each
    # in units of scale), x and y exact but for y's rounding to bf16
    tol = (2.0 ** -4 + 2.0 ** -7) * size + 6 * 2.0 ** -9 * scale + 2.0 ** -133
    assert ((y - w[:, 7].double()).abs() <= tol).all()


def test_products_without_channels():
    from latent_kv_decode_b200 import ops
    x = torch.zeros((2, 0), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((3, 0, 288), dtype=torch.uint8, device="cuda")
    with pytest.raises(ops.MlaError):
        ops.mla_fp4_linear(x, w)
    with pytest.raises(ops.MlaError):
        ops.mla_fp4_linear(x.view(2, 1, 0), w)
    x = torch.zeros((2, 0, 1, 512), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ops.MlaError):
        ops.mla_fp4_group_wo(x, torch.zeros((0, 8, 1, 288), dtype=torch.uint8, device="cuda"))

"""Codes of -0 in blocks that are not all zero: the code's sign bit is the sign
bit of x at every block scale, through every call that quantizes.  Where s_g has
few significant bits some block scales take a multiplier of two parts, whose two
products must not add up to +0."""
import numpy as np
import pytest
import torch

import oracle
import synthetic as S
from _gpu_util import bits_of, check_quantize, check_quantized, fh, quantize_tiled, to_dev
from test_gpu_kv_cache import check as check_cache

pytestmark = pytest.mark.gpu

GSCALES = [1.0, 0.0078125, 1.5, 1.25, 3.0, 0.1]


def block_scales():
    """The values of the 126 block scales above 0."""
    s = np.arange(1, 127)
    return np.where(s < 8, s * 2.0 ** -9, (8 + s % 8) * 2.0 ** (s // 8 - 10.0))


def signed_zeros(sg):
    """BF16 bits [126, 64]: a row a block scale, each of its four blocks with the largest element that has it, zeros and
    the smallest magnitudes of both signs, and elements of codes -0.5 .. -6."""
    s = block_scales()
    top = S.to_bf16_bits((6 * s * sg).astype(np.float32)).astype(np.uint16)
    part = S.to_bf16_bits((s[:, None] * sg * np.array([-0.5, -1.0, -2.0, -3.0, -6.0])).astype(np.float32)).astype(np.uint16)
    x = np.zeros((126, 4, 16), np.uint16)
    x[:, :, 0] = top[:, None]
    x[:, 1::2, 0] |= 0x8000
    x[:, :, 1:6] = 0x8000
    x[:, :, 6:8] = [0x0001, 0x8001]
    x[:, :, 8:13] = part[:, None]
    x[:, :, 13] = 0x8000
    rng = np.random.default_rng(0)
    for b in range(4):
        x[:, b] = x[:, b][:, rng.permutation(16)]
    return x.reshape(126, 64)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("sg", GSCALES)
def test_activations(sg, layout):
    check_quantize(signed_zeros(sg), sg, layout)


@pytest.mark.parametrize("sg", GSCALES)
def test_cache_write(sg):
    x = signed_zeros(sg).reshape(126, 1, 64)
    check_cache(126, 1, 64, 32, 9, k=x, v=x ^ 0x8000, gscales=(sg, sg))


def gelu_inputs():
    """Rows of 2048: a block a block scale of 2 and more (whose largest element GELU leaves alone) at s_g = 1, in turns,
    the rest so far below zero that GELU is -0, or -0 itself."""
    s = block_scales()
    s = s[s >= 2]
    x = np.full((128, 16), -200.0)
    x[:, 5] = 6 * np.resize(s, 128)
    x[:, 9] = -0.0
    return S.to_bf16_bits(x.astype(np.float32)).reshape(1, 2048)


def test_gelu_then_quantize():
    m = fh()
    x = to_dev(np.repeat(gelu_inputs(), 3, 0))
    g = torch.empty_like(x)
    m.fh_gelu_bf16(x, g)
    codes, scales = m.empty_quantized(3, 2048)
    clip = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.fh_gelu_quantize_act(x, 1.0, codes, scales, clip)
    assert (bits_of(g) == 0x8000).sum() >= 3 * 128 * 14
    check_quantized(codes, scales, int(clip), bits_of(g), 1.0)


def test_gelu_epilogue():
    """The layer's output is its bias: no weight is other than zero."""
    m = fh()
    a, w = (quantize_tiled(to_dev(np.zeros(shape, np.uint16)), 1.0) for shape in ((70, 128), (2048, 128)))
    bias = to_dev(gelu_inputs().reshape(2048))
    y = torch.empty((70, 2048), dtype=torch.bfloat16, device="cuda")
    m.fh_nvfp4_linear(a[0], a[1], 1.0, w[0], w[1], 1.0, bias, y)
    m.fh_gelu_bf16(y, y)
    codes, scales = m.empty_quantized(70, 2048)
    clip = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.fh_nvfp4_linear_gelu_quant(a[0], a[1], 1.0, w[0], w[1], 1.0, bias, 1.0, codes, scales, clip)
    m.fh_device_status()
    assert (bits_of(y) == 0x8000).sum() >= 70 * 128 * 14
    check_quantized(codes, scales, int(clip), bits_of(y), 1.0)

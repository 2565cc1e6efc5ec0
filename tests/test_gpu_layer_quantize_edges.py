"""The quantized norm and the cache write at the edges of their number range."""
import numpy as np
import pytest
import torch

from gpu_util import host, scalar

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _norm_fp8(lib, x, weight, group, eps=1e-6):
    m, k = x.shape
    q = torch.zeros((m, k), dtype=torch.uint8, device="cuda")
    s = torch.zeros((m, k // group if group else 1), device="cuda")
    lib.add_rms_norm_fp8_quantize(x, None, weight, scalar(eps), None, q, s, group, m, k)
    torch.cuda.synchronize()
    return q, s


def _rows(m, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("size", [1e-30, 1e-36, 1e-37, 2e-38])
@pytest.mark.parametrize("k", [256, 5120])
def test_fp8_scales_of_tiny_values(lib, group, size, k):
    """Values so small that 448 over their largest is past fp32: zeros stay
    zeros, and value times scale stands for y as elsewhere."""
    x = _rows(3, k, 5)
    x[:, ::3] = 0
    weight = torch.full((k,), size, device="cuda").to(torch.bfloat16)
    q, s = _norm_fp8(lib, x, weight, group)
    v, scale = host(q.view(torch.float8_e4m3fn).float()).astype(np.float64), host(s).astype(np.float64)
    f = host(x.double())
    y = f / np.sqrt((f * f).mean(-1, keepdims=True) + np.float64(np.float32(1e-6))) * host(weight.double())
    assert np.isfinite(v).all() and np.isfinite(scale).all() and (v[f == 0] == 0).all()
    scale = np.repeat(scale, group or k, axis=1)
    # E4M3: half a step is 2^-4 of a normal value and 2^-10 of a subnormal one;
    # the scale's own rounding moves value and scale together
    assert (np.abs(v * scale - y) <= np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) * 1.001).all()

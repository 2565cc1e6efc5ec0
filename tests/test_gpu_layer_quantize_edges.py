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


def _norm_nvfp4(lib, x, weight, layout):
    m, k = x.shape
    q = torch.zeros((m, k // 2), dtype=torch.uint8, device="cuda")
    sf = torch.zeros(lib.nvfp4_sf_bytes(m, k, layout), dtype=torch.uint8, device="cuda")
    lib.add_rms_norm_nvfp4_quantize(x, None, weight, scalar(1e-6), scalar(448.0), None, q, sf, layout, m, k)
    torch.cuda.synchronize()
    return q, sf


@pytest.mark.parametrize("k", [16, 256, 5120, 16384])
@pytest.mark.parametrize("m", [3, 200])
def test_nan_in_a_norm_is_not_lost(lib, m, k):
    """A NaN makes its row NaN, as a scale of 0x7F in every block of it, and no
    other row moves; a NaN weight the blocks of its column."""
    x, weight = _rows(m, k, 6), torch.ones(k, dtype=torch.bfloat16, device="cuda")
    q0, s0 = _norm_nvfp4(lib, x, weight, lib.SF_LINEAR)
    s0 = s0.reshape(m, -1)
    x[1, k // 2] = NAN
    q, s = _norm_nvfp4(lib, x, weight, lib.SF_LINEAR)
    s = s.reshape(m, -1)
    keep = torch.arange(m, device="cuda") != 1
    assert (s[1] == 0x7F).all()
    assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
    swizzled = _norm_nvfp4(lib, x, weight, lib.SF_SWIZZLED_128x4)[1]
    assert int((swizzled == 0x7F).sum()) == k // 16
    x = _rows(m, k, 6)
    weight[k - 1] = NAN
    q, s = _norm_nvfp4(lib, x, weight, lib.SF_LINEAR)
    s = s.reshape(m, -1)
    assert (s[:, -1] == 0x7F).all() and torch.equal(s[:, :-1], s0[:, :-1]) and torch.equal(q[:, :k // 2 - 8], q0[:, :k // 2 - 8])


@pytest.mark.parametrize("group", [0, 128])
def test_nan_in_an_fp8_norm(lib, group):
    """E4M3 has a NaN of its own: the row's values are it, its scales 1; a NaN
    weight is its column's values, and no scale's."""
    x, weight = _rows(4, 512, 7), torch.ones(512, dtype=torch.bfloat16, device="cuda")
    weight[7] = 0
    q0, s0 = _norm_fp8(lib, x, weight, group)
    x[2, 300] = NAN
    q, s = _norm_fp8(lib, x, weight, group)
    assert torch.isnan(q[2].view(torch.float8_e4m3fn).float()).all() and (s[2] == 1).all()
    keep = torch.arange(4, device="cuda") != 2
    assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
    x = _rows(4, 512, 7)
    weight[7] = NAN
    q, s = _norm_fp8(lib, x, weight, group)
    assert torch.isnan(q[:, 7].view(torch.float8_e4m3fn).float()).all() and torch.equal(s, s0)
    q[:, 7] = q0[:, 7]
    assert torch.equal(q, q0)


@pytest.mark.parametrize("d", [64, 128])
def test_cache_write_of_what_is_not_finite(lib, d):
    """Each block as nvfp4_quantize makes it: a NaN does not count for the
    block's largest magnitude, and the cache holds finite numbers only."""
    n, heads, page = 37, 2, 16
    k, v = _rows(n, heads * d, 8), _rows(n, heads * d, 9)
    k[1, 3], k[2, 16:32], v[3, 5], v[4, 16:32] = NAN, NAN, NAN, NAN
    k[5, 7], v[6, 8], k[7], v[7] = float("inf"), -float("inf"), NAN, NAN
    slots = torch.randperm(3 * page, device="cuda")[:n]
    gs = scalar(448.0)
    cache = torch.zeros(lib.nvfp4_kv_cache_bytes(3, page, heads, d), dtype=torch.uint8, device="cuda")
    lib.nvfp4_kv_cache_write(k, v, heads * d, heads * d, slots, gs, gs, cache, n, heads, d, 3, page)
    rec = cache.reshape(3, heads, 1, 18 * d)[slots // page, :, 0].reshape(n * heads, 18 * d).long()
    tok = (slots % 16).repeat_interleave(heads)[:, None]
    b, x = torch.arange(d // 16, device="cuda"), torch.arange(d // 2, device="cuda")
    got = [torch.gather(rec, 1, at) for at in (tok * (d // 2) + x, 8 * d + tok * (d // 16) + b,
                                               9 * d + (x // 8 * 16 + tok) * 8 + x % 8, 17 * d + b * 16 + tok)]
    for (codes, sf), t in ((got[:2], k), (got[2:], v)):
        q = torch.zeros((n * heads, d // 2), dtype=torch.uint8, device="cuda")
        s = torch.zeros((n * heads, d // 16), dtype=torch.uint8, device="cuda")
        lib.nvfp4_quantize(t.reshape(n * heads, d), n * heads, d, gs, q, s, lib.SF_LINEAR)
        assert torch.equal(codes, q.long()) and torch.equal(sf, s.long())
        assert ((sf & 0x7F) != 0x7F).all()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    lib.nvfp4_kv_cache_read(cache, slots, 1 / gs, 1 / gs, ko, vo, n, heads, d, 3, page)
    torch.cuda.synchronize()
    assert torch.isfinite(ko.float()).all() and torch.isfinite(vo.float()).all()

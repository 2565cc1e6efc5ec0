"""The decoder layer of examples/decoder_layer.py against the oracle, half by
half, on weights that the oracle dequantizes."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_host, host

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

HIDDEN, INTER, LENS = 512, 1024, [70, 33, 1]
# A requantized value moves by a code where products of other sizes sum in
# another order: at most 0.5 % of them (tolerance.MAX_FLIP_FRAC), by a quarter
# of their size on average (the steps of E2M1 are 1/6 to 1/2 of the value).
# Two requantized tensors enter each half, keys and values or the MLP's input
# and hidden values, and the half's result is rounded to bf16.
HALF = (2 * 0.005) ** 0.5 / 4 + 2.0 ** -8


class Plain:
    """A layer and, in plain numbers, its weights and one step's tensors."""

    def __init__(self, monkeypatch, hq, hkv, d):
        import decoder_layer as ex
        made, quantize = [], ex.quantize_weight

        def record(w):
            codes, sf, gs = quantize(w)
            made.append((host(codes).copy(), host(sf).copy()))
            return codes, sf, gs

        monkeypatch.setattr(ex, "quantize_weight", record)
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, ex.PAGE
        self.layer = ex.DecoderLayer(hidden=HIDDEN, inter=INTER, q_heads=hq, kv_heads=hkv, head_dim=d, pages=16, seed=5)
        self.w = dict(zip(("qkv", "o", "gate_up", "down"), made))
        g = torch.Generator(device="cuda").manual_seed(6)
        m = sum(LENS)
        # (small next to what the two halves add, so that the sums show it)
        self.x, self.res = ((0.1 * torch.randn((m, HIDDEN), generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
        for i, w in enumerate((self.layer.norm1, self.layer.norm2)):
            w.copy_(1 + 0.3 * torch.randn(HIDDEN, generator=g, device="cuda"))
        self.table = torch.tensor([[3, 9, 1], [5, 0, 2], [7, 8, 4]], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32, device="cuda")
        slots = [self.table[b].long()[p // self.page] * self.page + p % self.page
                 for b, p in enumerate(torch.arange(n, device="cuda") for n in LENS)]
        self.y, self.r = self.layer.step(self.x, self.res, self.table, self.lens, self.cu, max(LENS), torch.cat(slots))
        torch.cuda.synchronize()
        self.r1 = oracle.bf16_round(bf16_host(self.x) + bf16_host(self.res))

    def quantized_norm(self, r, weight):
        y = r / np.sqrt((r * r).mean(-1, keepdims=True) + np.float64(np.float32(1e-6))) * bf16_host(weight)
        return oracle.quantize_nvfp4(y.astype(np.float32), host(self.layer.gs_x)[0])


def _off(a, b, rounded):
    """|a - b| beyond the rounding of `rounded` to bf16, against |b|'s part."""
    return max(np.linalg.norm(a - b) - 2.0 ** -8 * np.linalg.norm(rounded), 0.0)


@pytest.fixture(params=[(8, 2, 128), (8, 8, 64)], ids=["gqa128", "mha64"])
def plain(request, lib, monkeypatch):
    return Plain(monkeypatch, *request.param)


def test_attention_half(plain):
    """norm, projections, cache, attention and output projection: what they
    add to the residual."""
    p, layer = plain, plain.layer
    qkv = oracle.gemm_w4a4(*p.quantized_norm(p.r1, layer.norm1), *p.w["qkv"], host(layer.alpha_qkv)[0])
    q, k, v = np.split(qkv, [p.hq * p.d, (p.hq + p.hkv) * p.d], axis=1)
    gs = host(layer.gs_kv)[0]
    kd, vd = (oracle.dequantize_nvfp4(*oracle.quantize_nvfp4(t.reshape(-1, p.d).astype(np.float32), gs)).reshape(-1, p.hkv, p.d) / gs
              for t in (k, v))
    q, out, at = q.reshape(-1, p.hq, p.d), np.zeros((len(q), p.hq, p.d)), 0
    for n in LENS:
        for h in range(p.hq):
            kv = h // (p.hq // p.hkv)
            s = q[at:at + n, h] @ kd[at:at + n, kv].T * p.d ** -0.5
            s[np.triu_indices(n, 1)] = -np.inf
            e = np.exp(s - s.max(-1, keepdims=True))
            out[at:at + n, h] = e @ vd[at:at + n, kv] / e.sum(-1, keepdims=True)
        at += n
    attn = oracle.gemm_w4a16(oracle.bf16_round(out).reshape(-1, p.hq * p.d), *p.w["o"], host(layer.alpha_o)[0])
    r = bf16_host(p.r)
    assert np.linalg.norm(attn) > 0.5 * np.linalg.norm(p.r1)
    assert _off(r, p.r1 + attn, r) <= HALF * np.linalg.norm(attn)


def test_mlp_half(plain):
    """The second norm, gate_up, SwiGLU and down_proj, from the residual that
    the layer returns."""
    p, layer = plain, plain.layer
    gate_up = oracle.gemm_w4a4(*p.quantized_norm(bf16_host(p.r), layer.norm2), *p.w["gate_up"],
                               host(layer.alpha_gate_up)[0], round_bf16=False)
    h = oracle.quantize_nvfp4(oracle.swiglu_h(gate_up), host(layer.gs_h)[0])
    y = oracle.gemm_w4a4(*h, *p.w["down"], host(layer.alpha_down)[0])
    assert np.linalg.norm(bf16_host(p.y) - y) <= HALF * np.linalg.norm(y)


def test_residual_bit_for_bit(plain, lib):
    """The returned residual is bf16(bf16(x + residual) + the attention's output)."""
    p, layer = plain, plain.layer
    m, wq, row = sum(LENS), p.hq * p.d, layer.qkv.n
    r1 = torch.empty_like(p.x)
    a, sf = layer.quantized_norm(p.x, p.res, layer.norm1, r1)
    assert np.array_equal(bf16_host(r1), p.r1)
    qkv = torch.empty((m, row), dtype=torch.bfloat16, device="cuda")
    ws, n = layer.workspace(lib.nvfp4_workspace_bytes(m, row, HIDDEN))
    lib.nvfp4_gemm(a, sf, layer.qkv.codes, layer.qkv.sf, layer.alpha_qkv, qkv, m, row, HIDDEN, ws, n)
    out = torch.empty((m, wq), dtype=torch.bfloat16, device="cuda")
    ws, n = layer.workspace(lib.nvfp4_kv_attention_workspace_bytes(m, 3, max(LENS), p.hq, p.hkv, p.d))
    lib.nvfp4_kv_attention(qkv, row, p.cu, layer.cache, p.table, p.lens, layer.qk_scale, layer.v_scale, out, None, m, 3,
                           max(LENS), p.hq, p.hkv, p.d, layer.pages, p.page, 3, 0, ws, n)
    attn = torch.empty((m, HIDDEN), dtype=torch.bfloat16, device="cuda")
    ws, n = layer.workspace(lib.bf16_fp4_gemm_workspace_bytes(m, HIDDEN, wq))
    lib.bf16_fp4_gemm(out, layer.o.codes, layer.o.sf, layer.alpha_o, attn, m, HIDDEN, wq, ws, n)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_host(p.r), oracle.bf16_round(p.r1 + bf16_host(attn)))

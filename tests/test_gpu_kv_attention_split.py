"""Units of the NVFP4 attention that several CTAs share: the plans that cut
them, the joins of their partial results, and waits that give up."""
import numpy as np
import pytest
import torch

from gpu_util import bf16_host, dev, host
from kv_util import check_attention
from test_gpu_kv_attention import Problem

pytestmark = pytest.mark.gpu


def _equal(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("seqs,hq,hkv,d", [
    ([(2600, 300)], 10, 2, 128), ([(1500, 300), (4000, 1), (900, 33)], 8, 2, 64), ([(9000, 40)], 8, 1, 128),
    ([(6000, 70)], 8, 1, 64), ([(5000, 4)] * 3, 16, 2, 128)])
def test_joins_take_this_calls_partial_results(lib, seqs, hq, hkv, d):
    """Two calls of one shape and different data take turns on one workspace:
    a partial result of the call before, read too early, would show."""
    ps = [Problem(seqs, hq, hkv, d, 16, seed=s, q_scale=q) for s, q in ((11, 1.0), (12, 5.0))]
    ts = [p.device() for p in ps]
    alone = [p.call(lib, t, p.workspace(lib)) for p, t in zip(ps, ts)]
    torch.cuda.synchronize()
    assert not _equal(*alone)
    ws = ps[0].workspace(lib)
    got = [(i, ps[i].call(lib, ts[i], ws)) for i in [0, 1] * 20]
    torch.cuda.synchronize()
    assert all(_equal(o, alone[i]) for i, o in got)
    assert not ws[:65536].any()


# What gives up first: the decode form's wait for its copies, the chunk form's
# for the first probabilities.
GIVES_UP = [([(9000, 1)] * 4, 8, 2, 128), ([(9000, 4)] * 2, 16, 2, 64), ([(2600, 700)], 8, 2, 128), ([(2600, 70)], 8, 2, 64)]


@pytest.mark.parametrize("seqs,hq,hkv,d", GIVES_UP)
def test_a_wait_that_runs_out_is_reported(lib, seqs, hq, hkv, d):
    """With a wait limit of one poll both forms record the timeout and return;
    after the workspace is zero-filled again the next call is right."""
    p = Problem(seqs, hq, hkv, d, 16, seed=13)
    t = p.device()
    ref = p.call(lib, t, p.workspace(lib))
    assert lib.nvfp4_get_device_status() == lib.OK
    ws = p.workspace(lib)
    lib.nvfp4_set_wait_limit(1)
    try:
        p.call(lib, t, ws)
        status = lib.nvfp4_get_device_status()
    finally:
        lib.nvfp4_set_wait_limit(0)
    assert status == lib.ERR_DEVICE_TIMEOUT
    ws.zero_()
    again = p.call(lib, t, ws)
    torch.cuda.synchronize()
    assert _equal(again, ref) and lib.nvfp4_get_device_status() == lib.OK


@pytest.mark.parametrize("seqs,hq,hkv,d", [([(4100, 1), (2050, 1)], 8, 1, 128), ([(5000, 4)] * 2, 8, 1, 64),
                                           ([(2600, 300)], 8, 2, 128)])
def test_a_workspace_that_is_too_small_splits_nothing(lib, seqs, hq, hkv, d):
    """Room for a few partial results is not room for the call's: units stay
    whole, as without a workspace, and every CTA works."""
    p = Problem(seqs, hq, hkv, d, 16, seed=14)
    t = p.device()
    whole = p.call(lib, t, None)
    full = p.workspace(lib)
    split = p.call(lib, t, full)
    torch.cuda.synchronize()
    assert not _equal(whole, split)
    for n in (65536 // 2, 65536 + (full.numel() - 65536) // 40, full.numel() - 16):
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        got = p.call(lib, t, ws)
        torch.cuda.synchronize()
        assert _equal(got, whole) and not ws.any()


@pytest.mark.parametrize("seqs,hq,hkv,d", [([(70, 20), (2, 2)], 64, 8, 128), ([(40, 33)], 64, 8, 64)])
def test_a_chunk_in_a_table_for_a_million_tokens(lib, seqs, hq, hkv, d):
    """The size of the table bounds the work that a call may have, counted in
    the tiles of the form that runs: chunks of 8192 of 64 heads fit."""
    p = Problem(seqs, hq, hkv, d, 16, seed=15)
    wide = np.full((len(seqs), (1 << 20) // 16), -1, dtype=np.int32)
    wide[:, :p.table.shape[1]] = p.table
    ref = p.reference()
    t = p.device()
    out = torch.empty((p.tokens, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((p.tokens, hq), device="cuda")
    n = lib.nvfp4_kv_attention_workspace_bytes(p.tokens, len(seqs), 8192, hq, hkv, d)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    lib.nvfp4_kv_attention(t["q"], hq * d, t["cu"], t["cache"], dev(wide), t["lens"], t["qk"], t["vs"], out, lse,
                           p.tokens, len(seqs), 8192, hq, hkv, d, p.pages, 16, wide.shape[1], 0, ws, n)
    torch.cuda.synchronize()
    check_attention(bf16_host(out), host(lse), ref)

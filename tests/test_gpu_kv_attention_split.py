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


# ---- batches of more units than CTAs, or of units that cut unevenly: the
# decode form lays them on a line and cuts that into equal parts

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _rows_of_tile(rows):
    tiles = -(-rows // 32)
    return 8 * -(-rows // (8 * tiles))


def takes_line(seqs, group, heads, d, table_tokens):
    """Whether the decode form lays this batch's units on a line: more units
    than CTAs, or pieces of units that come out too uneven."""
    nq = _rows_of_tile(max(n for _, n in seqs) * group) // 8
    ctas = {1: 4, 2: 3, 3: 2, 4: 2}[nq] + (d == 64 and nq == 2)
    cost = 8 if nq == 1 else 12
    tiles = [-(-n * group // (8 * nq)) for _, n in seqs]
    steps = [max(-(-ln // 32), 1) for ln, _ in seqs]
    places = heads * max(tiles) * (-(-table_tokens // 32) + cost)
    grid = min(torch.cuda.get_device_properties(0).multi_processor_count * ctas, int(places * len(seqs) / 8 + 1))
    units, work = heads * sum(tiles), heads * sum(t * s for t, s in zip(tiles, steps))
    if units >= grid:
        return True
    inv = min(grid / work, 1 / 8)
    cut = lambda s: 1 if s <= 16 else 1 + int((s - 1) * inv)  # noqa: E731
    if heads * sum(t * cut(s) for t, s in zip(tiles, steps)) > grid:
        inv = min((grid - units) / (1.001 * work), 1 / 8)
    longest = max(s / cut(s) for t, s in zip(tiles, steps) if t)
    return work >= 4 * grid and longest > max(work / grid + 0.8 * cost, 16)


class Batch:
    """Random sequences over a cache of random codes and scales, made on the
    GPU; everything that no sequence holds is NaN scales."""

    def __init__(self, seqs, group, heads, d, page, window=0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 + seed)
        self.seqs, self.group, self.heads, self.d, self.page, self.window = seqs, group, heads, d, page, window
        need = [-(-ln // page) for ln, _ in seqs]
        self.pages, self.width = sum(need) + 3, max(need) + 1
        order = torch.randperm(self.pages, generator=g, device="cuda").int()
        self.table = torch.full((len(seqs), self.width), -7, dtype=torch.int32, device="cuda")
        self.cache = torch.full((self.pages, heads, page // 16, 18 * d), 0xFF, dtype=torch.uint8, device="cuda")
        at, self.kv = 0, []
        lut = torch.cat([E2M1, -E2M1]).cuda()
        for b, (ln, _) in enumerate(seqs):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            t = torch.arange(ln, device="cuda")
            pg = self.table[b, t // page].long()
            codes = torch.randint(0, 16, (2, ln, heads, d), generator=g, device="cuda", dtype=torch.uint8)
            sf = torch.randint(0x20, 0x40, (2, ln, heads, d // 16), generator=g, device="cuda", dtype=torch.uint8)
            rec, tok = t % page // 16, t % 16
            packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
            h = torch.arange(heads, device="cuda")[None, :, None]
            put = lambda col, val: self.cache.__setitem__((pg[:, None, None], h, rec[:, None, None], col[:, None, :]), val)  # noqa: E731
            x, nb = torch.arange(d // 2, device="cuda"), torch.arange(d // 16, device="cuda")
            put(tok[:, None] * (d // 2) + x, packed[0])
            put(8 * d + tok[:, None] * (d // 16) + nb, sf[0])
            put(9 * d + (x // 8 * 16 + tok[:, None]) * 8 + x % 8, packed[1])
            put(17 * d + nb * 16 + tok[:, None], sf[1])
            val = lut[codes.long()] * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
            self.kv.append((val[0], val[1]))
        self.q_lens = [n for _, n in seqs]
        self.tokens, self.hq = sum(self.q_lens), heads * group
        self.q = (torch.randn((self.tokens, self.hq, d), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
        self.lens = torch.tensor([ln for ln, _ in seqs], dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.q_lens)]), dtype=torch.int32, device="cuda")
        self.qk = torch.full((1,), 0.5 * d ** -0.5, device="cuda")
        self.vs = torch.full((1,), 0.01, device="cuda")

    def workspace(self, lib):
        n = lib.nvfp4_kv_attention_workspace_bytes(self.tokens, len(self.seqs), max(self.q_lens), self.hq, self.heads, self.d)
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def call(self, lib, ws):
        out = torch.full((self.tokens, self.hq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.tokens, self.hq), float("nan"), device="cuda")
        lib.nvfp4_kv_attention(self.q, self.hq * self.d, self.cu, self.cache, self.table, self.lens, self.qk, self.vs,
                               out, lse, self.tokens, len(self.seqs), max(self.q_lens), self.hq, self.heads, self.d,
                               self.pages, self.page, self.width, self.window, ws, 0 if ws is None else ws.numel())
        return out, lse

    def reference(self):
        """(out, lse, spread, reach, mass) as kv_util.attention's."""
        got, at = [[] for _ in range(5)], 0
        qk, vs = self.qk.double(), self.vs.double()
        for (ln, n), (k, v) in zip(self.seqs, self.kv):
            if n == 0:
                continue
            q = self.q[at:at + n].double().reshape(n, self.heads, self.group, self.d)
            at += n
            pos, t = ln - n + torch.arange(n, device="cuda")[:, None], torch.arange(ln, device="cuda")
            see = (t <= pos) & (t > pos - (self.window or 1 << 40))
            hidden = ~see[:, None, None, :]
            s = (torch.einsum("nhgd,thd->nhgt", q, k) * qk).masked_fill(hidden, -torch.inf)
            reach = (torch.einsum("nhgd,thd->nhgt", q.abs(), k.abs()) * qk).masked_fill(hidden, 0.0)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
            out, spread = (torch.einsum("nhgt,thd->nhgd", p, x) * vs for x in (v, v.abs()))
            mass = torch.einsum("nt,thd->nhd", see.double(), v.abs())[:, :, None].expand_as(out) * vs
            top = reach.amax(-1) if ln else torch.zeros_like(lse)
            for to, x in zip(got, (out, lse, spread, top, mass)):
                to.append(x.reshape(n, self.hq, *x.shape[3:]))
        return tuple(torch.cat(x).cpu().numpy() for x in got)


def _mixed(n, lo, hi, queries, seed):
    """n sequences of lo to hi tokens; some empty, some without a query."""
    g = np.random.default_rng([31, n, lo, hi, seed])
    seqs = [(int(x), int(g.integers(1, queries + 1))) for x in np.exp(g.uniform(np.log(lo), np.log(hi), n))]
    seqs[3], seqs[n // 2], seqs[-2] = (0, 1), (lo, 0), (1, queries)
    seqs[5] = (hi, queries)
    return seqs


LINE = [
    # sequences, query heads a group, key/value heads, head_dim, page, window
    (_mixed(170, 200, 900, 1, 0), 5, 4, 128, 16, 0), (_mixed(170, 200, 900, 1, 1), 8, 4, 64, 32, 0),
    (_mixed(66, 100, 900, 1, 2), 12, 8, 128, 32, 0), (_mixed(90, 100, 700, 2, 3), 8, 8, 64, 16, 150),
    (_mixed(45, 100, 1200, 3, 4), 8, 8, 128, 16, 0), (_mixed(45, 100, 1200, 3, 5), 7, 8, 64, 48, 333),
    (_mixed(45, 100, 1200, 4, 6), 8, 8, 128, 64, 100), (_mixed(45, 100, 1200, 4, 7), 8, 8, 64, 16, 0),
    (_mixed(30, 100, 1200, 8, 8), 8, 8, 64, 16, 0),
    # fewer units than CTAs, cut unevenly; up to 32 sequences (a lane each) and more
    ([(1024, 4)] * 24, 8, 8, 128, 64, 0), ([(1500, 4)] * 24, 8, 8, 64, 16, 0), ([(800, 1)] * 50, 8, 8, 128, 32, 0),
    ([(900, 1)] * 49 + [(17, 1)], 4, 8, 64, 16, 500), ([(1300, 2)] * 29 + [(3, 1)], 8, 8, 128, 16, 0)]


@pytest.mark.parametrize("case", range(len(LINE)))
def test_batches_on_a_line(lib, case):
    """Against 64 bits, whole and split; equal bits from call to call, and the
    counters zero after each."""
    seqs, group, heads, d, page, window = LINE[case]
    b = Batch(seqs, group, heads, d, page, window, seed=case)
    assert window or takes_line(seqs, group, heads, d, b.width * page)      # (a window shortens the steps)
    ws = b.workspace(lib)
    ref = b.reference()
    first = b.call(lib, ws)
    for got in (first, b.call(lib, None)):
        torch.cuda.synchronize()
        check_attention(bf16_host(got[0]), host(got[1]), ref)
    for _ in range(5):
        assert _equal(b.call(lib, ws), first)
    torch.cuda.synchronize()
    assert not ws[:65536].any()
    assert lib.nvfp4_get_device_status() == lib.OK

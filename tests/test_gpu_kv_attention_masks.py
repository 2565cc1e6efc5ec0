"""What the NVFP4 attention must not use (tokens in front of a window), and
scale factors that are not numbers."""
import numpy as np
import pytest
import torch

from gpu_util import dev, scalar
from kv_util import offsets
from test_gpu_kv_attention import Problem

pytestmark = pytest.mark.gpu


def _visible(p, b, window):
    """Tokens that some query of sequence b sees."""
    n = int(p.lens[b])
    return range(max(n - p.q_lens[b] - window + 1, 0), n) if p.q_lens[b] else range(0)


def _filled(p, window, fill):
    """The cache with every byte of a token that no query sees set to `fill`."""
    c = np.full_like(p.cache.bytes, fill)
    for b in range(len(p.lens)):
        for t in _visible(p, b, window):
            at = int(p.table[b, t // p.page]), slice(None), t % p.page // 16
            for o in offsets(t % 16, p.d):
                c[at][:, o] = p.cache.bytes[at][:, o]
    return c


STALE = [
    # sequences (length, queries), query heads, key/value heads, page
    ([(300, 1)], 8, 2, 16), ([(300, 1), (90, 1), (41, 1)], 5, 1, 16), ([(300, 3), (77, 4)], 16, 2, 32),
    ([(700, 4)], 8, 1, 16), ([(300, 40)], 4, 1, 16), ([(600, 150), (310, 1), (333, 70)], 3, 1, 16),
    ([(900, 300)], 2, 2, 64)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [1, 7, 33, 100, 131, 270])
@pytest.mark.parametrize("seqs,hq,hkv,page", STALE)
def test_stale_bytes_in_front_of_a_window(lib, seqs, hq, hkv, page, window, d):
    """Tokens in front of every query's window may hold anything, NaN scales
    among it: a server has given their pages to others, or points their
    entries at one page that was never written."""
    p = Problem(seqs, hq, hkv, d, page, seed=21)
    t, ws = p.device(), p.workspace(lib)
    ref = p.call(lib, t, ws, window)
    torch.cuda.synchronize()
    assert torch.isfinite(ref[0]).all() and torch.isfinite(ref[1]).all()
    free = next(x for x in range(p.pages) if not any(
        x in p.table[b, :-(-int(n) // page)] for b, n in enumerate(p.lens)))
    table = p.table.copy()
    for b in range(len(p.lens)):
        seen = _visible(p, b, window)
        table[b, :(seen[0] if len(seen) else 0) // page] = free
    for fill in (0x7F, 0xFF, 0x7E):
        c = dev(_filled(p, window, fill))
        for tab in (t["table"], dev(table)):
            out, lse = p.call(lib, dict(t, cache=c, table=tab), ws, window)
            torch.cuda.synchronize()
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


SCALES = [([(40, 1), (300, 1), (0, 1)], 8, 2), ([(300, 4), (2, 4)], 8, 1), ([(300, 40), (20, 30)], 8, 2)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs,hq,hkv", SCALES)
def test_scales_that_are_nan(lib, seqs, hq, hkv, d):
    """A NaN score scale makes every row NaN that sees anything, log-sum-exp
    included; a NaN value scale the outputs alone."""
    p = Problem(seqs, hq, hkv, d, 16, seed=22)
    t, ws = p.device(), p.workspace(lib)
    ref = p.call(lib, t, ws)
    torch.cuda.synchronize()
    sees = torch.isfinite(ref[1])
    assert not sees.all() and sees.any()
    for sign in (1.0, -1.0):
        out, lse = p.call(lib, dict(t, qk=scalar(sign * float("nan"))), ws)
        torch.cuda.synchronize()
        assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
        assert (out[~sees] == 0).all() and torch.isneginf(lse[~sees]).all()
    out, lse = p.call(lib, dict(t, vs=scalar(float("nan"))), ws)
    torch.cuda.synchronize()
    assert torch.isnan(out[sees]).all() and (out[~sees] == 0).all()
    assert torch.equal(lse, ref[1])

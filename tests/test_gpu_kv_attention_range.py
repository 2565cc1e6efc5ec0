"""Scores that are large, alike or far apart: the NVFP4 attention's running
reference over long rows, and beyond fp32's integers."""
import numpy as np
import pytest
import torch

from gpu_util import bf16_host, host
from kv_util import check_attention
from test_gpu_kv_attention import Problem
from test_gpu_kv_attention_split import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("workspace", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,queries", [(5, 1), (12, 1), (8, 3), (8, 4), (16, 5)])
def test_long_rows_of_large_scores(lib, group, queries, d, workspace):
    """60,000 tokens whose scores are all near one large number, another one
    for each row: the probabilities are nearly flat, and every step's share of
    the sum and of the output has to keep its weight."""
    b = Batch([(60000, queries)], group, 1, d, 64, seed=40 + d + group)
    # the first block of every key is 4.0 * 0.5, the first block of a query row its own constant
    k = b.kv[0][0]
    t = torch.arange(60000, device="cuda")
    for i in range(16):                              # token i of every record
        at = t[t % 16 == i]
        page, g = b.table[0, at // 64].long(), at % 64 // 16
        b.cache[page, 0, g, i * (d // 2):i * (d // 2) + 8] = 0x66
        b.cache[page, 0, g, 8 * d + i * (d // 16)] = 0x30
    k[:, :, :16] = 2.0
    rows = b.q.view(-1, d)
    rows *= 0.05
    rows[:, :16] = (torch.linspace(300.0, 900.0, len(rows), device="cuda") / (32 * b.qk))[:, None].to(torch.bfloat16)
    out, lse = b.call(lib, b.workspace(lib) if workspace else None)
    torch.cuda.synchronize()
    ref = b.reference()
    assert ref[1].min() > 200
    check_attention(bf16_host(out), host(lse), ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_scale", [1e6, 1e7, 1e8, 1e9, 1e12, 1e20, 1e30], ids=str)
@pytest.mark.parametrize("seqs,hq,hkv", [([(50, 1), (300, 1)], 5, 1), ([(200, 4), (31, 4)], 8, 1), ([(300, 40), (90, 30)], 8, 2)])
def test_scores_past_the_integers(lib, seqs, hq, hkv, q_scale, d):
    """A finite score, however large, has a softmax: of a row whose largest
    score stands apart by more than fp32's roundings, its token's value."""
    p = Problem(seqs, hq, hkv, d, 16, seed=41, q_scale=q_scale)
    out, lse = p.call(lib, p.device(), p.workspace(lib))
    torch.cuda.synchronize()
    ref = p.reference()
    check_attention(bf16_host(out), host(lse), ref)
    got, sharp, at = bf16_host(out), 0, 0
    for b, n in enumerate(p.q_lens):
        kv = [p.cache.token(int(p.table[b, t // 16]) * 16 + t % 16) for t in range(int(p.lens[b]))]
        for i in range(at, at + n):
            last = int(p.lens[b]) - n + i - at + 1
            for h in range(hq):
                k = np.stack([x[0][h // (hq // hkv)] for x in kv[:last]])
                s = np.sort(k @ p.q[i, h]) * float(p.qk_scale)
                if last > 1 and s[-1] - s[-2] <= 40 + ref[3][i, h] * 2.0 ** -18:
                    continue
                sharp += 1
                v = kv[int(np.argmax(k @ p.q[i, h]))][1][h // (hq // hkv)] * float(p.v_scale)
                assert (np.abs(got[i, h] - v) <= np.abs(v) * 2.0 ** -8 * 1.01).all(), (i, h)
        at += n
    assert sharp > p.tokens * hq // 2

"""Scores that are large and alike: the NVFP4 attention's running reference over
long rows."""
import pytest
import torch

from gpu_util import bf16_host, host
from kv_util import check_attention
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

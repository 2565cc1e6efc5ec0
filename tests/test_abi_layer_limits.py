"""The layer operators' size limits, calls on nothing, and what the binding
takes for a pointer.  No GPU needed: a call that is accepted has no tokens."""
import numpy as np
import pytest

import nvfp4_quantized_dense_gb300 as nv
from nvfp4_quantized_dense_gb300 import build as nvbuild

FAKE = 1 << 20   # 16-byte aligned address that is never dereferenced
INV, SHAPE = nv.ERR_INVALID_ARG, nv.ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return nv.load()


def _attend(lib, max_q, hq, hkv, d, table_tokens, page=16):
    """Status of a call without tokens."""
    return lib.nvfp4_kv_attention(FAKE, hq * d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, 1, max_q, hq, hkv, d,
                                  9, page, table_tokens // page, 0, None, 0, None)


# Places on the line of one sequence: key/value heads * query tiles * (steps of
# the table + a unit's cost), below 2^31.
@pytest.mark.parametrize("max_q,hq,hkv,d,table", [
    (8192, 64, 8, 128, 1 << 20), (131072, 64, 8, 128, 131072), (131072, 40, 8, 128, 131072), (1 << 20, 8, 8, 128, 1 << 20),
    (1, 64, 8, 128, 1 << 30), (4, 64, 8, 128, 1 << 30), (8, 64, 8, 64, 1 << 30), (9, 64, 8, 64, 1 << 30),
    (1, 32, 32, 128, 1 << 30), (5, 64, 8, 128, 1 << 30)])
def test_sizes_that_fit(lib, max_q, hq, hkv, d, table):
    assert _attend(lib, max_q, hq, hkv, d, table) not in (INV, SHAPE)


@pytest.mark.parametrize("max_q,hq,hkv,d,table", [
    (1, 64, 64, 128, 1 << 30), (8, 256, 32, 64, 1 << 30), (1 << 28, 8, 8, 128, 1 << 20), (1 << 20, 1024, 8, 64, 1 << 20),
    (33, 256, 256, 128, 1 << 30)])
def test_sizes_that_do_not(lib, max_q, hq, hkv, d, table):
    assert _attend(lib, max_q, hq, hkv, d, table) == SHAPE


def test_workspace_of_sizes_that_are_refused(lib):
    """0 bytes for what the call would refuse, however large the numbers."""
    f = nv.nvfp4_kv_attention_workspace_bytes
    assert f(4, 4, 1, 8, 2, 128) > 65536
    for bad in ((4, 65537, 1, 8, 2, 128), (1 << 31, 4, 1, 8, 2, 128), (4, 4, (1 << 28) + 1, 8, 2, 128),
                (4, 4, 1 << 62, 8, 2, 128), (4, 4, 1, 2048, 2, 128), (4, 4, 1, 1 << 62, 1 << 61, 128),
                (4, 4, 1, 8, 8, 256)):
        assert f(*bad) == 0, bad

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


def test_calls_on_nothing(lib):
    """No rows, tokens or sequences: the tensors may have no memory (an empty
    tensor's address is NULL), and the answer is never a refusal."""
    refused = (INV, SHAPE)
    z = None
    assert lib.add_rms_norm_nvfp4_quantize(z, z, FAKE, FAKE, FAKE, z, z, z, 0, 0, 256, None) not in refused
    assert lib.add_rms_norm_nvfp4_quantize(z, z, z, z, z, z, z, z, 0, 0, 256, None) not in refused
    assert lib.add_rms_norm_fp8_quantize(z, z, FAKE, FAKE, z, z, z, 128, 0, 256, None) not in refused
    assert lib.nvfp4_kv_cache_write(z, z, 256, 256, z, FAKE, FAKE, FAKE, 0, 2, 128, 3, 16, None) not in refused
    assert lib.nvfp4_kv_cache_read(FAKE, z, FAKE, FAKE, z, z, 0, 2, 128, 3, 16, None) not in refused
    attend = lib.nvfp4_kv_attention
    #              q  qs    cu    cache table lens  qk    vs    out lse tok b mq hq hkv d  pages page maxp win ws ws_b st
    assert attend(z, 1024, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, z, z, 0, 4, 0, 8, 2, 128, 9, 16, 3, 0, z, 0, None) not in refused
    assert attend(z, 1024, z, FAKE, z, z, FAKE, FAKE, z, z, 0, 0, 1, 8, 2, 128, 9, 16, 3, 0, z, 0, None) not in refused
    # what does not depend on the number of tokens is checked all the same
    assert lib.add_rms_norm_nvfp4_quantize(z, z, FAKE, FAKE, FAKE, z, z, z, 0, 0, 250, None) == SHAPE
    assert lib.nvfp4_kv_cache_write(z, z, 256, 256, z, FAKE, FAKE, FAKE, 0, 2, 96, 3, 16, None) == SHAPE
    assert attend(z, 1024, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, z, z, 0, 4, -1, 8, 2, 128, 9, 16, 3, 0, z, 0, None) == INV
    assert attend(z, 1024, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, z, z, 0, 4, 1, 8, 3, 128, 9, 16, 3, 0, z, 0, None) == INV


@pytest.mark.parametrize("bad", [b"0123456789abcdef", "text", bytearray(16), 1.5, np.zeros(4, np.float32), [1]], ids=lambda x: type(x).__name__)
def test_pointers_are_tensors_integers_or_none(lib, bad):
    """Host memory never reaches a kernel by way of the binding."""
    with pytest.raises(AttributeError):
        nv.nvfp4_kv_cache_write(bad, FAKE, 256, 256, FAKE, FAKE, FAKE, FAKE, 0, 2, 96, 3, 16, stream=0)
    with pytest.raises(AttributeError):
        nv.nvfp4_quantize(bad, 0, 250, FAKE, FAKE, FAKE, stream=0)

"""The layer operators on nothing: no rows, no tokens, no sequences."""
import pytest
import torch

from gpu_util import scalar

pytestmark = pytest.mark.gpu


def test_empty_tensors(lib):
    """A step without new tokens, as the tensors of one come: nothing is
    launched and nothing refused."""
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    u8, one = torch.uint8, scalar(1.0)
    lib.add_rms_norm_nvfp4_quantize(e(0, 256), e(0, 256), e(256), one, one, e(0, 256), e(0, 128, dtype=u8), e(0, dtype=u8),
                                    lib.SF_SWIZZLED_128x4, 0, 256)
    lib.add_rms_norm_fp8_quantize(e(0, 256), None, e(256), one, None, e(0, 256, dtype=u8), e(0, 2, dtype=torch.float32), 128, 0, 256)
    cache = torch.zeros(lib.nvfp4_kv_cache_bytes(2, 16, 2, 64), dtype=u8, device="cuda")
    slots = e(0, dtype=torch.int64)
    lib.nvfp4_kv_cache_write(e(0, 128), e(0, 128), 128, 128, slots, one, one, cache, 0, 2, 64, 2, 16)
    lib.nvfp4_kv_cache_read(cache, slots, one, one, e(0, 128), e(0, 128), 0, 2, 64, 2, 16)
    zeros = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert lib.nvfp4_kv_attention_workspace_bytes(0, 3, 0, 4, 2, 64) == 0
    lib.nvfp4_kv_attention(e(0, 256), 256, zeros, cache, zeros[:3].reshape(3, 1), zeros[:3], one, one, e(0, 256), None, 0, 3,
                           0, 4, 2, 64, 2, 16, 1)
    lib.nvfp4_kv_attention(e(0, 256), 256, None, cache, e(0, 1, dtype=torch.int32), e(0, dtype=torch.int32), one, one,
                           e(0, 256), None, 0, 0, 1, 4, 2, 64, 2, 16, 1)
    torch.cuda.synchronize()
    assert not cache.any() and lib.nvfp4_get_device_status() == lib.OK

"""The attention's workspace stays bounded (no GPU)."""
import pytest

from skinny_gemm_gb300 import ops

GIB = 1 << 30


@pytest.mark.parametrize("T,max_len", [(2048, 131072), (8192, 131072), (8192, 8192), (32768, 32768), (100000, 1 << 20)])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 256), (32, 8, 128), (28, 4, 128), (12, 4, 64)])
@pytest.mark.parametrize("window", [0, 1000, 50000])
def test_long_prompts(T, max_len, hq, hkv, dim, window):
    """Partial results of at most 2^32 bytes, and of the rest (the parts of divided groups) a tenth."""
    n = ops.lib().w4a16_kv_attention_workspace_bytes(1, T, hq, hkv, dim, min(T, max_len), max_len, window)
    groups = min(-(-max_len // 1024), (window + T - 2) // 1024 + 2 if window else max_len)
    if groups * T * hq > 2 ** 31 - 1:
        assert n == 0
    else:
        assert 0 < n < 4.1 * GIB
        assert n >= min(2 * GIB, groups * T * hq * (4 * dim + 8))  # (launches of equal size)


def test_small_steps_have_a_slot_for_every_group_of_every_row():
    """What fits is taken in one launch."""
    for B, T, hq, hkv, dim, max_new, max_len in ((64, 64, 8, 2, 256, 1, 16000), (3, 900, 28, 4, 128, 300, 6300),
                                                 (1, 1, 8, 2, 256, 1, 131072)):
        n = ops.lib().w4a16_kv_attention_workspace_bytes(B, T, hq, hkv, dim, max_new, max_len, 0)
        need = -(-max_len // 1024) * T * hq * (4 * dim + 8)
        assert need <= n < need + 0.1 * GIB
    n = ops.lib().w4a16_kv_attention_workspace_bytes(4, 4096, 32, 8, 128, 1024, 1024, 0)
    assert n < 0.1 * GIB  # one group a row: written out at once

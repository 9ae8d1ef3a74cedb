"""The paged attention at the ends of its ranges: lengths, windows, offsets, scales and workspaces."""
import pytest
import torch

from kv_cases import Step, assert_close
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (4, 4, 64)])
def test_windows_longer_than_any_request(hq, hkv, dim):
    """A window up to 2^31 - 1 is no window: prompts of several row tiles from an empty cache, and beside others."""
    step = Step(hq, hkv, dim, 16, [0, 3, 200, 0], [300, 130, 40, 1], seed=dim)
    cache = step.cache()
    want = step.run(cache=cache)
    ref, bound = step.reference()
    assert_close(want, ref, bound)
    for window in (max(step.lens), TOP - 33, TOP - 8, TOP - 1, TOP):
        assert torch.equal(step.run(window=window, cache=cache), want), window
    assert ops.device_status() == 0

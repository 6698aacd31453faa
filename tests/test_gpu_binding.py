"""What the Python binding of the serving operators refuses, on both of its
routes (the C++ one, and the Python one that a stream argument takes)."""
import pytest
import torch

from gpu_util import require_gpu
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200.device import i32_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_count_without_an_element_copies_nothing(own_stream):
    """num_pairs without an element is no count; it must not mean "all"."""
    st = torch.cuda.current_stream() if own_stream else None
    kp = torch.arange(4 * 16 * 64, device="cuda").view(4, 16, 1, 64).to(
        torch.bfloat16)
    vp = -kp
    k0, v0 = kp.clone(), vp.clone()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="num_pairs"):
        _lib.tv_page_copy(kp, vp, i32_tensor([0]), i32_tensor([3]),
                          num_pairs=none, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(kp, k0) and torch.equal(vp, v0)

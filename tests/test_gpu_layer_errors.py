"""Errors that are neither the arguments' nor the library's."""
import pytest

import tensor_core_tiled_02_gb300 as tc

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def test_out_of_memory_is_torch_s_own_error():
    """An output of 8 TiB: nothing is launched, and what catches torch's error catches this one."""
    x = torch.zeros(1 << 21, 8, device="cuda", dtype=torch.float16)
    w = torch.zeros(8, 1 << 21, device="cuda", dtype=torch.float16)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        tc.linear(x, w)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        tc.gated_ffn(x, w, w, torch.zeros(1 << 21, 8, device="cuda", dtype=torch.float16))
    small = tc.linear(x[:8], w[:, :64])
    assert torch.count_nonzero(small) == 0

"""A call that finds no memory for its outputs raises what torch raises."""
import pytest
import torch

from test_gpu_serving_kv import bsq, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def test_out_of_memory_is_torchs_error(bsq):  # noqa: F811
    """The process's share of the memory ends before `out` fits: nothing runs, and the same call
    works once it may have the memory."""
    d = bsq.kv_cache(3, 1, 64)
    q = torch.zeros((1 << 17, 4, 64), dtype=torch.bfloat16, device="cuda")       # 64 MiB, as out
    args = (q, d, i32([0, 1]), i32([0]), i32([[0]]), 1, 1)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    held = []
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (32 << 20)) / total)
        # what earlier tests left in the allocator may be free for `out`: taken until nothing is
        with pytest.raises(torch.OutOfMemoryError):
            for _ in range(10000):
                held.append(torch.empty_like(q))
        with pytest.raises(torch.OutOfMemoryError):
            bsq.kv_cache_attention(*args)
    finally:
        del held
        torch.cuda.set_per_process_memory_fraction(1.0)
    out = bsq.kv_cache_attention(*args)
    torch.cuda.synchronize()
    assert torch.all(out[0] == 0)

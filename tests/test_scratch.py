"""The binding's kept scratch: its bookkeeping (no GPU needed)."""
import threading

import torch


def test_is_bounded_and_per_thread():
    """A program that goes through streams does not gather a megabyte for each: the oldest makes room."""
    from mxfp8_grouped_gemm_gb300 import _lib
    cache, cpu = _lib._ScratchCache(), torch.device("cpu")
    first = cache.get(cpu, 1)
    assert cache.get(cpu, 1) is first and first.numel() == cache.BYTES
    for handle in range(2, 200):
        assert cache.get(cpu, handle) is cache.get(cpu, handle)
        assert len(cache.kept) <= cache.MOST
    assert cache.get(cpu, 1) is not first
    seen = []
    t = threading.Thread(target=lambda: seen.append(cache.get(cpu, 1)))
    t.start()
    t.join()
    assert seen[0] is not cache.get(cpu, 1)

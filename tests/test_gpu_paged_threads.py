"""Paged calls from several host threads at once, each with its own cache and stream."""
import ctypes
import threading

import pytest

from test_gpu_paged import _cache, _i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402


def test_tables_of_other_sizes_from_several_threads():
    """8192 rows need more shared memory than 2500, and both more than a kernel has without asking.  The library is called without
    the layers above it, so that the calls meet inside it."""
    jobs = []
    for rows in (8192, 2500, 8192, 2500):
        cache = _cache(num_pages=rows + 8, num_seqs=rows, max_blocks=2, num_kv_heads=1)
        plan = cache.new_plan(rows)
        jobs.append((cache, plan, _i32([127] * rows), _i32([1] * rows), _i32([0] * rows), torch.cuda.Stream()))
    torch.cuda.synchronize()
    go, errors = threading.Barrier(len(jobs)), []

    call = kivi.load_library().kivi_paged_build_tables

    def work(cache, plan, lens, new, out, stream):
        queue = torch.zeros(2, dtype=torch.int64, device="cuda")
        args = (ctypes.byref(cache.cfg), ctypes.byref(cache.c), len(lens), lens.data_ptr(), new.data_ptr(), out.data_ptr(),
                queue.data_ptr(), ctypes.byref(plan.c), cache.status.data_ptr(), stream.cuda_stream)
        go.wait()
        errors.append(sum(call(*args) != 0 for _ in range(4000)))

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert errors == [0] * len(jobs)
    for cache, plan, lens, new, out, _ in jobs:
        assert (out == 128).all() and plan.counts.tolist() == [cache.cfg.num_seqs] * 2 and cache.read_status() == 0

"""Evictions of several host threads at once, each with its own workspace and stream."""

import ctypes
import threading

import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402
from decode_attention_13_b200 import binding  # noqa: E402
from tests.serving import workspace  # noqa: E402
from tests.test_gpu_evict import Codes, check_evict  # noqa: E402

pytestmark = pytest.mark.gpu


def test_two_threads_evict_caches_of_different_sizes():
    # the calls need different amounts of shared memory, in the search (length) and in the move (width, share kept)
    shapes = [([300], 3, 3, 200, 4, 8), ([40000], 2, 2, 900, 4, 64), ([5000], 8, 8, 77, 2, 5)]
    jobs = []
    for i, (lens, kb, vb, keep, first, recent) in enumerate(shapes):
        c = Codes(lens, 1, 2, kb, vb, seed=i)
        w = torch.rand((1, 1, c.cap), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda")
        dst = torch.full((c.plan.packed_bytes,), 0x5A, dtype=torch.uint8, device="cuda")
        new = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        kept = torch.full((1, 1, keep), -7, dtype=torch.int32, device="cuda")
        wo = torch.full((1, 1, keep), 77.0, device="cuda")
        jobs.append((c, w, keep, first, recent, dst, new, kept, wo, workspace(gtq.gtq_evict_workspace(c.plan, c.cap)),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed, begin = [], threading.Barrier(len(jobs))

    def loop(c, w, keep, first, recent, dst, new, kept, wo, ws, stream):
        # the library's own call, its arguments made beforehand: the threads are inside it nearly all of the time
        two = lambda x: (ctypes.c_int64 * 2)(x.stride(0), x.stride(1))  # noqa: E731
        ev = binding.gtq_eviction(keep, first, recent, w.data_ptr(), two(w), wo.data_ptr(), two(wo), kept.data_ptr(),
                                  new.data_ptr())
        args = (c.plan.handle, c.packed.data_ptr(), c.cap, ctypes.byref(c.layout), ctypes.byref(ev), dst.data_ptr(),
                dst.numel(), None, ws.data_ptr(), ws.numel(), stream.cuda_stream)
        call = binding.library().gtq_evict
        begin.wait()
        for i in range(6000):
            rc = call(*args)
            if rc != gtq.GTQ_OK:
                failed.append((c.cap, i, rc))
                return

    threads = [threading.Thread(target=loop, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for c, w, keep, first, recent, dst, new, kept, wo, ws, stream in jobs:
        assert gtq.gtq_status(c.plan) == gtq.GTQ_OK
        check_evict(c, w, keep, first, recent, dst, None, new, kept, wo)

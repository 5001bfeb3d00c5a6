"""The operators around the scan called by two host threads at once, each on a stream of its own.

The threads are native (a few lines of C++ compiled here): Python threads hold
the interpreter's lock between their calls and hardly ever meet inside the library."""
import ctypes
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <atomic>
#include <cstdint>
#include <thread>
typedef int (*Fwd)(const void*, const void*, const float*, void*, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float,
                   int, int, void*);
struct Call { const void *y, *z; const float* w; void* out; int64_t dim, len; void* stream; };
// Calls of `fwd` that failed, of n by each of two threads.
extern "C" int both(Fwd fwd, const Call* calls, int n) {
    std::atomic<int> failed{0}, ready{0};
    auto work = [&](const Call& c) {
        ++ready;
        while (ready < 2) {}
        for (int i = 0; i < n; ++i)
            failed += fwd(c.y, c.z, c.w, c.out, 1, c.dim, c.len, 1, c.dim * c.len, c.len, 1e-5f, 1, 0, c.stream) != 0;
    };
    std::thread other(work, calls[1]);
    work(calls[0]);
    other.join();
    return failed;
}
"""


class Call(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("y", "z", "w", "out")] + [("dim", ctypes.c_int64), ("len", ctypes.c_int64),
                                                                        ("stream", ctypes.c_void_p)]


def test_gated_norms_of_different_widths(tmp_path):
    """Wide groups take most of an SM's shared memory and narrow ones little: neither
    call may undo what the other needs between its set-up and its launch."""
    import linear_recurrence_gb300 as lr
    (tmp_path / "both.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "both.cpp", "-o", "both.so"], cwd=tmp_path, check=True)
    both = ctypes.CDLL(str(tmp_path / "both.so")).both
    g = torch.Generator(device="cuda").manual_seed(1)
    calls, keep = (Call * 2)(), []
    for i, dim in enumerate((8192, 64)):
        y, z = (torch.randn(1, dim, 16, generator=g, device="cuda").bfloat16() for _ in range(2))
        w, out, stream = torch.ones(dim, device="cuda"), torch.empty_like(y), torch.cuda.Stream()
        want = lr.gatenorm_fwd(y, z, w)
        calls[i] = Call(y.data_ptr(), z.data_ptr(), w.data_ptr(), out.data_ptr(), dim, 16, stream.cuda_stream)
        keep.append((y, z, w, out, stream, want))
    torch.cuda.synchronize()
    failed = both(ctypes.cast(lr.lib().gatenorm_fwd, ctypes.c_void_p), calls, 20000)
    torch.cuda.synchronize()
    assert failed == 0
    for *_, out, _, want in keep:
        assert torch.equal(out, want)

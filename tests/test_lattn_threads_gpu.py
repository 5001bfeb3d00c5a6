"""Moves of cache rows, norms of queries and keys, and packed prompts of linear attention called by two host
threads at once, a call that needs much shared memory beside one that needs little, each on a stream of its own:
neither may undo what the other needs between its set-up and its launch.

The threads are native (a few lines of C++ compiled here): Python threads hold
the interpreter's lock between their calls and hardly ever meet inside the library."""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <atomic>
#include <thread>
#include "sscan.h"

// Calls that failed: n by one thread, and another thread's for as long as these take.
template <typename F>
static int both(F call, int n) {
    std::atomic<int> failed{0}, ready{0};
    std::atomic<bool> done{false};
    auto meet = [&] { ++ready; while (ready < 2) {} };
    std::thread other([&] {
        meet();
        while (!done) failed += call(1) != 0;
    });
    meet();
    for (int i = 0; i < n; ++i) failed += call(0) != 0;
    done = true;
    other.join();
    return failed;
}

struct Move { void* cache; const int32_t *src, *dst; int64_t moves, layers, rows, row_bytes; void* stream; };
extern "C" int moves(decltype(&state_move) f, const Move* c, int n) {
    return both([&](int w) { return f(c[w].cache, c[w].src, c[w].dst, c[w].moves, c[w].layers, c[w].rows, c[w].row_bytes, c[w].stream); }, n);
}

// queries alone: [1, 2 heads, len], all frequencies
struct Norm { const void *q, *dout; const float *w, *freq; const int32_t* pos; void* out; float* dw; int64_t dim, len; int dtype; void* stream; };
extern "C" int norms(decltype(&qknorm_fwd) f, const Norm* c, int n) {
    return both([&](int w) {
        const Norm& x = c[w];
        const int64_t strides[4] = {2 * x.dim * x.len, x.len, 0, 0};
        return f(x.q, nullptr, x.w, nullptr, x.pos, x.freq, x.out, nullptr, 1, 2, 0, x.dim, x.len, x.dim / 2, strides, 1e-5f, x.dtype, x.stream);
    }, n);
}
extern "C" int norm_gradients(decltype(&qknorm_bwd) f, const Norm* c, int n) {
    return both([&](int w) {
        const Norm& x = c[w];
        const int64_t strides[4] = {2 * x.dim * x.len, x.len, 0, 0};
        return f(x.q, nullptr, x.w, nullptr, x.pos, x.freq, x.dout, nullptr, x.out, nullptr, x.dw, nullptr, 1, 2, 0, x.dim, x.len, x.dim / 2,
                 strides, 1e-5f, x.dtype, x.stream);
    }, n);
}

// prompts of 8 requests of 4 tokens, one head, steps of one, no rows continued
struct Prompt { const void *q, *k, *v; const float* A; const int32_t* cu; const uint8_t* has; float* state; void* out; int64_t key, value; void* stream; };
extern "C" int prompts(decltype(&lattn_prompt) f, const Prompt* c, int n) {
    return both([&](int w) {
        const Prompt& x = c[w];
        const int64_t strides[8] = {0, 32, 0, 32, 0, 32, 0, 0};
        return f(x.q, x.k, x.v, x.A, nullptr, nullptr, nullptr, x.cu, nullptr, x.has, x.state, x.out, 8, 8, 1, 1, x.key, x.value, 32, strides, 0.1f, 0,
                 0, 1, x.stream);
    }, n);
}
"""


class Move(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("cache", "src", "dst")] + [
        (n, ctypes.c_int64) for n in ("moves", "layers", "rows", "row_bytes")] + [("stream", ctypes.c_void_p)]


class Norm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "dout", "w", "freq", "pos", "out", "dw")] + [
        ("dim", ctypes.c_int64), ("len", ctypes.c_int64), ("dtype", ctypes.c_int), ("stream", ctypes.c_void_p)]


class Prompt(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "A", "cu", "has", "state", "out")] + [
        ("key", ctypes.c_int64), ("value", ctypes.c_int64), ("stream", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def threads(tmp_path_factory):
    where = tmp_path_factory.mktemp("threads")
    (where / "both.cpp").write_text(SOURCE)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I", include, "both.cpp", "-o", "both.so"], cwd=where, check=True)
    return ctypes.CDLL(str(where / "both.so"))


def entry(lr, name):
    return ctypes.cast(getattr(lr.lib(), name), ctypes.c_void_p)


@pytest.mark.parametrize("width", [64, 9], ids=["vectors", "words"])
def test_moves_of_many_rows_and_of_few(lr, threads, width):
    calls, keep = (Move * 2)(), []
    for i, (rows, count) in enumerate(((8000, 4000), (64, 2))):
        cache, stream = torch.randn(rows, width, device="cuda"), torch.cuda.Stream()
        src = torch.arange(count, device="cuda", dtype=torch.int32)
        dst = src + count
        want = cache.clone()
        want[count:2 * count] = cache[:count]
        calls[i] = Move(cache.data_ptr(), src.data_ptr(), dst.data_ptr(), count, 1, rows, 4 * width, stream.cuda_stream)
        keep.append((cache, src, dst, stream, want))
    torch.cuda.synchronize()
    failed = threads.moves(entry(lr, "state_move"), calls, 2000)
    torch.cuda.synchronize()
    assert failed == 0
    for cache, *_, want in keep:
        assert torch.equal(cache, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("length", [32, 33])
@pytest.mark.parametrize("gradients", [False, True], ids=["forward", "gradients"])
def test_norms_of_wide_heads_and_of_narrow(lr, threads, dtype, length, gradients):
    io = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    calls, keep = (Norm * 2)(), []
    for i, dim in enumerate((128, 66)):
        q, do = (torch.randn(1, 2 * dim, length, device="cuda").to(io) for _ in range(2))
        w, freq = torch.rand(dim, device="cuda"), torch.rand(dim // 2, device="cuda")
        pos = torch.arange(length, device="cuda", dtype=torch.int32)[None].contiguous()
        out, dw, stream = torch.empty_like(q), torch.empty_like(w), torch.cuda.Stream()
        if gradients:
            g = lr.qknorm_bwd(q, None, w, None, do, None, pos, freq)
            want = [(out, g["dq"]), (dw, g["dq_weight"])]
        else:
            want = [(out, lr.qknorm_fwd(q, None, w, None, pos, freq)[0])]
        calls[i] = Norm(q.data_ptr(), do.data_ptr(), w.data_ptr(), freq.data_ptr(), pos.data_ptr(), out.data_ptr(), dw.data_ptr(), dim, length,
                        lr.SSCAN_F32 if dtype == "f32" else lr.SSCAN_BF16, stream.cuda_stream)
        keep.append((q, do, w, freq, pos, stream, want))
    torch.cuda.synchronize()
    name = "qknorm_bwd" if gradients else "qknorm_fwd"
    failed = (threads.norm_gradients if gradients else threads.norms)(entry(lr, name), calls, 3000)
    torch.cuda.synchronize()
    assert failed == 0
    for *_, want in keep:
        for got, value in want:
            assert torch.equal(got, value)


def test_short_prompts_of_wide_heads_and_of_narrow(lr, threads):
    calls, keep = (Prompt * 2)(), []
    cu = torch.arange(0, 33, 4, device="cuda", dtype=torch.int32)
    has = torch.zeros(8, device="cuda", dtype=torch.bool)
    A = torch.tensor([-0.1], device="cuda")
    for i, (key, value) in enumerate(((128, 256), (68, 16))):
        q, k = (torch.randn(key, 32, device="cuda") for _ in range(2))
        v, stream = torch.randn(value, 32, device="cuda"), torch.cuda.Stream()
        state, held = (torch.zeros(8, value, key, device="cuda") for _ in range(2))
        out = torch.empty_like(v)
        want = lr.lattn_prompt(q, k, v, A, cu_seqlens=cu, state=held, has_state=has, scale=0.1, pieces=1)
        calls[i] = Prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), A.data_ptr(), cu.data_ptr(), has.data_ptr(), state.data_ptr(), out.data_ptr(),
                          key, value, stream.cuda_stream)
        keep.append((q, k, v, stream, (out, want), (state, held)))
    torch.cuda.synchronize()
    failed = threads.prompts(entry(lr, "lattn_prompt"), calls, 3000)
    torch.cuda.synchronize()
    assert failed == 0
    for *_, out, state in keep:
        assert torch.equal(*out) and torch.equal(*state)

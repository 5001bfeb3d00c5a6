"""The packed scan stages rows of u, delta and z in 16-byte pieces; no piece
that its kernels copy without a check may lie outside its array.  The rule is
integer arithmetic (csrc/row_pieces.cuh), so every piece is enumerated here, on
the host, for the rows a warp takes in each of the kernels' forms, and for rules
that are too weak, which the enumeration has to catch."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrence_gb300", "csrc")

# The number of unchecked pieces outside an array of dim rows whose base lies `base` elements past a
# 16-byte boundary.  rule 0: the scan pass; 1: the end-state pass (tiles of segments that end before
# the rows do); 2: checks for the warp of the last row alone; 3: checks for the first tile alone.
SOURCE = r"""
#include "row_pieces.cuh"
extern "C" long long leaks(int rule, int warp_rows, long long dim, int tokens, int vec, int base) {
    const int tile = 16;
    long long bad = 0;
    for (long long row0 = 0; row0 < dim; row0 += warp_rows) {
        const int rows = dim - row0 < warp_rows ? (int)(dim - row0) : warp_rows;
        const int last_inner = sscan::last_inner_tile(row0, rows, dim, tokens, tile, vec);
        for (int t0 = 0; t0 < tokens; t0 += tile) {
            if (rule == 1 && t0 + tile >= tokens) break;
            const bool edge = rule == 0   ? sscan::at_edge(t0, last_inner)
                              : rule == 1 ? sscan::inner_at_edge(row0, rows, dim, tokens, t0, tile, vec)
                              : rule == 2 ? (row0 == 0 && t0 == 0) || (row0 + rows >= dim && t0 + tile + vec > tokens)
                                          : t0 == 0;
            if (edge) continue;
            for (int r = 0; r < rows; ++r)
                for (int c = 0; c <= tile / vec; ++c) {
                    const long long row = (row0 + r) * tokens, phase = (base + row) & (vec - 1);
                    const long long from = row + t0 + c * vec - phase;
                    bad += from < 0 || from + vec > dim * tokens;
                }
        }
    }
    return bad;
}
// the tiles of a call whose pieces are checked
extern "C" long long checked(int warp_rows, long long dim, int tokens, int vec) {
    long long n = 0;
    for (long long row0 = 0; row0 < dim; row0 += warp_rows)
        for (int t0 = 0; t0 < tokens; t0 += 16)
            n += sscan::at_edge(t0, sscan::last_inner_tile(row0, dim - row0 < warp_rows ? (int)(dim - row0) : warp_rows, dim,
                                                           tokens, 16, vec));
    return n;
}
"""

WARP_ROWS = (2, 4, 8, 16, 32, 64)  # of the scan pass, by lanes a channel and channels a thread
END_ROWS = 32
DIMS = [*range(1, 131), 1536, 5120, 5121]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    folder = tmp_path_factory.mktemp("row_pieces")
    source, out = folder / "enumerate.cpp", folder / "enumerate.so"
    source.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", str(source), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.leaks.restype = lib.checked.restype = ctypes.c_longlong
    lib.leaks.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    lib.checked.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.mark.parametrize("vec", [4, 8])  # fp32, bf16
@pytest.mark.parametrize("rows", WARP_ROWS)
def test_scan_pass_stages_inside_its_arrays(lib, rows, vec):
    for dim in DIMS:
        for tokens in range(1, 41):
            for base in range(vec):
                assert lib.leaks(0, rows, dim, tokens, vec, base) == 0, (dim, tokens, base)


@pytest.mark.parametrize("vec", [4, 8])
def test_end_state_pass_stages_inside_its_arrays(lib, vec):
    for dim in DIMS:
        for tokens in range(17, 70):
            for base in range(vec):
                assert lib.leaks(1, END_ROWS, dim, tokens, vec, base) == 0, (dim, tokens, base)


def test_weaker_rules_are_caught(lib):
    """One token of 5120 bf16 or fp32 channels, and few tokens of odd counts, pass the end of more than the last rows."""
    assert lib.leaks(2, 8, 5120, 1, 8, 0) > 0 and lib.leaks(2, 8, 5120, 1, 4, 0) > 0
    assert lib.leaks(2, 8, 65, 7, 8, 0) > 0 and lib.leaks(2, 2, 40, 5, 8, 0) > 0
    assert lib.leaks(2, 2, 40, 1, 8, 4) > 0  # and rows after the first reach before the front
    assert lib.leaks(3, 8, 33, 17, 8, 0) > 0


def test_only_tiles_at_the_ends_are_checked(lib):
    """Long rows: the first tile of every warp's rows, and of the last warp's those that reach past the end (8192 and 8208)."""
    assert lib.checked(16, 2048, 8209, 8) == 2048 // 16 + 2
    assert lib.checked(8, 5120, 37, 8) <= 5120 // 8 + 2

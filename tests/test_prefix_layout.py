"""The places in a query tile of the tensor-core prefix kernel, from the kernel's
own address functions: a warp's query rows and the rows of the records that pass
through the same tile lie in bytes of that warp alone, for the warps of a stream
are not ordered with one another when one item ends and the next begins."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_paged_kv_zp_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "prefix_layout.h"
int main() {
    const int half = 128 * 128;
    for (int D = 64; D <= 128; D += 64)
        for (int row = 0; row < 128; ++row) {
            for (int c = 0; c < D / 8; ++c) std::printf("%d q %d %d\n", D, row, zp::pt_chunk(row, c, half));
            for (int c = 0; c < zp::pt_record_cols(D) / 4; ++c) std::printf("%d r %d %d\n", D, row, zp::pt_chunk(row, c, half));
        }
}
"""


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("layout")
    src, exe = where / "places.cpp", where / "places"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    got = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        D, kind, row, at = line.split()
        got.setdefault((int(D), kind, int(row) // 32), []).append(int(at))
    return got


@pytest.mark.parametrize("D", [64, 128])
def test_warps_stay_in_their_own_bytes(places, D):
    tile = D // 64 * 128 * 128
    for kind in "qr":
        every = [at for w in range(4) for at in places[D, kind, w]]
        assert sorted(every) == list(range(0, tile, 16)), "the chunks fill the tile, each once"
    for w in range(4):
        for other in range(4):
            shared = set(places[D, "q", w]) & set(places[D, "r", other])
            assert bool(shared) == (w == other), "warp %d's queries and warp %d's records" % (w, other)


@pytest.mark.parametrize("D", [64, 128])
def test_no_bank_conflicts(places, D):
    """Eight consecutive 16-byte accesses (a 128-byte phase) cover every bank: a column of chunks
    (a thread per row) and a row of chunks (the stores to memory)."""
    half = 128 * 128
    n = D // 8
    at = {(row, c): places[D, "q", row // 32][(row % 32) * n + c] for row in range(128) for c in range(n)}
    for c in range(n):
        for r0 in range(0, 128, 8):
            assert len({at[r, c] % 128 for r in range(r0, r0 + 8)}) == 8
    for row in range(128):
        for c0 in range(0, n, 8):
            assert len({at[row, c] % 128 for c in range(c0, c0 + 8)}) == 8
    assert max(at.values()) < D // 64 * half

"""CPU test of the attention kernels' work lists: every warp of either kernel has an entry of its own for its part of the sum,
beside the fields that the same function writes without a barrier in between."""
import os
import re
import subprocess

import pytest

from bit_quantized_skinny_gb300 import build_lib

PROGRAM = r"""
#include <cstddef>
#include <cstdio>
#include "q4k_attn_parts.cuh"
int main() {
  using q4k::Piece;
  std::printf("%zu %zu\n", offsetof(Piece, scan), offsetof(Piece, scan) + sizeof(Piece::scan));
  std::printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu\n", offsetof(Piece, w0), offsetof(Piece, w1), offsetof(Piece, per), offsetof(Piece, b),
              offsetof(Piece, rb), offsetof(Piece, h), offsetof(Piece, rows), offsetof(Piece, s), offsetof(Piece, unit));
  return 0;
}
"""


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    at = tmp_path_factory.mktemp("piece")
    source, program = at / "piece.cu", at / "piece"
    source.write_text(PROGRAM)
    r = subprocess.run([build_lib.NVCC, *build_lib.NVCC_FLAGS, str(source), "-o", str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    scan, fields = subprocess.run([str(program)], capture_output=True, text=True, check=True).stdout.splitlines()
    return [int(x) for x in scan.split()], [int(x) for x in fields.split()]


@pytest.mark.parametrize("source", ["qmm_attn.cu", "qmm_attn_fp4.cu"])
def test_every_warp_has_an_entry(layout, source):
    with open(os.path.join(build_lib.CSRC, source), encoding="utf-8") as fh:
        a, b = re.search(r"constexpr int kThreads = (\d+) \* (\d+)", fh.read()).groups()
    warps = int(a) * int(b) // 32
    (begin, end), fields = layout
    used = range(begin, begin + 8 * warps)
    assert used.stop <= end, f"{warps} warps, {(end - begin) // 8} entries"
    assert not [f for f in fields if f in used]

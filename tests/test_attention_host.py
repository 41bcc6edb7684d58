"""The visible keys of a row, evaluated on the host by the function that the attention kernels use (no GPU needed)."""
import os
import subprocess

import pytest

from block_quantized_weight_matmulnbits_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "attention.h"
int main(int argc, char** argv) {
    // quintuples: new tokens, keys, window, causal, row
    for (int i = 1; i + 4 < argc; i += 5) {
        mnb::attn::AttnParams p{};
        p.window = std::atoi(argv[i + 2]);
        p.causal = std::atoi(argv[i + 3]);
        const int row = std::atoi(argv[i + 4]);
        int lo, hi;
        mnb::attn::visible_range(p, std::atoi(argv[i]), std::atoi(argv[i + 1]), row, row + 1, &lo, &hi);
        std::printf("%d %d\n", lo, hi);
    }
}
"""


@pytest.fixture(scope="module")
def visible(tmp_path_factory):
    at = tmp_path_factory.mktemp("visible")
    (at / "visible.cu").write_text(PROGRAM)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fwrapv", "-I", _build.INCLUDE,
                    "-I", _build.CSRC, str(at / "visible.cu"), "-o", str(at / "visible")], check=True, capture_output=True)

    def run(cases):
        out = subprocess.run([str(at / "visible"), *[str(x) for c in cases for x in c]], check=True, capture_output=True, text=True).stdout
        return [tuple(int(x) for x in line.split()) for line in out.splitlines()]

    return run


def test_visible_range(visible):
    """j <= pos (causal) and j > pos - window, for windows up to the largest int and rows before the sequence."""
    cases = [(n, length, w, causal, row) for n, length in [(1, 1), (1, 777), (5, 2), (300, 130), (9, 0), (2 ** 29, 3)]
             for w in (0, 1, 2, 130, 2 ** 30, 2 ** 31 - 3, 2 ** 31 - 1) for causal in (0, 1) for row in sorted({0, n // 2, n - 1})]
    for (n, length, w, causal, row), (lo, hi) in zip(cases, visible(cases)):
        pos = length - n + row
        keys = [j for j in range(length) if (j <= pos or not causal) and (w == 0 or j > pos - w)]
        assert list(range(max(lo, 0), max(hi, 0))) == keys and lo >= 0, (n, length, w, causal, row, lo, hi)

"""Attention's host side (no GPU needed): the visible keys of a row, by the function that the kernels use, and workspaces."""
import ctypes
import subprocess

import pytest

import block_quantized_weight_matmulnbits_gb300 as mnb
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


def test_workspace_for_a_larger_call_is_enough_for_a_smaller_one(monkeypatch):
    """No call refuses a buffer that was sized for one with more of everything (the launch itself is not made)."""
    lib = mnb.load()
    monkeypatch.setenv("MNB_FAIL_LAUNCH", "1")
    heads, kv_heads, D = 32, 8, 128
    sizes = [(T, q, kv) for T in (1, 8, 500, 1000, 1024, 8192) for q in (1, 8, 500, 8192) for kv in (100, 9000, 32000, 131072) if q <= T]
    c = mnb.KvCache()
    c.k_pages = c.v_pages = c.tables = c.kv_lens = 4096
    c.batch, c.table_stride, c.num_pages, c.page_size, c.kv_heads, c.head_dim, c.dtype = 1, 9000, 9, 16, kv_heads, D, mnb.MNB_BF16
    c.page_stride, c.token_stride, c.head_stride = kv_heads * 16 * D, D, 16 * D
    a = mnb.AttentionArgs()
    a.q = a.o = a.q_start = a.workspace = 4096
    a.q_heads, a.scale, a.causal = heads, 0.1, 1
    a.q_token_stride = a.o_token_stride = heads * D
    a.q_head_stride = a.o_head_stride = D
    for big in sizes:
        a.workspace_bytes = mnb.mnb_attention_workspace_size(1, big[0], heads, kv_heads, D, big[1], big[2], mnb.MNB_BF16)
        for small in sizes:
            if all(x <= y for x, y in zip(small, big)):
                a.T, a.max_q, a.max_kv = small
                assert lib.mnb_paged_attention(ctypes.byref(a), ctypes.byref(c)) == mnb.MNB_ERR_CUDA, (big, small)
    a.workspace_bytes = 4 << 20
    assert lib.mnb_paged_attention(ctypes.byref(a), ctypes.byref(c)) == mnb.MNB_ERR_NO_MEM

"""A decoder layer's attention block on the library, as a server runs it: int4 projections, rotary positions, a paged
cache and attention over it.

    python examples/decoder_layer.py            # prefill two prompts, fork samples of one, decode, free and compact

Each step is a handful of calls on the current stream:

    mnb_cache_resize      pages for the step's new tokens (a fork's shared last page is copied first)
    mnb_matmul            QKV product with block-quantised weights
    mnb_rotary_append     queries and keys turned, keys and values written to the pages
    mnb_paged_attention   the new tokens over everything cached
    mnb_matmul            output product
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_matmulnbits_gb300 as mnb  # noqa: E402


def aligned(nbytes, align=256):
    raw = torch.empty(nbytes + align, dtype=torch.uint8, device="cuda")
    off = (-raw.data_ptr()) % align
    return raw[off:off + nbytes]


class Linear:
    """y = x . dequant(B)^T with int4 codes in blocks of 32 and f16 scales (random weights of a given deviation)."""

    def __init__(self, n, k, gen, deviation):
        self.n, self.k = n, k
        codes = torch.randint(0, 256, (n, k // 32, 16), generator=gen, device="cuda", dtype=torch.uint8)
        self.scales = torch.full((n, k // 32), deviation / 4.6, device="cuda", dtype=torch.float16)  # codes 0..15 deviate by 4.6
        self.packed = aligned(mnb.mnb_packed_size(n, k, 4, 32))
        mnb.mnb_pack_weights(codes, self.packed, n, k, 4, 32)

    def __call__(self, x):
        y = torch.empty((x.shape[0], self.n), dtype=torch.bfloat16, device="cuda")
        mnb.mnb_matmul(x, self.packed, self.scales, None, y, x.shape[0], self.n, self.k, 4, 32, mnb.MNB_BF16, mnb.MNB_BF16, mnb.MNB_F16)
        return y

    def dense(self):
        w = torch.empty((self.n, self.k), device="cuda")
        mnb.mnb_dequantize(self.packed, self.scales, None, w, self.n, self.k, 4, 32, mnb.MNB_F16)
        return w


class Layer:
    def __init__(self, hidden=512, heads=8, kv_heads=2, dim=64, page_size=16, num_pages=64, max_seqs=8, max_pages=16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page_size = heads, kv_heads, dim, page_size
        self.qkv = Linear((heads + 2 * kv_heads) * dim, hidden, gen, hidden ** -0.5)
        self.out = Linear(hidden, heads * dim, gen, (heads * dim) ** -0.5)
        n_pos = max_pages * page_size
        self.cos, self.sin = (torch.empty((n_pos, dim // 2), device="cuda") for _ in range(2))
        mnb.mnb_rotary_table(self.cos, self.sin, scaling=mnb.MNB_ROPE_BY_PARTS, factor=2.0, trained_len=n_pos / 2,
                             attn_factor=0.1 * math.log(2.0) + 1.0)
        # plane 0 the keys, plane 1 the values: pages of [kv_heads][page_size][dim]
        self.pool = torch.zeros((2, num_pages, kv_heads, page_size, dim), dtype=torch.bfloat16, device="cuda")
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        self.tables = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(max_seqs, dtype=torch.int32, device="cuda")
        self.planes = mnb.page_planes(self.pool)
        self.state = mnb.cache_state(self.refs, self.tables, self.lens, page_size)
        self.ws = aligned(mnb.mnb_cache_workspace_size(num_pages, max_seqs, max_pages))
        self.max_kv = n_pos

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def fork(self, src, dst):
        mnb.mnb_cache_fork(self.state, self.ints(src), self.ints(dst), workspace=self.ws)

    def resize(self, seqs, lens):
        mnb.mnb_cache_resize(self.state, self.planes, self.ints(seqs), self.ints(lens), workspace=self.ws)

    def compact(self):
        counts = torch.empty(2, dtype=torch.int32, device="cuda")
        mnb.mnb_cache_compact(self.state, self.planes, self.refs, self.tables, counts, workspace=self.ws)
        return counts

    def step(self, x, seqs, new, lens):
        """x [sum(new), hidden]: new[i] tokens of sequence seqs[i], which then holds lens[i] tokens."""
        self.resize(seqs, lens)
        rows = self.ints(seqs).long()
        start = torch.zeros(len(seqs) + 1, dtype=torch.int32, device="cuda")
        start[1:] = torch.cumsum(self.ints(new), 0)
        cache = mnb.kv_cache(self.pool[0], self.pool[1], self.tables[rows], self.lens[rows], "hnd", mnb.MNB_BF16)
        h, g, d = self.heads, self.kv_heads, self.dim
        y = self.qkv(x).view(-1, h + 2 * g, d)
        q, o = y[:, :h], torch.empty((x.shape[0], h, d), dtype=torch.bfloat16, device="cuda")
        mnb.mnb_rotary_append(q, q, y[:, h:h + g], y[:, h + g:], self.cos, self.sin, cache, start)
        ws = aligned(mnb.mnb_attention_workspace_size(len(seqs), x.shape[0], h, g, d, max(new), max(lens), mnb.MNB_BF16))
        mnb.mnb_paged_attention(q, o, cache, start, max(new), max(lens), d ** -0.5, workspace=ws)
        return self.out(o.view(-1, h * d))


def main():
    layer = Layer()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = lambda n: torch.randn((n, 512), generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    layer.step(x(37 + 90), [0, 1], [37, 90], [37, 90])            # two prompts in one call
    layer.fork([0, 0, 0], [2, 3, 4])                               # three samples of the first
    print("pages held after the fork:", int((layer.refs > 0).sum()), "for lengths", layer.lens.tolist())
    lens = {0: 37, 1: 90, 2: 37, 3: 37, 4: 37}
    for _ in range(5):                                             # decode: one token of each sequence a step
        lens = {b: n + 1 for b, n in lens.items()}
        y = layer.step(x(len(lens)), list(lens), [1] * len(lens), list(lens.values()))
    layer.resize([1, 3], [0, 0])                                   # two sequences end
    counts = layer.compact()
    print("pages held:", int(counts[0]), "moved:", int(counts[1]), "lengths:", layer.lens.tolist())
    assert mnb.mnb_get_device_error() == 0 and torch.isfinite(y).all()


if __name__ == "__main__":
    main()

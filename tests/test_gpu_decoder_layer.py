"""The operators together, as examples/decoder_layer.py runs them, against the layer in 64 bits over plain lists of
each sequence's tokens: prompts, forks that share pages, decode steps, freed sequences and a compaction."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import _decoder_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(mnb, example):
    example.main()


def test_layer_against_64_bits(mnb, example):
    L = example.Layer(seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    w_qkv, w_out = R.f64(L.qkv.dense()), R.f64(L.out.dense())
    cos, sin = R.f64(L.cos), R.f64(L.sin)
    h, g, d = L.heads, L.kv_heads, L.dim
    held = {}  # sequence -> the inputs of its tokens so far

    def reference(seq, n):
        """Output rows of the last n tokens of a sequence, everything in 64 bits from the bf16 inputs."""
        x = np.concatenate(held[seq])
        y = (x @ w_qkv.T).reshape(len(x), h + 2 * g, d)
        pos = np.arange(len(x))
        q, k = R.rotary(y[:, :h], cos, sin, pos, "half")[0], R.rotary(y[:, h:h + g], cos, sin, pos, "half")[0]
        o = np.zeros((n, h, d))
        for a in range(h):
            o[:, a] = R.attention(q[-n:, a], k[:, a // (h // g)], y[:, h + g + a // (h // g)], len(x) - n, d ** -0.5, True, 0)[0]
        return o.reshape(n, -1) @ w_out.T

    def step(seqs, new):
        x = torch.randn((sum(new), 512), generator=gen, device="cuda").to(torch.bfloat16)
        at = 0
        for b, n in zip(seqs, new):
            held.setdefault(b, []).append(R.f64(x[at:at + n]))
            at += n
        y = R.f64(L.step(x, seqs, new, [sum(len(t) for t in held[b]) for b in seqs]))
        ref = np.concatenate([reference(b, n) for b, n in zip(seqs, new)])
        # Four roundings to bf16 in a row (q, k, v; rotated q and k; p and o; the result), each 2^-8 of its value, the
        # values of order 1: sums over 512 products of them add in quadrature, so 2^-8 * (4 to 8) of the rows' deviation
        # on the worst element.
        assert np.abs(y - ref).max() <= 8 * 2.0 ** -8 * max(1.0, ref.std() * 4), np.abs(y - ref).max()

    step([0, 1], [37, 90])
    L.fork([0, 0, 1], [2, 3, 4])
    for a, b in ((2, 0), (3, 0), (4, 1)):
        held[a] = list(held[b])
    step([0, 1, 2, 3, 4], [1] * 5)
    step([3, 0, 2], [3, 1, 20])
    L.resize([1, 3], [0, 0])
    del held[1], held[3]
    L.compact()
    step([0, 2, 4], [1, 1, 1])
    L.fork([4, 0], [0, 4])  # trade places
    held[0], held[4] = list(held[4]), list(held[0])
    step([0, 4, 5], [2, 1, 33])
    assert mnb.mnb_get_device_error() == 0


def test_offsets_past_32_bits(mnb):
    """Pages that start more than 2^32 bytes into the cache: append, both attention kernels and the page copy."""
    D, ps, stride, pages = 64, 16, 1 << 29, 10  # elements between pages: the last starts at 4.8e9
    k, v = (torch.empty(stride * (pages - 1) + ps * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp, vp = (torch.as_strided(t, (pages, 1, ps, D), (stride, ps * D, D, 1)) for t in (k, v))
    rng = np.random.default_rng(1)
    for n, at in ((1, 100), (40, 140)):
        order = [9, 1, 8, 0, 7, 2, 6, 3, 5]
        tables = torch.tensor([order], dtype=torch.int32, device="cuda")
        lens = torch.tensor([at], dtype=torch.int32, device="cuda")
        cache = mnb.kv_cache(kp, vp, tables, lens, "hnd", 2)
        x = [torch.from_numpy(rng.standard_normal((at, 1, D))).to(torch.bfloat16).cuda() for _ in range(2)]
        one = torch.ones((200, D // 2), device="cuda")
        start = torch.tensor([0, at], dtype=torch.int32, device="cuda")
        mnb.mnb_rotary_append(None, None, x[0], x[1], one, torch.zeros_like(one), cache, start)
        q = torch.from_numpy(rng.standard_normal((n, 1, D))).to(torch.bfloat16).cuda()
        o = torch.empty_like(q)
        qs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ws = torch.empty(mnb.mnb_attention_workspace_size(1, n, 1, 1, D, n, at, 2), dtype=torch.uint8, device="cuda")
        mnb.mnb_paged_attention(q, o, cache, qs, n, at, D ** -0.5, workspace=ws)
        ref, _, bound, _ = R.attention(R.f64(q[:, 0]), R.f64(x[0][:, 0]), R.f64(x[1][:, 0]), at - n, D ** -0.5, True, 0)
        assert (np.abs(R.f64(o[:, 0]) - ref) <= bound["bf16"]).all()
    pool = torch.as_strided(k, (1, pages, ps * D), (0, stride, 1))
    mnb.mnb_pages_copy(mnb.page_planes(pool), torch.tensor([8], dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda"))
    assert torch.equal(kp[4], kp[8])
    assert mnb.mnb_get_device_error() == 0


def test_bounded_wait_timeout_reports_and_recovers(mnb, monkeypatch):
    """MNB_WAIT_LIMIT=1: the many-row attention kernel gives up at its first wait that is not already satisfied, lets its
    copies and MMAs finish and frees tensor memory; the next call is right."""
    from tests.test_gpu_paged_attention import Problem
    p = Problem(mnb, [200], [700], 4, 2, 128, "bf16", 16, "hnd", seed=11)
    monkeypatch.setenv("MNB_WAIT_LIMIT", "1")
    p.run()
    torch.cuda.synchronize()
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_TIMEOUT
    monkeypatch.delenv("MNB_WAIT_LIMIT")
    for _ in range(2):
        p.check(*p.run())

"""Refusals of the decoder-layer calls, before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

import block_quantized_weight_matmulnbits_gb300 as mnb


def _cache(**kw):
    c = mnb.KvCache()
    c.k_pages = c.v_pages = c.tables = c.kv_lens = 4096
    c.batch, c.table_stride, c.num_pages = 2, 4, 9
    c.page_stride, c.token_stride, c.head_stride = 4096, 128, 2048
    c.page_size, c.kv_heads, c.head_dim, c.dtype = 16, 2, 128, mnb.MNB_BF16
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHE = [{"page_size": 12}, {"page_size": 4}, {"page_size": 2048}, {"k_pages": None}, {"k_pages": 4104}, {"tables": 2},
             {"batch": 0}, {"num_pages": 0}, {"num_pages": 1 << 31}, {"page_stride": 4100}, {"token_stride": -128},
             {"dtype": 3}, {"kv_heads": 0}]


def _attention(**kw):
    a = mnb.AttentionArgs()
    a.q = a.o = a.q_start = 4096
    a.T, a.q_heads, a.max_q, a.max_kv, a.scale, a.causal = 2, 4, 1, 50, 0.1, 1
    a.q_token_stride = a.o_token_stride = 512
    a.q_head_stride = a.o_head_stride = 128
    a.workspace, a.workspace_bytes = 4096, 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", BAD_CACHE)
def test_cache_is_checked(bad):
    lib, c = mnb.load(), _cache(**bad)
    assert lib.mnb_paged_attention(ctypes.byref(_attention()), ctypes.byref(c)) == mnb.MNB_ERR_INVALID_ARG
    r = mnb.RotaryArgs()
    r.k = r.v = r.cos_table = r.sin_table = r.q_start = 4096
    r.T, r.rot_dim, r.n_pos = 1, 64, 10
    assert lib.mnb_rotary_append(ctypes.byref(r), ctypes.byref(c)) == mnb.MNB_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [{"q": None}, {"q": 4098}, {"o": None}, {"q_start": None}, {"T": -1}, {"q_heads": 3}, {"q_heads": 0},
                                 {"max_q": 0}, {"max_kv": -1}, {"window": -1}, {"causal": 2}, {"scale": float("nan")},
                                 {"q_token_stride": 4}, {"o_head_stride": -8}, {"workspace": 4100}, {"lse": 2}])
def test_attention_arguments(bad):
    assert mnb.load().mnb_paged_attention(ctypes.byref(_attention(**bad)), ctypes.byref(_cache())) == mnb.MNB_ERR_INVALID_ARG


@pytest.mark.parametrize("dim", [12, 264, 0])
def test_attention_head_dim(dim):
    assert mnb.load().mnb_paged_attention(ctypes.byref(_attention()), ctypes.byref(_cache(head_dim=dim))) == mnb.MNB_ERR_INVALID_ARG


def test_nothing_to_do_is_ok():
    lib = mnb.load()
    assert lib.mnb_paged_attention(ctypes.byref(_attention(T=0)), ctypes.byref(_cache())) == mnb.MNB_OK
    assert lib.mnb_rotary(None, None, None, None, None, 0, 1, 64, 64, 10, 64, 64, 64, 64, 0, 0, None) == mnb.MNB_OK


def test_attention_null_structs():
    lib = mnb.load()
    assert lib.mnb_paged_attention(None, ctypes.byref(_cache())) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_paged_attention(ctypes.byref(_attention()), None) == mnb.MNB_ERR_INVALID_ARG


@pytest.mark.parametrize("args", [(0, 64, 64, 10), (1, 0, 2, 10), (1, 64, 63, 10), (1, 64, 66, 10), (1, 64, 0, 10), (1, 64, 64, 0)])
def test_rotary_sizes(args):
    H, D, rot, n_pos = args
    p = 4096
    assert mnb.load().mnb_rotary(p, p, p, p, p, 1, H, D, rot, n_pos, D, D, D, D, 0, 0, None) == mnb.MNB_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(flags=4), dict(dtype=3), dict(x=4098), dict(ts=-1)])
def test_rotary_arguments(kw):
    p = 4096
    assert mnb.load().mnb_rotary(kw.get("x", p), p, p, p, p, 1, 2, 64, 64, 10, kw.get("ts", 128), 64, 128, 64, kw.get("dtype", 0),
                                 kw.get("flags", 0), None) == mnb.MNB_ERR_INVALID_ARG


@pytest.mark.parametrize("args", [(0, 64, 1e4, 0, 1.0, 0, 0, 0, 1.0), (9, 63, 1e4, 0, 1.0, 0, 0, 0, 1.0), (9, 64, -1.0, 0, 1.0, 0, 0, 0, 1.0),
                                  (9, 64, 1e4, 4, 1.0, 0, 0, 0, 1.0), (9, 64, 1e4, 1, 0.0, 0, 0, 0, 1.0), (9, 2, 1e4, 2, 2.0, 0, 0, 0, 1.0),
                                  (9, 64, 1e4, 3, 2.0, 0.0, 1, 32, 1.0), (9, 64, 1e4, 3, 2.0, 4096.0, 32, 32, 1.0)])
def test_rotary_table_arguments(args):
    assert mnb.load().mnb_rotary_table(4096, 4096, *args, None) == mnb.MNB_ERR_INVALID_ARG


def _state(**kw):
    s = mnb.CacheState()
    s.refs = s.tables = s.lens = 4096
    s.num_pages, s.num_seqs, s.table_stride, s.page_size = 9, 3, 4, 16
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _planes(**kw):
    p = mnb.PagePlanes()
    p.base, p.num_planes, p.plane_stride, p.page_stride, p.page_bytes, p.num_pages = 4096, 2, 9 * 64, 64, 64, 9
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("bad", [{"refs": None}, {"num_pages": 0}, {"num_seqs": 262145}, {"table_stride": 0}, {"page_size": 0}, {"lens": 2},
                                 {"table_stride": 1 << 30}])
def test_cache_state(bad):
    lib, s = mnb.load(), _state(**bad)
    assert lib.mnb_cache_fork(ctypes.byref(s), 4096, 4096, 1, 4096, 1 << 40, None) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_cache_resize(ctypes.byref(s), None, 4096, 4096, 1, 4096, 1 << 40, None) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_cache_compact(ctypes.byref(s), ctypes.byref(_planes()), 4096, 4096, 4096, 4096, 1 << 40, None) == mnb.MNB_ERR_INVALID_ARG


def test_cache_lists_and_workspace():
    lib, s = mnb.load(), _state()
    need = mnb.mnb_cache_workspace_size(9, 3, 4)
    assert need > 0 and need % 256 == 0
    assert lib.mnb_cache_fork(ctypes.byref(s), 4096, 4096, 4, 4096, need, None) == mnb.MNB_ERR_INVALID_ARG  # n > num_seqs
    assert lib.mnb_cache_fork(ctypes.byref(s), None, 4096, 1, 4096, need, None) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_cache_fork(ctypes.byref(s), 4096, 4096, 1, 4096, 16, None) == mnb.MNB_ERR_NO_MEM
    assert lib.mnb_cache_fork(ctypes.byref(s), 4096, 4096, 1, 4100, need, None) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_cache_fork(ctypes.byref(s), 4096, 4096, 0, None, 0, None) == mnb.MNB_OK
    assert mnb.mnb_cache_workspace_size(0, 3, 4) == 0 and mnb.mnb_cache_workspace_size(9, 1 << 20, 4) == 0


@pytest.mark.parametrize("bad", [{"base": None}, {"base": 4104}, {"page_bytes": 24}, {"page_bytes": 80}, {"plane_stride": 64},
                                 {"plane_stride": 0}, {"num_planes": 0}, {"page_stride": 1 << 62}])
def test_page_planes(bad):
    assert mnb.load().mnb_pages_copy(ctypes.byref(_planes(**bad)), 4096, 4096, 1, None) == mnb.MNB_ERR_INVALID_ARG


def test_page_planes_of_the_wrong_count():
    s = _state()
    assert mnb.load().mnb_cache_compact(ctypes.byref(s), ctypes.byref(_planes(num_pages=8, plane_stride=512)), 4096, 4096, 4096, 4096, 1 << 40,
                                        None) == mnb.MNB_ERR_INVALID_ARG


def test_binding_checks_tensors():
    t = torch.zeros((2, 3, 8))
    tab = torch.zeros((4, 2))
    with pytest.raises(ValueError):
        mnb.mnb_rotary(t, t[:, :2], torch.zeros(2, dtype=torch.int32), tab, tab, 0, stream=0)
    with pytest.raises(ValueError):
        mnb.mnb_rotary(t, t, torch.zeros(2, dtype=torch.int64), tab, tab, 0, stream=0)
    with pytest.raises(ValueError):
        mnb.mnb_rotary(t.bfloat16(), t, torch.zeros(2, dtype=torch.int32), tab, tab, 0, stream=0)
    pages = torch.zeros((3, 2, 16, 8))
    with pytest.raises(ValueError):
        mnb.kv_cache(pages, pages[:2], torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), "hnd", 0)
    with pytest.raises(ValueError):
        mnb.kv_cache(pages, pages, torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), "dhn", 0)
    c = mnb.kv_cache(pages, pages, torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), "hnd", 0)
    assert (c.num_pages, c.kv_heads, c.page_size, c.head_dim, c.token_stride, c.head_stride) == (3, 2, 16, 8, 8, 128)
    c = mnb.kv_cache(pages, pages, torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), "nhd", 0)
    assert (c.kv_heads, c.page_size, c.token_stride, c.head_stride) == (16, 2, 128, 8)
    with pytest.raises(ValueError):
        mnb.page_planes(torch.zeros((2, 3, 4, 5)).transpose(2, 3))
    p = mnb.page_planes(torch.zeros((2, 3, 4, 8)))
    assert (p.num_planes, p.num_pages, p.plane_stride, p.page_stride, p.page_bytes) == (2, 3, 384, 128, 128)

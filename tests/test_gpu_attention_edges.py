"""Attention over the paged cache at its edges: NaN and infinities in queries and keys, rows that see nothing beside
rows that do, windows wider than any sequence, batches wider than one look at them, workspaces of other calls."""

import math

import numpy as np
import pytest
import torch

from tests import _decoder_ref as R
from tests.test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu


def _rows(p):
    """(token, sequence, position) of each row of the call."""
    t = 0
    for b, (m, n) in enumerate(zip(p.q_lens, p.kv_lens)):
        for i in range(m):
            yield t, b, n - m + i
            t += 1


def _check(p, o, lse, nan_rows, empty_rows=(), window=0, heads=None):
    """Rows (token, head) of nan_rows are NaN in every depth and in lse, those of empty_rows 0 and -inf, and all others
    within the 64-bit form's bounds."""
    go, gl = R.f64(o), R.f64(lse)
    k, v = {}, {}
    for t, b, pos in _rows(p):
        for h in range(p.hq) if heads is None else heads:
            if (t, h) in nan_rows:
                assert np.isnan(go[t, h]).all() and np.isnan(gl[t, h]), ("NaN", t, h, go[t, h][:4], gl[t, h])
                continue
            if (t, h) in empty_rows:
                assert (go[t, h] == 0).all() and np.isneginf(gl[t, h]), ("empty", t, h, go[t, h][:4], gl[t, h])
                continue
            hk = h // (p.hq // p.hkv)
            if (b, hk) not in k:
                k[b, hk], v[b, hk] = p.rows(p.k, b, hk), p.rows(p.v, b, hk)
            lo = max(0, pos - window + 1) if window else 0
            ro, rl, bo, bl = R.attention(R.f64(p.q[t:t + 1, h]), k[b, hk][lo:pos + 1], v[b, hk][lo:pos + 1], pos - lo,
                                         np.float32(p.scale()).astype(np.float64), True, 0)
            assert (np.abs(go[t, h] - ro[0]) <= bo[p.dtype][0]).all(), (t, h)
            assert (np.isneginf(gl[t, h]) and np.isneginf(rl[0])) or abs(gl[t, h] - rl[0]) <= bl[0], (t, h, gl[t, h], rl[0])


def _set_keys(p, b, keys, value, what="k", head=slice(None)):
    """Keys (or values) of a sequence's tokens."""
    pages = p.k if what == "k" else p.v
    for j in keys:
        page, row = int(p.np_tables[b, j // p.page]), j % p.page
        if p.order == "hnd":
            pages[page, head, row] = value
        else:
            pages[page, row, head] = value


#: one call of each kernel and form: clusters, the even cut and its join, the many-row kernel whole and cut, f32
FORMS = [("bf16", [1, 1], [300, 40], 8, 2, 128), ("f16", [1] * 5, [9000, 31, 700, 64, 5], 8, 2, 64), ("bf16", [1], [3000], 2, 1, 256),
         ("bf16", [1] * 40, [37 * (i + 1) for i in range(40)], 16, 8, 128), ("bf16", [260], [260], 2, 1, 64), ("f16", [40], [2500], 4, 2, 128),
         ("bf16", [70, 3], [1900, 40], 6, 2, 96), ("bf16", [90], [100], 4, 2, 128), ("f32", [1, 9], [500, 30], 4, 2, 64)]


def _form(mnb, form, seed, **kw):
    dtype, q_lens, kv_lens, hq, hkv, D = form
    return Problem(mnb, q_lens, kv_lens, hq, hkv, D, dtype, 16, "hnd", seed=seed, **kw)


@pytest.mark.parametrize("form", FORMS)
def test_a_nan_query_gives_nan(mnb, form):
    """Never the zeros of a row that sees no key, however the keys are divided."""
    p = _form(mnb, form, 21)
    bad = {(0, 0), (p.T - 1, p.hq - 1), (p.T // 2, 1)}
    for t, h in bad:
        p.q[t, h, 3] = float("nan")
    o, _ = p.run()
    for t, h in bad:
        assert torch.isnan(o[t, h]).all(), (t, h, o[t, h, :4])
    o[torch.tensor([t for t, _ in bad]), torch.tensor([h for _, h in bad])] = 0
    assert not torch.isnan(o).any()


@pytest.mark.parametrize("tiles", [1, 2, 3, 4])
@pytest.mark.parametrize("form", [f for f in FORMS if max(f[2]) >= 1900])
def test_nan_in_every_key_of_a_range_gives_nan(mnb, form, tiles):
    """The first 128, 256, .. keys of the longest sequence hold NaN, so that for one of the counts at least a range of its
    keys holds nothing else: every row of the sequence is NaN, and none of the others."""
    p = _form(mnb, form, 22)
    b = int(np.argmax(p.kv_lens))
    _set_keys(p, b, range(128 * tiles), float("nan"))
    o, _ = p.run()
    for t, s, _ in _rows(p):
        assert torch.isnan(o[t]).all() if s == b else not torch.isnan(o[t]).any(), t


@pytest.mark.parametrize("form", FORMS)
def test_lse_of_a_nan_row_is_nan(mnb, form):
    """And not the -inf of a row that sees no key; the other rows keep theirs."""
    p = _form(mnb, form, 23)
    bad = {(0, 0), (p.T - 1, p.hq - 1), (p.T // 2, 1)}
    for t, h in bad:
        p.q[t, h, p.D - 1] = float("nan")
    o, lse = p.run()
    _check(p, o, lse, bad, heads=sorted({0, 1, p.hq - 1}) if p.T <= 10 else [0])


@pytest.mark.parametrize("form", FORMS)
def test_an_infinite_score_gives_nan(mnb, form):
    """exp(inf - inf): the row has no value, in o and in lse."""
    p = _form(mnb, form, 24)
    p.q[:, :, 0] = 1.0
    _set_keys(p, 0, [0], 0.0)
    p.k[int(p.np_tables[0, 0]), :, 0, 0] = float("inf")
    o, lse = p.run()
    for t, b, _ in _rows(p):
        bad = torch.isnan(o[t]).all() and torch.isnan(lse[t]).all()
        assert bad if b == 0 else not (torch.isnan(o[t]).any() or torch.isnan(lse[t]).any()), t


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
@pytest.mark.parametrize("dtype,q_lens,kv_lens,hq,hkv,D", [
    ("bf16", [5], [2], 4, 2, 128), ("f16", [5, 1], [2, 20000], 4, 2, 64), ("bf16", [300, 4], [130, 1], 4, 2, 128), ("f32", [5, 40], [2, 7], 2, 1, 64)])
def test_a_window_past_every_sequence_is_no_window(mnb, window, dtype, q_lens, kv_lens, hq, hkv, D):
    """The largest int stands for "no limit", and more new tokens than keys put the first rows before the sequence."""
    p = Problem(mnb, q_lens, kv_lens, hq, hkv, D, dtype, 16, "hnd", seed=25)
    p.check(*p.run(window=window), window=window)


@pytest.mark.parametrize("dtype,batch,q,hq,hkv,D", [
    ("bf16", 140, 1, 4, 1, 128), ("f16", 300, 1, 2, 1, 64),      # clusters
    ("bf16", 200, 1, 4, 4, 128), ("bf16", 150, 20, 2, 1, 128),   # the even cut, the many-row kernel
    ("f32", 140, 1, 2, 1, 64)])
@pytest.mark.parametrize("at", [0, 127, 128, -1])
def test_any_sequence_past_the_bounds_is_reported(mnb, dtype, batch, q, hq, hkv, D, at):
    lens = [q + (7 * i) % 90 for i in range(batch)]
    lens[at] = 300
    p = Problem(mnb, [q] * batch, lens, hq, hkv, D, dtype, 16, "hnd", seed=26)
    o, lse = p.run(max_kv=299)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    p.check(o, lse, seqs={0, 1, 63, 126, batch - 2} - {at % batch}, heads=[0, hq - 1])


@pytest.mark.parametrize("dtype,q", [("bf16", 1), ("bf16", 60), ("f32", 1)])
def test_a_sequence_without_new_tokens_is_reported_too(mnb, dtype, q):
    p = Problem(mnb, [q, 0, q], [80, 300, 70], 4, 2, 128, dtype, 16, "hnd", seed=27)
    o, lse = p.run(max_kv=200)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    p.check(o, lse, seqs=[0, 2])


def test_a_workspace_of_a_larger_call_serves_smaller_ones(mnb):
    """A server sizes its buffer once, for the largest call; that call may have units enough and cut none of them."""
    heads, kv_heads, D, code = 4, 2, 128, R.CODE["bf16"]
    size = mnb.mnb_attention_workspace_size(1, 8000, heads, kv_heads, D, 8000, 9000, code)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for q, kv in ((70, 9000), (300, 2500), (1, 9000), (20, 3000)):
        p = Problem(mnb, [q], [kv], heads, kv_heads, D, "bf16", 16, "hnd", seed=q)
        o, lse = torch.empty_like(p.q), torch.empty(p.q.shape[:2], device="cuda")
        mnb.mnb_paged_attention(p.q, o, p.cache, p.start, q, kv, p.scale(), lse=lse, workspace=ws)
        p.check(o, lse, heads=[0, heads - 1])


@pytest.mark.parametrize("part", [0.0, 0.3, 0.7, 1.0])
def test_a_smaller_workspace_cuts_into_fewer_ranges(mnb, part):
    """Between the least and the full size a call is cut as far as the buffer goes, and no byte past it is written."""
    p = Problem(mnb, [70], [9000], 4, 2, 128, "bf16", 16, "hnd", seed=28)
    full = mnb.mnb_attention_workspace_size(1, 70, 4, 2, 128, 70, 9000, R.CODE["bf16"])
    least = mnb.mnb_attention_workspace_size(1, 1, 4, 2, 128, 1, 9000, R.CODE["bf16"])
    size = least + int((full - least) * part) // 256 * 256
    ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(p.q), torch.empty(p.q.shape[:2], device="cuda")
    mnb.mnb_paged_attention(p.q, o, p.cache, p.start, 70, 9000, p.scale(), lse=lse, workspace=ws[:size])
    p.check(o, lse, heads=[0, 3])
    assert (ws[size:] == 0x5A).all()
    with pytest.raises(mnb.MnbError) as e:
        mnb.mnb_paged_attention(p.q, o, p.cache, p.start, 70, 9000, p.scale(), lse=lse, workspace=ws[:least - 256])
    assert e.value.status == mnb.MNB_ERR_NO_MEM


@pytest.mark.parametrize("causal", [True, False])
def test_under_a_window_the_cut_does_not_follow_the_context(mnb, causal):
    """A chunk under a window sees as many keys of a long context as of a short one: the same bits, whatever max_kv is."""
    p = Problem(mnb, [500], [3000], 32, 8, 128, "bf16", 16, "hnd", seed=29)
    got = [p.run(causal, 1024, max_kv=n) for n in (3000, 32000, 100000)]
    p.check(*got[0], causal=causal, window=1024, heads=[31])
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


def test_the_window_and_not_the_context_chooses_the_kernel(mnb, monkeypatch, capfd):
    """Drafted tokens (17 to 32 rows a key head) under a window read the same keys of a long context as of a short one."""
    families = []
    for kv in (2000, 40000):
        p = Problem(mnb, [8] * 16, [600] * 16, 16, 4, 64, "f16", 32, "nhd", seed=30)
        monkeypatch.setenv("MNB_PROFILE", "1")
        monkeypatch.setenv("MNB_PROFILE_EVERY", "1")
        capfd.readouterr()
        o, lse = p.run(window=500, max_kv=kv)
        torch.cuda.synchronize()
        p.run(window=500, max_kv=kv)
        monkeypatch.delenv("MNB_PROFILE")
        families.append({x for x in ("attn_mma", "attn_tc") if f"kernel={x} " in capfd.readouterr().err})
        p.check(o, lse, window=500, heads=[0, 15], seqs=[0, 15])
    assert families[0] and families[0] == families[1]


@pytest.mark.parametrize("mode", ["0", "1", "2"])
def test_roles_wait_while_a_large_batch_is_searched(mnb, monkeypatch, mode):
    """Four million sequences of which the last one alone has new tokens: the warps that wait for their unit do so for as
    long as the search takes, whatever the matmul kernels' way of waiting is."""
    batch, n, kv, page = 1 << 22, 60, 1000, 1024
    p = Problem(mnb, [n], [kv], 4, 1, 64, "bf16", page, "hnd", seed=38)
    start = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    lens, tables = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros((batch, 1), dtype=torch.int32, device="cuda")
    start[-1], lens[-1], tables[-1, 0] = n, kv, p.tables[0, 0]
    cache = mnb.kv_cache(p.k, p.v, tables, lens, "hnd", R.CODE["bf16"])
    o, lse = torch.empty_like(p.q), torch.empty(p.q.shape[:2], device="cuda")
    ws = torch.empty(mnb.mnb_attention_workspace_size(batch, n, 4, 1, 64, n, kv, R.CODE["bf16"]), dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("MNB_WAIT_MODE", mode)
    mnb.mnb_paged_attention(p.q, o, cache, start, n, kv, p.scale(), lse=lse, workspace=ws)
    torch.cuda.synchronize()
    p.check(o, lse)


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("dtype,page,q,kv,window", [
    ("bf16", 16, 1, 500, 97), ("f16", 64, 1, 5000, 1003), ("bf16", 128, 60, 900, 333), ("f16", 16, 60, 9000, 1003), ("f32", 32, 1, 500, 100),
    ("bf16", 8, 3, 77, 5)])
def test_a_nan_before_the_window_reaches_no_row(mnb, what, dtype, page, q, kv, window):
    """Tokens that no row of the call sees any more, up to the last of them: inside a page and a tile that rows do read."""
    p = Problem(mnb, [q], [kv], 4, 2, 128, dtype, page, "hnd", seed=31)
    gone = kv - q - window + 1
    _set_keys(p, 0, range(max(0, gone - 300), gone), float("nan"), what)
    o, lse = p.run(window=window)
    _set_keys(p, 0, range(max(0, gone - 300), gone), 0.0, what)  # (the plain form multiplies them by nought)
    p.check(o, lse, window=window)


@pytest.mark.parametrize("form", FORMS)
def test_scores_of_minus_infinity_alone_are_no_keys(mnb, form):
    """Every visible score -inf: nothing to weigh, o = 0 and lse = -inf, in every kernel; beside a finite score such keys
    weigh nothing."""
    p = _form(mnb, form, 32)
    p.q[:, :, 0] = 1.0
    n = p.kv_lens[0]
    _set_keys(p, 0, range(n), 0.0)
    keys = range(n) if p.q_lens[0] == 1 else range(n - p.q_lens[0] + 3)
    for j in keys:
        page, row = int(p.np_tables[0, j // p.page]), j % p.page
        p.k[page, :, row, 0] = float("-inf")
    o, lse = p.run()
    go, gl = R.f64(o), R.f64(lse)
    values = {hk: p.rows(p.v, 0, hk) for hk in range(p.hkv)}
    for t, b, pos in _rows(p):
        if b:
            continue
        left = np.arange(len(keys), pos + 1)  # these weigh alike: their scores are q . (0, ..) = 0
        for h in range(p.hq):
            if not len(left):
                assert (go[t, h] == 0).all() and np.isneginf(gl[t, h]), (t, h)
            else:
                v = values[h // (p.hq // p.hkv)][left]
                assert (np.abs(go[t, h] - v.mean(0)) <= 1.02 * R.ROUND[p.dtype] * np.abs(v).mean(0) + 2 * R.ROUND[p.dtype] * np.abs(v.mean(0))
                        + 2.0 ** -18).all()
                assert abs(gl[t, h] - math.log(len(left))) <= 2.0 ** -18


@pytest.mark.parametrize("dtype,q_lens,kv_lens,hq,hkv", [
    ("bf16", [5], [3], 4, 2), ("f16", [7, 1], [3, 9000], 2, 1), ("bf16", [300], [200], 4, 2), ("bf16", [300], [100], 4, 2), ("f16", [60, 1], [40, 3000], 4, 2), ("f32", [5], [3], 4, 2)])
def test_a_row_without_a_key_is_zero_beside_rows_that_are_nan(mnb, dtype, q_lens, kv_lens, hq, hkv):
    p = Problem(mnb, q_lens, kv_lens, hq, hkv, 128, dtype, 16, "hnd", seed=33)
    _set_keys(p, 0, [0], float("nan"), "v")
    o, lse = p.run()
    none = q_lens[0] - kv_lens[0]
    assert (o[:none] == 0).all() and torch.isneginf(lse[:none]).all()
    assert torch.isnan(o[none:q_lens[0]]).all() and torch.isfinite(lse[none:q_lens[0]]).all()
    assert not torch.isnan(o[q_lens[0]:]).any()


@pytest.mark.parametrize("q,dtype", [(1, "bf16"), (60, "f16"), (1, "f32")])
def test_a_row_of_a_strided_table_ends_with_its_columns(mnb, q, dtype):
    """Tables that are some columns of a wider array: a length past them sets the status, and what stands behind them is
    not taken for pages."""
    p = Problem(mnb, [q, q], [200, 90], 4, 2, 128, dtype, 16, "hnd", seed=34)
    wide = torch.full((2, 40), 1, dtype=torch.int32, device="cuda")
    cols = wide[:, 3:3 + 13]
    cols.copy_(p.tables[:, :13])
    p.cache = mnb.kv_cache(p.k, p.v, cols, p.lens, "hnd", R.CODE[dtype])
    p.check(*p.run())
    cols = wide[:, 3:3 + 12]  # a page short for the first sequence, and enough for the second
    p.cache = mnb.kv_cache(p.k, p.v, cols, p.lens, "hnd", R.CODE[dtype])
    o, lse = p.run()
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    p.check(o, lse, seqs=[1])
    before = p.k.clone(), p.v.clone()
    x = torch.ones((2, 2, 128), dtype=p.k.dtype, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    one = torch.ones((300, 64), device="cuda")
    mnb.mnb_rotary_append(None, None, x, x, one, torch.zeros_like(one), p.cache, start)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    page, row = int(p.np_tables[1, 89 // 16]), 89 % 16
    before[0][page, :, row], before[1][page, :, row] = 1, 1
    assert torch.equal(torch.nan_to_num(before[0]), torch.nan_to_num(p.k)) and torch.equal(torch.nan_to_num(before[1]), torch.nan_to_num(p.v))


@pytest.mark.parametrize("dtype,page,order", [("bf16", 64, "nhd"), ("f16", 16, "hnd"), ("f32", 32, "nhd")])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D", [
    ([1, 1], [500, 64], 8, 2, 128), ([1], [6000], 4, 1, 64), ([150, 20, 0, 7], [400, 20, 9, 3], 2, 1, 64), ([4, 1], [300, 2], 8, 1, 128),
    ([90], [1500], 4, 2, 96), ([3, 40], [90, 700], 2, 2, 256)])
@pytest.mark.parametrize("window", [0, 65])
def test_not_causal(mnb, dtype, page, order, q_lens, kv_lens, hq, hkv, D, window):
    """Encoders and cross attention: every row sees every key (from its window on)."""
    p = Problem(mnb, q_lens, kv_lens, hq, hkv, D, dtype, page, order, seed=35)
    p.check(*p.run(False, window), causal=False, window=window)


@pytest.mark.parametrize("dtype,page,order", [("f16", 32, "nhd"), ("f32", 8, "nhd"), ("bf16", 128, "nhd")])
@pytest.mark.parametrize("window", [1, 64, 200])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D", [([1, 1], [500, 64], 8, 2, 128), ([150, 20], [400, 20], 2, 1, 64), ([4, 1], [2, 300], 8, 1, 80)])
def test_windows_of_other_types_and_orders(mnb, dtype, page, order, window, q_lens, kv_lens, hq, hkv, D):
    p = Problem(mnb, q_lens, kv_lens, hq, hkv, D, dtype, page, order, seed=window)
    p.check(*p.run(window=window), window=window)


@pytest.mark.parametrize("form", FORMS)
def test_nan_in_a_key_reaches_the_rows_that_see_it(mnb, form):
    """And no other row: the scores of keys that a row does not see are not looked at."""
    p = _form(mnb, form, 36)
    b = len(p.q_lens) - 1
    j = p.kv_lens[b] - max(1, p.q_lens[b] // 2)
    _set_keys(p, b, [j], float("nan"))
    heads = [0, p.hq - 1]
    bad = {(t, h) for t, s, pos in _rows(p) for h in heads if s == b and pos >= j}
    o, lse = p.run()
    if p.T > 60:  # many rows: who is NaN, and no row in part
        assert all(torch.isnan(o[t, h]).all() and torch.isnan(lse[t, h]) for t, h in bad)
        assert torch.isnan(o[:, heads]).all(-1).sum() == len(bad) and torch.equal(torch.isnan(o).any(-1), torch.isnan(o).all(-1))
        return
    _check(p, o, lse, bad, heads=heads)


@pytest.mark.parametrize("form", [("bf16", [1] * 200, [1 + (11 * i) % 250 for i in range(200)], 2, 1, 64),
                                  ("f16", [1] * 150, [1 + (13 * i) % 400 for i in range(150)], 4, 1, 128)])
def test_clusters_of_more_than_128_sequences(mnb, form):
    p = _form(mnb, form, 37)
    p.check(*p.run(), seqs=set(range(0, len(p.q_lens), 9)) | {127, 128, 129, len(p.q_lens) - 1})

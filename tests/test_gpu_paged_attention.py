"""Attention of new tokens over a paged cache against the 64-bit form, per row and depth, with bounds that follow from
the roundings: single tokens to long chunks, shared heads, odd lengths, windows, rows without a key, both page orders."""
import numpy as np
import pytest
import torch

from tests import _decoder_ref as R

pytestmark = pytest.mark.gpu


class Problem:
    def __init__(self, mnb, q_lens, kv_lens, hq, hkv, D, dtype, page, order, seed=0, spread=2.0, pad=0, poison=True):
        rng = np.random.default_rng(seed)
        self.mnb, self.dtype, self.q_lens, self.kv_lens = mnb, dtype, q_lens, kv_lens
        self.hq, self.hkv, self.D, self.page = hq, hkv, D, page
        held = [-(-n // page) for n in kv_lens]
        pages = sum(held) + 2
        shape = (pages, hkv, page, D) if order == "hnd" else (pages, page, hkv, D)
        k, v = rng.standard_normal(shape), rng.standard_normal(shape)
        perm = rng.permutation(pages).astype(np.int32)
        tables = np.full((len(held), max(held + [1]) + 1), 2 ** 30, dtype=np.int32)  # never to be read past a sequence's pages
        at = 0
        used = np.zeros(shape[:1] + (page,), dtype=bool)
        for b, n in enumerate(held):
            tables[b, :n] = perm[at:at + n]
            at += n
            for j in range(n):
                used[tables[b, j], :min(page, kv_lens[b] - j * page)] = True
        if poison:  # rows that no sequence holds are NaN
            view = (lambda a: a.transpose(0, 2, 1, 3)) if order == "hnd" else (lambda a: a)
            view(k)[~used] = np.nan
            view(v)[~used] = np.nan
        self.k, self.v = (torch.from_numpy(a).to(R.DT[dtype]).cuda() for a in (k, v))
        self.tables, self.np_tables = torch.from_numpy(tables).cuda(), tables
        self.lens = torch.tensor(kv_lens, dtype=torch.int32).cuda()
        self.start = torch.tensor(np.cumsum([0] + q_lens), dtype=torch.int32).cuda()
        self.T = sum(q_lens)
        self.q = torch.from_numpy(rng.standard_normal((self.T + pad, hq, D)) * spread).to(R.DT[dtype]).cuda()
        self.cache = mnb.kv_cache(self.k, self.v, self.tables, self.lens, order, R.CODE[dtype])
        self.order = order

    def rows(self, pages, b, h):
        p = self.np_tables[b, :-(-self.kv_lens[b] // self.page)]
        x = pages[p][:, h] if self.order == "hnd" else pages[p][:, :, h]
        return R.f64(x).reshape(-1, self.D)[:self.kv_lens[b]]

    def run(self, causal=True, window=0, scale=None, q=None, max_q=None, max_kv=None, stream=None):
        mnb = self.mnb
        q = self.q if q is None else q
        o = torch.full(self.q.shape, 9.0, dtype=self.q.dtype, device="cuda")
        lse = torch.full(self.q.shape[:2], 9.0, device="cuda")
        mq, mk = max(self.q_lens + [1]) if max_q is None else max_q, max(self.kv_lens + [1]) if max_kv is None else max_kv
        ws = torch.empty(mnb.mnb_attention_workspace_size(len(self.q_lens), q.shape[0], self.hq, self.hkv, self.D, mq, mk,
                                                          R.CODE[self.dtype]) + 256, dtype=torch.uint8, device="cuda").fill_(0xFF)
        mnb.mnb_paged_attention(q, o, self.cache, self.start, mq, mk, self.scale(scale), lse=lse, causal=causal, window=window,
                                workspace=ws, stream=stream)
        return o, lse

    def scale(self, scale=None):
        return self.D ** -0.5 if scale is None else scale

    def check(self, o, lse, causal=True, window=0, scale=None, seqs=None, heads=None):
        t = 0
        for b, (m, n) in enumerate(zip(self.q_lens, self.kv_lens)):
            if m and (seqs is None or b in seqs):
                for h in range(self.hq) if heads is None else heads:
                    hk = h // (self.hq // self.hkv)
                    ro, rl, bo, bl = R.attention(R.f64(self.q[t:t + m, h]), self.rows(self.k, b, hk), self.rows(self.v, b, hk),
                                                 n - m, np.float32(self.scale(scale)).astype(np.float64), causal, window)
                    go, gl = R.f64(o[t:t + m, h]), R.f64(lse[t:t + m, h])
                    bad = np.abs(go - ro) > bo[self.dtype]
                    assert not bad.any() and not np.isnan(go).any(), (b, h, np.argwhere(bad)[:4], go[bad][:4], ro[bad][:4], bo[self.dtype][bad][:4])
                    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
                    fin = np.isfinite(rl)
                    assert (np.abs(gl[fin] - rl[fin]) <= bl[fin]).all(), (b, h, gl[fin], rl[fin])
            t += m
        assert (o[self.T:] == 9).all() and (lse[self.T:] == 9).all()
        assert self.mnb.mnb_get_device_error() == 0


SHAPES = [  # q_lens, kv_lens, hq, hkv, D
    ([1], [1], 1, 1, 64), ([1], [777], 8, 2, 128), ([1, 1, 1, 1], [1, 63, 64, 65], 4, 4, 128),
    ([1, 1, 1], [2000, 17, 513], 16, 2, 64), ([3, 1, 8], [3, 40, 130], 12, 4, 128), ([2, 0, 5], [300, 20, 5], 6, 2, 80),
    ([40], [170], 7, 1, 96), ([129, 70], [129, 301], 4, 2, 128), ([260], [260], 2, 1, 64), ([200], [450], 3, 1, 256),
    ([1, 1], [128, 129], 64, 2, 128), ([5], [600], 10, 2, 8), ([300, 1, 17], [300, 900, 40], 8, 4, 128)]


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D", SHAPES)
@pytest.mark.parametrize("dtype,page,order", [("bf16", 16, "hnd"), ("f16", 64, "nhd"), ("f32", 32, "hnd"), ("bf16", 128, "nhd"), ("f16", 8, "hnd")])
def test_causal(mnb, q_lens, kv_lens, hq, hkv, D, dtype, page, order):
    p = Problem(mnb, q_lens, kv_lens, hq, hkv, D, dtype, page, order, seed=D + len(q_lens), pad=2)
    p.check(*p.run())


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D", [([1, 1], [500, 64], 8, 2, 128), ([150, 20], [400, 20], 2, 1, 64), ([4, 1], [300, 2], 8, 1, 128)])
def test_window(mnb, window, causal, q_lens, kv_lens, hq, hkv, D):
    p = Problem(mnb, q_lens, kv_lens, hq, hkv, D, "bf16", 16, "hnd", seed=window)
    p.check(*p.run(causal, window), causal, window)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [0, 5]), ([5, 300], [2, 130]), ([0, 0, 1], [0, 9, 3]), ([4], [0]), ([300], [0])])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_a_key(mnb, q_lens, kv_lens, dtype):
    """More new tokens than keys: the first rows stand before the sequence and see nothing."""
    p = Problem(mnb, q_lens, kv_lens, 4, 2, 128, dtype, 16, "hnd", seed=3)
    p.check(*p.run())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [3000]), ([200], [1500])])
def test_scores_far_apart(mnb, dtype, q_lens, kv_lens):
    """Peaked rows: maxima that keep growing along the context, and scores hundreds apart."""
    p = Problem(mnb, q_lens, kv_lens, 2, 1, 128, dtype, 16, "nhd", seed=4, spread=1.0)
    n = kv_lens[0]
    order = torch.arange(n, device="cuda", dtype=torch.float32) / n * 6  # keys grow along the sequence
    pages = p.tables[0, :-(-n // 16)].long()
    k = p.k[pages].float().reshape(-1, 1, 128)
    k[:n] += order[:, None, None]
    p.k[pages] = k.view(-1, 16, 1, 128).to(p.k.dtype)
    p.q += 1.0
    p.check(*p.run())
    p.check(*p.run(scale=-0.3), scale=-0.3)
    p.check(*p.run(scale=0.0), scale=0.0)


def test_strided_queries_and_another_stream(mnb):
    p = Problem(mnb, [1, 30, 150], [70, 30, 400], 6, 3, 128, "bf16", 32, "hnd", seed=5)
    wide = torch.zeros((p.T, 11, 128), dtype=p.q.dtype, device="cuda")
    wide[:, 2:8] = p.q
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = p.run(q=wide[:, 2:8], stream=s)
    s.synchronize()
    p.check(o, lse)


def test_sequences_past_the_bounds_set_the_status(mnb):
    p = Problem(mnb, [1, 3], [50, 90], 4, 2, 128, "bf16", 16, "hnd", seed=6)
    o, lse = p.run(max_kv=60)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    o, lse = p.run(max_q=2)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    p.check(o, lse, seqs=[0]) if True else None


@pytest.mark.parametrize("q,kv", [(1, 300), (200, 200)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_page_that_does_not_exist_sets_the_status(mnb, q, kv, dtype):
    p = Problem(mnb, [q, q], [kv, kv], 4, 2, 128, dtype, 16, "hnd", seed=7)
    p.tables[1, 3] = 2 ** 30
    o, lse = p.run()
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    p.check(o, lse, seqs=[0])


@pytest.mark.parametrize("q,kv,batch", [(1, 1500, 3), (64, 700, 2), (300, 900, 1)])
def test_repeats_give_the_same_bits(mnb, q, kv, batch):
    p = Problem(mnb, [q] * batch, [kv] * batch, 8, 2, 128, "bf16", 16, "hnd", seed=8)
    a, b = p.run(), p.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_in_a_graph_with_lengths_that_change(mnb):
    """A captured step replays with other lengths and tables under the same bounds."""
    p = Problem(mnb, [1, 1], [400, 90], 8, 2, 128, "bf16", 16, "hnd", seed=9, poison=False)
    o, lse = torch.zeros_like(p.q), torch.zeros(p.q.shape[:2], device="cuda")
    ws = torch.empty(mnb.mnb_attention_workspace_size(2, 2, 8, 2, 128, 1, 400, 2) + 256, dtype=torch.uint8, device="cuda")
    step = lambda: mnb.mnb_paged_attention(p.q, o, p.cache, p.start, 1, 400, p.scale(), lse=lse, workspace=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([400, 90], [17, 1], [321, 0]):
        p.kv_lens = lens
        p.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        p.check(o, lse)


def _ragged(n, most, seed):
    return [int(x) for x in np.random.default_rng(seed).integers(0, most + 1, n)]


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page,window", [
    ([1], [20011], 8, 2, 128, 16, 0),                                   # one context over every CTA, joined
    ([1, 1], [9001, 12], 12, 2, 80, 32, 0),
    ([1] * 40, _ragged(40, 700, 1), 16, 8, 128, 16, 0),                 # many short units: ranges that hold several, empty ones
    ([1] * 70, _ragged(70, 90, 2), 10, 10, 64, 8, 0),
    ([1] * 90, _ragged(90, 300, 3), 16, 2, 256, 64, 0),
    ([20, 3], [2500, 30], 4, 4, 64, 16, 300),                           # two row tiles of few rows
    ([3] * 50, [n + 3 for n in _ragged(50, 400, 4)], 6, 3, 128, 16, 100),
    ([40], [9000], 4, 2, 128, 16, 0),                                   # many rows, keys cut into ranges
    ([70, 1, 0, 33], [5000, 40, 0, 33], 6, 2, 96, 32, 0),
    ([500], [2100], 4, 1, 64, 128, 777)])
def test_long_and_many(mnb, q_lens, kv_lens, hq, hkv, D, page, window):
    p = Problem(mnb, q_lens, kv_lens, hq, hkv, D, "bf16", page, "hnd", seed=D + len(q_lens))
    heads = sorted({0, hq // 2, hq - 1})
    some = range(0, len(q_lens), max(1, len(q_lens) // 25))
    p.check(*p.run(window=window), window=window, heads=heads, seqs=set(some) | {len(q_lens) - 1})


@pytest.mark.parametrize("q,hq,dtype", [(1, 8, "bf16"), (1, 8, "f32"), (60, 8, "f16")])
def test_pages_before_the_window_are_not_read(mnb, q, hq, dtype):
    """A server under a sliding window frees the pages that no row sees any more."""
    n, window, page = 3000, 500, 16
    p = Problem(mnb, [q], [n], hq, 2, 128, dtype, page, "hnd", seed=13)
    gone = (n - q - window + 1) // page
    keep = p.np_tables[0, :gone].copy()
    p.tables[0, :gone] = -1
    p.k[torch.from_numpy(keep).long().cuda()] = float("nan")
    p.v[torch.from_numpy(keep).long().cuda()] = float("nan")
    o, lse = p.run(window=window)
    # (the plain form reads the freed pages' places, masked: give it zeros)
    p.k[torch.from_numpy(keep).long().cuda()] = 0
    p.v[torch.from_numpy(keep).long().cuda()] = 0
    p.check(o, lse, window=window)


@pytest.mark.parametrize("q,kv", [(120, 900), (300, 300)])
def test_many_rows_in_a_graph_with_lengths_that_change(mnb, q, kv):
    p = Problem(mnb, [q, 7], [kv, 90], 8, 2, 128, "bf16", 16, "hnd", seed=14, poison=False)
    o, lse = torch.zeros_like(p.q), torch.zeros(p.q.shape[:2], device="cuda")
    ws = torch.empty(mnb.mnb_attention_workspace_size(2, p.T, 8, 2, 128, q, kv, 2) + 256, dtype=torch.uint8, device="cuda")
    step = lambda: mnb.mnb_paged_attention(p.q, o, p.cache, p.start, q, kv, p.scale(), lse=lse, workspace=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([kv, 90], [q, 7], [kv - 13, 30]):
        p.kv_lens = lens
        p.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        p.check(o, lse, heads=[0, 5])


@pytest.mark.parametrize("T,q_lens", [(3, [0, 0]), (300, [0, 0]), (0, [0, 0])])
def test_padding_alone(mnb, T, q_lens):
    """Nothing but tokens past q_start[batch]: nothing is written."""
    p = Problem(mnb, q_lens, [5, 40], 4, 2, 128, "bf16", 16, "hnd", seed=15, pad=T)
    o, lse = p.run(max_q=max(1, T))
    p.check(o, lse)


def test_strides_along_one_token_or_head_do_not_matter(mnb):
    p = Problem(mnb, [1], [45], 1, 1, 64, "bf16", 16, "hnd", seed=16)
    q = torch.as_strided(p.q.clone(), (1, 1, 64), (3, 5, 1))
    p.check(*p.run(q=q))


@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("inside", ["page pairs", "padded heads", "padded pages", "one head of many"])
@pytest.mark.parametrize("q_lens,kv_lens", [([70, 40], [70, 333]), ([1, 1], [45, 700])])
def test_pools_with_gaps(mnb, order, inside, q_lens, kv_lens):
    """Keys and values of a page side by side, and strides that are no multiples of each other."""
    hkv = 1 if inside == "one head of many" else 2
    p = Problem(mnb, q_lens, kv_lens, 4, hkv, 128, "bf16", 16, order, seed=17)
    pages, b, c, D = p.k.shape
    if inside == "page pairs":
        pool = torch.full((pages, 2, b, c, D), float("nan"), dtype=p.k.dtype, device="cuda")
        k, v = pool[:, 0], pool[:, 1]
    elif inside == "one head of many":
        at = 1 if order == "hnd" else 2
        wide = list(p.k.shape)
        wide[at] = 3
        k, v = (torch.full(wide, float("nan"), dtype=p.k.dtype, device="cuda").narrow(at, 1, 1) for _ in range(2))
    else:
        pad = 8 if inside == "padded pages" else 0
        row = D + 8 if inside == "padded heads" else D
        k, v = (torch.full((pages * (b * c * row + pad),), float("nan"), dtype=p.k.dtype, device="cuda").as_strided(
            p.k.shape, (b * c * row + pad, c * row, row, 1)) for _ in range(2))
    k.copy_(p.k)
    v.copy_(p.v)
    p.cache = mnb.kv_cache(k, v, p.tables, p.lens, order, R.CODE["bf16"])
    p.check(*p.run())


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("scale", [-0.3, 0.0, -1e-38])
def test_many_rows_under_scales_that_are_not_positive(mnb, D, scale):
    p = Problem(mnb, [90], [400], 4, 2, D, "f16", 16, "hnd", seed=18)
    p.check(*p.run(scale=scale), scale=scale)

"""Copying, forking, resizing and compacting the pages of a cache against plain lists: every array equal after every
step, for random histories and for the cases where a parallel step can go wrong."""
import numpy as np
import pytest
import torch

from tests import _decoder_ref as R

pytestmark = pytest.mark.gpu


class Cache:
    def __init__(self, mnb, pages, seqs, stride, ps, planes=3, elems=24, seed=0):
        self.mnb, self.ps = mnb, ps
        rng = np.random.default_rng(seed)
        self.pool = torch.from_numpy(rng.integers(-30000, 30000, (planes, pages, elems)).astype(np.int16)).cuda()
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.tables = torch.full((seqs, stride), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.planes = mnb.page_planes(self.pool)
        self.state = mnb.cache_state(self.refs, self.tables, self.lens, ps)
        self.ws = torch.empty(mnb.mnb_cache_workspace_size(pages, seqs, stride), dtype=torch.uint8, device="cuda").fill_(0xEE)
        self.ref = R.Pages(self.refs, self.tables, self.lens, ps, self.pool.cpu().numpy())

    def same(self):
        assert self.refs.tolist() == self.ref.refs
        assert self.lens.tolist() == self.ref.lens
        assert self.tables.tolist() == self.ref.tables
        assert np.array_equal(self.pool.cpu().numpy(), self.ref.pool)

    def fork(self, src, dst):
        self.mnb.mnb_cache_fork(self.state, _i(src), _i(dst), workspace=self.ws)
        self.ref.fork(src, dst)

    def resize(self, seqs, lens):
        self.mnb.mnb_cache_resize(self.state, self.planes, _i(seqs), _i(lens), workspace=self.ws)
        assert self.ref.resize(seqs, lens) == (self.mnb.mnb_get_device_error() == 0)

    def compact(self, in_place=False):
        refs = self.refs if in_place else torch.empty_like(self.refs)
        tables = self.tables if in_place else torch.empty_like(self.tables)
        counts = torch.empty(2, dtype=torch.int32, device="cuda")
        self.mnb.mnb_cache_compact(self.state, self.planes, refs, tables, counts, workspace=self.ws)
        assert counts.tolist() == list(self.ref.compact())
        self.refs.copy_(refs)
        self.tables.copy_(tables)


def _i(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("pages,seqs,stride,ps,planes,elems", [
    (1, 1, 1, 1, 1, 8), (40, 6, 8, 16, 3, 24), (700, 33, 40, 4, 2, 8), (5000, 300, 20, 8, 1, 2056), (300, 3, 130, 1, 5, 8)])
def test_random_history(mnb, pages, seqs, stride, ps, planes, elems):
    c = Cache(mnb, pages, seqs, stride, ps, planes, elems, pages)
    rng = np.random.default_rng(pages + 1)
    for step in range(14):
        what = rng.integers(0, 4)
        n = int(rng.integers(1, seqs + 1))
        dst = [int(x) for x in rng.permutation(seqs)[:n]]
        if what == 0:
            c.fork([int(x) for x in rng.integers(0, seqs, n)], dst)
        elif what == 3:
            c.compact(in_place=bool(step & 1))
        else:
            most = min(stride * ps, max(1, 2 * pages * ps // seqs))
            c.resize(dst, [int(x) for x in rng.integers(0, most + 1, n)])
        c.same()


def test_swap_and_self_fork(mnb):
    c = Cache(mnb, 20, 4, 5, 4)
    c.resize([0, 1, 2], [9, 14, 4])
    c.fork([1, 0, 2, 0], [0, 1, 2, 3])  # 0 and 1 trade places, 2 stays, 3 takes the old 0
    c.same()
    assert c.lens.tolist() == [14, 9, 4, 9]


def test_every_holder_of_a_shared_page_grows(mnb):
    c = Cache(mnb, 30, 5, 6, 4)
    c.resize([0], [6])
    c.fork([0, 0, 0], [1, 2, 3])
    c.resize([3, 0, 1, 2], [7, 7, 9, 12])
    c.same()
    c.resize([0, 1], [0, 0])  # freed
    c.same()
    c.resize([4, 2], [11, 12])
    c.same()


def test_growing_from_a_full_last_page_copies_nothing(mnb):
    c = Cache(mnb, 10, 2, 4, 4)
    c.resize([0], [8])
    c.fork([0], [1])
    c.resize([1], [9])
    c.same()
    assert (c.refs > 1).sum() == 2


def test_too_few_pages_change_nothing(mnb):
    c = Cache(mnb, 4, 3, 4, 4)
    c.resize([0, 1], [8, 4])
    c.resize([2, 0], [5, 9])  # needs three of one free page
    c.same()
    c.mnb.mnb_cache_resize(c.state, c.planes, _i([2]), _i([5]), workspace=c.ws)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_NO_MEM
    c.same()


@pytest.mark.parametrize("seqs,lens", [([0, 0], [1, 2]), ([3], [1]), ([-1], [1]), ([0], [17]), ([0], [-1])])
def test_invalid_lists_change_nothing(mnb, seqs, lens):
    c = Cache(mnb, 9, 3, 4, 4)
    c.resize([1], [7])
    c.mnb.mnb_cache_resize(c.state, c.planes, _i(seqs), _i(lens), workspace=c.ws)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    c.same()
    if lens[0] == 1:
        c.mnb.mnb_cache_fork(c.state, _i([1] * len(seqs)), _i(seqs), workspace=c.ws)
        assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
        c.same()


def test_without_planes_a_shared_partial_page_is_refused(mnb):
    c = Cache(mnb, 9, 3, 4, 4)
    c.mnb.mnb_cache_resize(c.state, None, _i([0]), _i([6]), workspace=c.ws)
    c.ref.resize([0], [6])
    c.fork([0], [1])
    c.mnb.mnb_cache_resize(c.state, None, _i([1]), _i([7]), workspace=c.ws)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    c.same()


@pytest.mark.parametrize("elems,planes,n", [(8, 1, 1), (24, 3, 7), (2056, 2, 5), (16384, 4, 3)])
def test_pages_copy(mnb, elems, planes, n):
    c = Cache(mnb, 3 * n, 1, 1, 1, planes, elems, n)
    perm = np.random.default_rng(n).permutation(3 * n)
    src, dst = perm[:n], perm[n:2 * n]
    mnb.mnb_pages_copy(c.planes, _i(src), _i(dst))
    c.ref.pool[:, dst] = c.ref.pool[:, src]
    c.same()
    # a strided view: planes inside pages ([pages, planes, n] storage)
    t = c.pool.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    mnb.mnb_pages_copy(mnb.page_planes(t), _i(dst), _i(perm[2 * n:]))
    c.ref.pool[:, perm[2 * n:]] = c.ref.pool[:, dst]
    assert np.array_equal(t.cpu().numpy(), c.ref.pool)
    # a page that does not exist is skipped
    mnb.mnb_pages_copy(c.planes, _i([0, 3 * n]), _i([-1, 0])) if n > 1 else None
    if n > 1:
        assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG


def test_repeats_give_the_same_bits(mnb):
    """Which page a sequence gets does not depend on how threads run."""
    got = []
    for _ in range(3):
        c = Cache(mnb, 4000, 200, 30, 4, 1, 8, 5)
        c.resize(range(200), [(i * 7) % 60 for i in range(200)])
        c.fork(range(100), range(199, 99, -1))
        c.resize(range(0, 200, 3), [(i * 11) % 100 for i in range(0, 200, 3)])
        got.append((c.refs.tolist(), c.tables.tolist(), c.pool.cpu().numpy().tobytes()))
    assert got[0] == got[1] == got[2]

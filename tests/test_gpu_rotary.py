"""Rotary positions and the append to the paged cache against their 64-bit forms: layouts, partial rotations, types,
strides and alignments that force every access width, the inverse as the gradient, ragged batches, refused places."""
import math

import numpy as np
import pytest
import torch

from tests import _decoder_ref as R

pytestmark = pytest.mark.gpu


def _tables(n_pos, rot):
    t = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.cos(t)).float().cuda(), torch.from_numpy(np.sin(t)).float().cuda()


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(R.DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot,pad,off", [
    (1, 1, 64, 64, 0, 0), (3, 5, 128, 128, 0, 0), (7, 3, 96, 64, 2, 0), (33, 9, 80, 40, 1, 0), (5, 2, 10, 6, 0, 0),
    (4, 3, 97, 64, 0, 0), (6, 2, 64, 32, 1, 1), (2, 3, 72, 72, 0, 4), (2, 1, 2, 2, 0, 0), (700, 40, 128, 128, 0, 0)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(mnb, dtype, layout, T, H, D, rot, pad, off, inverse):
    n_pos = 517
    cos, sin = _tables(n_pos, rot)
    flat = _rand((T * (H + pad) * D + off,), dtype, T + D).cuda()
    x = flat[off:].view(T, H + pad, D)[:, :H]
    pos = torch.from_numpy(np.random.default_rng(T).integers(0, n_pos, T).astype(np.int32)).cuda()
    y = torch.full((T, H + 1, D), 7.0, dtype=R.DT[dtype], device="cuda")
    flags = (mnb.MNB_ROTARY_INTERLEAVED if layout == "interleaved" else 0) | (mnb.MNB_ROTARY_INVERSE if inverse else 0)
    mnb.mnb_rotary(x, y[:, 1:], pos, cos, sin, R.CODE[dtype], flags=flags)
    ref, mag = R.rotary(R.f64(x), R.f64(cos), R.f64(sin), pos.cpu().numpy(), layout, inverse)
    assert (np.abs(R.f64(y[:, 1:]) - ref) <= R.rotary_bound(ref, mag, dtype)).all()
    assert (y[:, 0] == 7).all()  # nothing beside the output is written
    x2 = x.clone()
    mnb.mnb_rotary(x2, x2, pos, cos, sin, R.CODE[dtype], flags=flags)  # in place
    assert torch.equal(x2, y[:, 1:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradient_is_the_inverse_rotation(mnb, layout):
    """d/dx <w, rotary(x)> against differences of <w, rotary(x)>, which is linear in x."""
    T, H, D, rot = 3, 2, 24, 16
    cos, sin = _tables(50, rot)
    pos = torch.tensor([0, 17, 49], dtype=torch.int32).cuda()
    flags = mnb.MNB_ROTARY_INTERLEAVED if layout == "interleaved" else 0
    w, x = _rand((T, H, D), "f32", 1).cuda(), _rand((T, H, D), "f32", 2).cuda()
    grad = torch.empty_like(x)
    mnb.mnb_rotary(w, grad, pos, cos, sin, 0, flags=flags | mnb.MNB_ROTARY_INVERSE)
    w64 = R.f64(w)
    for t, h, d in [(0, 0, 0), (1, 1, 3), (1, 0, 8), (2, 1, 15), (2, 0, 20)]:
        out = []
        for step in (0.5, -0.5):  # exact steps
            z = x.clone()
            z[t, h, d] = step
            y = torch.empty_like(z)
            mnb.mnb_rotary(z, y, pos, cos, sin, 0, flags=flags)
            out.append((w64 * R.f64(y)).sum())
        # each y of the pair is within 3 * 2^-24 of |a| + |b| <= 5, on both sides; w within 5
        assert abs(out[0] - out[1] - float(grad[t, h, d])) <= 4 * 3 * 2.0 ** -24 * 25


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("q_lens,kv_lens,page,hq,hkv,D,rot,layout", [
    ([1], [1], 16, 4, 1, 64, 64, "half"), ([1, 1, 1], [17, 1, 300], 16, 4, 2, 128, 128, "half"),
    ([5, 0, 40, 1], [5, 9, 90, 32], 8, 6, 2, 80, 40, "interleaved"), ([130, 3], [130, 257], 128, 3, 3, 24, 8, "half"),
    ([300, 600], [300, 777], 32, 32, 8, 128, 128, "interleaved")])
def test_rotary_append(mnb, dtype, order, q_lens, kv_lens, page, hq, hkv, D, rot, layout):
    B, T = len(q_lens), sum(q_lens)
    held = [-(-n // page) for n in kv_lens]
    pages = sum(held) + 2
    rng = np.random.default_rng(D)
    perm = rng.permutation(pages).astype(np.int32)
    tables = np.full((B, max(held) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(held):
        tables[b, :n] = perm[at:at + n]
        at += n
    shape = (pages, hkv, page, D) if order == "hnd" else (pages, page, hkv, D)
    kp, vp = _rand(shape, dtype, 5).cuda(), _rand(shape, dtype, 6).cuda()
    qkv = _rand((T + 2, hq + 2 * hkv, D), dtype, 7).cuda()  # two tokens of padding
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cos, sin = _tables(1000, rot)
    start = torch.tensor(np.cumsum([0] + q_lens), dtype=torch.int32).cuda()
    cache = mnb.kv_cache(kp, vp, torch.from_numpy(tables).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(), order, R.CODE[dtype])
    out = torch.full((T + 2, hq, D), 3.0, dtype=R.DT[dtype], device="cuda")
    pos = np.concatenate([np.arange(n - m, n) for m, n in zip(q_lens, kv_lens)]).astype(np.int64)
    kref, vref = R.f64(kp), R.f64(vp)
    mnb.mnb_rotary_append(q, out, k, v, cos, sin, cache, start, flags=mnb.MNB_ROTARY_INTERLEAVED if layout == "interleaved" else 0)
    qr, qm = R.rotary(R.f64(q[:T]), R.f64(cos), R.f64(sin), pos, layout)
    kr, km = R.rotary(R.f64(k[:T]), R.f64(cos), R.f64(sin), pos, layout)
    kb = np.zeros_like(kref)
    seq = np.repeat(np.arange(B), q_lens)
    for t in range(T):
        p, r = tables[seq[t], pos[t] // page], pos[t] % page
        at = (p, slice(None), r) if order == "hnd" else (p, r)
        kref[at], kb[at], vref[at] = kr[t], R.rotary_bound(kr[t], km[t], dtype), R.f64(v[t])
    assert (np.abs(R.f64(out[:T]) - qr) <= R.rotary_bound(qr, qm, dtype)).all()
    assert (out[T:] == 3).all()
    assert (np.abs(R.f64(kp) - kref) <= kb).all() and np.array_equal(R.f64(vp), vref)
    # append alone writes the same bits
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    cache2 = mnb.kv_cache(kp2, vp2, cache.tensors[2], cache.tensors[3], order, R.CODE[dtype])
    mnb.mnb_rotary_append(None, None, k, v, cos, sin, cache2, start, flags=mnb.MNB_ROTARY_INTERLEAVED if layout == "interleaved" else 0)
    for t in range(0, T, 7):
        p, r = tables[seq[t], pos[t] // page], pos[t] % page
        at = (p, slice(None), r) if order == "hnd" else (p, r)
        assert torch.equal(kp2[at], kp[at]) and torch.equal(vp2[at], vp[at])
    assert mnb.mnb_get_device_error() == 0


def test_explicit_positions_and_another_stream(mnb):
    cos, sin = _tables(300, 32)
    kp, vp = torch.zeros((4, 2, 16, 32), device="cuda"), torch.zeros((4, 2, 16, 32), device="cuda")
    tables = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32).cuda()
    lens = torch.tensor([20, 5], dtype=torch.int32).cuda()
    start = torch.tensor([0, 2, 3], dtype=torch.int32).cuda()
    pos = torch.tensor([250, 7, 0], dtype=torch.int32).cuda()
    k, v = _rand((3, 2, 32), "f32", 1).cuda(), _rand((3, 2, 32), "f32", 2).cuda()
    cache = mnb.kv_cache(kp, vp, tables, lens, "hnd", 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mnb.mnb_rotary_append(None, None, k, v, cos, sin, cache, start, positions=pos, stream=s)
    s.synchronize()
    ref, mag = R.rotary(R.f64(k), R.f64(cos), R.f64(sin), pos.cpu().numpy(), "half")
    for t, (p, r) in enumerate([(0, 2), (0, 3), (3, 4)]):
        assert (np.abs(R.f64(kp[p, :, r]) - ref[t]) <= R.rotary_bound(ref[t], mag[t], "f32")).all()
        assert torch.equal(vp[p, :, r], v[t])


def test_places_out_of_range_set_the_status_and_write_nothing(mnb):
    cos, sin = _tables(10, 32)
    x = _rand((3, 2, 32), "f32", 1).cuda()
    y = torch.zeros_like(x)
    mnb.mnb_rotary(x, y, torch.tensor([3, 10, -1], dtype=torch.int32).cuda(), cos, sin, 0)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    assert (y[1:] == 0).all() and (y[0] != 0).any()
    kp, vp = torch.zeros((2, 1, 8, 32), device="cuda"), torch.zeros((2, 1, 8, 32), device="cuda")
    start = torch.tensor([0, 1, 2, 3], dtype=torch.int32).cuda()
    k, v = x[:, :1], x[:, 1:]
    # a page number past the pool, an empty sequence that is given a token, a place past its table
    tables = torch.tensor([[2], [0], [1]], dtype=torch.int32).cuda()
    lens = torch.tensor([1, 0, 9], dtype=torch.int32).cuda()
    mnb.mnb_rotary_append(None, None, k, v, cos, sin, mnb.kv_cache(kp, vp, tables, lens, "hnd", 0), start)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    assert (kp == 0).all() and (vp == 0).all()


@pytest.mark.parametrize("kind", ["none", "linear", "ntk", "by_parts"])
def test_rotary_table(mnb, kind):
    n_pos, rot, base, s, L = 20000, 96, 10000.0, 4.0, 4096.0
    cos, sin = torch.empty((n_pos, rot // 2), device="cuda"), torch.empty((n_pos, rot // 2), device="cuda")
    code = {"none": mnb.MNB_ROPE_NONE, "linear": mnb.MNB_ROPE_LINEAR, "ntk": mnb.MNB_ROPE_NTK, "by_parts": mnb.MNB_ROPE_BY_PARTS}[kind]
    attn = 0.1 * math.log(s) + 1
    mnb.mnb_rotary_table(cos, sin, base, code, factor=s, trained_len=L, low=1.0, high=32.0, attn_factor=attn)
    b = base * s ** (rot / (rot - 2)) if kind == "ntk" else base
    f = b ** (-np.arange(0, rot, 2) / rot)
    if kind == "linear":
        f = f / s
    if kind == "by_parts":
        g = np.clip((L * f / (2 * math.pi) - 1) / 31, 0, 1)
        f = g * f + (1 - g) * f / s
    t = np.arange(n_pos)[:, None] * f
    # f64 frequencies within 2^-48, times positions below 2^15, then one rounding to f32
    tol = 2.0 ** -33 + 2.0 ** -24 * attn
    assert np.abs(R.f64(cos) - attn * np.cos(t)).max() <= tol
    assert np.abs(R.f64(sin) - attn * np.sin(t)).max() <= tol


def test_zero_tokens(mnb):
    cos, sin = _tables(10, 32)
    x = torch.empty((0, 2, 32), device="cuda")
    mnb.mnb_rotary(x, x, torch.empty(0, dtype=torch.int32, device="cuda"), cos, sin, 0)


def test_no_tokens(mnb):
    """An empty batch is a call that does nothing, whatever its tensors' strides are (numpy's empty ones have zeros)."""
    cos, sin = _tables(50, 64)
    none = torch.from_numpy(np.zeros((0, 2, 64), dtype=np.float32)).cuda()
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    mnb.mnb_rotary(none, torch.empty_like(none), pos, cos, sin, 0)
    pages = torch.full((2, 2, 16, 64), 5.0, device="cuda")
    start, lens = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32).cuda()
    cache = mnb.kv_cache(pages, pages.clone(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), lens, "hnd", 0)
    mnb.mnb_rotary_append(none, none.clone(), none, none, cos, sin, cache, start)
    mnb.mnb_rotary_append(None, None, none, none, cos, sin, cache, start)
    torch.cuda.synchronize()
    assert (pages == 5).all()

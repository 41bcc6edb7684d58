"""mnb_rms_norm against its definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests import _step_ref as R

pytestmark = pytest.mark.gpu

# The sum of squares of a row: each term and each addition rounds, at most 32 in a thread, 5 + 5 in the trees and the
# mean, eps and root: below 64 * 2^-24 of a positive sum, half of that for the root; S, the two products and 1 + w add
# 4 * 2^-24 (the rounding of S is relative to S; the inputs are not near cancellation but for single values, which the
# rounding of x + r, relative to the sum, covers).
REL = 40 * 2.0 ** -24


def make(t, h, dtype, gen, pad=0, scale=1.0):
    return (torch.randn((t, h + pad), generator=gen, device="cuda") * scale).to(R.DT[dtype])[:, :h]


def check(y, ref, rel=REL):
    err = np.abs(R.f64(y) - ref)
    tol = np.abs(ref) * (rel + R.half_step(y) * (1 + rel)) + R.smallest(y)
    assert (err <= tol).all(), (err - tol).max()


def check_codes(codes, scales, ref, bs):
    t, h = ref.shape
    kb = -(-h // bs)
    padded = np.zeros((t, kb * bs))
    padded[:, :h] = ref
    blocks = padded.reshape(t, kb, bs)
    a = np.abs(blocks).max(2) / 127
    got_a, q = R.f64(scales), R.f64(codes).reshape(t, kb, bs)
    assert (np.abs(got_a - a) <= a * (REL + 2.0 ** -23) + 2.0 ** -149).all()
    # a code is within half a step of y / a, whose own error is that of y and of a, at most 127 steps of 2 REL + 2^-22
    assert (np.abs(q * got_a[..., None] - blocks) <= a[..., None] * (0.5 + 127 * (2 * REL + 2.0 ** -22))).all()
    assert (np.abs(q) <= 127).all() and (q.reshape(t, -1)[:, h:] == 0).all()


CASES = [  # rows, width, dtype, residual, weight type, unit offset, block, pad
    (1, 1, "f32", False, "f32", False, 16, 0), (1, 4096, "bf16", True, "bf16", False, 32, 0), (3, 7, "f16", True, "f32", True, 16, 0),
    (5, 100, "bf16", True, "f32", False, 64, 3), (2, 1000, "f32", True, "f32", True, 128, 1), (2, 1000, "f32", True, "f32", True, 256, 24),
    (700, 4096, "bf16", True, "bf16", True, 256, 0), (313, 5120, "f16", True, "f16", False, 512, 24), (900, 72, "f16", False, "bf16", False, 64, 0),
    (2, 32768, "bf16", True, "bf16", False, 32768, 0), (2, 32767, "f32", True, "f32", False, 4096, 0), (4, 20000, "f32", False, None, False, 16, 0),
    (311, 8192, "f32", True, "f32", False, 2048, 0), (305, 9001, "bf16", True, "bf16", True, 1024, 0),
]


@pytest.mark.parametrize("rows,width,dtype,residual,wt,unit,bs,pad", CASES)
def test_norm(mnb, rows, width, dtype, residual, wt, unit, bs, pad):
    gen = torch.Generator(device="cuda").manual_seed(rows * width)
    x = make(rows, width, dtype, gen, pad)
    r = make(rows, width, dtype, gen, 0, 3.0) if residual else None
    w = (1 + 0.3 * torch.randn(width, generator=gen, device="cuda")).to(R.DT[wt]) if wt else None
    s_out = torch.full_like(r, float("nan")) if residual else None
    y = torch.full((rows, width), float("nan"), dtype=R.DT[dtype], device="cuda")
    kb = -(-width // bs)
    codes = torch.full((rows, kb * bs), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((rows, kb), float("nan"), device="cuda")
    flags = mnb.MNB_NORM_UNIT_OFFSET if unit else 0
    mnb.mnb_rms_norm(x, w, 1e-5, residual=r, residual_out=s_out, y=y, codes=codes, scales=scales, block_size=bs, flags=flags)
    s_ref, ref = R.rms_norm(R.f64(x), None if r is None else R.f64(r), None if w is None else R.f64(w), float(np.float32(1e-5)), unit)
    if residual:
        check(s_out, s_ref, 2.0 ** -24)
    check(y, ref)
    check_codes(codes, scales, ref, bs)
    # each output alone, and the sum alone, are the same bits
    y2, s2 = torch.empty_like(y), None if s_out is None else torch.empty_like(s_out)
    mnb.mnb_rms_norm(x, w, 1e-5, residual=r, y=y2, flags=flags)
    assert torch.equal(y2, y)
    c2, a2 = torch.empty_like(codes), torch.empty_like(scales)
    mnb.mnb_rms_norm(x, w, 1e-5, residual=r, residual_out=s2, codes=c2, scales=a2, block_size=bs, flags=flags)
    assert torch.equal(c2, codes) and torch.equal(a2, scales) and (s2 is None or torch.equal(s2, s_out))
    assert mnb.mnb_get_device_error() == 0


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_output_of_another_type(mnb, out):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = make(9, 520, "f16", gen, 8)
    y = torch.empty((9, 520), dtype=R.DT[out], device="cuda")
    mnb.mnb_rms_norm(x, None, 0.0, y=y)
    check(y, R.rms_norm(R.f64(x), None, None, 0.0, False)[1])


def test_in_place_and_wider_rows(mnb):
    """The sum takes the residual's place, the norm takes x's; both are slices of wider buffers that stay as they are."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    xb, rb = (torch.randn((37, 640), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    x0, r0 = xb.clone(), rb.clone()
    x, r = xb[:, 64:576], rb[:, 8:520]
    mnb.mnb_rms_norm(x, None, 1e-6, residual=r, residual_out=r, y=x)
    s_ref, ref = R.rms_norm(R.f64(x0[:, 64:576]), R.f64(r0[:, 8:520]), None, float(np.float32(1e-6)), False)
    check(r, s_ref, 2.0 ** -24)
    check(x, ref)
    for now, was, lo, hi in ((xb, x0, 64, 576), (rb, r0, 8, 520)):
        assert torch.equal(now[:, :lo], was[:, :lo]) and torch.equal(now[:, hi:], was[:, hi:])


def test_codes_are_those_of_the_quantiser(mnb):
    """From the same f32 values mnb_quantize_activations gives the same codes and scales."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = make(6, 500, "bf16", gen)
    y = torch.empty((6, 500), dtype=torch.float32, device="cuda")
    codes, scales = torch.empty((6, 512), dtype=torch.int8, device="cuda"), torch.empty((6, 16), device="cuda")
    mnb.mnb_rms_norm(x, None, 1e-6, y=y, codes=codes, scales=scales, block_size=32)
    qa, sa = torch.empty_like(codes), torch.empty_like(scales)
    mnb.mnb_quantize_activations(y, qa, sa, 6, 500, 32, mnb.MNB_F32)
    assert torch.equal(qa, codes) and torch.equal(sa, scales)


@pytest.mark.parametrize("bs", [32, 1024])
def test_infinities_and_nan_show(mnb, bs):
    x = torch.ones((4, 2048), dtype=torch.bfloat16, device="cuda")
    x[1, 5], x[2, 7], x[3] = float("nan"), float("inf"), 0.0
    kb = 2048 // bs
    y, codes = torch.empty_like(x), torch.empty((4, 2048), dtype=torch.int8, device="cuda")
    scales = torch.empty((4, kb), device="cuda")
    mnb.mnb_rms_norm(x, None, 1e-6, y=y, codes=codes, scales=scales, block_size=bs)
    assert torch.isfinite(y[0]).all() and (codes[0] == 127).all()
    assert torch.isnan(y[1]).all() and torch.isnan(scales[1]).all() and (codes[1] == 0).all()
    # 1 / inf = 0 beside the infinity, inf / inf = NaN at it
    assert torch.isnan(y[2, 7]) and (y[2, :7] == 0).all() and torch.isnan(scales[2, 0]) and (scales[2, 1:] == 0).all()
    assert (codes[2] == 0).all()
    assert (y[3] == 0).all() and (codes[3] == 0).all() and (scales[3] == 0).all()  # an empty row


def test_streams_and_graphs(mnb):
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, r = make(20, 4096, "bf16", gen), make(20, 4096, "bf16", gen)
    y, s = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mnb.mnb_rms_norm(x, None, 1e-6, residual=r, residual_out=s, y=y)
    side.synchronize()
    want_y, want_s = y.clone(), s.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mnb.mnb_rms_norm(x, None, 1e-6, residual=r, residual_out=s, y=y)
        mnb.mnb_rms_norm(x, None, 1e-6, residual=s, residual_out=s, y=y)
    x.neg_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    s1 = (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(s, (x.float() + s1.float()).to(torch.bfloat16))
    x.neg_()
    mnb.mnb_rms_norm(x, None, 1e-6, residual=r, residual_out=s, y=y)
    assert torch.equal(y, want_y) and torch.equal(s, want_s)


def test_nothing_to_do_and_refusals(mnb):
    x = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    mnb.mnb_rms_norm(x[:0], None, 1e-6, y=torch.empty_like(x[:0]))
    with pytest.raises(ValueError):
        mnb.mnb_rms_norm(x, None, 1e-6, y=torch.empty((2, 63), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        mnb.mnb_rms_norm(x, None, 1e-6, y=x.cpu())
    with pytest.raises(mnb.MnbError):
        mnb.mnb_rms_norm(x, None, 1e-6)
    with pytest.raises(mnb.MnbError) as e:
        wide = torch.ones((1, 32769), dtype=torch.bfloat16, device="cuda")
        mnb.mnb_rms_norm(wide, None, 1e-6, y=torch.empty_like(wide))
    assert e.value.status == mnb.MNB_ERR_UNSUPPORTED

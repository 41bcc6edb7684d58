"""mnb_moe_route and mnb_moe against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

from tests import _step_ref as R

pytestmark = pytest.mark.gpu


def scratch(mnb, t, s, e, k, i):
    from tests import _gpu as G
    return G.aligned_empty(mnb.mnb_moe_workspace_size(t, s, e, k, i))


def check_route(ids, weights, logits, s, bias, sigmoid, renorm, scale):
    want, w = R.route(R.f64(logits), s, None if bias is None else R.f64(bias), sigmoid, renorm, scale)
    assert (R.f64(ids) == want).all()
    # exp to 2 ulp of an argument good to 2^-24 of up to 32, sums of up to 1024 terms, a division: 2^-17
    got = R.f64(weights)
    assert (np.isnan(got) == np.isnan(w)).all()
    assert (np.abs(got - w) <= np.abs(w) * 2.0 ** -17 + 1e-30)[~np.isnan(w)].all()
    return want, w


ROUTES = [(1, 1, 1, "f32", False, True), (1, 64, 8, "bf16", False, True), (5, 60, 4, "f16", True, True), (300, 128, 8, "f32", False, False),
          (9, 257, 6, "f32", True, False), (3, 1000, 32, "bf16", True, True), (2, 7, 7, "f32", False, False)]


@pytest.mark.parametrize("t,e,s,dtype,sigmoid,renorm", ROUTES)
def test_route(mnb, t, e, s, dtype, sigmoid, renorm):
    gen = torch.Generator(device="cuda").manual_seed(t * e)
    logits = (torch.randn((t, e + 3), generator=gen, device="cuda") * 2).to(R.DT[dtype])[:, :e]
    bias = torch.randn(e, generator=gen, device="cuda") * 0.1 if sigmoid and e % 2 == 0 else None
    ids = torch.full((t, s), -5, dtype=torch.int32, device="cuda")
    w = torch.full((t, s), float("nan"), device="cuda")
    mnb.mnb_moe_route(logits, ids, w, bias=bias, scoring=mnb.MNB_MOE_SIGMOID if sigmoid else mnb.MNB_MOE_SOFTMAX, renormalize=renorm, scale=2.5)
    check_route(ids, w, logits, s, bias, sigmoid, renorm, 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_ties_masks_and_nan(mnb, sigmoid):
    inf, nan = float("inf"), float("nan")
    rows = [[0.0] * 6, [1.0, 2.0, 2.0, -0.0, 0.0, 1.0], [-inf] * 6, [-inf, -inf, 3.0, -inf, -inf, -inf], [-3.0e38] * 6, [nan, -inf, 1.0, nan, nan, nan],
            [-65504.0, 1.0, -65504.0, -65504.0, 1.0, 1.0]]
    logits = torch.tensor(rows, device="cuda")
    ids, w = torch.empty((7, 3), dtype=torch.int32, device="cuda"), torch.empty((7, 3), device="cuda")
    mnb.mnb_moe_route(logits, ids, w, scoring=mnb.MNB_MOE_SIGMOID if sigmoid else mnb.MNB_MOE_SOFTMAX)
    check_route(ids, w, logits, 3, None, sigmoid, True, 1.0)
    assert ids[0].tolist() == [0, 1, 2] and ids[1].tolist() == [1, 2, 0] and (w[2] == 0).all()


# tokens, top_k, experts, hidden, inner, bits, bs, act, scale type, zp, sigmoid, gelu, out, pad of x and y
CASES = [
    (1, 2, 4, 256, 128, 4, 32, "bf16", "f16", True, False, False, "bf16", 0),
    (1, 8, 64, 512, 256, 4, 32, "bf16", "f16", False, False, False, "bf16", 0),
    (1, 1, 1, 1, 1, 4, 16, "bf16", "f32", False, False, False, "f32", 0),
    (2, 3, 5, 100, 37, 8, 16, "f16", "f32", True, True, False, "f32", 5),
    (3, 2, 6, 1000, 616, 8, 16, "bf16", "f32", True, True, False, "bf16", 0),
    (4, 2, 8, 384, 640, 2, 32, "f16", "bf16", True, False, True, "f16", 8),
    (5, 4, 16, 136, 72, 2, 16, "bf16", "f16", True, False, False, "f32", 0),
    (7, 2, 3, 1001, 300, 4, 64, "bf16", "bf16", False, False, False, "f32", 0),
    (8, 8, 9, 512, 384, 4, 128, "f16", "f16", True, True, False, "f16", 24),
    (9, 2, 4, 256, 256, 4, 256, "bf16", "f16", False, False, False, "f32", 0),
    (16, 4, 24, 640, 160, 4, 32, "bf16", "f16", True, False, False, "bf16", 0),
    (16, 2, 2, 128, 1024, 8, 64, "bf16", "bf16", True, False, False, "f32", 0),
    (33, 1, 4, 264, 80, 4, 32, "f16", "f32", True, False, True, "f32", 8),
    (64, 16, 20, 144, 48, 4, 16, "bf16", "f16", False, True, False, "f32", 0),
    (1, 2, 4, 4096, 96, 8, 128, "bf16", "f16", True, False, False, "f32", 0),
    (2, 2, 4, 96, 4096, 2, 1024, "bf16", "f16", True, False, False, "f32", 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_layer(mnb, case):
    t, s, e, k, i, bits, bs, act, sdt, zp, sigmoid, gelu, out, pad = case
    gen = torch.Generator(device="cuda").manual_seed(t * k + i)
    gate, up = (R.Experts(mnb, e, i, k, bits, bs, sdt, zp, gen, 256 if pad == 0 else 1) for _ in range(2))
    down = R.Experts(mnb, e, k, i, bits, bs, sdt, zp, gen, 256 if pad == 0 else 1)
    x = torch.randn((t, k + pad), generator=gen, device="cuda").to(R.DT[act])[:, :k]
    yb = torch.full((t, k + pad), 7.0, dtype=R.DT[out], device="cuda")
    y = yb[:, :k]
    logits = torch.randn((t, e), generator=gen, device="cuda")
    bias = torch.randn(e, generator=gen, device="cuda") * 0.1 if sigmoid else None
    ids, w = torch.empty((t, s), dtype=torch.int32, device="cuda"), torch.empty((t, s), device="cuda")
    kw = dict(bias=bias, scoring=mnb.MNB_MOE_SIGMOID if sigmoid else mnb.MNB_MOE_SOFTMAX, scale=1.5,
              activation=mnb.MNB_ACT_GELU_TANH if gelu else mnb.MNB_ACT_SILU, workspace=scratch(mnb, t, s, e, k, i))
    mnb.mnb_moe(x, logits, gate.handle, up.handle, down.handle, y, s, ids=ids, weights=w, **kw)
    want, wts = check_route(ids, w, logits, s, bias, sigmoid, True, 1.5)
    ref, tol = R.moe(R.f64(x), want, wts, gate.w, up.w, down.w, gelu)
    tol = tol + np.abs(ref) * 2.0 ** -16  # the weights' own error, see check_route
    err = np.abs(R.f64(y) - ref)
    tol = tol + (np.abs(ref) + tol) * R.half_step(y) + R.smallest(y)
    assert (err <= tol).all(), (err / tol).max()
    assert (yb[:, k:] == 7.0).all()
    y2 = torch.empty((t, k), dtype=R.DT[out], device="cuda")
    mnb.mnb_moe(x, logits, gate.handle, up.handle, down.handle, y2, s, **kw)
    assert torch.equal(y2, y)  # results repeat, with and without the selection's outputs
    assert mnb.mnb_get_device_error() == 0


@pytest.fixture(scope="module")
def small(mnb):
    gen = torch.Generator(device="cuda").manual_seed(77)
    return tuple(R.Experts(mnb, 6, n, k, 4, 32, "f16", True, gen) for n, k in ((192, 256), (192, 256), (256, 192)))


def layer(mnb, small, x, logits, y, ws, **kw):
    mnb.mnb_moe(x, logits, small[0].handle, small[1].handle, small[2].handle, y, 2, workspace=ws, **kw)


@pytest.mark.parametrize("t", [1, 6, 12])
def test_every_token_on_one_expert_and_masked_tokens(mnb, small, t):
    """All tokens pick experts 3 and 5; the last has no expert at all: y = 0."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randn((t, 256), generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.full((t, 6), float("-inf"), device="cuda")
    logits[:, 3], logits[:, 5] = 1.0, 0.5
    logits[t - 1] = float("-inf")
    y = torch.empty((t, 256), device="cuda")
    layer(mnb, small, x, logits, y, scratch(mnb, t, 2, 6, 256, 192))
    ids, w = R.route(R.f64(logits), 2, None, False, True, 1.0)
    ref, tol = R.moe(R.f64(x), ids, w, small[0].w, small[1].w, small[2].w, False)
    assert (np.abs(R.f64(y) - ref) <= tol + np.abs(ref) * 2.0 ** -16 + 1e-37).all()
    assert (y[t - 1] == 0).all()


@pytest.mark.parametrize("t", [1, 4, 16])
def test_chained_calls_share_a_workspace_and_replay(mnb, small, t):
    """Layers in a row on one workspace, the output of one the input of the next, eagerly, captured and replayed with
    other logits; a second stream with a workspace of its own at the same time."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randn((t, 256), generator=gen, device="cuda").to(torch.bfloat16)
    logits = [torch.randn((t, 6), generator=gen, device="cuda") for _ in range(4)]
    ws, ws2 = scratch(mnb, t, 2, 6, 256, 192), scratch(mnb, t, 2, 6, 256, 192)
    y = [torch.empty_like(x) for _ in range(4)]

    def chain(ys, w):
        h = x
        for lg, to in zip(logits, ys):
            layer(mnb, small, h, lg, to, w)
            h = to

    def one_by_one():
        h, out = x, []
        for lg in logits:
            to = torch.empty_like(x)
            layer(mnb, small, h, lg, to, scratch(mnb, t, 2, 6, 256, 192))
            torch.cuda.synchronize()
            out.append(to)
            h = to
        return out

    want = one_by_one()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = [torch.empty_like(x) for _ in range(4)]
    for _ in range(5):
        chain(y, ws)
        with torch.cuda.stream(side):
            chain(y2, ws2)
    torch.cuda.synchronize()
    for a, b, c in zip(want, y, y2):
        assert torch.equal(a, b) and torch.equal(a, c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(y, ws)
    for lg in logits:
        lg.copy_(torch.randn((t, 6), generator=gen, device="cuda"))
    x.neg_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(one_by_one(), y):
        assert torch.equal(a, b)
    assert mnb.mnb_get_device_error() == 0


def test_matches_the_grouped_product(mnb, small):
    """The routing with mnb_matmul_grouped and torch between gives the layer, to the roundings of its bf16 steps."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = 4
    x = torch.randn((t, 256), generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn((t, 6), generator=gen, device="cuda")
    ids, w = torch.empty((t, 2), dtype=torch.int32, device="cuda"), torch.empty((t, 2), device="cuda")
    y = torch.empty((t, 256), device="cuda")
    layer(mnb, small, x, logits, y, scratch(mnb, t, 2, 6, 256, 192), ids=ids, weights=w)

    def grouped(x, m, n, k, per_slot):
        out = torch.empty((t, 2, n), device="cuda")
        d = m.handle
        mnb.mnb_matmul_grouped(x, ids, d.tensors[0], d.tensors[1], d.tensors[2], out, t, 2, 6, n, k, 4, 32, mnb.MNB_BF16, mnb.MNB_F32,
                               mnb.MNB_F16, x_per_slot=per_slot)
        return out

    g, u = grouped(x, small[0], 192, 256, False), grouped(x, small[1], 192, 256, False)
    h = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
    ref = (w[..., None] * grouped(h.view(t * 2, 192), small[2], 256, 192, True)).sum(1)
    # h rounded to bf16 here, 192 products of it: 2^-9 of a value's deviation on average, four deviations on the worst
    assert (y - ref).abs().max() <= 4 * 2.0 ** -9 * float(ref.std()) * 2


def test_nan_and_infinities_stay_with_their_token(mnb, small):
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((4, 256), generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.zeros((4, 6), device="cuda")  # all on experts 0 and 1
    ws = scratch(mnb, 4, 2, 6, 256, 192)
    clean, y = torch.empty((4, 256), device="cuda"), torch.empty((4, 256), device="cuda")
    layer(mnb, small, x, logits, clean, ws)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    layer(mnb, small, x, logits, y, ws)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[3], clean[3])
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()


def test_large_intermediate_values_fit(mnb, small):
    """f16 activations whose gate and up pass the largest f16 value: the layer's own parts do not overflow."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = (torch.randn((2, 256), generator=gen, device="cuda") * 3000).to(torch.float16)
    logits = torch.randn((2, 6), generator=gen, device="cuda")
    y = torch.empty((2, 256), device="cuda")
    layer(mnb, small, x, logits, y, scratch(mnb, 2, 2, 6, 256, 192))
    ids, w = R.route(R.f64(logits), 2, None, False, True, 1.0)
    ref, tol = R.moe(R.f64(x), ids, w, small[0].w, small[1].w, small[2].w, False)
    assert np.abs(ref).max() > 65504
    assert (np.abs(R.f64(y) - ref) <= tol + np.abs(ref) * 2.0 ** -16).all()


@pytest.mark.parametrize("size", [2.0 ** -28, 2.0 ** 30])
@pytest.mark.parametrize("t", [2, 20])
def test_range_of_bf16(mnb, small, size, t):
    """Values near both ends of the documented range: h is of the order of size^2."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = (torch.randn((t, 256), generator=gen, device="cuda") * size).to(torch.bfloat16)
    logits = torch.randn((t, 6), generator=gen, device="cuda")
    y = torch.empty((t, 256), device="cuda")
    layer(mnb, small, x, logits, y, scratch(mnb, t, 2, 6, 256, 192))
    ids, w = R.route(R.f64(logits), 2, None, False, True, 1.0)
    ref, tol = R.moe(R.f64(x), ids, w, small[0].w, small[1].w, small[2].w, False)
    # (and 2^-17 of each expert's share, the weights' own bound, which test_layer counts from the kernel's weights)
    share = sum(R.moe(R.f64(x), ids[:, s:s + 1], w[:, s:s + 1], small[0].w, small[1].w, small[2].w, False)[0].__abs__() for s in range(2))
    assert (np.abs(R.f64(y) - ref) <= tol + share * 2.0 ** -16).all()


def test_weights_of_another_device_are_refused(mnb, small, monkeypatch):
    x, logits = torch.ones((1, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 6), device="cuda")
    monkeypatch.setattr(small[1].handle, "dev", 1)  # as expert_weights() on that device would note it
    with pytest.raises(ValueError):
        layer(mnb, small, x, logits, torch.empty((1, 256), device="cuda"), scratch(mnb, 1, 2, 6, 256, 192))


def test_wrong_headers_are_reported(mnb, small):
    x, logits = torch.ones((1, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 6), device="cuda")
    y, ws = torch.empty((1, 256), device="cuda"), scratch(mnb, 1, 2, 6, 256, 192)
    packed = small[2].handle.tensors[0]
    keep = packed[:16].clone()
    packed[8:12] = 255
    layer(mnb, small, x, logits, y, ws)
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_LAYOUT_MISMATCH
    packed[:16] = keep
    layer(mnb, small, x, logits, y, ws)
    assert mnb.mnb_get_device_error() == 0


def test_refusals(mnb, small):
    x, logits = torch.ones((1, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 6), device="cuda")
    y, ws = torch.empty((1, 256), device="cuda"), scratch(mnb, 1, 2, 6, 256, 192)
    with pytest.raises(mnb.MnbError) as e:
        layer(mnb, small, x, logits, y, ws[:256])
    assert e.value.status == mnb.MNB_ERR_NO_MEM
    with pytest.raises(mnb.MnbError) as e:
        layer(mnb, small, x.float(), logits, y, ws)
    assert e.value.status == mnb.MNB_ERR_UNSUPPORTED
    with pytest.raises(mnb.MnbError) as e:
        layer(mnb, small, x, logits[:, :5], y, ws)
    assert e.value.status == mnb.MNB_ERR_INVALID_ARG
    for bad in (dict(x=x[:, :255]), dict(logits=logits.cpu()), dict(y=y[:, :100]), dict(x=x.expand(2, 256))):
        with pytest.raises(ValueError):
            layer(mnb, small, **{**dict(x=x, logits=logits, y=y, ws=ws), **bad})
    layer(mnb, small, x[:0], logits[:0], y[:0], ws)

"""mnb_sample against its definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests import _step_ref as R

pytestmark = pytest.mark.gpu

# Weights are good to 2^-34.5 (and half a unit of 2^-43, which averages out over a row); a sum up to a place and the share
# of the whole that it is held against both move by that: a place whose 64-bit sum is closer than 2^-33 to a border is the
# reference's to choose as much as the kernel's.
NEAR = 2.0 ** -33


def run(mnb, logits, t=None, k=None, p=None, m=None, u=None, seed=0):
    b = logits.shape[0]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda v: None if v is None else torch.tensor(np.broadcast_to(v, b).copy(), dtype=torch.float32, device="cuda")  # noqa: E731
    ut = torch.rand(b, generator=gen, device="cuda") if u is None else f(u)
    kt = None if k is None else torch.tensor(np.broadcast_to(k, b).copy(), dtype=torch.int32, device="cuda")
    tt, pt, mt = f(t), f(p), f(m)
    tokens = torch.full((b,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((b,), float("nan"), device="cuda")
    mnb.mnb_sample(logits, ut, tokens, temperature=tt, top_k=kt, top_p=pt, min_p=mt, probs=probs)
    again = torch.empty_like(tokens)
    mnb.mnb_sample(logits, ut, again, temperature=tt, top_k=kt, top_p=pt, min_p=mt)
    assert torch.equal(tokens, again)
    x, uu = R.f64(logits), R.f64(ut)
    at = lambda v, i, d: d if v is None else float(R.f64(v)[i])  # noqa: E731
    for i in range(b):
        token, prob, near = R.sample(x[i], at(tt, i, 1.0), int(at(kt, i, 0)), at(pt, i, 1.0), at(mt, i, 0.0), uu[i])
        if near < NEAR:
            continue
        # the probability: a weight and a sum good to 2^-34 of what they are, rounded to f32; a unit of 2^-43 for tiny ones
        got = float(probs[i])
        assert int(tokens[i]) == token, (i, int(tokens[i]), token, near)
        assert abs(got - prob) <= prob * (2.0 ** -24 + 2.0 ** -33) + 2.0 ** -42, (i, got, prob)
    return tokens, probs


def logits_of(b, v, dtype, seed, scale=2.0, pad=0, mean=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((b, v + pad), generator=gen, device="cuda") * scale + mean
    x[:, : v // 50 + 1] += 4.0
    return x.to(R.DT[dtype])[:, pad // 2: pad // 2 + v]


SHAPES = [(1, 1, "f32", 0), (3, 2, "bf16", 1), (5, 33, "f16", 3), (4, 1000, "f32", 5), (7, 4097, "bf16", 0), (2, 50257, "f16", 0),
          (3, 128000, "bf16", 0), (2, 200003, "f32", 0), (40, 20001, "f16", 7), (320, 3000, "f32", 2), (1, 700001, "f32", 3)]


@pytest.mark.parametrize("b,v,dtype,pad", SHAPES)
@pytest.mark.parametrize("cut", ["none", "k", "big_k", "p", "m", "all", "hot", "cold"])
def test_rows(mnb, b, v, dtype, pad, cut):
    if b * v > 300_000 and cut in ("cold", "m", "hot") and v > 300_000:
        pytest.skip("covered by the smaller rows")
    x = logits_of(b, v, dtype, b * v, pad=pad)
    kw = {"none": {}, "k": dict(k=max(1, min(40, v // 2))), "big_k": dict(k=max(1, v * 2 // 3), p=0.97), "p": dict(t=0.8, p=0.9), "m": dict(m=0.05),
          "all": dict(t=0.7, k=50, p=0.9, m=0.02), "hot": dict(t=50.0, p=0.8), "cold": dict(t=0.01, m=0.001)}[cut]
    run(mnb, x, **kw, seed=v)
    assert mnb.mnb_get_device_error() == 0


def test_each_row_its_own(mnb):
    """Parameters of all kinds side by side, off values among them."""
    x = logits_of(12, 32000, "bf16", 1)
    run(mnb, x, t=[0, 1, 0.5, 2, 1e-30, 1e30, float("inf"), 1, 1, 1, 0, 1], k=[5, 0, -3, 32000, 7, 99999, 3, 1, 2, 20000, 0, 1500],
        p=[0.5, 1, 2, 0.3, 0.9, 0.5, 0.5, 0.9, 0.0, 0.99, 1, -1], m=[0, 1, 2, 0.1, 0, 0, 0, 0, 0, 1e-9, 0.5, 0])


@pytest.mark.parametrize("v", [900, 5000, 70000, 400000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits(mnb, v, dtype):
    """All equal (the j-th of equal tokens), two values, and a few values with thousands of tokens each."""
    x = torch.zeros((6, v), device="cuda")
    x[1] = -1.5
    x[2, ::3] = 1.0
    x[3] = (torch.arange(v, device="cuda") % 5).float() * 0.125
    x[4] = -3.0e38
    x[5] = torch.where(torch.arange(v, device="cuda") % 2 == 0, 0.0, -0.0)
    x = x.to(R.DT[dtype])
    run(mnb, x, u=[0.0, 0.999999, 0.4, 0.77, 0.5, 0.31])
    run(mnb, x, k=[v // 2, 3, v // 3 + 5, v - 1, 1, v // 2 + 1], p=[0.9, 1, 0.99, 0.6, 0.7, 0.3], u=0.9)


@pytest.mark.parametrize("v", [3000, 100000])
def test_masks_infinities_and_nan(mnb, v):
    inf, nan = float("inf"), float("nan")
    x = logits_of(8, v, "f32", 9)
    x[0] = -inf
    x[1] = nan
    x[2] = -inf
    x[2, v - 2] = 0.5
    x[3, ::2] = nan
    x[4, 5] = x[4, v - 7] = inf
    x[5, 3:] = torch.finfo(torch.float32).min
    x[6] = torch.finfo(torch.float32).min
    x[6, 11] = -inf
    x[7, 1::2] = -inf
    for kw in (dict(), dict(k=20, p=0.9, m=0.01), dict(p=0.95), dict(t=0.0), dict(t=100.0, k=v // 2)):
        tokens, probs = run(mnb, x, **kw, seed=v)
        assert tokens[:2].tolist() == [-1, -1] and probs[:2].tolist() == [0.0, 0.0]
        assert int(tokens[2]) == v - 2 and int(tokens[4]) in (5, v - 7) and 0 <= int(tokens[5]) < 3 and int(tokens[6]) != 11
    assert mnb.mnb_get_device_error() == 0


def test_close_and_far_values(mnb):
    """Tokens whose logits differ in the last bits (bins of one value at first sight), at all magnitudes."""
    v = 60000
    i = torch.arange(v, device="cuda", dtype=torch.float32)
    x = torch.stack([1000.0 + i * 2.0 ** -14, 1.0 + (i % 4096) * 2.0 ** -23, -(i + 1) * 1e-30, torch.where(i < 3, 80.0, i * 1e-4)])
    run(mnb, x)
    run(mnb, x, k=[30000, 20, 50000, 4], p=0.9)
    run(mnb, x * 1e-3, t=[1e-3, 5e-4, 1.0, 1e-3])


def test_distribution(mnb):
    """Evenly spaced numbers draw each token as often as its probability says, to one draw at each border."""
    n = 20000
    x = torch.tensor([1.0, 3.0, 2.0, -1.0, 3.0, 0.0], device="cuda")
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tokens = torch.empty(n, dtype=torch.int32, device="cuda")
    mnb.mnb_sample(x.expand(n, 6).contiguous(), u, tokens)
    count = torch.bincount(tokens.long(), minlength=6).double()
    assert ((count / n - torch.softmax(x.double(), 0)).abs() <= 2 / n).all()


def test_wrong_parameters_are_reported(mnb):
    x = logits_of(6, 500, "f32", 3)
    nan = float("nan")
    b, f = 6, lambda *v: torch.tensor(v, device="cuda")  # noqa: E731
    tokens, probs = torch.empty(b, dtype=torch.int32, device="cuda"), torch.empty(b, device="cuda")
    mnb.mnb_sample(x, f(0.5, 0.5, 0.5, 0.5, 1.0, -0.1), tokens, temperature=f(-1.0, nan, 1.0, 1.0, 1.0, 1.0), top_p=f(0.9, 0.9, nan, 0.9, 0.9, 0.9),
                   min_p=f(0.0, 0.0, 0.0, nan, 0.0, 0.0), probs=probs)
    assert tokens.tolist() == [-1] * 6 and probs.tolist() == [0.0] * 6
    assert mnb.mnb_get_device_error() == mnb.MNB_ERR_INVALID_ARG
    mnb.mnb_sample(x, f(0.5, 0.5, 0.5, 0.5, 0.0, 0.1), tokens)
    assert (tokens >= 0).all() and mnb.mnb_get_device_error() == 0


@pytest.mark.parametrize("v", [600, 30000])
def test_edges_of_the_parameters(mnb, v):
    """-0 is 0; the largest u below 1; a share of 0 keeps one token; the smallest and largest temperatures."""
    x = logits_of(6, v, "f32", 7)
    zero, one = [-0.0] * 6, [1 - 2.0 ** -24] * 6
    first = torch.argmax(x, 1).int()
    for p in ([-0.0] * 6, None, [2.0 ** -149] * 6, [1.0 - 2.0 ** -24] * 6):
        tokens, _ = run(mnb, x, u=zero, p=p, m=zero)
        assert torch.equal(tokens, first)
        run(mnb, x, u=one, p=p)
    tokens, _ = run(mnb, x, u=one, p=[-1.0] * 6, m=[-1.0] * 6, k=-5)
    assert torch.equal(tokens, first)
    run(mnb, x, t=[2.0 ** -149, 1e-30, 1e-3, 1e30, 3e38, float("inf")])


def test_streams_and_graphs(mnb):
    x = logits_of(9, 30001, "bf16", 5)
    u, t = torch.rand(9, device="cuda"), torch.empty(9, dtype=torch.int32, device="cuda")
    k, p = torch.full((9,), 2000, dtype=torch.int32, device="cuda"), torch.full((9,), 0.9, device="cuda")
    g = torch.cuda.CUDAGraph()
    mnb.mnb_sample(x, u, t, top_k=k, top_p=p)
    with torch.cuda.graph(g):
        mnb.mnb_sample(x, u, t, top_k=k, top_p=p)
    x.copy_(logits_of(9, 30001, "bf16", 6))
    p.fill_(0.5)
    g.replay()
    side, t2 = torch.cuda.Stream(), torch.empty_like(t)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mnb.mnb_sample(x, u, t2, top_k=k, top_p=p)
    torch.cuda.synchronize()
    assert torch.equal(t, t2)


def test_refusals(mnb):
    x, u = logits_of(2, 100, "f32", 1), torch.zeros(2, device="cuda")
    t = torch.empty(2, dtype=torch.int32, device="cuda")
    mnb.mnb_sample(x[:0], u[:0], t[:0])
    for bad in (dict(u=u[:1]), dict(tokens=t.long()), dict(logits=x.double()), dict(logits=x.T), dict(temperature=t), dict(top_k=u),
                dict(probs=t), dict(top_p=u.cpu()), dict(u=None)):
        with pytest.raises(ValueError):
            mnb.mnb_sample(**{**dict(logits=x, u=u, tokens=t), **bad})

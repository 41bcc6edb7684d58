"""mnb_sample where many tokens are far below the largest: sums of up to 2^24 tiny weights against their values."""
import math

import numpy as np
import pytest
import torch

from tests import _step_ref as R

pytestmark = pytest.mark.gpu

# A weight is good to 2^-34 of itself; the sum up to a place is floored to a unit of at most 2^-37 of the largest weight, as
# is the share of the whole that it is held against, and weights below 2^-36 / V of the largest (and 2^-44) are left out,
# 2^-36 in all: 2^-34 + 2 * 2^-37 + 2^-36 = 1.5 * 2^-34 of what is kept, which holds the largest weight.
SUMS = 2.0 ** -33


def call(mnb, x, u, **kw):
    b = x.shape[0]
    f = lambda v: torch.full((b,), v, device="cuda")  # noqa: E731
    tokens, probs = torch.full((b,), -7, dtype=torch.int32, device="cuda"), torch.full((b,), float("nan"), device="cuda")
    k = torch.full((b,), kw.pop("top_k"), dtype=torch.int32, device="cuda") if "top_k" in kw else None
    mnb.mnb_sample(x, u, tokens, top_k=k, probs=probs, **{n: f(v) for n, v in kw.items()})
    assert mnb.mnb_get_device_error() == 0
    return tokens.tolist(), probs.tolist()


def near_one(share):
    """f32 numbers below 1 around `share`, and the largest."""
    at = np.float32(min(share, 1 - 2.0 ** -24))
    near, lo, hi = [at], at, at
    for _ in range(3):
        lo, hi = np.nextafter(lo, np.float32(0)), np.nextafter(hi, np.float32(2))
        near += [lo, hi]
    wide = [share + (1 - share) * f for f in (0.01, 0.3, 0.5, 0.9, 0.999)]
    return torch.tensor([float(v) for v in near + wide + [0.0, 1 - 2.0 ** -24] if 0 <= np.float32(v) < 1], dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("below", [24.3, 35.0, 36.5, 37.9, 40.4, 42.5, 43.4, 43.98, 44.1, 47.6, 50.5])
@pytest.mark.parametrize("v", [5001, 128000, 1 << 20, 1 << 24])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_and_many_equal(mnb, v, below, dtype):
    """One token and v - 1 equal ones 2^-below of it: the token drawn from the tail is the one that u names."""
    if v == 1 << 24 and dtype == "bf16" and below not in (36.5, 42.5):
        pytest.skip("as in f32")
    top = v // 3
    value = torch.tensor(-below * math.log(2.0)).to(R.DT[dtype])
    w = math.exp(float(value))
    total = 1 + (v - 1) * w
    u = near_one(1 / total)
    x = torch.full((len(u), v), float(value), dtype=R.DT[dtype], device="cuda")
    x[:, top] = 0.0
    tokens, probs = call(mnb, x, u)
    for i, token in enumerate(tokens):
        s = float(u[i]) * total
        # tokens before it in the order: the maximum comes first, the equal ones by their index
        place = 0 if token == top else token + 1 - (1 if token > top else 0)
        lo, hi = (0.0, 1.0) if token == top else (1 + (place - 1) * w, 1 + place * w)
        assert lo - SUMS * total <= s <= hi + SUMS * total, (i, float(u[i]), token, lo - s, s - hi)
        want = (1.0 if token == top else w) / total
        assert abs(probs[i] - want) <= want * (2.0 ** -24 + 2.0 ** -32)


@pytest.mark.parametrize("v", [128000, 1 << 20])
@pytest.mark.parametrize("share", [1e-3, 1e-9, 3e-12])
def test_many_beside_min_p(mnb, v, share):
    """v - 1 equal tokens just above or just below min_p: all kept or none."""
    share = float(np.float32(share))
    at = np.float32(math.log(share))
    while math.exp(float(at)) >= share:
        at = np.nextafter(at, np.float32(-100))
    under, over = at, np.nextafter(at, np.float32(0))
    while math.exp(float(over)) < share:
        over = np.nextafter(over, np.float32(0))
    for value, kept in ((under, False), (over, True)):
        # (a weight that is nearer to min_p than its own error says nothing)
        assert abs(math.exp(float(value)) / share - 1) > 2.0 ** -33
        w = math.exp(float(value))
        total = 1 + (v - 1) * w if kept else 1.0
        u = near_one(1 / (1 + (v - 1) * w))
        x = torch.full((len(u), v), float(value), device="cuda")
        x[:, 7] = 0.0
        for more in ({}, {"top_p": 1 - 2.0 ** -24}, {"top_k": v - 5}):
            tokens, probs = call(mnb, x, u, min_p=share, **more)
            if more:
                continue  # (their borders are among the equal tokens: that they run and stay in range)
            for i, token in enumerate(tokens):
                s = float(u[i]) * total
                place = 0 if token == 7 else token + 1 - (1 if token > 7 else 0)
                lo, hi = (0.0, 1.0) if token == 7 else (1 + (place - 1) * w, 1 + place * w)
                assert (kept or token == 7) and lo - SUMS * total <= s <= hi + SUMS * total, (value, i, token)


def exact(x, t, k, p, m, u):
    """(token, distance to the nearest border) of a float64 row, its sums in two whole numbers each."""
    order = np.lexsort((np.arange(len(x)), -x))
    w = np.exp(-(x.max() - x[order]) / t)
    w = w[:k] if 0 < k < len(w) else w
    hi = np.floor(w * 2.0 ** 50)  # (sums below 2^60: a row's whole is a few times its largest)
    lo = np.floor((w * 2.0 ** 50 - hi) * 2.0 ** 40)
    sums = np.cumsum(hi.astype(np.int64)).astype(np.longdouble) + np.cumsum(lo.astype(np.int64)).astype(np.longdouble) * 2.0 ** -40
    near, n = 1.0, len(sums)

    def border(target):
        at = int(np.searchsorted(sums, target))
        return min(abs(float(sums[i] - target)) for i in (at - 1, at, at + 1) if 0 <= i < len(sums)) / float(sums[-1])

    if p < 1:
        target = np.longdouble(p) * sums[-1]
        near = min(near, border(target))
        n = min(n, int(np.searchsorted(sums, target)) + 1)
    if m > 0:
        near = min(near, float(np.abs(w / m - 1).min()))
        n = min(n, int((w >= m).sum()))
    target = np.longdouble(u) * sums[n - 1]
    return int(order[min(int(np.searchsorted(sums, target, side="right")), n - 1)]), min(near, border(target)), n


@pytest.mark.parametrize("v,dtype", [(100000, "f32"), (300000, "f16"), (1 << 20, "f32"), (700000, "bf16")])
def test_wide_rows(mnb, v, dtype):
    """Rows whose bulk is 2^-20 to 2^-45 of the largest token and still holds a share."""
    gen = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn((5, v), generator=gen, device="cuda") * 2.0
    x[:, 11] = torch.tensor([18.0, 22.0, 26.0, 30.0, 14.0], device="cuda")
    x = x.to(R.DT[dtype])
    kept = x.double().cpu().numpy()
    for kw in ({}, dict(top_p=0.99999), dict(min_p=1e-12), dict(top_k=v // 2), dict(top_k=v // 3, top_p=0.9999999, min_p=1e-8)):
        u = torch.tensor([1 - 2.0 ** -20, 1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -24, 0.6], dtype=torch.float32, device="cuda")
        tokens, _ = call(mnb, x, u, **kw)
        f = lambda n, d: float(np.float32(kw.get(n, d)))  # noqa: E731
        for i in range(5):
            token, near, n = exact(kept[i], 1.0, kw.get("top_k", 0), f("top_p", 1.0), f("min_p", 0.0), float(u[i]))
            assert near < SUMS or tokens[i] == token, (kw, i, tokens[i], token, near, n)

"""Weights of experts whose sigmoids are at the low end of f32: the ratios of what was selected, as the definition has them."""
import numpy as np
import pytest
import torch

from tests import _step_ref as R
from tests.test_gpu_moe import scratch

pytestmark = pytest.mark.gpu

INF = float("inf")
ROWS = [[-90.0, -92.5, -91.0, -200.0, -95.0, -120.0], [-300.0, -301.0, -302.5, -299.5, -400.0, -5000.0], [-87.5, -88.5, -89.5, -104.0, -60.0, -61.0],
        [-1e30, -1e30, -2e30, -INF, -INF, -INF], [-INF] * 6, [-40.0, -59.0, -61.0, -85.0, -100.0, -45.0], [3.0, -100.0, -200.0, -300.0, -400.0, -88.0],
        [-102.0, -103.0, -104.5, -130.0, -131.0, -102.5]]


def weights(row, ids, scale):
    """The selected sigmoids over their sum, by their logarithms; 0 where 64 bits have no sigmoid above 0."""
    l = np.array(row)[ids]
    if (l < -745).all():
        return np.zeros(len(ids))
    log = -np.logaddexp(0.0, -l)
    w = np.exp(log - log.max())
    return w / w.sum() * scale


@pytest.mark.parametrize("bias", [False, True])
def test_route(mnb, bias):
    logits = torch.tensor(ROWS, device="cuda")
    b = torch.tensor([0.0, 0.1, 0.2, 0.3, 0.25, 0.05], device="cuda") if bias else None
    ids, w = torch.empty((8, 3), dtype=torch.int32, device="cuda"), torch.empty((8, 3), device="cuda")
    mnb.mnb_moe_route(logits, ids, w, bias=b, scoring=mnb.MNB_MOE_SIGMOID, scale=2.0)
    want_ids, _ = R.route(R.f64(logits), 3, R.f64(b) if bias else None, True, True, 2.0)
    for i, row in enumerate(ROWS):
        assert ids[i].tolist() == want_ids[i].tolist()
        want = weights(row, want_ids[i], 2.0)
        # exp to 2 ulp of a difference of logits that is exact or far below 0, a sum of three, a division, the scale; what is
        # below 2^-40 of the sum may be left out
        assert (np.abs(R.f64(w[i]) - want) <= want * 2.0 ** -20 + 2.0 ** -40).all(), (i, w[i].tolist(), want)


def test_as_they_are(mnb):
    """Not divided by their sum: the sigmoids themselves, subnormal ones too."""
    logits = torch.tensor(ROWS, device="cuda")
    ids, w = torch.empty((8, 3), dtype=torch.int32, device="cuda"), torch.empty((8, 3), device="cuda")
    mnb.mnb_moe_route(logits, ids, w, scoring=mnb.MNB_MOE_SIGMOID, renormalize=False)
    want = np.exp(-np.logaddexp(0.0, -np.take_along_axis(np.array(ROWS), ids.cpu().long().numpy(), 1)))
    # (subnormal numbers are 2^-149 apart)
    assert (np.abs(R.f64(w) - want) <= want * 2.0 ** -20 + 2.0 ** -148).all()


@pytest.mark.parametrize("t", [8, 40])
def test_layer(mnb, t):
    """The same weights inside mnb_moe, which routes for itself (8 tokens) or by a launch ahead of it."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    gate, up, down = (R.Experts(mnb, 6, n, k, 4, 32, "f16", True, gen).handle for n, k in ((64, 128), (64, 128), (128, 64)))
    logits = torch.tensor(ROWS * (t // 8), device="cuda")
    x, y = torch.randn((t, 128), generator=gen, device="cuda").to(torch.bfloat16), torch.empty((t, 128), device="cuda")
    ids, w = torch.empty((t, 3), dtype=torch.int32, device="cuda"), torch.empty((t, 3), device="cuda")
    mnb.mnb_moe(x, logits, gate, up, down, y, 3, ids=ids, weights=w, scoring=mnb.MNB_MOE_SIGMOID, workspace=scratch(mnb, t, 3, 6, 128, 64))
    for i in range(t):
        want = weights(ROWS[i % 8], ids[i].cpu().numpy(), 1.0)
        assert (np.abs(R.f64(w[i]) - want) <= want * 2.0 ** -20 + 2.0 ** -40).all(), (i, w[i].tolist(), want)
    assert torch.isfinite(y).all() and (y[4::8] == 0).all() and mnb.mnb_get_device_error() == 0

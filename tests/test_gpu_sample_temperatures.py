"""mnb_sample at temperatures and logits of the largest and smallest sizes that f32 has."""
import pytest
import torch

from tests.test_gpu_sample import run

pytestmark = pytest.mark.gpu

LOWEST, INF = torch.finfo(torch.float32).min, float("inf")


@pytest.mark.parametrize("v", [40, 3001, 30000])
def test_far_logits_under_a_high_temperature(mnb, v):
    """A mask of the lowest value is a weight like any other once the temperature is as large; so are both ends of f32."""
    x = torch.zeros((6, v), device="cuda")
    x[:, ::3] = LOWEST
    x[1, 1::3] = -LOWEST
    x[2] = torch.linspace(-3.4e38, 3.4e38, v, device="cuda")
    x[3, ::5] = -INF
    x[4, 1::3] = 1e30
    x[5, 1::3] = torch.arange(len(x[5, 1::3]), device="cuda") * 1e20
    u = [0.9, 0.7, 0.35, 0.95, 0.999, 0.6]
    for t in (1e19, 1.9e19, 1e30, 1e37, 1e38, 3.4e38, INF):
        for kw in ({}, dict(p=0.9), dict(k=v // 2), dict(m=0.1), dict(k=v // 2, p=0.95, m=0.02)):
            run(mnb, x, t=t, u=u, **kw)
            run(mnb, x, t=t, u=[1 - a for a in u], **kw)
    assert mnb.mnb_get_device_error() == 0


@pytest.mark.parametrize("v", [40, 3001, 30000])
def test_tiny_logits_under_a_low_temperature(mnb, v):
    """Differences as small as f32 has, under temperatures as small; large logits beside them are equal or nothing."""
    i = torch.arange(v, device="cuda", dtype=torch.float64)
    for size, ts in ((2.0 ** -149, (2.0 ** -149, 2.0 ** -146, 2.0 ** -140)), (2.0 ** -135, (2.0 ** -135, 2.0 ** -126)), (2.0 ** -104, (2.0 ** -104, 2.0 ** -99))):
        x = torch.stack([(i % 50) * size, -(i % 7) * size, i * size * 0.25, (i % 3) * size + (i % 2) * 1e-3, (i % 2) * -3e38 + (i % 5) * size,
                         torch.where(i % 4 == 0, 1.5, (i % 5) * size)]).float()
        for t in ts:
            for kw in ({}, dict(p=0.9), dict(k=v // 2), dict(m=0.1), dict(k=v // 2, p=0.95, m=0.02)):
                run(mnb, x, t=t, u=[0.9, 0.7, 0.35, 0.95, 0.99, 0.6], **kw)
    assert mnb.mnb_get_device_error() == 0

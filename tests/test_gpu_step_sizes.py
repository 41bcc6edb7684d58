"""Sizes at which mnb_moe and mnb_sample take another launch: wide hidden sizes (no cluster), many experts, wide batches;
rows that stay in L2, rows of more than 65536 tokens a CTA."""
import numpy as np
import pytest
import torch

from tests import _step_ref as R
from tests.test_gpu_moe import check_route, scratch

pytestmark = pytest.mark.gpu

# tokens, top_k, experts, hidden, inner, bits, bs, act
LAYERS = [(2, 2, 4, 5120, 48, 4, 32, "bf16"), (20, 2, 4, 5120, 48, 4, 32, "f16"), (3, 2, 3, 4999, 40, 8, 64, "bf16"), (17, 3, 4, 7001, 24, 2, 16, "f16"),
          (1, 8, 128, 256, 64, 4, 32, "bf16"), (1, 8, 256, 256, 64, 4, 32, "f16"), (2, 8, 128, 256, 64, 4, 32, "bf16"), (8, 8, 256, 128, 32, 4, 32, "bf16"),
          (33, 4, 16, 1024, 512, 4, 32, "bf16"), (64, 2, 8, 2048, 768, 4, 64, "f16"), (64, 8, 128, 512, 96, 8, 32, "bf16")]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(str(v) for v in c))
def test_layer(mnb, case):
    t, s, e, k, i, bits, bs, act = case
    gen = torch.Generator(device="cuda").manual_seed(t * k + i)
    gate, up = (R.Experts(mnb, e, i, k, bits, bs, "f16", True, gen) for _ in range(2))
    down = R.Experts(mnb, e, k, i, bits, bs, "f16", True, gen)
    x = torch.randn((t, k), generator=gen, device="cuda").to(R.DT[act])
    logits = torch.randn((t, e), generator=gen, device="cuda")
    y, again = torch.empty((t, k), device="cuda"), torch.empty((t, k), device="cuda")
    ids, w = torch.empty((t, s), dtype=torch.int32, device="cuda"), torch.empty((t, s), device="cuda")
    ws = scratch(mnb, t, s, e, k, i)
    mnb.mnb_moe(x, logits, gate.handle, up.handle, down.handle, y, s, ids=ids, weights=w, workspace=ws)
    mnb.mnb_moe(x, logits, gate.handle, up.handle, down.handle, again, s, workspace=ws)
    want, wts = check_route(ids, w, logits, s, None, False, True, 1.0)
    ref, tol = R.moe(R.f64(x), want, wts, gate.w, up.w, down.w, False)
    share = np.abs(ref) * 2.0 ** -16  # the weights' own error, see check_route
    assert (np.abs(R.f64(y) - ref) <= tol + share + np.abs(ref) * 2.0 ** -24 + 1e-37).all()
    assert torch.equal(y, again) and mnb.mnb_get_device_error() == 0


def rows_of(b, v, dtype, pad):
    gen = torch.Generator(device="cuda").manual_seed(b + v)
    x = torch.randn((b, v + pad), generator=gen, device="cuda") * 2.0
    x[:, :v // 50 + 1] += 4.0
    x = x.to(R.DT[dtype])[:, pad // 2:pad // 2 + v]
    inf, nan = float("inf"), float("nan")
    x[0] = 0.5
    x[1] = (torch.arange(v, device="cuda") % 5).float() * 0.125
    x[2, 1::2] = nan
    x[3] = -inf
    x[4, 5] = x[4, v - 7] = inf
    x[5] = nan
    x[6, 3:] = torch.finfo(x.dtype).min
    x[7] = -inf
    x[7, v - 2] = 0.5
    return x


@pytest.mark.parametrize("b,v,dtype,pad", [(64, 80001, "f32", 5), (160, 70001, "bf16", 3), (160, 40003, "f32", 0), (80, 100001, "f16", 9),
                                           (20, 300001, "bf16", 1), (3, 1000003, "f32", 7)])
@pytest.mark.parametrize("cut", ["none", "k", "big_k", "p", "m", "all", "hot", "greedy"])
def test_rows_that_stay_in_memory(mnb, b, v, dtype, pad, cut):
    x = rows_of(b, v, dtype, pad) if b >= 8 else rows_of(8, v, dtype, pad)[:b]
    kw = {"none": {}, "k": dict(k=40), "big_k": dict(k=v * 2 // 3, p=0.97), "p": dict(t=0.8, p=0.9), "m": dict(m=0.05),
          "all": dict(t=0.7, k=50, p=0.9, m=0.02), "hot": dict(t=50.0, p=0.8), "greedy": dict(t=0.0)}[cut]
    gen = torch.Generator(device="cuda").manual_seed(v)
    u = torch.rand(b, generator=gen, device="cuda")
    f = lambda n, d, dt: torch.full((b,), kw[n], dtype=dt, device="cuda") if n in kw else d  # noqa: E731
    tokens, probs = torch.full((b,), -7, dtype=torch.int32, device="cuda"), torch.full((b,), float("nan"), device="cuda")
    mnb.mnb_sample(x, u, tokens, temperature=f("t", None, torch.float32), top_k=f("k", None, torch.int32), top_p=f("p", None, torch.float32),
                   min_p=f("m", None, torch.float32), probs=probs)
    assert mnb.mnb_get_device_error() == 0
    at = lambda n, d: float(np.float32(kw.get(n, d)))  # noqa: E731
    for i in [*range(min(b, 8)), *range(8, b, 19)]:
        token, prob, near = R.sample(R.f64(x[i]), at("t", 1.0), kw.get("k", 0), at("p", 1.0), at("m", 0.0), float(u[i]))
        if near >= 2.0 ** -33:  # as tests/test_gpu_sample.py has it
            assert int(tokens[i]) == token, (i, int(tokens[i]), token, near)
            assert abs(float(probs[i]) - prob) <= prob * (2.0 ** -24 + 2.0 ** -33) + 2.0 ** -42

"""Norms, experts and the draw of tokens run together as examples/decoder_layer.py runs them: each stage against its
definition in 64 bits from what the stage before it left, the same step captured and replayed, and on two streams at once."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import _step_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rows(n, seed, hidden=512):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, attended = (torch.randn((n, hidden), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    f = lambda lo, hi: torch.rand(n, generator=gen, device="cuda") * (hi - lo) + lo  # noqa: E731
    cuts = dict(temperature=f(0.5, 1.5), top_k=torch.randint(0, 300, (n,), generator=gen, device="cuda", dtype=torch.int32),
                top_p=f(0.7, 1.0), min_p=f(0.0, 0.02))
    return x, attended, f(0.0, 0.999), cuts


def dense(mnb, handle):
    """[count] float64 [n, k] weights of an expert_weights descriptor."""
    packed, scales, _ = handle.tensors
    size, out = packed.numel() // handle.E, []
    for e in range(handle.E):
        w = torch.empty((handle.N, handle.K), device="cuda")
        mnb.mnb_dequantize(packed[e * size:(e + 1) * size], scales[e], None, w, handle.N, handle.K, 4, 32, mnb.MNB_F16)
        out.append(R.f64(w))
    return out


def norm_check(x, residual, gain, eps, sums, y):
    s, want = R.rms_norm(R.f64(x), R.f64(residual), R.f64(gain), eps, False)
    half = 2.0 ** -8  # one rounding to bf16, f32 arithmetic below 2^-16 of the value beside it
    assert (np.abs(R.f64(sums) - s) <= np.abs(s) * half * 1.01 + 1e-30).all()
    assert (np.abs(R.f64(y) - want) <= np.abs(want) * half * 1.01 + 1e-30).all()


@pytest.mark.parametrize("n", [1, 3, 17, 64])
def test_stages(mnb, example, n):
    model = example.Decoder(None, seed=2)
    x, attended, u, cuts = rows(n, n)
    seen = {}

    def spy(name, keep):
        inner = getattr(mnb, name)

        def call(*a, **k):
            before = [t.clone() if isinstance(t, torch.Tensor) else t for t in a] + [k["residual"].clone() if "residual" in k else None]
            inner(*a, **k)
            seen.setdefault(name, []).append((before, [t.clone() for t in keep(a, k)]))
        return call

    names = {"mnb_rms_norm": lambda a, k: (k["residual_out"], k["y"]), "mnb_moe": lambda a, k: (a[5],), "mnb_sample": lambda a, k: (a[2],)}
    real = {name: getattr(mnb, name) for name in names}
    try:
        for name, keep in names.items():
            setattr(mnb, name, spy(name, keep))
        tokens = model.after(x.clone(), attended, u, **cuts)
    finally:
        for name, f in real.items():
            setattr(mnb, name, f)
    assert mnb.mnb_get_device_error() == 0
    for i, ((a, out), gain) in enumerate(zip(seen["mnb_rms_norm"], model.gains[1:])):
        norm_check(a[0], a[-1], gain, model.eps, *out)
        assert i > 0 or torch.equal(a[-1], x)
    (a, (mixed,)), = seen["mnb_moe"]
    ids, weights = R.route(R.f64(a[1]), model.top_k, None, False, True, 1.0)
    want, tol = R.moe(R.f64(a[0]), ids, weights, *(dense(mnb, w) for w in (model.gate, model.up, model.down)), False)
    # and 2^-17 of each expert's share (the weights' own bound), one rounding to bf16
    assert (np.abs(R.f64(mixed) - want) <= tol + np.abs(want) * (2.0 ** -8) * 1.01 + 2.0 ** -16 * np.abs(want).max()).all()
    (a, (drawn,)), = seen["mnb_sample"]
    logits, uu, c = R.f64(a[0]), R.f64(u), {k: R.f64(v) for k, v in cuts.items()}
    assert torch.equal(drawn, tokens)
    for i in range(n):
        token, _, near = R.sample(logits[i], c["temperature"][i], int(c["top_k"][i]), c["top_p"][i], c["min_p"][i], uu[i])
        assert near < 2.0 ** -33 or int(drawn[i]) == token


def test_captured_step(mnb, example):
    model = example.Decoder(None, seed=3)
    x, attended, u, cuts = rows(8, 5)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        model.after(x.clone(), attended, u, **cuts)
    torch.cuda.synchronize()
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tokens = model.after(held, attended, u, **cuts)
    for seed in (5, 6, 7):
        x2, attended2, u2, cuts2 = rows(8, seed)
        held.copy_(x2), attended.copy_(attended2), u.copy_(u2)
        for k, v in cuts2.items():
            cuts[k].copy_(v)
        graph.replay()
        eager = x2.clone()
        want = model.after(eager, attended2, u2, **cuts2)
        assert torch.equal(want, tokens) and torch.equal(eager, held)


def test_two_streams(mnb, example):
    """Two steps in flight at once, a workspace each."""
    models = [example.Decoder(None, seed=4) for _ in range(2)]
    data = [rows(16, 8 + i) for i in range(2)]
    want = [models[0].after(x.clone(), a, u, **c) for x, a, u, c in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (x, a, u, c) in enumerate(data):
            with torch.cuda.stream(streams[i]):
                got[i].append(models[i].after(x.clone(), a, u, **c))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])


def test_prompt_and_single_tokens(mnb, example):
    """A whole step from token to token, as a prompt and one token at a time (their roundings differ: only that both run)."""
    tokens = torch.tensor([5, 900, 31, 77, 1200, 6], dtype=torch.int32, device="cuda")
    cuts, u = dict(temperature=torch.zeros(1, device="cuda")), torch.zeros(1, device="cuda")
    model = example.Decoder(example.Layer(seed=6), seed=6)
    whole = model.step(tokens, [0], [6], [6], u, **cuts)
    for i in range(6):
        last = model.step(tokens[i:i + 1], [1], [1], [i + 1], u, **cuts)
    assert 0 <= int(whole) < 2000 and 0 <= int(last) < 2000
    assert mnb.mnb_get_device_error() == 0


def test_rows_that_lie_far_apart(mnb):
    """Row strides past 2^31 elements: the same results as from rows side by side."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    far = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    apart = lambda: far.as_strided((2, 256), (2 ** 31, 1), 0)  # noqa: E731
    x = torch.randn((2, 256), generator=gen, device="cuda").to(torch.bfloat16)
    apart().copy_(x)
    y, z = torch.empty_like(x), far.as_strided((2, 256), (2 ** 31, 1), 1024)
    mnb.mnb_rms_norm(x, None, 1e-5, y=y)
    mnb.mnb_rms_norm(apart(), None, 1e-5, y=z)
    assert torch.equal(y, z)
    u = torch.rand(2, generator=gen, device="cuda")
    a, b = (torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(2))
    mnb.mnb_sample(x, u, a)
    mnb.mnb_sample(apart(), u, b)
    assert torch.equal(a, b)
    gate, up, down = (R.Experts(mnb, 4, n, k, 4, 32, "f16", True, gen).handle for n, k in ((64, 256), (64, 256), (256, 64)))
    logits = torch.randn((2, 4), generator=gen, device="cuda").to(torch.bfloat16)
    spread = far.as_strided((2, 4), (2 ** 31, 1), 2048)
    spread.copy_(logits)
    from tests import _gpu as G
    ws = G.aligned_empty(mnb.mnb_moe_workspace_size(2, 2, 4, 256, 64))
    mnb.mnb_moe(x, logits, gate, up, down, y, 2, workspace=ws)
    mnb.mnb_moe(apart(), spread, gate, up, down, z, 2, workspace=ws)
    assert torch.equal(y, z) and mnb.mnb_get_device_error() == 0

"""Calls of two host threads at once, each on a stream of its own, whose launches need shared memory of other sizes."""
import ctypes
import threading

import pytest
import torch

from tests import _gpu as G
from tests import _step_ref as R

pytestmark = pytest.mark.gpu


def together(calls, rounds=4000):
    """Runs each call `rounds` times on a thread of its own (call(stream) gives a function without arguments), all at once; what
    came back that was not 0."""
    answers, gate = set(), threading.Barrier(len(calls))

    def work(make):
        stream = torch.cuda.Stream()
        call = make(stream.cuda_stream)
        gate.wait()
        for i in range(rounds):
            answers.add(call())
            if i % 100 == 99:
                stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return answers - {0, None}


def test_sample(mnb):
    gen = torch.Generator(device="cuda").manual_seed(1)
    calls, done = [], []
    for b, v in ((1, 3000), (1, 200003), (2, 60001), (1, 150000)):
        x, u = torch.randn((b, v), generator=gen, device="cuda"), torch.rand(b, generator=gen, device="cuda")
        want, got = torch.empty(b, dtype=torch.int32, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")
        mnb.mnb_sample(x, u, want)

        def make(stream, x=x, u=u, got=got, b=b, v=v):
            a = mnb.SampleArgs(x.data_ptr(), u.data_ptr(), None, None, None, None, got.data_ptr(), None, b, v, v, mnb.MNB_F32, stream)
            return lambda: mnb.load().mnb_sample(a)

        calls.append(make)
        done.append((got, want))
    assert together(calls) == set()
    assert all(torch.equal(a, b) for a, b in done) and mnb.mnb_get_device_error() == 0


def test_experts(mnb):
    gen = torch.Generator(device="cuda").manual_seed(2)
    gate, up, down = (R.Experts(mnb, 4, n, k, 4, 32, "f16", True, gen).handle for n, k in ((64, 128), (64, 128), (128, 64)))
    calls, done = [], []
    for t in (1, 64, 20, 2):
        x = torch.randn((t, 128), generator=gen, device="cuda").to(torch.bfloat16)
        logits = torch.randn((t, 4), generator=gen, device="cuda")
        ws = G.aligned_empty(mnb.mnb_moe_workspace_size(t, 3, 4, 128, 64))
        want, got = torch.empty((t, 128), device="cuda"), torch.empty((t, 128), device="cuda")
        mnb.mnb_moe(x, logits, gate, up, down, want, 3, workspace=ws)

        def make(stream, t=t, x=x, lg=logits, ws=ws, got=got):
            r = mnb.MoeRouteArgs(lg.data_ptr(), None, None, None, t, 4, 3, 4, mnb.MNB_F32, mnb.MNB_MOE_SOFTMAX, 1, 1.0, stream)
            a = mnb.MoeArgs(x.data_ptr(), got.data_ptr(), ctypes.pointer(gate), ctypes.pointer(up), ctypes.pointer(down), 128, 128, mnb.MNB_BF16,
                            mnb.MNB_F32, mnb.MNB_ACT_SILU, ws.data_ptr(), ws.numel(), stream)
            return lambda: mnb.load().mnb_moe(a, r)

        calls.append(make)
        done.append((got, want))
    assert together(calls) == set()
    assert all(torch.equal(a, b) for a, b in done) and mnb.mnb_get_device_error() == 0


@pytest.mark.parametrize("m", [1, 2, 8, 64])
@pytest.mark.parametrize("acc", [0, 4])
def test_products(mnb, m, acc):
    """Products of few and many rows whose shared memory goes by K."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    calls, done = [], []
    for n, k in ((256, 256), (256, 8192)):
        codes = torch.randint(0, 256, (n, k // 32, 16), generator=gen, device="cuda", dtype=torch.uint8)
        scales = (torch.rand((n, k // 32), generator=gen, device="cuda") * 0.01).half()
        packed = G.aligned_empty(mnb.mnb_packed_size(n, k, 4, 32))
        mnb.mnb_pack_weights(codes, packed, n, k, 4, 32)
        x = torch.randn((m, k), generator=gen, device="cuda").half()
        want, got = torch.empty((m, n), dtype=torch.float16, device="cuda"), torch.empty((m, n), dtype=torch.float16, device="cuda")
        ws = G.aligned_empty(max(256, mnb.mnb_workspace_size(m, n, k, 4, 32, acc)))

        def make(stream, x=x, packed=packed, scales=scales, n=n, k=k, ws=ws, y=got):
            a = mnb._matmul_args(x, packed, scales, None, y, m, n, k, 4, 32, mnb.MNB_F16, mnb.MNB_F16, mnb.MNB_F16, None, None, mnb.MNB_F32,
                                 acc, ws, "auto", stream, 0)
            return lambda: mnb.load().mnb_matmul_ex(a)

        mnb.mnb_matmul_ex(x, packed, scales, None, want, m, n, k, 4, 32, mnb.MNB_F16, mnb.MNB_F16, mnb.MNB_F16, accuracy_level=acc, workspace=ws)
        calls.append(make)
        done.append((got, want))
    assert together(calls) == set()
    assert all(torch.equal(a, b) for a, b in done) and mnb.mnb_get_device_error() == 0

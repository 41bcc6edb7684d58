"""Refusals of the norm, expert and sampling calls, before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

import block_quantized_weight_matmulnbits_gb300 as mnb


def _norm(**kw):
    a = mnb.RmsNormArgs()
    a.x = a.y = a.residual = a.residual_out = a.weight = a.codes = a.scales = 4096
    a.T, a.width, a.block_size = 2, 64, 32
    a.x_stride = a.residual_stride = a.residual_out_stride = a.y_stride = 64
    a.dtype = a.weight_dtype = a.out_dtype = mnb.MNB_BF16
    a.eps = 1e-6
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [{"x": None}, {"x": 4097}, {"T": -1}, {"width": 0}, {"dtype": 3}, {"weight_dtype": -1}, {"out_dtype": 7},
                                 {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"flags": 2}, {"residual": None},
                                 {"codes": None}, {"scales": None}, {"codes": 4104}, {"scales": 4098}, {"block_size": 24},
                                 {"block_size": 8}, {"x_stride": 63}, {"y_stride": -64}, {"residual": 4097}, {"y": 4097}, {"weight": 4097}])
def test_norm_arguments(bad):
    assert mnb.load().mnb_rms_norm(ctypes.byref(_norm(**bad))) == mnb.MNB_ERR_INVALID_ARG


def test_norm_limits():
    lib = mnb.load()
    assert lib.mnb_rms_norm(None) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_rms_norm(ctypes.byref(_norm(T=0))) == mnb.MNB_OK
    assert lib.mnb_rms_norm(ctypes.byref(_norm(width=32769, x_stride=40000, y_stride=40000, residual_stride=40000,
                                               residual_out_stride=40000))) == mnb.MNB_ERR_UNSUPPORTED
    assert lib.mnb_rms_norm(ctypes.byref(_norm(block_size=65536))) == mnb.MNB_ERR_UNSUPPORTED
    none = dict(y=None, residual=None, residual_out=None, codes=None, scales=None)
    assert lib.mnb_rms_norm(ctypes.byref(_norm(**none))) == mnb.MNB_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [{"y": 4096, "out_dtype": mnb.MNB_F32}, {"y": 4096, "y_stride": 128},
                                 {"residual_out": 4096, "residual_out_stride": 128}, {"y": 12288, "out_dtype": mnb.MNB_F32}])
def test_norm_output_over_an_input_of_another_layout(bad):
    a = _norm(**{**dict(x=4096, residual=12288, residual_out=16384, y=20480, dtype=mnb.MNB_BF16, out_dtype=mnb.MNB_BF16), **bad})
    assert mnb.load().mnb_rms_norm(ctypes.byref(a)) == mnb.MNB_ERR_INVALID_ARG


def test_norm_binding_checks():
    x = torch.ones((2, 64))
    for kw in (dict(y=torch.ones((2, 63))), dict(residual=torch.ones((2, 64), dtype=torch.float16), y=x), dict(codes=x, y=x),
               dict(y=torch.ones((64, 2)).T), dict(y=x)):  # the last: not on a GPU
        with pytest.raises(ValueError):
            mnb.mnb_rms_norm(x, None, 1e-6, **kw)


def _route(**kw):
    a = mnb.MoeRouteArgs()
    a.logits = a.ids = a.weights = 4096
    a.T, a.E, a.S, a.logits_stride = 2, 8, 2, 8
    a.dtype, a.renormalize, a.scale = mnb.MNB_F32, 1, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_ROUTE = [{"logits": None}, {"logits": 4098}, {"T": -1}, {"E": 0}, {"S": 0}, {"S": 9}, {"dtype": 5}, {"scoring": 2}, {"renormalize": 2},
             {"scale": float("nan")}, {"scale": float("inf")}, {"bias": 4096}, {"bias": 4097, "scoring": 1}, {"logits_stride": 7},
             {"ids": 4097}, {"weights": 4098}]


def _experts(n, k, **kw):
    w = mnb.ExpertWeights()
    w.packed_b = w.scales = w.zero_points = 4096
    w.E, w.N, w.K, w.bits, w.block_size, w.scale_dtype = 8, n, k, 4, 32, mnb.MNB_F16
    for key, v in kw.items():
        setattr(w, key, v)
    return w


def _moe(gate=None, up=None, down=None, **kw):
    a = mnb.MoeArgs()
    a.keep = tuple(_experts(*s, **(d or {})) for s, d in (((96, 64), gate), ((96, 64), up), ((64, 96), down)))
    a.gate, a.up, a.down = (ctypes.pointer(w) for w in a.keep)
    a.x = a.y = a.workspace = 4096
    a.x_stride = a.y_stride = 64
    a.act_dtype = a.out_dtype = mnb.MNB_BF16
    a.workspace_bytes = 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", BAD_ROUTE)
def test_route_arguments(bad):
    lib = mnb.load()
    assert lib.mnb_moe_route(ctypes.byref(_route(**bad))) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_moe(ctypes.byref(_moe()), ctypes.byref(_route(**bad))) == mnb.MNB_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [{"x": None}, {"x": 4097}, {"y": 4097}, {"x_stride": 63}, {"y_stride": -1}, {"act_dtype": 4}, {"out_dtype": -1},
                                 {"activation": 2}, {"gate": {"N": 95}}, {"up": {"K": 63}}, {"down": {"K": 95}}, {"down": {"N": 65}},
                                 {"gate": {"E": 7}}, {"up": {"packed_b": 4100}}, {"down": {"packed_b": None}}, {"down": {"scales": 4097}},
                                 {"gate": {"bits": 3}}, {"gate": {"block_size": 8}}, {"down": {"scale_dtype": 9}}, {"workspace": 4100}])
def test_moe_arguments(bad):
    assert mnb.load().mnb_moe(ctypes.byref(_moe(**bad)), ctypes.byref(_route())) == mnb.MNB_ERR_INVALID_ARG


def test_moe_limits():
    lib = mnb.load()
    call = lambda a, r: lib.mnb_moe(ctypes.byref(a), ctypes.byref(r))  # noqa: E731
    assert lib.mnb_moe(None, ctypes.byref(_route())) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_moe(ctypes.byref(_moe()), None) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_moe_route(ctypes.byref(_route(T=0))) == mnb.MNB_OK and call(_moe(), _route(T=0)) == mnb.MNB_OK
    assert lib.mnb_moe_route(ctypes.byref(_route(ids=None, weights=None))) == mnb.MNB_ERR_INVALID_ARG
    for r in (dict(T=65), dict(E=2000, logits_stride=2000), dict(E=64, S=33, logits_stride=64)):
        e = r.get("E", 8)
        a = _moe(*({"E": e} for _ in range(3)))
        assert call(a, _route(**r)) == mnb.MNB_ERR_UNSUPPORTED
    assert call(_moe(act_dtype=mnb.MNB_F32), _route()) == mnb.MNB_ERR_UNSUPPORTED
    assert call(_moe(up={"bits": 8}), _route()) == mnb.MNB_ERR_UNSUPPORTED
    assert call(_moe(down={"block_size": 16}), _route()) == mnb.MNB_ERR_UNSUPPORTED
    need = mnb.mnb_moe_workspace_size(2, 2, 8, 64, 96)
    assert need >= 2 * 2 * 2 * 96 * 2
    assert call(_moe(workspace_bytes=need - 1), _route()) == mnb.MNB_ERR_NO_MEM
    assert call(_moe(workspace=None), _route()) == mnb.MNB_ERR_NO_MEM
    for bad in ((0, 2, 8, 64, 96), (65, 2, 8, 64, 96), (2, 9, 8, 64, 96), (2, 2, 8, 0, 96), (64, 32, 64, 64, 96), (2, 2, 8, 64, 0)):
        assert mnb.mnb_moe_workspace_size(*bad) == 0


def test_moe_counts_fit_32_bits():
    assert mnb.mnb_moe_workspace_size(64, 16, 64, 64, 1 << 24) > 0
    for hidden, inner in ((64, 1 << 25), (1 << 25, 64)):
        assert mnb.mnb_moe_workspace_size(64, 16, 64, hidden, inner) == 0


def _sample(**kw):
    a = mnb.SampleArgs()
    a.logits = a.u = a.tokens = a.temperature = a.top_k = a.top_p = a.min_p = a.probs = 4096
    a.B, a.V, a.row_stride, a.dtype = 2, 100, 100, mnb.MNB_F32
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [{"logits": None}, {"logits": 4098}, {"u": None}, {"tokens": None}, {"tokens": 4097}, {"probs": 4098}, {"B": -1},
                                 {"V": 0}, {"row_stride": 99}, {"dtype": 3}, {"top_k": 4097}, {"top_p": 4097}, {"min_p": 4097}, {"temperature": 4097}])
def test_sample_arguments(bad):
    assert mnb.load().mnb_sample(ctypes.byref(_sample(**bad))) == mnb.MNB_ERR_INVALID_ARG


def test_sample_limits():
    lib = mnb.load()
    assert lib.mnb_sample(None) == mnb.MNB_ERR_INVALID_ARG
    assert lib.mnb_sample(ctypes.byref(_sample(B=0))) == mnb.MNB_OK
    assert lib.mnb_sample(ctypes.byref(_sample(V=(1 << 24) + 1, row_stride=1 << 25))) == mnb.MNB_ERR_UNSUPPORTED

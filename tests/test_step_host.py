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


def test_norm_binding_checks():
    x = torch.ones((2, 64))
    for kw in (dict(y=torch.ones((2, 63))), dict(residual=torch.ones((2, 64), dtype=torch.float16), y=x), dict(codes=x, y=x),
               dict(y=torch.ones((64, 2)).T), dict(y=x)):  # the last: not on a GPU
        with pytest.raises(ValueError):
            mnb.mnb_rms_norm(x, None, 1e-6, **kw)

"""Plain 64-bit definitions of the norm, expert and sampling operators, and helpers.  Test code only."""
import numpy as np
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(t):
    """Largest relative error of one rounding to the type of a tensor (or to dtype t)."""
    return torch.finfo(t if isinstance(t, torch.dtype) else t.dtype).eps / 2


def smallest(t):
    """Half the spacing of the type's subnormal numbers: the absolute error of a rounding near zero."""
    f = torch.finfo(t if isinstance(t, torch.dtype) else t.dtype)
    return f.smallest_normal * f.eps / 2


def rms_norm(x, residual, weight, eps, unit):
    """(sum, norm), float64 arrays."""
    s = x if residual is None else x + residual
    with np.errstate(all="ignore"):
        y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps)
        if weight is not None:
            y = y * (weight + 1 if unit else weight)
    return s, y

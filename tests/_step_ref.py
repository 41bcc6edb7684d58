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


def route(logits, S, bias, sigmoid, renorm, scale):
    """Experts and weights of float64 logits [T, E] (ties to the lowest expert, NaN last)."""
    T, E = logits.shape
    ids, weights = np.zeros((T, S), dtype=np.int64), np.zeros((T, S))
    with np.errstate(all="ignore"):
        for t in range(T):
            score = 1 / (1 + np.exp(-logits[t])) if sigmoid else logits[t]
            key = score + bias if sigmoid and bias is not None else logits[t]
            order = sorted(range(E), key=lambda e: (np.isnan(key[e]), 0.0 if np.isnan(key[e]) else -key[e], e))[:S]
            ids[t] = order
            if sigmoid:
                w = score[order]
                total = w.sum() if renorm else 1.0
            else:
                top = logits[t, order[0]]
                ex = np.where(logits[t] == -np.inf, 0.0, np.exp(logits[t] - top))
                w, total = ex[order], ex[order].sum() if renorm else ex.sum()
            weights[t] = (w / total if total != 0 else 0 * w) * scale
    return ids, weights


def codes_to_weights(codes, scales, zp, n, k, bits, bs):
    """codes uint8 [N, KB, blob], scales [N, KB], zp uint8 [N, ...] or None -> float64 [N, K]."""
    per, mask = 8 // bits, 2 ** bits - 1
    kb = scales.shape[1]
    q = np.stack([(codes >> (bits * j)) & mask for j in range(per)], -1).reshape(n, kb, bs).astype(np.float64)
    z = 2.0 ** (bits - 1)
    if zp is not None:
        z = np.stack([(zp >> (bits * j)) & mask for j in range(per)], -1).reshape(n, -1)[:, :kb, None].astype(np.float64)
    return ((q - z) * scales[..., None]).reshape(n, -1)[:, :k]


class Experts:
    """E random [N, K] weights: device buffers, the library's descriptor, and their values."""

    def __init__(self, mnb, e, n, k, bits, bs, sdt, zp, gen, align=256):
        from tests import _gpu as G
        kb = -(-k // bs)
        codes = torch.randint(0, 256, (e, n, kb, bs * bits // 8), generator=gen, device="cuda", dtype=torch.uint8)
        scales = ((torch.rand((e, n, kb), generator=gen, device="cuda") + 0.5) * (k ** -0.5 * 3.4 / 2 ** bits)).to(DT[sdt])
        zps = torch.randint(0, 256, (e, n, -(-kb * bits // 8)), generator=gen, device="cuda", dtype=torch.uint8) if zp else None
        size = mnb.mnb_packed_size(n, k, bits, bs)
        packed = G.aligned_empty(e * size)
        for i in range(e):
            mnb.mnb_pack_weights(codes[i], packed[i * size:(i + 1) * size], n, k, bits, bs)
        if align != 256:  # scales and zero points on their natural alignment only
            scales = torch.cat([scales.flatten()[:1], scales.flatten()])[1:].view(e, n, kb)
            if zp:
                zps = torch.cat([zps.flatten()[:1], zps.flatten()])[1:].view(e, n, -1)
        self.handle = mnb.expert_weights(packed, scales, zps, e, n, k, bits, bs)
        s = f64(scales)
        self.w = [codes_to_weights(codes[i].cpu().numpy(), s[i], None if zps is None else zps[i].cpu().numpy(), n, k, bits, bs) for i in range(e)]


def moe(x, ids, weights, gate, up, down, gelu):
    """(y, bound): the layer in 64 bits, and how far f32 sums and a 16-bit h may be from it."""
    T, K = x.shape
    inner = gate[0].shape[0]
    y, tol = np.zeros((T, K)), np.zeros((T, K))
    # An MMA adds 16 products and the running sum with an error of at most 2^-22 of what they come to in magnitude; a
    # dot product of depth d is d / 16 of them, a scaling each 1 or 2, and joins: below (d / 16 + 40) * 2^-21 of sum |x w|.
    unit = lambda d: (d / 16 + 40) * 2.0 ** -21  # noqa: E731
    with np.errstate(all="ignore"):
        for t in range(T):
            for e, w in zip(ids[t], weights[t]):
                g, u = gate[e] @ x[t], up[e] @ x[t]
                dg, du = unit(K) * (np.abs(gate[e]) @ np.abs(x[t])), unit(K) * (np.abs(up[e]) @ np.abs(x[t]))
                if gelu:
                    a = 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
                else:
                    a = g / (1 + np.exp(-g))
                h = w * a * u
                # |act'| <= 1.2; the function itself, the products and w: 2^-19 of h (and of g for tanh's cancellation);
                # two bf16 parts: 2^-18
                dh = abs(w) * (1.2 * dg * (np.abs(u) + du) + np.abs(a) * du) + np.abs(h) * (2.0 ** -18 + 2.0 ** -19) \
                    + abs(w) * np.abs(g * u) * 2.0 ** -21
                y[t] += down[e] @ h
                tol[t] += np.abs(down[e]) @ dh + unit(inner) * (np.abs(down[e]) @ np.abs(h))
    return y, tol


def sample(x, t, k, p, m, u):
    """(token, probability, distance): the draw from a float64 row; the distance of its sums from the nearest border that
    would change it, relative to what is kept."""
    x = np.where(np.isnan(x), -np.inf, x)
    if x.max() == -np.inf:
        return -1, 0.0, 1.0
    order = np.lexsort((np.arange(len(x)), -x))
    if t == 0:
        return int(order[0]), 1.0, 1.0
    with np.errstate(invalid="ignore"):
        d = np.where(x[order] == x.max(), 0.0, x.max() - x[order])
        w = np.where(np.isinf(d), 0.0, np.exp(-np.where(np.isinf(d), 0.0, d) / t))
    near = 1.0
    if 0 < k < len(x):
        w[k:] = 0.0
    if p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep = before < p * w.sum()
        keep[0] = True
        near = min(near, np.abs(np.cumsum(w) - p * w.sum()).min() / w.sum())
        w[~keep] = 0.0
    if m > 0:
        near = min(near, np.abs(w - min(m, 1.0))[w != 1].min(initial=1.0))
        w[w < min(m, 1.0)] = 0.0
    upto = np.cumsum(w)
    near = min(near, np.abs(upto - u * upto[-1]).min() / upto[-1]) if u > 0 else near
    at = int((upto <= u * upto[-1]).sum())
    return int(order[at]), float(w[at] / upto[-1]), near

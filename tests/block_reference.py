"""Plain definitions of the block norm, the int8 quantiser and product, and
expert routing, on the CPU: elementwise steps in binary32 one rounding at a
time, statistics, sums and choices in binary64."""
import math

import numpy as np
import torch

F32, F64 = torch.float32, torch.float64
TINY = 2.0 ** -119


def rstd(v, eps):
    return (1.0 / torch.sqrt(v.to(F64).square().sum(-1, keepdim=True) / v.shape[-1] + eps)).to(F32)


def quantize(v):
    """codes int8, scales f32 of the rows of v, whose type is exact in f32."""
    v = v.to(F32)
    amax = v.abs().amax(-1, keepdim=True)          # NaN if the row holds one
    a = torch.clamp(amax, min=TINY)
    most = torch.full_like(a, 127.0)               # tensors: a quotient with a plain number is a
    codes = torch.round(v * (most / a))            # product with a reciprocal, rounded twice
    fine = torch.isfinite(amax)
    codes = torch.where(fine, codes, torch.zeros_like(codes))
    assert codes.abs().max() <= 127
    return codes.to(torch.int8), torch.where(fine, a / most, torch.full_like(a, math.nan))[:, 0]


def block_norm(x, gamma, y, gamma_post, gate, residual_scale, branch_scale, eps=1e-6):
    """(residual_out or None, norm or None) with the kernel's roundings."""
    eps = float(np.float32(eps))
    r = x
    if y is not None:
        p = y.to(F32)
        if gamma_post is not None:
            p = (p * rstd(p, eps)) * gamma_post.to(F32)
        if gate is not None:
            p = p * gate.to(F32)
        f = lambda s: torch.tensor(s, dtype=F32)  # noqa: E731
        r = (f(residual_scale) * x.to(F32) + f(branch_scale) * p).to(x.dtype)
    if gamma is None:
        return r, None
    v = r.to(F32)
    return (r if y is not None else None), ((v * rstd(v, eps)) * gamma.to(F32)).to(gamma.dtype)


def int8_sums(a, b):
    """Exact sums (binary64 holds every one of them)."""
    return a.to(F64) @ b.to(F64).t()


def int8_gemm(a, sa, b, sb, bias, dtype):
    v = (int8_sums(a, b).to(F32) * sa[:, None]) * sb
    return (v if bias is None else v + bias).to(dtype)


def route(logits, k, scoring, bias, groups, keep, top, renorm, scale):
    """One token and one choice at a time."""
    T, E = logits.shape
    L = logits.to(F64).numpy()
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        l = L[t].copy()
        out = np.isnan(l) | ((scoring == "softmax") & (l == np.inf))
        poisoned = out.any()
        out = out | (l == -np.inf)
        l[out] = -np.inf
        with np.errstate(over="ignore"):
            if scoring == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-l))
            elif out.all():
                s = np.zeros(E)
            else:
                e = np.exp(l - l.max())
                s = e / math.fsum(e)
        score = s + (0.0 if bias is None else bias.to(F64).numpy())
        key = l.copy() if bias is None else score.copy()
        key[out] = -np.inf
        score[out] = -np.inf
        if groups > 1:
            size = E // groups
            sums = []
            for g in range(groups):
                best = sorted((key if top == 1 else score)[g * size:(g + 1) * size], reverse=True)[:top]
                sums.append(best[0] if top == 1 else sum(-1e30 if v == -np.inf else v for v in best))
            order = sorted(range(groups), key=lambda g: (-sums[g], g))
            for g in order[keep:]:
                key[g * size:(g + 1) * size] = -np.inf
        order = sorted((e for e in range(E) if key[e] != -np.inf), key=lambda e: (-key[e], e))[:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[order]
        if renorm:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
        w[t] *= scale
        if poisoned:
            w[t] = np.nan
    return torch.from_numpy(w), torch.from_numpy(ids)


def route_rows(logits, k, scoring, bias, groups, keep, top, renorm, scale):
    """route() for many tokens at once, on the device the logits are on."""
    T, E = logits.shape
    inf = math.inf
    l = logits.to(F64)
    bad = l.isnan() | ((l == inf) if scoring == "softmax" else torch.zeros_like(l, dtype=torch.bool))
    l = l.masked_fill(bad, -inf)
    out = l == -inf
    if scoring == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True).clamp_min(torch.finfo(F64).min))
        s = e / e.sum(1, keepdim=True).clamp_min(torch.finfo(F64).tiny)
    score = (s if bias is None else s + bias.to(F64)).masked_fill(out, -inf)
    key = l.clone() if bias is None else score.clone()
    if groups > 1:
        by_group = (key if top == 1 else score).view(T, groups, E // groups)
        best = by_group.sort(dim=2, descending=True).values[..., :top]
        if top == 2:
            best = best.masked_fill(best == -inf, -1e30)
        order = best.sum(2).sort(dim=1, descending=True, stable=True).indices
        shut = torch.ones(T, groups, dtype=torch.bool, device=l.device).scatter_(1, order[:, :keep], False)
        key.view(T, groups, -1).masked_fill_(shut[..., None], -inf)
    order = key.sort(dim=1, descending=True, stable=True)
    ids, none = order.indices[:, :k], order.values[:, :k] == -inf
    w = s.gather(1, ids).masked_fill(none, 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    w = (w * scale).masked_fill(bad.any(1, keepdim=True), math.nan)
    return w, ids.masked_fill(none, -1).to(torch.int32)

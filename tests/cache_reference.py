"""Plain definitions of the rotary positions, the 4-bit cache and the attention
over it, on the CPU in binary64, one row at a time."""
import math

import numpy as np
import torch

F64 = torch.float64
GRID = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), dtype=F64)
EXPONENTS = {torch.bfloat16: (-125, 125), torch.float16: (-23, 13)}


def rope(x, positions, inv_freq, axes=None, interleaved=False, inverse=False, scale=1.0):
    """x [T, H, D] turned, in binary64, not rounded."""
    at = positions if positions.dim() == 2 else positions[None]
    out = x.to(F64).clone()
    pairs = len(inv_freq)
    for i in range(pairs):
        theta = at[0 if axes is None else axes[i]].to(F64) * inv_freq[i].to(F64)
        c, s = torch.cos(theta)[:, None] * scale, torch.sin(theta)[:, None] * scale * (-1 if inverse else 1)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        u, w = x[..., a].to(F64), x[..., b].to(F64)
        out[..., a], out[..., b] = u * c - w * s, w * c + u * s
    return out


def groups(v, low, high):
    """(codes, scale byte) of one group of 32 binary64 values, by search."""
    if not torch.isfinite(v).all():
        return [0] * 32, 255
    most = v.abs().max().item()
    e = low
    while e < high and 6.0 * 2.0 ** e < most:
        e += 1
    codes = []
    for x in v.tolist():
        y = min(abs(x) / 2.0 ** e, 6.0)
        best = min(range(8), key=lambda i: (abs(y - GRID[i].item()), i % 2))
        codes.append(best | (8 if math.copysign(1.0, x) < 0 else 0))
    return codes, e + 127


def decode(codes, byte):
    if byte == 255:
        return [math.nan] * 32
    return [(-1.0 if c & 8 else 1.0) * GRID[c & 7].item() * 2.0 ** (byte - 127) for c in codes]


def quantized(x):
    """Values [.., D] that x [.., D] is held as, in binary64."""
    low, high = EXPONENTS[x.dtype]
    flat = x.to(F64).reshape(-1, 32)
    return torch.tensor([decode(*groups(g, low, high)) for g in flat], dtype=F64).reshape(x.shape)


def quantized_fast(x):
    """The same for finite x, all groups at once."""
    low, high = EXPONENTS[x.dtype]
    v = x.to(F64).unflatten(-1, (-1, 32))
    most = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(most / 6).clamp(min=-1000))
    e = torch.where(6.0 * torch.exp2(e - 1) >= most, e - 1, e)      # logarithms off by a last place
    e = torch.where(6.0 * torch.exp2(e) < most, e + 1, e).clamp(low, high)
    y = (v.abs() * torch.exp2(-e)).clamp(max=6.0)
    d = (y[..., None] - GRID).abs() + 1e-9 * (torch.arange(8) % 2)   # ties, and only those, to the even code
    return torch.copysign(GRID[d.argmin(-1)] * torch.exp2(e), v).flatten(-2)


class Cache:
    """The cache's bytes, one slot at a time."""

    def __init__(self, pages, heads, D, ps):
        self.pages, self.heads, self.D, self.ps = pages, heads, D, ps
        self.bytes = np.zeros((pages, heads, ps * (D + D // 16)), np.uint8)

    def parts(self, slot, kind):
        """Byte numbers of a slot's codes and scales in its page."""
        ps, D, at = self.ps, self.D, slot % self.ps
        codes = kind * ps * D // 2 + at * D // 2 + np.arange(D // 2)
        scales = ps * D + kind * ps * D // 32 + np.arange(D // 32) * ps + at
        return slot // ps, codes, scales

    def write(self, slot, kind, rows):
        """rows [heads, D] of bf16 or fp16."""
        if slot < 0 or slot >= self.pages * self.ps:
            return
        page, codes, scales = self.parts(slot, kind)
        for h in range(self.heads):
            made = [groups(g, *EXPONENTS[rows.dtype]) for g in rows[h].to(F64).reshape(-1, 32)]
            c = np.array([x for g in made for x in g[0]], np.uint8)
            self.bytes[page, h, codes] = c[0::2] | c[1::2] << 4
            self.bytes[page, h, scales] = [g[1] for g in made]

    def read(self, slot, kind):
        """[heads, D] in binary64."""
        if slot < 0 or slot >= self.pages * self.ps:
            return torch.zeros(self.heads, self.D, dtype=F64)
        page, codes, scales = self.parts(slot, kind)
        out = []
        for h in range(self.heads):
            c = self.bytes[page, h, codes]
            c = np.stack((c & 15, c >> 4), 1).reshape(-1, 32)
            out.append([x for g, b in zip(c, self.bytes[page, h, scales]) for x in decode(g.tolist(), int(b))])
        return torch.tensor(out, dtype=F64)


def packed(k, v, order, pages, ps):
    """(cache bytes, values of k, values of v): token t of k and v [n, H, D] in
    slot order[t], written as a whole from finite values."""
    n, H, D = k.shape
    cache = torch.zeros(pages, H, ps * (D + D // 16), dtype=torch.uint8)
    page, at = order // ps, order % ps
    held = []
    for kind, x in enumerate((k, v)):
        q = quantized_fast(x)
        g = q.unflatten(-1, (-1, 32))
        low, high = EXPONENTS[x.dtype]
        most = x.to(F64).abs().unflatten(-1, (-1, 32)).amax(-1)
        e = torch.full_like(most, float(low))
        for i in range(low, high):
            e = torch.where(most > 6.0 * 2.0 ** i, torch.full_like(e, i + 1.0), e)
        code = (g.abs()[..., None] * torch.exp2(-e)[..., None, None] - GRID).abs().argmin(-1) + 8 * torch.signbit(g)
        code = code.to(torch.uint8).flatten(-2)
        codes = cache[:, :, kind * ps * D // 2:(kind + 1) * ps * D // 2].unflatten(2, (ps, D // 2))
        scales = cache[:, :, ps * D + kind * ps * D // 32:ps * D + (kind + 1) * ps * D // 32].unflatten(2, (D // 32, ps))
        codes[page, :, at] = code[..., 0::2] | code[..., 1::2] << 4
        scales[page, :, :, at] = (e + 127).to(torch.uint8)
        held.append(q)
    return cache, *held


def attention(q, keys, values, lens, q_starts, visible=None, scale=None, causal=True, window=0, softcap=0.0,
              relative=False):
    """keys[b], values[b] [len, Hkv, D] in binary64 (as many tokens as lens[b] says at least); visible[b] bool [len]
    or None.  Returns (out, lse, bound, lse_bound): bound is how far the output in q's type may be off.  relative: a
    capped score is off by a part of itself, not of the cap."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2
    out = torch.full((T, Hq, D), math.nan, dtype=F64)
    bound = torch.zeros_like(out)
    lse = torch.full((T, Hq), math.nan, dtype=F64)
    lse_bound = torch.zeros_like(lse)
    for b, L in enumerate(lens):
        first, n = q_starts[b], q_starts[b + 1] - q_starts[b]
        L = max(L, 0)
        Hk = keys[b].shape[1] if keys[b] is not None else 1
        for i in range(n):
            p = L - n + i
            t = torch.arange(L)
            seen = torch.ones(L, dtype=torch.bool) if visible is None or visible[b] is None else visible[b][:L].clone()
            if causal:
                seen &= t <= p
            if window:
                seen &= t > p - window
            if not seen.any():
                out[first + i], lse[first + i] = 0.0, -math.inf
                continue
            K, V = keys[b][:L][seen], values[b][:L][seen]
            K = K.repeat_interleave(Hq // Hk, 1)
            V = V.repeat_interleave(Hq // Hk, 1)
            x = q[first + i].to(F64)
            s = torch.einsum("hd,thd->ht", x, K) * scale
            # scores: D products and sums of 24 bits, then a product and exp2's argument, times 2
            off = 2 * (D + 4) * 2.0 ** -24 * (torch.einsum("hd,thd->ht", x.abs(), K.abs()) * abs(scale))
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                # relative: with h = 2^-24 for a rounding, fewer than 32 of them.  Up to c / 4 tanh's series: 7 with
                # constants and factors.  Above, 1 - 2 / (e + 1): x is off by 2, 2 |x| log2 e by 2 more, so e by 8 |x|
                # and exp2's 2, which sum and reciprocal take times e / (e + 1) and add 3: 5.5 at c / 4, times
                # 2 / (e - 1) = 3.1, less farther on; then 4 with c log2 e
                off = off + (s.abs() * 2.0 ** -19 if relative else softcap * 2.0 ** -21)
            off = off + 2.0 ** -22 * (s.abs() + 1)
            off = off.amax(1, keepdim=True)                      # [Hq, 1]
            e = torch.softmax(s, 1)
            out[first + i] = torch.einsum("ht,thd->hd", e, V)
            size = torch.einsum("ht,thd->hd", e, V.abs())
            count = K.shape[0]
            # the output's rounding, the weights', the scores', the sums'
            bound[first + i] = u * out[first + i].abs() + (u + 2 * off + 2 * count * 2.0 ** -24 + 2.0 ** -21) * size \
                + count * 2.0 ** -34 * V.abs().amax(0) + torch.finfo(q.dtype).tiny
            lse[first + i] = torch.logsumexp(s, 1)
            lse_bound[first + i] = off[:, 0] + count * 2.0 ** -23 + 2.0 ** -21 * (1 + lse[first + i].abs())
    return out, lse, bound, lse_bound

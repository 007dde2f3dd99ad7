"""Cases and plain forms of the rotary positions, of writing and reading a key/value cache held in 4 bits, and of
attention over that cache.

``run`` computes an operator in elementary torch operations, or, where ``own`` is true, calls this package's kernel
for it on the same inputs.

The cache is uint8 [pages, heads, page_size (D + D / 16)]. For each page and head it holds the keys' codes
[page_size, D / 2], the values' codes, the keys' scales [D / 32, page_size] and the values' scales. A code is four
bits (e2m1; channel 2 j is the low half of byte j), a scale one byte e + 127 for 32 channels: value = code 2^e. Byte 255
stands for NaN.
"""
import math
import random

import torch

own = False

F32, F64 = torch.float32, torch.float64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# exponents of the scales whose whole grid the type holds
EXPONENTS = {"bf16": (-125, 125), "f16": (-23, 13)}


# ------------------------------------------------------------------ cases --

def listed():
    """40 query heads of 128 channels are the package's width 5120; T = 4, 4160 and 16384 are its workloads' tokens; the
    rest is generic."""
    return [
        # a decode step's four tokens, far along in their sequences
        rope_case("rope_decode", T=4, Hq=40, Hk=8, D=128, R=128, dtype="bf16", order="one", far=1 << 20),
        # the gradient of a vision encoder's rotation: rows and columns, neighbouring pairs, no key heads beside it
        rope_case("rope_image_back", T=4160, Hq=16, Hk=0, D=96, R=96, dtype="f16", order="blocks2", far=128,
                  interleaved=True, inverse=True),
        # a long prefill of text, images and video: time, height and width in turn, scaled, heads inside a qkv product
        rope_case("rope_prefill", T=16384, Hq=40, Hk=8, D=128, R=128, dtype="bf16", order="cyclic3", far=1 << 15,
                  scale=1.2, fused=True),
        # a decode step of 64 sequences, some of them padding
        cache_case("write_decode", "write", T=64, H=8, D=128, ps=64, dtype="bf16", skip=0.1),
        # a long prefill's keys and values, inside the qkv product's rows
        cache_case("write_prefill", "write", T=16384, H=8, D=128, ps=64, dtype="bf16", fused=True),
        # a short prefix taken back out, odd sizes, some slots empty
        cache_case("read_ragged", "read", T=1037, H=3, D=64, ps=48, dtype="f16", skip=0.1),
        # long prefixes taken back out
        cache_case("read_prefix", "read", T=131072, H=8, D=128, ps=64, dtype="bf16"),
        # one token of one sequence: latency
        attend_case("attend_token", B=1, Q=1, L=1003, Hq=16, Hk=2, D=64, ps=16, dtype="bf16"),
        # a decode step of 64 ragged sequences, five query heads to a key head
        attend_case("attend_decode", B=64, Q=1, L=8192, Hq=40, Hk=8, D=128, ps=64, dtype="bf16"),
        # drafted tokens under a sliding window with capped scores, wide heads
        attend_case("attend_draft", B=16, Q=5, L=4099, Hq=8, Hk=4, D=256, ps=32, dtype="f16", softcap=30.0, window=1024),
        # two very long sequences, with the logarithm of the sums that another part's result is joined by
        attend_case("attend_long", B=2, Q=1, L=131071, Hq=32, Hk=4, D=128, ps=256, dtype="f16", lse=True),
        # a chunk of a long prompt behind what its cache holds already
        attend_case("attend_chunk", B=1, Q=4096, L=16384, Hq=40, Hk=8, D=128, ps=64, dtype="bf16"),
    ]


def named(name, c):
    return dict(c, name=name) if name else c


def rope_case(name, T, Hq, Hk, D, R, dtype, order, far, interleaved=False, inverse=False, scale=1.0, fused=False):
    return named(name, {"op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "dtype": dtype, "order": order,
                        "far": far, "interleaved": interleaved, "inverse": inverse, "scale": scale, "fused": fused})


def cache_case(name, op, T, H, D, ps, dtype, skip=0.0, fused=False):
    return named(name, {"op": op, "T": T, "H": H, "D": D, "ps": ps, "dtype": dtype, "skip": skip, "fused": fused})


def attend_case(name, B, Q, L, Hq, Hk, D, ps, dtype, softcap=0.0, window=0, causal=True, lse=False):
    return named(name, {"op": "attend", "B": B, "Q": Q, "L": L, "Hq": Hq, "Hk": Hk, "D": D, "ps": ps, "dtype": dtype,
                        "softcap": softcap, "window": window, "causal": causal, "lse": lse})


def spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("rope", "write", "read", "attend", "attend", "attend"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "rope":
        D = rng.choice((64, 80, 96, 128, 128, 256))
        Hq = spread(rng, 1, 48)
        Hk = rng.choice((0, Hq, spread(rng, 1, Hq)))
        return rope_case(None, spread(rng, 1, min(16384, 16384 * 48 * 128 // ((Hq + Hk) * D))), Hq, Hk, D,
                         rng.choice((D, D, D // 2, D // 4)), dtype, rng.choice(("one", "blocks2", "blocks3", "cyclic3")),
                         spread(rng, 16, 1 << 20), rng.random() < 0.4, rng.random() < 0.4, rng.choice((1.0, 1.2)),
                         rng.random() < 0.5)
    if op != "attend":
        D, H = rng.choice((64, 128, 128, 256)), spread(rng, 1, 32)
        most = (16384 if op == "write" else 131072) * 8 * 128 // (H * D)
        return cache_case(None, op, spread(rng, 1, min(131072, most)), H, D, rng.choice((16, 48, 64, 256)), dtype,
                          rng.choice((0.0, 0.1)), rng.random() < 0.5)
    D, Hk, group = rng.choice((64, 128, 128, 256)), spread(rng, 1, 16), rng.choice((1, 2, 4, 5, 8, 16))
    B = spread(rng, 1, 64)
    kind = rng.choice(("token", "token", "draft", "chunk"))
    # what the listed decode step reads, and what the listed chunk computes, over the batch
    L = spread(rng, 1, min(131072, 64 * 8192 * 8 * 128 // (B * Hk * D)))
    Q = 1 if kind == "token" else rng.randint(2, 8)
    if kind == "chunk":
        L = min(L, 16384)
        Q = spread(rng, 1, max(1, min(4096, L, 4096 * 16384 * 40 * 128 // (B * L * Hk * group * D))))
    return attend_case(None, B, Q, max(L, Q), Hk * group, Hk, D, rng.choice((16, 48, 64, 256)), dtype,
                       rng.choice((0.0, 0.0, 30.0)), rng.choice((0, 0, 1000)), rng.random() < 0.85, rng.random() < 0.3)


def lengths(case):
    """Query rows and cached tokens of each sequence: the case's own, whatever the seed."""
    rng = random.Random("%(B)d %(Q)d %(L)d" % case)
    rows, lens = [case["Q"]], [case["L"]]           # the longest one stands first
    for _ in range(case["B"] - 1):
        rows.append(case["Q"] if case["Q"] <= 8 else spread(rng, 1, case["Q"]))
        lens.append(max(rows[-1], spread(rng, max(1, case["L"] // 8), case["L"])))
    return rows, lens


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=F32)

    s, dt, D = dict(case), DTYPES[case["dtype"]], case["D"]

    def heads(T, counts, fused):
        """Tensors [T, H, D], apart or side by side in the rows of one product."""
        if not fused:
            return [normal(T, H, D).to(dt) for H in counts]
        rows = normal(T, sum(counts) * D).to(dt)
        return [r.view(T, H, D) for r, H in zip(rows.split([H * D for H in counts], 1), counts)]

    if case["op"] == "rope":
        T, pairs = case["T"], case["R"] // 2
        s["q"], s["k"] = heads(T, [case["Hq"], case["Hk"]], case["fused"])
        if not case["Hk"]:
            s["k"] = None
        n = {"one": 1, "blocks2": 2, "blocks3": 3, "cyclic3": 3}[case["order"]]
        start = torch.randint(0, case["far"], (n, 1), generator=g, device="cuda")
        step = torch.randint(0, 3, (n, T), generator=g, device="cuda")
        s["positions"] = (start + step.cumsum(1)).to(torch.int32)
        s["axes"] = None if n == 1 else tuple(i % n if "cyclic" in case["order"] else i * n // pairs
                                              for i in range(pairs))
        s["axis_of"] = torch.tensor(s["axes"] or [0] * pairs, device="cuda")
        base = torch.arange(pairs, device="cuda", dtype=F64) / pairs
        s["inv_freq"] = (10000.0 ** -base).to(F32)
        return s

    # keys have a few loud channels, values none
    loud = 1.0 + 8.0 * (torch.rand(D, generator=g, device="cuda") < 0.03)
    ps, lo_hi = case["ps"], EXPONENTS[case["dtype"]]
    if case["op"] != "attend":
        T, H = case["T"], case["H"]
        pages = -(-T // ps) + 2                     # the last one is nobody's
        slots = torch.arange((pages - 1) * ps, device="cuda").view(-1, ps)
        order = torch.randperm(pages - 1, generator=g, device="cuda")
        slots = slots[order].flatten()[:T]
        if case["skip"]:
            slots = slots.masked_fill(torch.rand(T, generator=g, device="cuda") < case["skip"], -1)
        s["slots"] = slots
        k, v = heads(T if case["op"] == "write" else pages * ps, [H, H], case["fused"])
        if case["op"] == "write":
            s["k"], s["v"] = k, v
            s["k"].mul_(loud.to(dt))
            s["cache"] = torch.zeros(pages, H, ps * (D + D // 16), dtype=torch.uint8, device="cuda")
        else:
            s["cache"] = packed((k * loud).to(dt), v, pages, ps, lo_hi)
        return s

    B, Hk = case["B"], case["Hk"]
    rows, lens = lengths(case)
    most = -(-case["L"] // ps)
    pages = sum(-(-n // ps) for n in lens) + 1
    s["cache"] = torch.empty(pages, Hk, ps * (D + D // 16), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (ps * Hk * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        s["cache"][at:at + n] = packed(normal(n * ps, Hk, D) * loud, normal(n * ps, Hk, D), n, ps, lo_hi)
    order = torch.randperm(pages - 1, generator=g, device="cuda").to(torch.int32)
    s["tables"] = torch.full((B, most), pages - 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        n = -(-n // ps)
        s["tables"][b, :n] = order[at:at + n]
        at += n
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    s["q_starts"] = None if case["Q"] == 1 else torch.tensor(starts, dtype=torch.int32, device="cuda")
    # queries lean on the keys' loud channels as much as on the others
    s["q"] = (1.5 * normal(starts[-1], case["Hq"], D) / loud).to(dt)
    return s


def run(s):
    if own:
        return run_own(s)
    return {"rope": plain_rope, "write": plain_write, "read": plain_read, "attend": plain_attend}[s["op"]](s)


def run_own(s):
    from layer_mhc_seam_amd import seam
    if s["op"] == "rope":
        q, k = seam.rope(s["q"], s["k"], s["positions"], s["inv_freq"], axes=s["axes"], interleaved=s["interleaved"],
                         inverse=s["inverse"], scale=s["scale"])
        return {"q": q} if k is None else {"q": q, "k": k}
    if s["op"] == "attend":
        r = seam.cache_attention(s["q"], s["cache"], s["tables"], s["lens"], q_starts=s["q_starts"], causal=s["causal"],
                                 window=s["window"], softcap=s["softcap"], lse=s["lse"])
        return {"out": r[0], "lse": r[1]} if s["lse"] else {"out": r}
    if s["op"] == "write":
        seam.cache_write(s["cache"], s["k"], s["v"], s["slots"])
    k, v = seam.cache_read(s["cache"], s["slots"], s["D"], dtype=s["dtype"])
    return {"k": k, "v": v}


# ------------------------------------------------------------ plain forms --

def plain_rope(s):
    # angles in 64 bits: a far position times a frequency has more than 24 of them before the point
    at = s["positions"].to(F64)                                             # [A, T]
    angle = at[s["axis_of"]].t() * s["inv_freq"].to(F64)                    # [T, pairs]
    c, n = torch.cos(angle).to(F32)[:, None], torch.sin(angle).to(F32)[:, None]
    n = -n if s["inverse"] else n
    return {name: turned(s[name], c, n, s) for name in ("q", "k") if s[name] is not None}


def turned(x, c, n, s):
    R, x32 = s["R"], x.to(F32)
    if s["interleaved"]:
        a, b = x32[..., 0:R:2], x32[..., 1:R:2]
    else:
        a, b = x32[..., :R // 2], x32[..., R // 2:R]
    a, b = s["scale"] * (a * c - b * n), s["scale"] * (b * c + a * n)
    r = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((r, x32[..., R:]), -1).to(x.dtype)


def power(e):
    """2^e in 32 bits for whole e from -126 to 127, by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(F32)


def quantized(x, lo_hi):
    """Codes [..., D / 2] and scales [..., D / 32] of [..., D]: the smallest exponent at which 6 reaches the group's
    largest, within the type's; the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    v = x.to(F32).unflatten(-1, (-1, 32))
    most = v.abs().amax(-1)
    fine = torch.isfinite(most)
    mantissa, e = torch.frexp(torch.where(fine, most, torch.zeros_like(most)))
    e = e - 2 - (mantissa <= 0.75).to(e.dtype)
    e = torch.where(most == 0, torch.full_like(e, lo_hi[0]), e).clamp(*lo_hi)
    y = (v * power(-e)[..., None]).abs().clamp(max=6.0)
    # two whole steps a binade: codes count them
    code = torch.where(y < 2, torch.round(2 * y), torch.where(y < 4, torch.round(y) + 2, torch.round(y / 2) + 4))
    code = (code + 8 * torch.signbit(v)).masked_fill(~fine[..., None], 0).to(torch.uint8).flatten(-2)
    scale = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def packed(k, v, pages, ps, lo_hi):
    """A cache of those pages whose slots hold k and v [pages ps, H, D] in order."""
    parts = []
    for x in (k, v):
        codes, scales = quantized(x.unflatten(0, (pages, ps)).transpose(1, 2), lo_hi)     # [pages, H, ps, ..]
        parts.append((codes.flatten(2), scales.transpose(2, 3).flatten(2)))
    return torch.cat((parts[0][0], parts[1][0], parts[0][1], parts[1][1]), 2)


def views(cache, D):
    """(codes [pages, H, ps, D / 2], scales [pages, H, D / 32, ps]) of the keys and of the values, in place."""
    ps = cache.shape[2] // (D + D // 16)
    c, s = ps * D // 2, ps * D // 32
    at = (0, c, 2 * c, 2 * c + s, 2 * c + 2 * s)
    part = [cache[:, :, at[i]:at[i + 1]] for i in range(4)]
    return ps, [(part[i].unflatten(2, (ps, D // 2)), part[2 + i].unflatten(2, (D // 32, ps))) for i in range(2)]


def values(codes, scales):
    """32-bit values [..., D] of codes [..., D / 2] and scales [..., D / 32]."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int64)
    grid = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), device=codes.device)
    v = torch.cat((grid, -grid))[code].unflatten(-1, (-1, 32))
    e = scales.to(torch.int32) - 127
    v = v * power(e.clamp(-126, 127))[..., None]
    return torch.where((scales == 255)[..., None], torch.full_like(v, math.nan), v).flatten(-2)


def plain_write(s):
    ps, parts = views(s["cache"], s["D"])
    slots = s["slots"]
    to = torch.where(slots < 0, s["cache"].shape[0] * ps - 1, slots)       # a slot that is nobody's
    page, at = to // ps, to % ps
    for x, (codes, scales) in zip((s["k"], s["v"]), parts):
        c, e = quantized(x, EXPONENTS[s["dtype"]])
        codes[page, :, at] = c
        scales[page, :, :, at] = e
    return plain_read(s)


def plain_read(s):
    ps, parts = views(s["cache"], s["D"])
    slots, out = s["slots"], []
    from_ = slots.clamp(min=0)
    page, at = from_ // ps, from_ % ps
    none = (slots < 0)[:, None, None]
    for codes, scales in parts:
        out.append(values(codes[page, :, at], scales[page, :, :, at]).masked_fill(none, 0.0).to(DTYPES[s["dtype"]]))
    return {"k": out[0], "v": out[1]}


def plain_attend(s):
    B, Q, L, Hk, D = s["B"], s["Q"], s["L"], s["Hk"], s["D"]
    G, dev = s["Hq"] // Hk, s["q"].device
    ps, parts = views(s["cache"], D)
    t = torch.arange(L, device=dev)
    page = s["tables"][:, t // ps].long()                                   # [B, L]
    k, v = (values(codes[page, :, t % ps], scales[page, :, :, t % ps]).transpose(1, 2) for codes, scales in parts)
    # queries padded to Q rows a sequence
    starts = s["q_starts"] if s["q_starts"] is not None else torch.arange(B + 1, device=dev)
    n = (starts[1:] - starts[:-1])[:, None]
    i = torch.arange(Q, device=dev)
    at = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"].to(F32)[at].view(B, Q, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * Q, D)
    score = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
    if s["softcap"]:
        score = s["softcap"] * torch.tanh(score / s["softcap"])
    last = s["lens"][:, None] - n + i if s["causal"] else (s["lens"][:, None] - 1).expand(B, Q)
    seen = (t <= last[..., None]) & (t < s["lens"][:, None, None])          # [B, Q, L]
    if s["window"]:
        seen = seen & (t > (s["lens"][:, None] - n + i)[..., None] - s["window"])
    score = score.view(B, Hk, G, Q, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hk, G * Q, L), v).view(B, Hk, G, Q, D)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1)
    # back to the rows there are: row r is row r - start of the last sequence that starts at or before it
    r = torch.arange(s["q"].shape[0], device=dev)
    b = (torch.searchsorted(starts, r.to(starts.dtype), right=True) - 1).long()
    j = r - starts[b]
    out = out[b, :, :, j].flatten(1, 2).to(s["q"].dtype)
    return {"out": out, "lse": lse[b, :, :, j].flatten(1, 2)} if s["lse"] else {"out": out}


# ------------------------------------------------------------------- work --

def work(case):
    D = case["D"]
    if case["op"] == "rope":
        H = case["Hq"] + case["Hk"]
        n = 1 if case["order"] == "one" else 2 if case["order"] == "blocks2" else 3
        return {"bytes": 4 * case["T"] * H * D + 4 * n * case["T"] + 2 * case["R"],
                "flops": 4 * case["T"] * H * case["R"]}
    if case["op"] != "attend":
        each = case["T"] * case["H"]
        # written and then read, or read: values of two bytes, codes with their scales
        passes = 2 if case["op"] == "write" else 1
        return {"bytes": passes * (each * (4 * D + D + D // 16) + 8 * case["T"]), "flops": passes * 4 * each * D}
    rows, lens = lengths(case)
    pairs = kept = 0
    for n, L in zip(rows, lens):
        reach = case["window"] or L
        if case["causal"]:
            pairs += sum(min(L - n + i + 1, reach) for i in range(n))
        else:
            pairs += sum(L - max(0, L - n + i + 1 - reach) for i in range(n))
        kept += min(L, n - 1 + reach)
    return {"bytes": kept * case["Hk"] * (D + D // 16) + 4 * sum(rows) * case["Hq"] * D
            + 4 * case["lse"] * sum(rows) * case["Hq"] + 4 * sum(-(-n // case["ps"]) for n in lens),
            "flops": 4 * pairs * case["Hq"] * D}


# ------------------------------------------------------------------ exact --
# From the definitions in 64 bits.

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": exact_rope, "write": exact_write, "read": exact_read, "attend": exact_attend}[case["op"]](s)


def exact_rope(s):
    T, R = s["T"], s["R"]
    angle = torch.empty(T, R // 2, dtype=F64, device="cuda")
    for i in range(R // 2):
        angle[:, i] = s["positions"][0 if s["axes"] is None else s["axes"][i]].double() * s["inv_freq"][i].double()
    turn = torch.polar(torch.full_like(angle, s["scale"]), -angle if s["inverse"] else angle).unsqueeze(1)
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        x = s[name].double()
        if s["interleaved"]:
            z = torch.view_as_complex(x[..., :R].reshape(T, -1, R // 2, 2).contiguous()) * turn
            x[..., 0:R:2], x[..., 1:R:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
            x[..., :R // 2], x[..., R // 2:R] = z.real, z.imag
        out[name] = x
    return out


def exact_write(s):
    lo, hi = EXPONENTS[s["dtype"]]
    grid = torch.tensor(GRID, dtype=F64, device="cuda")
    none = (s["slots"] < 0)[:, None, None]
    out = {}
    for name in ("k", "v"):
        x = s[name].double()
        group = x.reshape(*x.shape[:-1], -1, 32)
        most = group.abs().max(-1, keepdim=True).values
        e = torch.full_like(most, float(lo))
        for k in range(lo, hi):                     # up while 6 2^k does not reach
            e = torch.where(most > 6.0 * 2.0 ** k, k + 1.0, e)
        unit = torch.pow(torch.full_like(e, 2.0), e)
        y = (group.abs() / unit).clamp_max(6.0)
        below = (torch.searchsorted(grid, y.contiguous(), right=True) - 1).clamp(0, 7)
        above = (below + 1).clamp_max(7)
        down, up = y - grid[below], grid[above] - y
        code = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
        q = torch.copysign(grid[code] * unit, group).reshape(x.shape)
        out[name] = torch.where(none, 0.0, q)
    return out


def exact_rows(cache, D, slots):
    """Keys and values [n, H, D] of those slots, none of them negative."""
    ps = cache.shape[2] * 16 // (17 * D)
    half, few = ps * D // 2, ps * D // 32
    page, at = slots // ps, slots % ps
    rows = cache[page]                              # [n, H, bytes]
    H = rows.shape[1]
    out = []
    for kind in range(2):
        byte = kind * half + at[:, None] * (D // 2) + torch.arange(D // 2, device="cuda")
        code = rows.gather(2, byte[:, None].expand(-1, H, -1)).long()
        byte = 2 * half + kind * few + torch.arange(D // 32, device="cuda") * ps + at[:, None]
        scale = rows.gather(2, byte[:, None].expand(-1, H, -1)).double()
        code = torch.stack((code % 16, code // 16), 3).reshape(len(slots), H, D)
        v = torch.tensor(GRID, dtype=F64, device="cuda")[code % 8] * (1 - 2 * (code // 8)).double()
        out.append(v * torch.exp2(scale - 127).repeat_interleave(32, 2))
    return out


def exact_read(s):
    out = {"k": [], "v": []}
    for part in s["slots"].split(4096):
        rows = exact_rows(s["cache"], s["D"], torch.where(part < 0, 0, part))
        for name, x in zip(("k", "v"), rows):
            out[name].append(torch.where((part < 0)[:, None, None], 0.0, x))
    return {name: torch.cat(x) for name, x in out.items()}


def exact_attend(s):
    """One sequence and one key head at a time, its keys in pieces."""
    rows, lens = lengths(s)
    D, Hk, G = s["D"], s["Hk"], s["Hq"] // s["Hk"]
    out = torch.empty(sum(rows), s["Hq"], D, dtype=F64, device="cuda")
    lse = torch.empty(sum(rows), s["Hq"], dtype=F64, device="cuda")
    first = 0
    for b, (n, L) in enumerate(zip(rows, lens)):
        t = torch.arange(L, device="cuda")
        slots = s["tables"][b].long()[t // s["ps"]] * s["ps"] + t % s["ps"]
        pieces = [exact_rows(s["cache"], D, part) for part in slots.split(4096)]
        K, V = (torch.cat([p[i] for p in pieces]) for i in range(2))
        place = torch.arange(L - n, L, device="cuda")[:, None]
        hidden = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        if s["causal"]:
            hidden |= t > place
        if s["window"]:
            hidden |= t <= place - s["window"]
        for h in range(Hk):
            q = s["q"][first:first + n, h * G:h * G + G].double()           # [n, G, D]
            for j in range(G):
                x = q[:, j] @ K[:, h].t() / math.sqrt(D)
                if s["softcap"]:
                    x = torch.tanh(x / s["softcap"]) * s["softcap"]
                x = x.masked_fill(hidden, -math.inf)
                out[first:first + n, h * G + j] = torch.softmax(x, 1) @ V[:, h]
                lse[first:first + n, h * G + j] = torch.logsumexp(x, 1)
        first += n
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}

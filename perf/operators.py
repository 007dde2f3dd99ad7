"""Cases and plain forms of the one-stream block norm, the int8 quantiser, the int8 product and the expert router.

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, calls this package's kernel for it on the same inputs.
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
TINY = 2.0 ** -119          # the int8 quantiser's smallest row maximum


# ------------------------------------------------------------------ cases --

def listed():
    """The sizes are the package's own workloads (T = 1, 4, 384, 4160, 16384
    at H = 5120, the width 7168 of its tests) and generic odd ones."""
    return [
        # a decode step's boundary: four tokens, LayerScale-like gate, int8 operand for the next product
        norm_case("norm_decode", T=4, H=5120, dtype="bf16", x_dtype="bf16", post=True, gate="channel", int8=True),
        # a prompt's boundary with an fp32 residual stream, fp16 activations, a scalar gate for each token, no
        # normalisation of the block's output
        norm_case("norm_f32_stream", T=384, H=7168, dtype="f16", x_dtype="f32", post=False, gate="token", int8=False),
        # a long prefill: norms on both sides, a gate for each element, norm and int8 operand both written
        norm_case("norm_prefill", T=16384, H=5120, dtype="bf16", x_dtype="bf16", post=True, gate="element", int8=True),
        # the int8 operand of an activation of odd row count and of a width that is no multiple of a vector
        {"name": "quant_ragged", "op": "quant", "T": 1037, "H": 1027, "dtype": "f16"},
        # the int8 operand of the four-stream seam's norm at its prefill workload
        {"name": "quant_prefill", "op": "quant", "T": 16384, "H": 5120, "dtype": "bf16"},
        # a projection of one token: the weights' bytes
        {"name": "gemm_token", "op": "gemm", "T": 1, "N": 5120, "K": 5120, "out": "bf16", "bias": False},
        # a prompt's projection, odd column count, depth that ends inside a tile, with a bias
        {"name": "gemm_prompt_odd", "op": "gemm", "T": 384, "N": 5117, "K": 5136, "out": "f16", "bias": True},
        # expert logits of a prefill in fp32
        {"name": "gemm_logits", "op": "gemm", "T": 4160, "N": 256, "K": 5120, "out": "f32", "bias": False},
        # a projection of a long prefill: the matrix cores
        {"name": "gemm_prefill", "op": "gemm", "T": 16384, "N": 5120, "K": 5120, "out": "bf16", "bias": False},
        # a decode step's choice among 256 experts in 8 groups
        route_case("route_decode", T=4, E=256, k=8, dtype="f32", scoring="sigmoid", bias=True, groups=8, keep=4, top=2),
        # a prefill chunk's choice among experts without groups, bf16 logits (many exact ties), some experts masked
        route_case("route_softmax", T=4160, E=160, k=6, dtype="bf16", scoring="softmax", bias=False, masked=True),
        # a long prefill's choice with the balance bias and groups
        route_case("route_prefill", T=16384, E=256, k=8, dtype="f32", scoring="sigmoid", bias=True, groups=8, keep=4,
                   top=2),
    ]


def norm_case(name, T, H, dtype, x_dtype, post, gate, int8):
    c = {"op": "norm", "T": T, "H": H, "dtype": dtype, "x_dtype": x_dtype, "post": post, "gate": gate, "int8": int8}
    return dict(c, name=name) if name else c


def route_case(name, T, E, k, dtype, scoring, bias, groups=1, keep=1, top=1, masked=False):
    c = {"op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "scoring": scoring, "bias": bias, "groups": groups,
         "keep": keep, "top": top, "masked": masked}
    return dict(c, name=name) if name else c


def spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def width(rng, lo, hi):
    """A row width: a multiple of 64, of 8, or any."""
    w = spread(rng, lo, hi)
    m = rng.choice((64, 64, 8, 1))
    return max(lo, w // m * m)


def draw(rng):
    op = rng.choice(("norm", "quant", "gemm", "gemm", "route"))
    if op == "norm":
        H = width(rng, 64, 8192)
        T = spread(rng, 1, 16384 * 5120 // max(H, 5120))
        dtype = rng.choice(("bf16", "bf16", "f16"))
        return norm_case(None, T, H, dtype, rng.choice((dtype, dtype, "f32")), rng.random() < 0.6,
                         rng.choice(("none", "token", "channel", "element")), rng.random() < 0.5)
    if op == "quant":
        H = width(rng, 64, 8192)
        return {"op": "quant", "T": spread(rng, 1, 16384 * 5120 // max(H, 5120)), "H": H,
                "dtype": rng.choice(("bf16", "f16"))}
    if op == "gemm":
        K = spread(rng, 64, 8192) // 16 * 16
        N = width(rng, 16, 8192)
        T = spread(rng, 1, min(16384, 16384 * 5120 * 5120 // (max(N, 2560) * max(K, 2560))))
        return {"op": "gemm", "T": T, "N": N, "K": K, "out": rng.choice(("bf16", "bf16", "f16", "f32")),
                "bias": rng.random() < 0.3}
    groups = rng.choice((1, 1, 4, 8))
    E = groups * spread(rng, 8, 512 // groups)
    keep = rng.randint(1, groups)
    k = rng.randint(1, min(10, E // groups * keep))
    return route_case(None, spread(rng, 1, 16384), E, k, rng.choice(("f32", "bf16", "f16")),
                      rng.choice(("softmax", "sigmoid")), rng.random() < 0.6, groups, keep,
                      rng.choice((1, 2)) if groups > 1 else 1, rng.random() < 0.3)


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=F32)

    s = dict(case)
    T = case["T"]
    if case["op"] == "norm":
        H, dt = case["H"], DTYPES[case["dtype"]]
        # a residual stream grows with depth and has a few loud channels
        loud = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.003)
        s["x"] = (4.0 * normal(T, H) * loud).to(DTYPES[case["x_dtype"]])
        s["y"] = normal(T, H).to(dt)
        s["gamma"] = (1.0 + 0.1 * normal(H)).to(dt)
        s["gamma_post"] = (1.0 + 0.1 * normal(H)).to(dt) if case["post"] else None
        s["gate"] = {"none": lambda: None,
                     "token": lambda: torch.sigmoid(normal(T, 1)),
                     "channel": lambda: 0.5 + 0.1 * normal(H),
                     "element": lambda: torch.sigmoid(normal(T, H)).to(dt)}[case["gate"]]()
        s["residual_scale"], s["branch_scale"] = 1.0, 0.22
    elif case["op"] == "quant":
        s["x"] = (normal(T, case["H"]) * torch.exp(normal(T, 1))).to(DTYPES[case["dtype"]])
    elif case["op"] == "gemm":
        N, K = case["N"], case["K"]
        # codes of Gaussian rows: their largest is 127, their deviation about a quarter of it
        s["a"] = (32.0 * normal(T, K)).round().clamp(-127, 127).to(torch.int8)
        s["b"] = (32.0 * normal(N, K)).round().clamp(-127, 127).to(torch.int8)
        s["a_scales"] = 0.03 * torch.exp(0.3 * normal(T))
        s["b_scales"] = 0.03 / math.sqrt(K) * torch.exp(0.3 * normal(N))
        s["bias_vec"] = normal(N) if case["bias"] else None
    else:
        E = case["E"]
        l = 1.5 * normal(T, E)
        if case["masked"]:
            # experts out of reach, another share in each row; some rows keep fewer than k, some none
            share = torch.rand(T, 1, generator=g, device="cuda")
            share = torch.where(share > 0.97, torch.ones_like(share), 0.5 * share)
            l = l.masked_fill(torch.rand(T, E, generator=g, device="cuda") < share, -math.inf)
        s["logits"] = l.to(DTYPES[case["dtype"]])
        s["bias_vec"] = 0.05 * normal(E) if case["bias"] else None
        s["scale"] = 2.5 if case["scoring"] == "sigmoid" else 1.0
    return s


def run(s):
    if own:
        return run_own(s)
    return {"norm": plain_norm, "quant": plain_quant, "gemm": plain_gemm, "route": plain_route}[s["op"]](s)


def run_own(s):
    from layer_mhc_seam_amd import seam
    if s["op"] == "norm":
        return seam.block_norm(s["x"], s["gamma"], s["y"], gamma_post=s["gamma_post"], gate=s["gate"],
                               residual_scale=s["residual_scale"], branch_scale=s["branch_scale"], eps=EPS,
                               int8=s["int8"])
    if s["op"] == "quant":
        codes, scales = seam.int8_quantize(s["x"])
        return {"codes": codes, "scales": scales}
    if s["op"] == "gemm":
        return seam.int8_gemm(s["a"], s["a_scales"], s["b"], s["b_scales"], s["bias_vec"], out_dtype=s["out"])
    weights, ids = seam.route(s["logits"], s["k"], scoring=s["scoring"], bias=s["bias_vec"], groups=s["groups"],
                              topk_groups=s["keep"], group_top=s["top"], scale=s["scale"])
    return {"weights": weights, "ids": ids}


# ------------------------------------------------------------ plain forms --
# Statistics and choices are held in 64 bits: a norm's last bit decides on
# which side of a code's border a value falls, and a score's last bit which of
# two experts is chosen.

def rstd(v):
    return (1.0 / torch.sqrt(v.to(F64).square().mean(-1, keepdim=True) + EPS)).to(F32)


def plain_codes(v):
    v = v.to(F32)
    amax = v.abs().amax(-1, keepdim=True)
    a = amax.clamp_min(TINY)
    # quotients of two tensors: one with a plain number is taken by way of a reciprocal, which is rounded twice
    most = torch.full_like(a, 127.0)
    codes = torch.round(v * (most / a))
    fine = torch.isfinite(amax)
    codes = torch.where(fine, codes, torch.zeros_like(codes)).to(torch.int8)
    return codes, torch.where(fine, a / most, torch.full_like(a, math.nan)).squeeze(-1)


def plain_norm(s):
    p = s["y"].to(F32)
    if s["gamma_post"] is not None:
        p = p * rstd(p) * s["gamma_post"].to(F32)
    if s["gate"] is not None:
        p = p * s["gate"].to(F32)
    r = (s["residual_scale"] * s["x"].to(F32) + s["branch_scale"] * p).to(s["x"].dtype)
    v = r.to(F32)
    norm = (v * rstd(v) * s["gamma"].to(F32)).to(s["y"].dtype)
    out = {"residual_out": r, "norm": norm}
    if s["int8"]:
        out["codes"], out["scales"] = plain_codes(norm)
    return out


def plain_quant(s):
    codes, scales = plain_codes(s["x"])
    return {"codes": codes, "scales": scales}


def plain_gemm(s):
    # whole numbers below 2^24 in practice: exact in 32 bits
    r = (s["a"].to(F32) @ s["b"].to(F32).t()) * s["a_scales"][:, None] * s["b_scales"]
    if s["bias_vec"] is not None:
        r = r + s["bias_vec"]
    return r.to(DTYPES[s["out"]])


def plain_route(s):
    l = s["logits"].to(F64)
    masked = l == -math.inf
    if s["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(-1, keepdim=True)
        e = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = e.sum(-1, keepdim=True)
        score = e / torch.where(total == 0, torch.ones_like(total), total)
    key = score if s["bias_vec"] is None else score + s["bias_vec"].to(F64)
    key = key.masked_fill(masked, -math.inf)
    if s["groups"] > 1:
        T, E = key.shape
        by_group = key.view(T, s["groups"], E // s["groups"])
        of_group = by_group.sort(dim=-1, descending=True, stable=True).values[..., :s["top"]]
        of_group = of_group.masked_fill(of_group == -math.inf, -1e30).sum(-1)
        kept = of_group.sort(dim=-1, descending=True, stable=True).indices[:, :s["keep"]]
        open_ = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, kept, True)
        key = by_group.masked_fill(~open_[..., None], -math.inf).view(T, E)
    order = key.sort(dim=-1, descending=True, stable=True)
    ids, none = order.indices[:, :s["k"]], order.values[:, :s["k"]] == -math.inf
    w = score.gather(1, ids).masked_fill(none, 0.0)
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total == 0, torch.ones_like(total), total) * s["scale"]
    return {"weights": w.to(F32), "ids": ids.masked_fill(none, -1).to(torch.int32)}


# ------------------------------------------------------------------- work --

def work(case):
    T = case["T"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "norm":
        H, e, x = case["H"], size[case["dtype"]], size[case["x_dtype"]]
        gate = {"none": 0, "token": 4 * T, "channel": 4 * H, "element": T * H * e}[case["gate"]]
        return {"bytes": T * H * (2 * x + 2 * e) + gate + H * e * (1 + case["post"]) + case["int8"] * T * (H + 4),
                "flops": T * H * (8 + 4 * case["post"] + 3 * case["int8"])}
    if case["op"] == "quant":
        return {"bytes": T * case["H"] * (size[case["dtype"]] + 1) + 4 * T, "flops": 3 * T * case["H"]}
    if case["op"] == "gemm":
        N, K = case["N"], case["K"]
        return {"bytes": T * K + N * K + T * N * size[case["out"]] + 4 * (T + N * (1 + case["bias"])),
                "flops": 2 * T * N * K}
    return {"bytes": T * case["E"] * size[case["dtype"]] + 8 * T * case["k"] + 4 * case["E"] * case["bias"],
            "flops": 8 * T * case["E"]}


# ------------------------------------------------------------------ exact --
# From the definitions in 64 bits, without the roundings to 8 or 16 bits on
# the way. Codes and ids are whole numbers and have no such value.

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    if case["op"] == "norm":
        branch = d["y"]
        if d["gamma_post"] is not None:
            ms = torch.einsum("th,th->t", branch, branch) / case["H"]
            branch = branch * (ms + EPS).rsqrt().unsqueeze(1) * d["gamma_post"]
        if d["gate"] is not None:
            branch = branch * d["gate"]
        r = torch.add(d["x"] * d["residual_scale"], branch, alpha=d["branch_scale"])
        n = r * (torch.einsum("th,th->t", r, r) / case["H"] + EPS).rsqrt().unsqueeze(1) * d["gamma"]
        out = {"residual_out": r, "norm": n}
        if case["int8"]:
            out |= {"codes": None, "scales": None}      # of the norm as rounded
        return out
    if case["op"] == "quant":
        return {"codes": None, "scales": torch.clamp(d["x"].abs().max(1).values, min=TINY) / 127}
    if case["op"] == "gemm":
        r = torch.matmul(d["a"] * d["a_scales"][:, None], (d["b"] * d["b_scales"][:, None]).t())
        return r if d["bias_vec"] is None else r + d["bias_vec"]
    return {"weights": exact_weights(case, d), "ids": None}


def exact_weights(case, d):
    """One choice at a time: the largest key, of the lowest index, k times."""
    l, E, groups = d["logits"], case["E"], case["groups"]
    T = l.shape[0]
    if case["scoring"] == "sigmoid":
        score = torch.special.expit(l)
    else:
        score = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    low = torch.finfo(F64).min
    key = score + (d["bias_vec"] if d["bias_vec"] is not None else 0.0)
    key = torch.where(torch.isneginf(l), torch.full_like(key, low), key)
    if groups > 1:
        best = key.reshape(T, groups, -1).topk(case["top"], 2).values.clamp_min(-1e30).sum(2)
        rank = (best.unsqueeze(1) > best.unsqueeze(2)).sum(2) \
            + torch.tril((best.unsqueeze(1) == best.unsqueeze(2)).to(torch.int64), -1).sum(2)
        shut = (rank >= case["keep"]).repeat_interleave(E // groups, 1)
        key = torch.where(shut, torch.full_like(key, low), key)
    w = torch.zeros(T, case["k"], dtype=F64, device=l.device)
    index = torch.arange(E, device=l.device)
    for j in range(case["k"]):
        best = key.amax(1, keepdim=True)
        at = torch.where(key == best, index, E).amin(1, keepdim=True)
        w[:, j:j + 1] = torch.where(best == low, 0.0, score.gather(1, at))
        key = key.scatter(1, at, low)
    total = w.sum(1, keepdim=True)
    return torch.where(total > 0, w / total, 0.0) * d["scale"]

"""The block norm and the int8 quantiser on the GPU.

Two bars.  Bit for bit against the definition with its roundings
(block_reference): statistics are binary64 on both sides, so the order of
sums reaches a result only when a row's mean lies within 2^-46 or so of a
rounding border of binary32.  And against the formula in 64 bits, with
    residual_out: eps_x / 2 |r| + 2^-24 (|residual_scale x| + 6 |branch_scale p gate| + |r|)
(the stream's rounding; one rounding of the first product, six on the
branch's way -- rstd, three factors, the scale, and that of a binary32 scale
-- and one of the sum), and for norm, from the stored residual_out,
    eps / 2 |n| + 4 2^-24 |n|
(its rounding; rstd and two products, and one for second order), each plus
the type's smallest subnormal.
"""
import math

import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def seam():
    from layer_mhc_seam_amd import seam as S
    return S


def inputs(T, H, dt, xdt, gate, post, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    c = dict(x=(3 * n(T, H)).to(xdt), y=n(T, H).to(dt), gamma=(1 + 0.2 * n(H)).to(dt),
             gamma_post=(1 + 0.2 * n(H)).to(dt) if post else None)
    c["gate"] = {"none": None, "token": n(T, 1), "channel": n(H), "element": n(T, H).to(dt)}[gate]
    return c


def dev(c):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}


def bits(t):
    t = t.detach().cpu()
    return t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(got, want):
    """Equal bit for bit, NaN for NaN."""
    g, w = got.detach().cpu(), want
    if g.is_floating_point():
        assert torch.equal(g.isnan(), w.isnan())
        keep = ~w.isnan()
        g, w = g[keep], w[keep]
    bad = (bits(g) != bits(w)).nonzero()
    assert not len(bad), f"{len(bad)} differ, first at {bad[:4].tolist()}"


def near_formula(o, c, rs, bs, eps=1e-6):
    d = {k: v.to(F64) if torch.is_tensor(v) else None for k, v in c.items()}
    x, p = d["x"] * rs, d["y"]
    if d["gamma_post"] is not None:
        p = p / torch.sqrt(p.square().mean(1, keepdim=True) + eps) * d["gamma_post"]
    p = p * bs * (1.0 if d["gate"] is None else d["gate"])
    r, got = x + p, o["residual_out"].cpu().to(F64)
    fx, fe = torch.finfo(c["x"].dtype), torch.finfo(c["y"].dtype)
    tol = fx.eps / 2 * r.abs() + 2.0 ** -24 * (x.abs() + 6 * p.abs() + r.abs()) + fx.smallest_normal * fx.eps
    assert ((got - r).abs() <= tol).all()
    n = got / torch.sqrt(got.square().mean(1, keepdim=True) + eps) * d["gamma"]
    tol = (fe.eps / 2 + 4 * 2.0 ** -24) * n.abs() + fe.smallest_normal * fe.eps
    assert ((o["norm"].cpu().to(F64) - n).abs() <= tol).all()


# widths: below a vector, ragged on either side of a wave's and of every
# change of the launch's shape, the package's own, the widest
WIDTHS = [1, 7, 8, 64, 100, 505, 509, 512, 1017, 1027, 2040, 2041, 2042, 2048, 2056, 5120, 7168, 8185, 8192, 8200,
          20481, 32751, 32768]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt,xdt", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
def test_block_norm_matches_definition(H, dt, xdt):
    for k, (gate, post) in enumerate([("none", True), ("token", False), ("channel", True), ("element", True)]):
        T = (1, 3, 5, 2)[k]
        c = inputs(T, H, dt, xdt, gate, post, seed=H + k)
        o = seam().block_norm(**dev(c), residual_scale=0.75, branch_scale=0.22, int8=True)
        r, n = ref.block_norm(**c, residual_scale=0.75, branch_scale=0.22)
        same(o["residual_out"], r)
        same(o["norm"], n)
        codes, scales = ref.quantize(n)
        same(o["codes"], codes)
        same(o["scales"], scales)
        near_formula(o, c, 0.75, 0.22)


@pytest.mark.parametrize("T", [1, 4, 63, 384, 4160])
def test_block_norm_token_counts(T):
    c = inputs(T, 512, BF16, BF16, "element", True, seed=T)
    o = seam().block_norm(**dev(c), int8=True)
    r, n = ref.block_norm(**c, residual_scale=1.0, branch_scale=1.0)
    same(o["residual_out"], r)
    same(o["norm"], n)
    codes, scales = ref.quantize(n)
    same(o["codes"], codes)
    same(o["scales"], scales)


def test_block_norm_output_sets():
    """Norm alone, residual alone, codes without the norm, the first block,
    in place, given outputs."""
    c = inputs(9, 1000, BF16, F32, "channel", True, seed=1)
    d = dev(c)
    r, n = ref.block_norm(**c, residual_scale=1.0, branch_scale=0.5)
    o = seam().block_norm(**d, branch_scale=0.5)
    assert set(o) == {"residual_out", "norm"}
    o = seam().block_norm(d["x"], None, d["y"], gamma_post=d["gamma_post"], gate=d["gate"], branch_scale=0.5)
    assert set(o) == {"residual_out"}
    same(o["residual_out"], r)
    o = seam().block_norm(**d, branch_scale=0.5, int8=True, norm=False)
    assert set(o) == {"residual_out", "codes", "scales"}
    same(o["codes"], ref.quantize(n)[0])
    _, n0 = ref.block_norm(c["x"], c["gamma"], None, None, None, 1.0, 1.0)
    o = seam().block_norm(d["x"], d["gamma"])
    assert set(o) == {"norm"}
    same(o["norm"], n0)
    given = {"residual_out": d["x"], "norm": torch.empty_like(d["y"])}
    o = seam().block_norm(**d, branch_scale=0.5, out=given)
    assert o["residual_out"].data_ptr() == d["x"].data_ptr()
    same(d["x"], r)
    same(given["norm"], n)


@pytest.mark.parametrize("H", [100, 509, 5120])
def test_block_norm_special_rows(H):
    """Zero rows, infinities, NaN, values whose squares leave binary32's
    range, subnormals: what the arithmetic gives, row by row."""
    c = inputs(10, H, BF16, F32, "token", True, seed=H)
    x, y, gate = c["x"], c["y"], c["gate"]
    x[0] = 0.0
    y[0] = 0.0
    x[1, H // 2] = math.inf
    x[2, 0] = math.nan
    y[3, H - 1] = -math.inf
    x[4] *= 1e30
    x[5] *= 1e-30
    y[5] *= 1e-38
    y[6] *= 1e35
    gate[7] = 0.0
    gate[8] = math.nan
    o = seam().block_norm(**dev(c), int8=True)
    r, n = ref.block_norm(**c, residual_scale=1.0, branch_scale=1.0)
    codes, scales = ref.quantize(n)
    for k, want in (("residual_out", r), ("norm", n), ("codes", codes), ("scales", scales)):
        same(o[k], want)
    assert o["scales"].isnan()[[1, 2, 3, 8]].all() and not o["scales"].isnan()[[0, 4, 5, 6, 7, 9]].any()


def test_block_norm_writes_nothing_else():
    """The elements behind the last row stay as they were."""
    T, H = 5, 509
    c = dev(inputs(T, H, BF16, BF16, "none", True, seed=3))
    def room(t, n):
        return torch.full((n + 64,), 7, dtype=t, device="cuda")
    buf = {"residual_out": room(BF16, T * H), "norm": room(BF16, T * H), "codes": room(torch.int8, T * H),
           "scales": room(F32, T)}
    out = {k: (v[:T] if k == "scales" else v[:T * H].view(T, H)) for k, v in buf.items()}
    seam().block_norm(**c, int8=True, out=out)
    for k, v in buf.items():
        assert (v[-64:] == 7).all(), k


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_int8_quantize_matches_definition(H, dt):
    g = torch.Generator().manual_seed(H)
    for T in (1, 6):
        v = (torch.randn(T, H, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))).to(dt)
        codes, scales = seam().int8_quantize(v.cuda())
        want = ref.quantize(v)
        same(codes, want[0])
        same(scales, want[1])
        # the formula: a code times its scale is within half a scale (and the
        # roundings of 127 / a, of its product and of the scale) of the value
        err = (codes.cpu().to(F64) * scales.cpu().to(F64)[:, None] - v.to(F64)).abs()
        assert (err <= scales.cpu().to(F64)[:, None] * (0.5 + 127 * 3 * 2.0 ** -24)).all()


def test_int8_quantize_every_value():
    """Every finite bf16 and fp16 value in rows of every largest value's
    exponent, and ties."""
    for dt in (BF16, F16):
        b = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
        v = b[b.isfinite()]
        mag = v.abs().sort().values
        tops = mag[:: max(1, len(mag) // 300)]
        rows = torch.where(v.abs()[None] <= tops[:, None], v[None], torch.zeros((), dtype=dt))
        rows[:, 0] = tops
        for part in rows.split(20000, dim=1):
            part = part.contiguous()
            codes, scales = seam().int8_quantize(part.cuda())
            want = ref.quantize(part)
            same(codes, want[0])
            same(scales, want[1])


def test_int8_quantize_special_rows_and_empty():
    v = torch.randn(5, 300).to(BF16)
    v[0] = 0
    v[1, 299] = math.inf
    v[2, 0] = math.nan
    v[3] *= 1e-38
    codes, scales = seam().int8_quantize(v.cuda())
    want = ref.quantize(v)
    same(codes, want[0])
    same(scales, want[1])
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    codes, scales = seam().int8_quantize(e)
    assert codes.shape == (0, 64) and scales.shape == (0,)
    assert seam().block_norm(e, torch.ones(64, dtype=BF16, device="cuda"))["norm"].shape == (0, 64)


def test_block_norm_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31 bytes and beyond 2^31 elements."""
    H, T = 32768, 70000
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    at = [0, 32767, 32768, 65535, 65536, 65537, T - 1]
    g = torch.Generator().manual_seed(5)
    v = torch.randn(len(at), H, generator=g).to(BF16)
    x[at] = v.cuda()
    codes, scales = seam().int8_quantize(x)
    want = ref.quantize(v)
    same(codes[at], want[0])
    same(scales[at], want[1])
    del codes, scales
    gamma = torch.ones(H, dtype=BF16, device="cuda")
    o = seam().block_norm(x, gamma, x.view(T, H).clone(), out={"residual_out": x})
    r, n = ref.block_norm(v, gamma.cpu(), v, None, None, 1.0, 1.0)
    same(x[at], r)
    same(o["norm"][at], n)


def test_block_norm_stream_and_graph():
    """On a stream of its own, and captured: every replay, with eager calls
    between, gives the eager bits."""
    c = dev(inputs(33, 5120, BF16, BF16, "element", True, seed=8))
    want = seam().block_norm(**c, int8=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = {k: torch.empty_like(v) for k, v in want.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        seam().block_norm(**c, int8=True, out=out, stream=s)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        seam().block_norm(**c, int8=True)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(bits(out[k]), bits(want[k]))


def test_block_norm_refusals():
    S = seam()
    c = dev(inputs(4, 128, BF16, BF16, "none", True, seed=9))
    x, y, g = c["x"], c["y"], c["gamma"]
    bad = [
        lambda: S.block_norm(x, g, y[:3]), lambda: S.block_norm(x, g[:64], y),
        lambda: S.block_norm(x.t(), g, y), lambda: S.block_norm(x.half(), g, y),
        lambda: S.block_norm(x, g, y.half()), lambda: S.block_norm(x.double(), g, y),
        lambda: S.block_norm(x, g, y, gate=torch.ones(4, device="cuda")),
        lambda: S.block_norm(x, g, y, gate=torch.ones(128, dtype=F16, device="cuda")),
        lambda: S.block_norm(x, None, y, int8=True), lambda: S.block_norm(x, g, y.cpu()),
        lambda: S.block_norm(x, g, out={"residual_out": torch.empty_like(x)}),
        lambda: S.block_norm(x, g, y, out={"nrom": torch.empty_like(x)}),
        lambda: S.block_norm(x[:, ::2], g[:64], y[:, ::2])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: S.block_norm(x, g, out={"norm": x}), lambda: S.block_norm(x, g, y, out={"norm": y}),
                 lambda: S.block_norm(x, g, branch_scale=0.5), lambda: S.block_norm(x, g, y, eps=-1.0),
                 lambda: S.block_norm(x, g, norm=False)):
        with pytest.raises(S.SeamError):
            call()


def test_results_do_not_depend_on_the_width_of_the_launch():
    """Zero columns behind a row change nothing but the mean's divisor: with
    gamma scaled for it, codes of the same row at widths of every launch
    shape are those of the definition (the bits of binary64 sums)."""
    g = torch.Generator().manual_seed(11)
    row = torch.randn(1, 500, generator=g).to(BF16)
    for H in (500, 1000, 4000, 10000, 30000):
        v = torch.zeros(1, H, dtype=BF16)
        v[:, :500] = row
        codes, scales = seam().int8_quantize(v.cuda())
        want = ref.quantize(row)
        same(codes[:, :500], want[0])
        assert not codes[:, 500:].any()
        same(scales, want[1])
    assert np.isfinite(float(want[1]))


def test_more_rows_than_a_grid_line_holds():
    """Rows whose threads number past 2^32: the last ones too."""
    T, H = 70_000_001, 8
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    at = [0, 1, 8388607, 8388608, 33554431, 33554432, 67108863, 67108864, 67108865, T - 2, T - 1]
    v = torch.randn(len(at), H).to(BF16)
    x[at] = v.cuda()
    codes, scales = seam().int8_quantize(x)
    want = ref.quantize(v)
    same(codes[at], want[0])
    same(scales[at], want[1])
    del codes, scales
    g = torch.ones(H, dtype=BF16, device="cuda")
    o = seam().block_norm(x, g)
    _, n = ref.block_norm(v, g.cpu(), None, None, None, 1.0, 1.0)
    same(o["norm"][at], n)


@pytest.mark.parametrize("H0,dt,xdt", [(500, BF16, BF16), (512, F16, F32), (509, BF16, F32), (512, BF16, BF16)])
def test_norms_do_not_depend_on_the_width_of_the_launch(H0, dt, xdt):
    """The same values among zeros, at random places of rows 4, 16 and 64
    times as wide: a row's mean is then 4^k times smaller, which eps 4^-k and
    gammas of 2^-k times take back without a rounding.  The sums of squares
    go over other lanes, waves and workgroup sizes each time, and every
    output has the bits of the narrow row's and of the definition."""
    T = 7
    c = inputs(T, H0, dt, xdt, "channel", True, seed=H0)
    first = None
    for k in range(4):
        H = H0 * 4 ** k
        if H > (32768 if H % 8 == 0 else 32752):
            break
        g = torch.Generator().manual_seed(k)
        at = torch.randperm(H, generator=g)[:H0].sort().values if k else torch.arange(H0)
        w = {}
        for name, v in c.items():
            w[name] = torch.zeros(*v.shape[:-1], H, dtype=v.dtype)
            w[name][..., at] = v / 2 ** k if name in ("gamma", "gamma_post") else v
        eps = 2.0 ** -20 / 4 ** k
        o = seam().block_norm(**dev(w), branch_scale=0.5, eps=eps, int8=True)
        r, n = ref.block_norm(**w, residual_scale=1.0, branch_scale=0.5, eps=eps)
        codes, scales = ref.quantize(n)
        for name, want in (("residual_out", r), ("norm", n), ("codes", codes), ("scales", scales)):
            same(o[name], want)
        got = [o[name].cpu()[:, at] for name in ("residual_out", "norm", "codes")] + [o["scales"].cpu()]
        if first is None:
            first = got
        for a, b in zip(got, first):
            same(a, b)
    assert k >= 2

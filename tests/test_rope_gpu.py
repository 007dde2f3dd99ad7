"""Rotary positions against their definition in 64 bits: widths, head layouts,
strides, axes and orders of pairs, far positions, gradients.

Tolerance of an output o = s (a cos - b sin): half a step of its type, and in
binary32 the angle's 2^-22 (sine and cosine), three roundings and scale's."""
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F64 = torch.bfloat16, torch.float16, torch.float64


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def freqs(pairs, base=10000.0):
    return (base ** -(torch.arange(pairs, dtype=F64) / pairs)).float()


def check(got, x, positions, inv_freq, scale=1.0, **kw):
    want = ref.rope(x, positions, inv_freq, scale=scale, **kw)
    u = torch.finfo(x.dtype).eps / 2
    pairs = len(inv_freq)
    a = x.to(F64).abs()
    size = a.clone()
    if kw.get("interleaved"):
        both = a[..., 0:2 * pairs:2] + a[..., 1:2 * pairs:2]
        size[..., 0:2 * pairs:2] = size[..., 1:2 * pairs:2] = both
    else:
        both = a[..., :pairs] + a[..., pairs:2 * pairs]
        size[..., :pairs] = size[..., pairs:2 * pairs] = both
    bound = u * want.abs() + abs(scale) * size * 2.0 ** -20 + torch.finfo(x.dtype).tiny
    off = (got.cpu().to(F64) - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    assert torch.equal(got.cpu()[..., 2 * pairs:], x[..., 2 * pairs:])       # copied


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [
    (1, 1, 1, 64, 64), (4, 40, 8, 128, 128), (37, 5, 1, 80, 80), (3, 3, 0, 96, 96), (129, 7, 7, 128, 32),
    (2, 2, 1, 256, 64), (5, 2, 2, 50, 18), (6, 1, 1, 7, 6), (9, 3, 2, 2, 2), (2, 70, 70, 512, 512), (700, 9, 3, 72, 36),
    (1, 1, 0, 100, 4)])
def test_rope(T, Hq, Hk, D, R, interleaved, dt):
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(T + D)
    q, k = torch.randn(T, Hq, D, generator=g).to(dt), torch.randn(T, Hk, D, generator=g).to(dt)
    pos = torch.randint(0, 5000, (T,), generator=g)
    f = freqs(R // 2)
    gq, gk = S.rope(q.cuda(), k.cuda() if Hk else None, pos.cuda(), f.cuda(), interleaved=interleaved)
    check(gq, q, pos, f, interleaved=interleaved)
    assert (gk is None) == (Hk == 0)
    if Hk:
        check(gk, k, pos, f, interleaved=interleaved)


@pytest.mark.parametrize("axes,pairs", [([0] * 8 + [1] * 12 + [2] * 12, 32), ([i % 3 for i in range(32)], 32),
                                        ([3, 1, 0, 2, 2, 1, 1, 0, 3], 9), ([1] * 64, 64),
                                        ([i * 7 % 4 for i in range(256)], 256)])
@pytest.mark.parametrize("whole", [torch.int32, torch.int64])
def test_rope_axes(axes, pairs, whole):
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(pairs)
    T, D = 21, min(2 * pairs + 6, 512)      # the widest head there is
    q = torch.randn(T, 3, D, generator=g).to(BF)
    pos = torch.randint(-300, 3000, (max(axes) + 1, T + 5), generator=g).to(whole)
    f = freqs(pairs)
    wide = pos.cuda()
    got, none = S.rope(q.cuda(), None, wide[:, 2:2 + T], f.cuda(), axes=axes, scale=1.3)   # rows of a wider table
    assert none is None
    check(got, q, pos[:, 2:2 + T], f, scale=1.3, axes=axes)


@pytest.mark.parametrize("start", [(1 << 20) + 1, (1 << 31) - 40, -(1 << 31), (1 << 40) + 3])
def test_rope_far_positions(start):
    """Nothing is lost far along: |p f| 2^-52 is below 2^-12 at 2^40, and far below the tolerance up to 2^31."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(5)
    T, D = 33, 128
    q = torch.randn(T, 2, D, generator=g).to(F16)
    pos = start + torch.arange(T)
    # frequencies of few bits: their products with positions are exact, and so are the reference's angles but for one
    # rounding of 2^-53
    f = (freqs(64) * 2 ** 10).round().clamp(min=1) / 2 ** 10
    if abs(start) < 1 << 32:
        got = S.rope(q.cuda(), None, pos.cuda(), f.cuda())[0]
        check(got, q, pos, f)
        if start <= (1 << 31) - 40:
            same = S.rope(q.cuda(), None, pos.to(torch.int32).cuda(), f.cuda())[0]
            assert torch.equal(got, same)
        return
    # beyond, the turn is still that of the angle to 2^-12: rotations that compose
    a = S.rope(q.cuda(), None, pos.cuda(), f.cuda())[0]
    b = S.rope(a, None, pos.cuda(), f.cuda(), inverse=True)[0]
    assert (b.cpu().float() - q.float()).abs().max() <= 2.0 ** -9 * q.abs().max()


@pytest.mark.parametrize("D,R,offset", [(128, 128, 0), (64, 32, 0), (96, 96, 4), (40, 20, 2), (34, 30, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inside_a_product(D, R, offset, interleaved):
    """q and k side by side in the rows of one product (starting anywhere), to dense outputs and in place; what lies
    beside them stays."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(D)
    T, Hq, Hk = 19, 6, 2
    width = (Hq + 2 * Hk) * D + 2 * offset
    rows = torch.randn(T, width, generator=g).to(BF)
    split = lambda r: (r[:, offset:offset + Hq * D].view(T, Hq, D),                          # noqa: E731
                       r[:, offset + Hq * D:offset + (Hq + Hk) * D].view(T, Hk, D))
    pos, f = torch.randint(0, 999, (T,), generator=g), freqs(R // 2)
    dev = rows.cuda()
    q, k = split(dev)
    dense = S.rope(q, k, pos.cuda(), f.cuda(), interleaved=interleaved)
    assert torch.equal(dev.cpu(), rows)
    for got, x in zip(dense, split(rows)):
        check(got, x, pos, f, interleaved=interleaved)
    there = S.rope(q, k, pos.cuda(), f.cuda(), interleaved=interleaved, out=(q, k))
    assert there[0] is q and torch.equal(q, dense[0]) and torch.equal(k, dense[1])
    left = dev.cpu()
    assert torch.equal(left[:, :offset], rows[:, :offset])
    assert torch.equal(left[:, offset + (Hq + Hk) * D:], rows[:, offset + (Hq + Hk) * D:])
    # heads first: tokens inside a head
    q2 = rows[:, offset:offset + Hq * D].reshape(T, Hq, D).transpose(0, 1).contiguous().cuda().transpose(0, 1)
    got = S.rope(q2, None, pos.cuda(), f.cuda(), interleaved=interleaved)[0]
    assert torch.equal(got, dense[0])


def test_rope_gradient():
    """The inverse is the gradient: by the formula, and by differences of the definition."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(8)
    T, H, D, R = 6, 2, 64, 48
    x, grad = torch.randn(T, H, D, generator=g).to(F16), torch.randn(T, H, D, generator=g).to(F16)
    pos, f = torch.randint(0, 9999, (T,), generator=g), freqs(R // 2)
    for interleaved in (False, True):
        kw = dict(interleaved=interleaved, scale=1.25)
        got = S.rope(grad.cuda(), None, pos.cuda(), f.cuda(), inverse=True, **kw)[0].cpu().double()
        leaf = x.double().requires_grad_()
        a = torch.zeros(T, R // 2, dtype=F64) + pos[:, None] * f.double()
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        u, w = (leaf[..., 0:R:2], leaf[..., 1:R:2]) if interleaved else (leaf[..., :R // 2], leaf[..., R // 2:R])
        p, m = 1.25 * (u * c - w * s), 1.25 * (w * c + u * s)
        y = torch.cat((torch.stack((p, m), -1).flatten(-2) if interleaved else torch.cat((p, m), -1),
                       leaf[..., R:]), -1)
        # channels past R are copied, so their gradient is the outputs'
        (y * grad.double()).sum().backward()
        # half a step, and the 2^-20 of two values that check() allows
        assert ((got - leaf.grad).abs() <= 2.0 ** -11 * leaf.grad.abs() + 2.0 ** -17).all()
        # differences: the map is linear, so a whole step of one input is exact
        for t, h, d in ((0, 0, 0), (3, 1, 17), (5, 1, R - 1), (2, 0, R)):
            step = torch.zeros_like(x)
            step[t, h, d] = 1.0
            moved = (ref.rope(step, pos, f, **kw) * grad.double()).sum()
            assert abs(got[t, h, d] - moved) <= 2.0 ** -11 * abs(moved) + 2.0 ** -17


def test_rope_special_values():
    """Infinities and NaN go through the arithmetic of their own pair only; T = 0."""
    from layer_mhc_seam_amd import seam as S
    x = torch.ones(3, 1, 64, dtype=BF)
    x[0, 0, 0], x[1, 0, 3], x[2, 0, 40] = float("nan"), float("inf"), -float("inf")
    got = S.rope(x.cuda(), None, torch.tensor([1, 2, 3]).cuda(), freqs(32).cuda())[0].cpu()
    odd = ~got.isfinite()
    want = torch.zeros(3, 1, 64, dtype=torch.bool)
    want[0, 0, [0, 32]] = want[1, 0, [3, 35]] = want[2, 0, [8, 40]] = True
    assert torch.equal(odd, want)
    q, k = S.rope(x[:0].cuda(), x[:0].cuda(), torch.zeros(0, dtype=torch.int64).cuda(), freqs(32).cuda())
    assert q.shape == k.shape == (0, 1, 64)


def test_rope_refuses_on_the_device():
    from layer_mhc_seam_amd import seam as S
    q, pos, f = torch.zeros(4, 2, 64, dtype=BF).cuda(), torch.arange(4).cuda(), freqs(32).cuda()
    for call in (lambda: S.rope(q, None, pos[:3], f), lambda: S.rope(q, None, pos, f.double()),
                 lambda: S.rope(q, q.half(), pos, f), lambda: S.rope(q, q[:3], pos, f),
                 lambda: S.rope(q, None, pos.float(), f), lambda: S.rope(q, None, pos, f, axes=[0] * 31),
                 lambda: S.rope(q, None, pos, f, axes=[1] * 32), lambda: S.rope(q.transpose(1, 2), None, pos, f),
                 lambda: S.rope(q, None, pos, f, out=(q, q)), lambda: S.rope(q, q[:, :0], pos, f)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: S.rope(q, None, pos, torch.ones(33).cuda()), lambda: S.rope(q, q, pos, f, out=(q, q)),
                 lambda: S.rope(q, None, pos, f, scale=float("inf")), lambda: S.rope(q, None, pos, f, scale=float("nan"))):
        with pytest.raises(S.SeamError):
            call()


@pytest.mark.parametrize("start", [(1 << 32) + 7, -(1 << 33), (1 << 40) + 3, -(1 << 40)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_positions_past_32_bits(start, interleaved):
    """Turns by the whole of a long position, each against the definition: an angle is off by 2^-51 of itself (three
    roundings of 2^-53), which moves an output by as much of its pair's size."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(7)
    T, D = 33, 128
    q = torch.randn(T, 2, D, generator=g).to(F16)
    pos = start + torch.arange(T)
    f = (freqs(64) * 2 ** 10).round().clamp(min=1) / 2 ** 10       # their products with positions are exact
    got = S.rope(q.cuda(), None, pos.cuda(), f.cuda(), interleaved=interleaved)[0].cpu()
    want = ref.rope(q, pos, f, interleaved=interleaved)
    a = q.to(F64).abs()
    if interleaved:
        size = (a[..., 0::2] + a[..., 1::2]).repeat_interleave(2, -1)
        angle = (pos[:, None] * f.to(F64)).repeat_interleave(2, -1)
    else:
        size = (a[..., :64] + a[..., 64:]).repeat(1, 1, 2)
        angle = (pos[:, None] * f.to(F64)).repeat(1, 2)
    bound = 2.0 ** -11 * want.abs() + size * (2.0 ** -20 + angle.abs()[:, None] * 2.0 ** -51) + 2.0 ** -14
    assert ((got.to(F64) - want).abs() <= bound).all()
    short = S.rope(q.cuda(), None, (pos % (1 << 32)).cuda(), f.cuda(), interleaved=interleaved)[0].cpu()
    assert ((got - short).abs().amax((1, 2)) > 0.1).all()          # not their low 32 bits

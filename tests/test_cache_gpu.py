"""Writing the 4-bit cache and reading it back, bit for bit against the definition: every value of both types, ties,
groups at the borders of two scales, special values, slots of padding, strides, far pages."""
import math

import numpy as np
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F64 = torch.bfloat16, torch.float16, torch.float64
NAMES = {BF: "bf16", F16: "f16"}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def cuda_cache(c):
    return torch.from_numpy(c.bytes).cuda()


def same(a, b):
    return torch.equal(a.nan_to_num(nan=-77.0), b.nan_to_num(nan=-77.0)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,pages,H,D,ps", [(1, 1, 1, 64, 16), (37, 4, 3, 128, 16), (50, 2, 2, 256, 48),
                                            (3, 7, 5, 64, 512), (130, 3, 1, 128, 64)])
def test_write_and_read(T, pages, H, D, ps, dt):
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(T + D)
    k, v = ((torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))).to(dt) for _ in "kv")
    slots = torch.randperm(pages * ps, generator=g)[:T]
    slots[1::7] += pages * ps                    # past the cache
    slots[::5] = -1 - slots[::5]                 # padding
    there = slots[(slots >= 0) & (slots < pages * ps)]
    assert len(there.unique()) == len(there)     # no slot twice
    c = ref.Cache(pages, H, D, ps)
    c.bytes[:] = np.random.default_rng(T).integers(0, 250, c.bytes.shape)   # what was there stays
    dev = cuda_cache(c)
    for t, s in enumerate(slots.tolist()):
        c.write(s, 0, k[t])
        c.write(s, 1, v[t])
    assert S.cache_write(dev, k.cuda(), v.cuda(), slots.cuda()) is dev
    assert torch.equal(dev.cpu(), torch.from_numpy(c.bytes))
    for whole in (torch.int64, torch.int32):
        gk, gv = S.cache_read(dev, slots.to(whole).cuda(), D, dtype=NAMES[dt])
        for kind, got in ((0, gk), (1, gv)):
            want = torch.stack([c.read(s, kind) for s in slots.tolist()])
            assert got.dtype == dt and torch.equal(got.cpu().to(F64), want)
    # any slots of the cache, twice too, in any order
    some = torch.randint(-2, pages * ps + 2, (T + 3,), generator=g)
    gk, gv = S.cache_read(dev, some.cuda(), D, dtype="bf16")
    want = torch.stack([c.read(s, 1) for s in some.tolist()])
    assert torch.equal(gv.cpu(), want.to(BF))


@pytest.mark.parametrize("dt", [BF, F16])
def test_every_value(dt):
    """Each finite number of the type in a group under each of the scales that groups of it meet: as its largest, and
    below 6 2^e for the e of the next powers."""
    from layer_mhc_seam_amd import seam as S
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
    x = x[x.isfinite()]
    most = torch.stack([x.abs() * f for f in (1.0, 1.5, 2.0, 3.0, 4.5, 7.0, 12.0, 20.0)], 1)
    keep = most.isfinite().all(1)
    x, most = x[keep], most[keep]
    rows = torch.zeros(len(x), 256, dtype=dt)
    rows[:, 0::32] = most
    rows[:, 5::32] = x[:, None].expand(-1, 8)
    rows[:, 30::32] = -x[:, None].expand(-1, 8)
    T = len(x)
    dev = S.kv_cache(-(-T // 512), 1, 256, 512)
    slots = torch.arange(T).cuda()
    r = rows[:, None].cuda()
    S.cache_write(dev, r, r.flip(0), slots)
    k, v = S.cache_read(dev, slots, 256, dtype=NAMES[dt])
    assert torch.equal(k, v.flip(0))
    want = torch.cat([ref.quantized_fast(p) for p in rows.split(8192)])
    assert torch.equal(k[:, 0].cpu().to(F64), want)


@pytest.mark.parametrize("dt", [BF, F16])
def test_groups_at_two_scales(dt):
    """A group's largest at 6 2^e and a step to either side."""
    from layer_mhc_seam_amd import seam as S
    low, high = ref.EXPONENTS[dt]
    e = torch.arange(low, high + 1, dtype=F64)
    edge = (6 * torch.exp2(e)).to(dt)
    bits = edge.view(torch.int16)
    most = torch.stack([(bits + d).view(dt) for d in (-1, 0, 1)], 1).flatten()
    most = most[most.isfinite()]
    rows = torch.zeros(len(most), 1, 64, dtype=dt)
    rows[:, 0, 31], rows[:, 0, 40] = most, -most
    rows[:, 0, 1] = (most.double() * 0.4).to(dt)
    slots = torch.arange(len(most)).cuda()
    dev = S.kv_cache(-(-len(most) // 16), 1, 64, 16)
    S.cache_write(dev, rows.cuda(), rows.cuda(), slots)
    k, _ = S.cache_read(dev, slots, 64, dtype=NAMES[dt])
    assert torch.equal(k.cpu().to(F64), ref.quantized(rows))


@pytest.mark.parametrize("dt", [BF, F16])
def test_special_values(dt):
    """A group with an infinity or NaN reads as NaN, the others are as ever; the type's smallest and largest."""
    from layer_mhc_seam_amd import seam as S
    x = torch.randn(9, 1, 64, generator=torch.Generator().manual_seed(0)).to(dt)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 31] = math.nan, math.inf, -math.inf
    x[3] = 0
    x[4] = -0.0
    x[5] = torch.finfo(dt).max
    x[6, 0, ::3] = torch.finfo(dt).tiny
    x[7] = torch.tensor([1], dtype=torch.int16).view(dt)            # the smallest subnormal
    x[8, 0, 7] = torch.finfo(dt).min
    slots = torch.arange(9).cuda()
    dev = S.kv_cache(2, 1, 64, 16)
    S.cache_write(dev, x.cuda(), x.cuda(), slots)
    k, v = S.cache_read(dev, slots, 64, dtype=NAMES[dt])
    assert same(k.cpu().to(F64), ref.quantized(x)) and same(v.cpu(), k.cpu())
    assert k[0, 0, :32].isnan().all() and k[0, 0, 32:].isfinite().all() and k[5].isfinite().all()


def test_slices_of_a_product():
    """k and v side by side in wider rows, read back into such rows; what lies beside them stays."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(4)
    T, H, D = 45, 3, 128
    rows = torch.randn(T, 5 * H * D, generator=g).to(BF).cuda()
    k, v = (rows[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in (3, 1))
    slots = torch.randperm(96, generator=g)[:T].cuda()
    a, b = S.kv_cache(2, H, D, 48), S.kv_cache(2, H, D, 48)
    S.cache_write(a, k, v, slots)
    S.cache_write(b, k.contiguous(), v.contiguous(), slots)
    assert torch.equal(a, b) and a.any()
    heads_first = k.transpose(0, 1).contiguous().transpose(0, 1)
    c = S.cache_write(S.kv_cache(2, H, D, 48), heads_first, v, slots)
    assert torch.equal(a, c)
    dense = S.cache_read(a, slots, D)
    back = torch.full_like(rows, 5.0)
    ok, ov = (back[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in (0, 4))
    assert S.cache_read(a, slots, D, out=(ok, ov))[0] is ok
    assert torch.equal(ok, dense[0]) and torch.equal(ov, dense[1])
    assert (back[:, H * D:4 * H * D] == 5.0).all()


def test_no_tokens():
    from layer_mhc_seam_amd import seam as S
    none = torch.zeros(0, dtype=torch.int64).cuda()
    x = torch.zeros(0, 2, 64, dtype=BF).cuda()
    c = S.kv_cache(2, 2, 64, 16)
    S.cache_write(c, x, x, none)
    assert not c.any() and S.cache_read(c, none, 64)[0].shape == (0, 2, 64)


def test_far_pages():
    """Pages past 4 GiB, and slots past 2^31 are refused or held by their whole number."""
    from layer_mhc_seam_amd import seam as S
    pages, H, D, ps = 5000, 16, 128, 512
    dev = S.kv_cache(pages, H, D, ps)
    assert dev.numel() > 5 << 30
    g = torch.Generator().manual_seed(6)
    T = 40
    slots = torch.cat((torch.randint(pages * ps - 9000, pages * ps, (T - 2,), generator=g).unique(),
                       torch.tensor([0, 1 << 40, (1 << 32) + 5])))
    T = len(slots)
    k, v = torch.randn(T, H, D, generator=g).to(BF), torch.randn(T, H, D, generator=g).to(BF)
    S.cache_write(dev, k.cuda(), v.cuda(), slots.cuda())
    gk, gv = S.cache_read(dev, slots.cuda(), D)
    there = (slots < pages * ps)[:, None, None]
    for got, x in ((gk, k), (gv, v)):
        assert torch.equal(got.cpu().to(F64), torch.where(there, ref.quantized_fast(x), torch.zeros(1, dtype=F64)))
    assert not dev[1:pages - 20].any()


def test_device_refusals():
    from layer_mhc_seam_amd import seam as S
    c = S.kv_cache(2, 2, 64, 16)
    x, s = torch.zeros(4, 2, 64, dtype=BF).cuda(), torch.arange(4).cuda()
    for call in (lambda: S.cache_write(c, x, x[:3], s), lambda: S.cache_write(c, x, x.half(), s),
                 lambda: S.cache_write(c, x, x, s[:3]), lambda: S.cache_write(c, x, x, s.float()),
                 lambda: S.cache_write(c, x[:, :1], x[:, :1], s), lambda: S.cache_write(c, x, x, s.cpu()),
                 lambda: S.cache_write(c.cpu(), x, x, s), lambda: S.cache_write(c[:, :, ::2], x, x, s),
                 lambda: S.cache_read(c, s.view(2, 2), 64), lambda: S.cache_read(c, s, 128),
                 lambda: S.cache_read(c, s, 64, out=(x, x.half())), lambda: S.cache_read(c, s, 64, out=(x[:3], x))):
        with pytest.raises(ValueError):
            call()
    y = torch.zeros(4, 2, 68, dtype=BF).cuda()[:, :, 2:66]
    for call in (lambda: S.cache_write(c, y, y, s), lambda: S.cache_read(c, s, 64, out=(x, x))):
        with pytest.raises(S.SeamError):
            call()


@pytest.mark.parametrize("H,D", [(1, 64), (5, 128), (3, 256)])
def test_keys_or_values_alone(H, D):
    """The C entry reads only what it is given a place for; what lies where the other would go stays."""
    import ctypes
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(D)
    T, ps, pages = 70, 16, 6
    x = torch.randn(2, T, H, D, generator=g).to(BF).cuda()
    slots = torch.randperm(pages * ps, generator=g)[:T]
    slots[::9] = -1
    slots = slots.cuda()
    c = S.cache_write(S.kv_cache(pages, H, D, ps), x[0], x[1], slots)
    want = S.cache_read(c, slots, D)
    for kind in range(2):
        out = torch.full((2, T, H, D), 7.0, dtype=BF).cuda()
        at = [out[kind].data_ptr() if i == kind else None for i in range(2)]
        for other in ((0, 0), (H * D, D)):              # the absent one's strides say nothing
            strides = [(H * D, D) if i == kind else other for i in range(2)]
            a = S.CacheArgs(T, pages, ps, H, D, 0, 8, 0, *strides[0], *strides[1], c.data_ptr(), slots.data_ptr(), *at)
            assert S.lib().mhc_cache_read(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == S.OK
        torch.cuda.synchronize()
        assert torch.equal(out[kind], want[kind]) and (out[1 - kind] == 7.0).all()

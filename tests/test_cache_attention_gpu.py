"""Attention over the 4-bit cache against its definition in 64 bits: head layouts and widths, lengths from none to
several thousand, ragged queries, masks that leave rows empty, NaN where nobody looks, bad pages, both ways the work
is split.  The tolerance is derived in cache_reference.attention: a rounding of the output and of the weights, and
the binary32 sums."""
import math

import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F64 = torch.bfloat16, torch.float16, torch.float64


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def batch(lens, rows, Hq, Hk, D, ps, dt, seed=0, width=None, sharp=1.0):
    """A cache of shuffled pages: (device tensors, host keys, values)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    width = width or max(max(need), 1)
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g)
    tables = torch.full((len(lens), width), -7, dtype=torch.int32)
    at, keys, values, slots, ks, vs = 0, [], [], [], [], []
    for b, n in enumerate(lens):
        mine = order[at:at + need[b]]
        at += need[b]
        tables[b, :need[b]] = mine.to(torch.int32)
        ks.append(torch.randn(n, Hk, D, generator=g).to(dt))
        vs.append((torch.randn(n, Hk, D, generator=g) * torch.exp(torch.randn(n, Hk, 1, generator=g))).to(dt))
        t = torch.arange(n)
        slots.append(mine[t // ps] * ps + t % ps if n else t)
    cache, hk, hv = ref.packed(torch.cat(ks), torch.cat(vs), torch.cat(slots), pages, ps)
    first = 0
    for n in lens:
        keys.append(hk[first:first + n])
        values.append(hv[first:first + n])
        first += n
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    q = (sharp * torch.randn(starts[-1], Hq, D, generator=g)).to(dt)
    return dict(q=q, cache=cache, tables=tables, lens=torch.tensor(lens, dtype=torch.int32),
                starts=starts, ps=ps), keys, values


def run(d, single=False, **kw):
    from layer_mhc_seam_amd import seam as S
    starts = None if single else torch.tensor(d["starts"], dtype=torch.int32).cuda()
    return S.cache_attention(d["q"].cuda(), d["cache"].cuda(), d["tables"].cuda(), d["lens"].cuda(),
                             q_starts=starts, lse=True, **kw)


def check(got, want, first=0):
    out, lse = (x.cpu().to(F64) for x in got)
    w, l, bound, lbound = want
    assert torch.equal(out.isnan(), w.isnan())
    off = (out - w).abs().nan_to_num(0)
    assert (off <= bound.nan_to_num(0)).all(), (off / bound).nan_to_num(0).max()
    fine = l.isfinite()
    assert torch.equal(lse[~fine].nan_to_num(nan=5.0), l[~fine].nan_to_num(nan=5.0))
    assert ((lse - l).abs()[fine] <= lbound[fine]).all(), ((lse - l).abs() / lbound)[fine].max()


def widened(d, tokens=4200):
    """The same behind tables for that many tokens, with which the work may be split."""
    B, width = d["tables"].shape
    ps = d["ps"]
    if width * ps >= tokens:
        return d
    tables = torch.full((B, -(-tokens // ps)), -5, dtype=torch.int32)
    tables[:, :width] = d["tables"]
    return dict(d, tables=tables)


def headed(d, n):
    """The same with every kv head and its query heads n times."""
    return dict(d, q=d["q"].repeat(1, n, 1), cache=d["cache"].repeat(1, n, 1))


def ways(d):
    """(the same case, how often its heads are in it): behind tables as they are, for 4200 tokens, with which work may
    be split, and where there are rows enough for 2^20 tokens, with which it is as a long prompt's: of few row blocks,
    shared out, and of more than there are workers."""
    yield d, 1
    yield widened(d), 1
    T, Hq, D = d["q"].shape
    B, Hk = len(d["lens"]), d["cache"].shape[1]
    if T * Hq // Hk >= 64 * B:
        yield widened(d, 1 << 20), 1
        n = 1100 // ((T * (Hq // Hk) // 128 + B) * Hk) + 1
        yield widened(headed(d, n), 1 << 20), n


def check_ways(d, want, single=False, **kw):
    for case, n in ways(d):
        got = run(case, single=single, **kw)
        check(got, tuple(x.repeat(1, n, *[1] * (x.dim() - 2)) for x in want))
        if n == 1:
            last = got
    return last


def both(lens, rows, Hq, Hk, D, ps, dt, seed=0, sharp=1.0, width=None, visible=None, **kw):
    """The definition's result, in all the ways the work is split."""
    d, keys, values = batch(lens, rows, Hq, Hk, D, ps, dt, seed, sharp=sharp, width=width)
    single = all(n == 1 for n in rows)
    want = ref.attention(d["q"], keys, values, lens, d["starts"], visible, **kw)
    got = check_ways(d, want, single, **kw)
    if single:
        again = run(widened(d), **kw)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    return d, got


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 8), (10, 2), (16, 1), (40, 2)])
def test_one_token(D, Hq, Hk, dt):
    both([1, 200, 33, 0, 64], [1] * 5, Hq, Hk, D, 16, dt)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 1003, 4097])
@pytest.mark.parametrize("dt", [BF, F16])
def test_lengths(L, dt):
    both([L], [1], 6, 2, 128, 48, dt, seed=L)


@pytest.mark.parametrize("ps", [16, 32, 48, 80, 256, 512])
def test_page_sizes(ps):
    both([700, 3, ps, ps + 1], [1] * 4, 4, 1, 64, ps, BF)


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal,window,softcap", [(True, 0, 0.0), (False, 0, 0.0), (True, 50, 0.0), (False, 20, 8.0),
                                                   (True, 1, 30.0), (True, 0, 5.0)])
def test_ragged_rows(causal, window, softcap, D, dt):
    """One to many query rows a sequence, none too, and more than its tokens."""
    both([90, 200, 41, 5, 0, 130], [7, 1, 41, 0, 3, 20], 6, 2, D, 32, dt, causal=causal, window=window,
         softcap=softcap)
    both([3, 70], [9, 2], 5, 5, D, 16, dt, causal=causal, window=window, softcap=softcap)


@pytest.mark.parametrize("T,L,Hq,Hk", [(200, 333, 4, 1), (64, 64, 8, 1), (300, 300, 3, 3), (17, 1500, 16, 2)])
@pytest.mark.parametrize("dt", [BF, F16])
def test_prompts(T, L, Hq, Hk, dt):
    both([L, 20, 77], [T, 20, 1], Hq, Hk, 128, 64, dt)


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal,window,softcap,scale", [(True, 0, 0.0, None), (False, 0, 0.0, None), (True, 50, 0.0, -0.2),
                                                         (False, 70, 8.0, None), (True, 1, 30.0, -0.1),
                                                         (True, 400, 5.0, None), (True, 0, 0.0, 0.0)])
def test_prompt_masks(causal, window, softcap, scale, D, dt):
    """Rows for several workgroups, of heads in threes and more, some with more rows than tokens."""
    both([190, 130, 64, 5, 0, 333], [150, 130, 1, 90, 3, 0], 6, 2, D, 48, dt, causal=causal, window=window,
         softcap=softcap, scale=scale)


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,rows,window", [([5000], [70], 0), ([100, 3000, 0, 2100], [1, 100, 2, 260], 0),
                                              ([2500, 2500], [300, 90], 700), ([3000, 1, 40, 700], [70, 1, 40, 300], 0),
                                              ([5000, 40, 3000], [300, 40, 3], 2100)])
def test_prompt_shares(lens, rows, window, D, dt):
    """Few blocks of long sequences, whose tiles several workers share; heads enough that a window leaves it so."""
    d, keys, values = batch(lens, rows, 3, 1, D, 64, dt, width=80)
    want = ref.attention(d["q"], keys, values, lens, d["starts"], window=window)
    check_ways(d, want, window=window)
    check(run(headed(d, 12), window=window), tuple(x.repeat(1, 12, *[1] * (x.dim() - 2)) for x in want))


@pytest.mark.parametrize("dt", [BF, F16])
def test_sharp_scores(dt):
    """Scores far apart: a maximum that moves often, weights that vanish."""
    both([600, 50], [3, 50], 4, 2, 128, 16, dt, sharp=30.0)
    both([600, 250], [100, 250], 4, 2, 128, 16, dt, sharp=30.0)
    both([600], [90], 2, 1, 256, 16, dt, sharp=100.0)
    both([600, 50], [1, 1], 4, 2, 64, 16, dt, sharp=200.0)
    both([600, 50], [1, 1], 4, 2, 64, 16, dt, scale=-0.3)
    both([600, 50], [1, 1], 4, 2, 64, 16, dt, scale=0.0)


def test_rising_maximum():
    """Scores that rise along the sequence, by less and by more than the slack, and fall again."""
    for slope in (0.02, 0.3, 5.0, -0.3):
        d, keys, values = batch([900], [1], 1, 1, 64, 16, BF, seed=3)
        k = torch.zeros(900, 1, 64, dtype=BF)
        k[:, 0, 0] = (torch.arange(900) * slope).to(BF)
        v = torch.randn(900, 1, 64, generator=torch.Generator().manual_seed(1)).to(BF)
        t = torch.arange(900)
        slots = d["tables"][0][t // 16].long() * 16 + t % 16
        d["cache"], hk, hv = ref.packed(k, v, slots, d["cache"].shape[0], 16)
        for n in (1, 100):
            d["q"] = torch.zeros(n, 1, 64, dtype=BF)
            d["q"][:, 0, 0] = 1.0
            d["starts"] = [0, n]
            check(run(d, scale=1.0), ref.attention(d["q"], [hk], [hv], [900], [0, n], scale=1.0))


def test_many_tiny_weights():
    """One token far above thousands of others, whose weights of 2^-22 and below add up: fp16 keeps them."""
    n = 6000
    d, _, _ = batch([n], [1], 1, 1, 64, 512, F16, seed=3)
    k = torch.zeros(n, 1, 64, dtype=F16)
    k[0, 0, 0] = 1.0
    v = torch.ones(n, 1, 64, dtype=F16)
    v[0] = 0
    t = torch.arange(n)
    slots = d["tables"][0][t // 512].long() * 512 + t % 512
    d["cache"], hk, hv = ref.packed(k, v, slots, d["cache"].shape[0], 512)
    for gap, rows in ((14.0, 1), (17.0, 1), (19.0, 1), (17.0, 70)):
        d["q"] = torch.zeros(rows, 1, 64, dtype=F16)
        d["q"][:, 0, 0] = gap
        d["starts"] = [0, rows]
        got = run(d, scale=1.0)
        want = ref.attention(d["q"], [hk], [hv], [n], [0, rows], scale=1.0)
        check(got, want)
        assert ((got[0].cpu().double() / want[0] - 1).abs() < 2.0 ** -8).all() or want[0].max() < 2.0 ** -14


def put(d, b, t, kind, D, ps, block, byte=255):
    """A scale byte of one token, in the bytes."""
    page, at = int(d["tables"][b, t // ps]), t % ps
    base = ps * D + kind * ps * D // 32
    d["cache"][page, :, base + block * ps + at] = byte
    codes = kind * ps * D // 2 + at * D // 2 + block * 16
    d["cache"][page, :, codes:codes + 16] = 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("lens,rows,window,width", [
    ((70, 140, 300), (30, 4, 1), 0, None), ((170, 240, 300), (130, 100, 1), 0, None),
    ((170, 240, 300), (130, 100, 1), 60, None), ((170, 240, 300), (130, 100, 1), 0, 130)])
def test_nan_reaches_who_sees_it(lens, rows, window, width, D, dt):
    """A NaN in a key makes the rows that see it NaN, one in a value only its 32 channels of them."""
    ps = 16
    d, keys, values = batch(lens, rows, 4, 2, D, ps, dt, seed=9, width=width)
    for b, t, kind, block in ((0, lens[0] - 25, 1, 1), (0, lens[0] - 10, 0, 0), (1, lens[1] - 2, 1, D // 32 - 1),
                              (1, lens[1] - 1, 0, 1), (2, 20, 1, 0), (2, 260, 1, 1), (1, 20, 1, 0)):
        put(d, b, t, kind, D, ps, block)
        (values if kind else keys)[b][t, :, block * 32:block * 32 + 32] = math.nan
    want = ref.attention(d["q"], keys, values, lens, d["starts"], window=window)
    for case, n in ways(d):
        got = run(case, window=window)
        out, lse = got[0].cpu().to(F64), got[1].cpu().to(F64)
        w, l, bound, lbound = (x.repeat(1, n, *[1] * (x.dim() - 2)) for x in want)
        assert torch.equal(out.isnan(), w.isnan()) and torch.equal(lse.isnan(), l.isnan())
        assert w.isnan().any() and not w.isnan().all(dim=(1, 2)).all()
        fine = ~w.isnan()
        assert ((out - w).abs()[fine] <= bound[fine]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [(1, 3, 1, 2), (70, 129, 1, 100)])
def test_what_nobody_sees_may_be_anything(rows, D):
    """Bytes of 255 everywhere but in the tokens: behind the last one, in other pages, before a window."""
    lens, ps = [70, 129, 1, 260], 32
    for kw in ({}, dict(window=40)):
        d, keys, values = batch(lens, rows, 4, 2, D, ps, BF, seed=2)
        clean = run(d, **kw)
        dirty = torch.full_like(d["cache"], 255)
        for b, n in enumerate(lens):
            for t in range(max(0, n - rows[b] + 1 - kw.get("window", n)), n):
                page, at = int(d["tables"][b, t // ps]), t % ps
                for kind in range(2):
                    c = kind * ps * D // 2 + at * D // 2
                    s = ps * D + kind * ps * D // 32 + torch.arange(D // 32) * ps + at
                    dirty[page, :, c:c + D // 2] = d["cache"][page, :, c:c + D // 2]
                    dirty[page, :, s] = d["cache"][page, :, s]
        d["cache"] = dirty
        wide = torch.full((len(lens), 100), 2 ** 31 - 1, dtype=torch.int32)
        wide[:, :d["tables"].shape[1]] = d["tables"]
        long = run(dict(d, tables=wide), **kw)
        check(long, ref.attention(d["q"], keys, values, lens, d["starts"], **kw))
        got = run(d, **kw)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
        check_ways(d, ref.attention(d["q"], keys, values, lens, d["starts"], **kw), **kw)


@pytest.mark.parametrize("rows", [(3, 1, 1), (80, 60, 33)])
def test_bad_pages_hide_their_tokens(rows):
    for width in (None, 200):
        bad_pages(rows, width)


def bad_pages(rows, width):
    lens, ps, D = [100, 64, 40], 16, 128
    d, keys, values = batch(lens, rows, 4, 2, D, ps, BF, seed=4, width=width)
    seen = [torch.ones(n, dtype=torch.bool) for n in lens]
    pages = d["cache"].shape[0]
    for b, page, bad in ((0, 2, -1), (0, 6, pages), (1, 0, 2 ** 31 - 1), (1, 3, -2 ** 31), (2, 0, pages + 5),
                         (2, 1, -3), (2, 2, 10 ** 6)):
        d["tables"][b, page] = bad
        seen[b][page * ps:(page + 1) * ps] = False
    want = ref.attention(d["q"], keys, values, lens, d["starts"], seen)
    assert (want[0][-1] == 0).all()               # a sequence with no page left
    check_ways(d, want)


def test_lengths_and_rows_that_do_not_fit():
    """Lengths below none and past the table, starts that fall or pass the rows, rows behind the last sequence."""
    from layer_mhc_seam_amd import seam as S
    lens, rows, ps, D = [64, 64, 30], [1, 1, 1], 16, 64
    d, keys, values = batch(lens, rows, 4, 2, D, ps, BF, seed=5)
    want = ref.attention(d["q"], keys, values, [64, 0, 30], d["starts"])
    d["lens"] = torch.tensor([1000, -5, 30], dtype=torch.int32)
    check(run(d, single=True), want)
    want = ref.attention(d["q"], keys, values, [20, 0, 20], d["starts"])
    check(run(d, single=True, max_len=20), want)
    # rows 0 and 4 belong to nobody, and stay
    q = torch.randn(5, 4, D, generator=torch.Generator().manual_seed(7)).to(BF)
    d["lens"] = torch.tensor([64, 64, 30], dtype=torch.int32)
    out = torch.full((5, 4, D), 7.0, dtype=BF).cuda()
    lse = torch.full((5, 4), 9.0).cuda()
    starts = torch.tensor([1, 3, 3, 4], dtype=torch.int32).cuda()
    got = S.cache_attention(q.cuda(), d["cache"].cuda(), d["tables"].cuda(), d["lens"].cuda(), q_starts=starts,
                            lse=True, out=(out, lse))
    assert got[0] is out and (out[[0, 4]] == 7.0).all() and (lse[[0, 4]] == 9.0).all()
    w = ref.attention(q, keys, values, lens, [1, 3, 3, 4])
    check((out[1:4], lse[1:4]), tuple(x[1:4] for x in w))
    # falling starts, and ones outside the rows: nothing is written outside, nothing read
    many = torch.randn(200, 4, D).to(BF)
    for rows in (q, many):
        T = len(rows)
        guard = torch.full((T + 64, 4, D), 7.0, dtype=BF).cuda()
        for bad in ([3, 1, 0, 2], [0, 9, 9, 9], [-4, 2, 1, 5], [2 ** 31 - 1, 0, 5, 2 ** 31 - 1], [-9, -8, -7, -6],
                    [0, T, T // 2, 2 * T]):
            S.cache_attention(rows.cuda(), d["cache"].cuda(), d["tables"].cuda(), d["lens"].cuda(), out=guard[32:T + 32],
                              q_starts=torch.tensor(bad, dtype=torch.int32).cuda())
        assert (guard[:32] == 7.0).all() and (guard[T + 32:] == 7.0).all()


def test_slices():
    """q inside a product's rows, tables inside wider ones."""
    from layer_mhc_seam_amd import seam as S
    lens, rows, ps, D, Hq = [64, 90, 30], [2, 5, 1], 16, 128, 6
    d, keys, values = batch(lens, rows, Hq, 2, D, ps, BF, seed=6, width=9)
    want = ref.attention(d["q"], keys, values, lens, d["starts"])
    wide = torch.randn(8, 10 * D).to(BF).cuda()
    q = wide[:, 2 * D:2 * D + Hq * D].view(8, Hq, D)
    q.copy_(d["q"])
    tables = torch.full((3, 20), 2 ** 30, dtype=torch.int32).cuda()
    tables[:, 5:14] = d["tables"].cuda()
    starts = torch.tensor(d["starts"], dtype=torch.int32).cuda()
    got = S.cache_attention(q, d["cache"].cuda(), tables[:, 5:14], d["lens"].cuda(), q_starts=starts, lse=True)
    check(got, want)
    plain = S.cache_attention(q, d["cache"].cuda(), tables[:, 5:14], d["lens"].cuda(), q_starts=starts)
    assert torch.equal(plain, got[0])


def test_many_sequences():
    """More sequences than a worker adds up, and blocks for every CU many times over."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 60, (1500,), generator=g).tolist()
    both(lens, [1] * 1500, 2, 1, 64, 16, BF)
    rows = torch.randint(0, 4, (1500,), generator=g).tolist()
    both(lens, rows, 4, 2, 64, 16, BF)
    both([40] * 300, [1] * 300, 16, 16, 64, 16, F16)


@pytest.mark.parametrize("B", [1, 3, 64, 65, 200])
def test_shares(B):
    """Workers' shares that begin and end anywhere in blocks of very unequal sequences."""
    g = torch.Generator().manual_seed(B)
    lens = (torch.rand(B, generator=g) ** 6 * 9000).long().tolist()
    lens[-1] = 5000
    both(lens, [1] * B, 2, 1, 64, 64, BF)


def test_far_pages():
    """A cache past 4 GiB whose last pages are read."""
    from layer_mhc_seam_amd import seam as S
    ps, D, Hk, L = 512, 128, 16, 1100
    pages = 5000
    cache = S.kv_cache(pages, Hk, D, ps)
    assert cache.numel() > 5 << 30
    g = torch.Generator().manual_seed(8)
    k, v = torch.randn(L, Hk, D, generator=g).to(BF), torch.randn(L, Hk, D, generator=g).to(BF)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32)
    t = torch.arange(L)
    small, hk, hv = ref.packed(k, v, (table[0][t // ps].long() - (pages - 3)) * ps + t % ps, 3, ps)
    cache[pages - 3:] = small.cuda()
    q = torch.randn(1, 32, D, generator=g).to(BF)
    got = S.cache_attention(q.cuda(), cache, table.cuda(), torch.tensor([L], dtype=torch.int32).cuda(), lse=True)
    check(got, ref.attention(q, [hk], [hv], [L], [0, 1]))


def test_device_refusals():
    from layer_mhc_seam_amd import seam as S
    d, _, _ = batch([64, 30], [1, 1], 4, 2, 64, 16, BF)
    q, c, tb, n = (d[k].cuda() for k in ("q", "cache", "tables", "lens"))
    for call in (lambda: S.cache_attention(q, c, tb.long(), n), lambda: S.cache_attention(q, c, tb, n.long()),
                 lambda: S.cache_attention(q, c, tb, n[:1]), lambda: S.cache_attention(q, c, tb.cpu(), n),
                 lambda: S.cache_attention(q, c, tb, n, q_starts=n), lambda: S.cache_attention(q, c, tb, n, max_len=0),
                 lambda: S.cache_attention(q, c[:, :, :-1].contiguous(), tb, n),
                 lambda: S.cache_attention(q, c, tb, n, out=q.half()),
                 lambda: S.cache_attention(q, c, tb, n, lse=True, out=(q.clone(), q)),
                 lambda: S.cache_attention(q, c, tb.t().contiguous().t(), n)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: S.cache_attention(q[:1], c, tb, n), lambda: S.cache_attention(q[:, :3].contiguous(), c, tb, n),
                 lambda: S.cache_attention(q, c, tb, n, out=q), lambda: S.cache_attention(q, c, tb, n, window=-1),
                 lambda: S.cache_attention(q, c, tb, n, softcap=-1.0)):
        with pytest.raises(S.SeamError):
            call()


def test_nothing_to_do():
    from layer_mhc_seam_amd import seam as S
    d, _, _ = batch([64], [1], 4, 2, 64, 16, BF)
    none = torch.zeros(0, dtype=torch.int32).cuda()
    out = S.cache_attention(d["q"][:0].cuda(), d["cache"].cuda(), d["tables"][:0].cuda(), none)
    assert out.shape == (0, 4, 64)
    out = S.cache_attention(d["q"][:0].cuda(), d["cache"].cuda(), d["tables"].cuda(), d["lens"].cuda(),
                            q_starts=torch.zeros(2, dtype=torch.int32).cuda())
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("T,B", [(5, 3), (40, 64), (300, 4), (300, 40), (2000, 130), (2000, 4), (40000, 3)])
def test_starts_that_fall_where_work_is_shared(T, B):
    """Tables for 4096 tokens, starts to and fro: blocks that two sequences have, or none, and more work than there
    are rows for.  Whatever the rows hold then, nothing is written outside of them and the call ends."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(T)
    ps, D, pages = 16, 64, 300
    cache = S.kv_cache(pages, 2, D, ps)
    cache.fill_(0)
    tables = torch.randint(-2, pages + 2, (B, 256), generator=g).to(torch.int32).cuda()
    lens = torch.randint(0, 4097, (B,), generator=g).to(torch.int32).cuda()
    q = torch.randn(T, 4, D, generator=g).to(BF).cuda()
    guard = torch.full((T + 64, 4, D), 7.0, dtype=BF).cuda()
    sums = torch.full((T + 64, 4), 9.0).cuda()
    for starts in ([0, T] * (B // 2 + 1), [T, 0, T // 2] * B, torch.randint(-3, T + 4, (B + 1,), generator=g).tolist()):
        S.cache_attention(q, cache, tables, lens, q_starts=torch.tensor(starts[:B + 1], dtype=torch.int32).cuda(),
                          lse=True, out=(guard[32:T + 32], sums[32:T + 32]))
    torch.cuda.synchronize()
    assert (guard[:32] == 7.0).all() and (guard[T + 32:] == 7.0).all()
    assert (sums[:32] == 9.0).all() and (sums[T + 32:] == 9.0).all()


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("cap", [5.0, 64.0, 65.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("lens,rows", [((300, 41), (1, 1)), ((250, 90), (100, 5)), ((330, 140), (200, 140))])
def test_capped_scores(lens, rows, cap, dt):
    """A capped score is good to its own bits, however large the cap: far above the scores it changes nothing."""
    for D, sharp in ((64, 1.0), (128, 4.0), (256, 30.0)):
        d, keys, values = batch(lens, rows, 4, 2, D, 16, dt, seed=D, sharp=sharp)
        want = ref.attention(d["q"], keys, values, lens, d["starts"], softcap=cap, relative=cap > 64)
        check_ways(d, want, single=max(rows) == 1, softcap=cap)
        if cap >= 1e30:
            free = ref.attention(d["q"], keys, values, lens, d["starts"])
            assert torch.equal(free[0], want[0]) or (free[0] - want[0]).abs().max() < 1e-12


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [(1, 3, 1, 2), (70, 129, 1, 100)])
@pytest.mark.parametrize("dt,byte", [(BF, 254), (F16, 254), (F16, 150)])
def test_what_nobody_sees_may_be_infinite(dt, byte, rows, D):
    """Codes and scales that are past the type's range everywhere but in the tokens, before a window above all."""
    lens, ps = [70, 129, 1, 260], 32
    for kw in ({}, dict(window=40), dict(window=33, causal=False), dict(window=7, softcap=20.0)):
        d, keys, values = batch(lens, rows, 4, 2, D, ps, dt, seed=2)
        dirty = torch.full_like(d["cache"], 0x77)            # 6, and 6
        dirty[:, :, ps * D:] = byte
        for b, n in enumerate(lens):
            for t in range(max(0, n - rows[b] + 1 - kw.get("window", n)), n):
                page, at = int(d["tables"][b, t // ps]), t % ps
                for kind in range(2):
                    c = kind * ps * D // 2 + at * D // 2
                    s = ps * D + kind * ps * D // 32 + torch.arange(D // 32) * ps + at
                    dirty[page, :, c:c + D // 2] = d["cache"][page, :, c:c + D // 2]
                    dirty[page, :, s] = d["cache"][page, :, s]
        d["cache"] = dirty
        check_ways(d, ref.attention(d["q"], keys, values, lens, d["starts"], **kw), **kw)


def test_longest_length_past_the_table():
    """max_len beyond what the tables hold says nothing new, whatever the workspace of such a length would be."""
    for B, Hq, Hk, n in ((64, 40, 8, 0), (1, 8, 2, 0), (3, 12, 4, 150)):
        lens = [200 - b for b in range(B)] if n == 0 else [n + 30, n, n + 7]
        rows = [1] * B if n == 0 else [n] * B
        d, keys, values = batch(lens, rows, Hq, Hk, 64, 64, BF, seed=B)
        d = widened(d, 8192)
        want = ref.attention(d["q"], keys, values, lens, d["starts"])
        plain = run(d, single=n == 0)
        check(plain, want)
        for most in (8193, 1 << 20, 1 << 29, 1 << 30, (1 << 31) - 1, 1 << 40):
            got = run(d, single=n == 0, max_len=most)
            assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("rows", [1, 400])
def test_workspace_refusals(rows):
    """A workspace that is missing, too small, or over what the call reads or writes: refused, and nothing is done."""
    import ctypes
    from layer_mhc_seam_amd import seam as S
    B, Hq, Hk, D, ps, width = 2, 8, 2, 128, 64, 80
    T = B * rows
    size = S.cache_attention_workspace(T, B, Hq, Hk, D, S._compute_units(0), width * ps)
    assert size > 0
    q = torch.randn(T, Hq, D).to(BF).cuda()
    cache = S.kv_cache(8, Hk, D, ps)
    tables, lens = torch.zeros(B, width, dtype=torch.int32).cuda(), torch.full((B,), 256, dtype=torch.int32).cuda()
    starts = torch.arange(0, T + 1, rows, dtype=torch.int32).cuda()
    out, lse = torch.full_like(q, 3.0), torch.full((T, Hq), 4.0).cuda()
    space = torch.empty(size, dtype=torch.uint8).cuda()

    def call(workspace, nbytes):
        a = S.CacheAttentionArgs(T, 0, 8, Hq * D, D, width, B, Hq, Hk, D, ps, width, 0, 1, 0, 0.1, 0.0, 0, q.data_ptr(),
                                 cache.data_ptr(), tables.data_ptr(), lens.data_ptr(), starts.data_ptr(), out.data_ptr(),
                                 lse.data_ptr(), workspace, nbytes)
        return S.lib().mhc_cache_attention(ctypes.byref(a), torch.cuda.current_stream().cuda_stream)

    for t in (q, cache, tables, lens, starts, out, lse):
        assert call(t.data_ptr(), size) == S.INVALID_ARG
        # ends inside the tensor, by 16 bytes
        assert call((t.data_ptr() + 15) // 16 * 16 - size // 16 * 16 - (16 if size % 16 else 0) + 16, size) == S.INVALID_ARG
    assert call(None, size) == call(space.data_ptr(), size - 1) == call(space.data_ptr() + 4, size) == S.INVALID_ARG
    torch.cuda.synchronize()
    assert (out == 3.0).all() and (lse == 4.0).all()
    assert call(space.data_ptr(), size) == S.OK
    torch.cuda.synchronize()
    assert not (out == 3.0).any() and not (lse == 4.0).any()

"""Expert routing on the GPU against the plain definition in binary64.

Ids are equal: both sides choose by binary64 keys, and inputs whose keys
differ by less than a few of its last places are exact ties (equal logits).
Weights are binary64 until their one rounding: 2^-24 relative, and 2^-40 for
the difference of two binary64 evaluations."""
import math
import random

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(logits, k, scoring="softmax", bias=None, groups=1, keep=1, top=1, renorm=True, scale=1.0):
    from layer_mhc_seam_amd.seam import route
    w, ids = route(logits.cuda(), k, scoring=scoring, bias=None if bias is None else bias.cuda(), groups=groups,
                   topk_groups=keep, group_top=top, renormalize=renorm, scale=scale)
    w, ids = w.cpu().double(), ids.cpu()
    want_w, want = ref.route(logits, k, scoring, bias, groups, keep, top, renorm, scale)
    bad = (ids != want).any(1).nonzero()
    assert not len(bad), f"{len(bad)} rows differ, first {bad[0].item()}: {ids[bad[0]]} for {want[bad[0]]}"
    nan = want_w.isnan()
    assert torch.equal(w.isnan(), nan)
    err = (w - want_w).abs()[~nan]
    assert (err <= (2.0 ** -24 + 2.0 ** -40) * want_w.abs()[~nan] + 2.0 ** -149).all()
    return w, ids


# experts: one, below, at and past a wave's and every change of the
# kernel's; groups of one, odd and even sizes, as many as there may be
@pytest.mark.parametrize("E,k,groups,keep,top", [
    (1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (8, 2, 1, 1, 1), (8, 2, 4, 2, 1), (63, 5, 1, 1, 1), (64, 6, 8, 3, 1),
    (64, 64, 1, 1, 1), (64, 64, 64, 64, 1), (65, 8, 5, 2, 2), (100, 7, 4, 1, 2), (127, 3, 1, 1, 1),
    (128, 8, 8, 4, 2), (129, 8, 3, 2, 2), (160, 6, 8, 3, 1), (160, 6, 1, 1, 1), (256, 8, 8, 4, 2),
    (256, 8, 1, 1, 1), (257, 9, 1, 1, 1), (384, 8, 1, 1, 1), (384, 8, 8, 4, 2), (512, 10, 16, 5, 2),
    (513, 4, 27, 9, 2), (700, 33, 7, 3, 2), (1000, 1, 1, 1, 1), (1024, 64, 64, 13, 2), (1024, 8, 1, 1, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_matches_definition(E, k, groups, keep, top, scoring):
    g = torch.Generator().manual_seed(E + k)
    for i, dt in enumerate(DTYPES):
        T = (1, 5, 67)[i]
        logits = (1.5 * torch.randn(T, E, generator=g)).to(dt)
        bias = 0.1 * torch.randn(E, generator=g)
        check(logits, k, scoring, None, groups, keep, top)
        check(logits, k, scoring, bias, groups, keep, top, renorm=i != 1, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_route_ties_go_to_the_lowest_index(scoring, groups, keep, top):
    """All equal; few distinct values; equal rows but one."""
    g = torch.Generator().manual_seed(1)
    l = torch.randint(-2, 3, (40, 128), generator=g).float()
    l[0] = 0.25
    l[1] = 0.25
    l[1, 77] = 0.5
    w, ids = check(l, 6, scoring, None, groups, keep, top)
    assert ids[0].tolist() == [0, 1, 2, 3, 4, 5]
    check(l, 6, scoring, torch.zeros(128), groups, keep, top)
    check(l, 6, scoring, torch.randint(-1, 2, (128,), generator=g).float() * 0.25, groups, keep, top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_near_ties(scoring, bias):
    """Logits one or two units of the last place apart, in a shuffled order:
    scores that binary32 cannot tell from each other."""
    g = torch.Generator().manual_seed(2)
    base = torch.tensor([0.7, 1.3, -2.1, 5.5]).repeat_interleave(10)[:, None]
    bits = base.expand(40, 96).contiguous().view(torch.int32) + torch.stack(
        [torch.randperm(96, generator=g) for _ in range(40)]).int()
    check(bits.view(torch.float32), 8, scoring, 0.01 * torch.ones(96) if bias else None)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (8, 2, 1), (8, 2, 2)])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masks(scoring, groups, keep, top, bias):
    """Experts out by -inf logits and by -inf bias: fewer than k left, one,
    none; whole groups out; groups with a single expert left."""
    g = torch.Generator().manual_seed(3)
    E = 64
    l = torch.randn(60, E, generator=g)
    share = torch.linspace(0, 1, 60)[:, None]
    l = l.masked_fill(torch.rand(60, E, generator=g) < share, -math.inf)
    l[0] = -math.inf
    l[1] = -math.inf
    l[1, 63] = -3.0
    l[2, :56] = -math.inf
    b = 0.1 * torch.randn(E, generator=g) if bias else None
    if bias:
        b[5] = -math.inf
        b[40:48] = -math.inf
    w, ids = check(l, 5, scoring, b, groups, keep, top)
    assert (ids[0] == -1).all() and (w[0] == 0).all()
    assert ids[1].tolist() == [63, -1, -1, -1, -1]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_lowest_values_infinities_and_nan(scoring):
    """The types' lowest and largest values, infinities and NaN: ids distinct
    and in range always."""
    for dt in DTYPES:
        f = torch.finfo(dt)
        l = torch.randn(12, 40).to(dt)
        l[0] = f.min
        l[1, 3:] = f.min
        l[2, 7] = f.max
        l[3] = f.max
        l[4, 9] = math.inf
        l[5, 9] = math.nan
        l[6] = math.nan
        l[7] = math.inf
        l[8, 0], l[8, 1], l[8, 2] = math.nan, math.inf, -math.inf
        l[9] = 60000.0
        l[10] = -60000.0
        w, ids = check(l, 6, scoring)
        assert w[5].isnan().all() and (ids[6] == -1).all()
        check(l, 6, scoring, torch.randn(40), 4, 2, 2)
    b = torch.zeros(40)
    b[3] = math.inf
    _, ids = check(torch.randn(3, 40), 4, scoring, b)
    assert (ids[:, 0] == 3).all()


def test_route_vanishing_scores():
    """Sigmoid scores that vanish in binary64: their sum is 0, weights are 0
    and ids stay those of the lowest indices."""
    w, ids = check(torch.full((2, 16), -800.0), 3, "sigmoid")
    assert ids[0].tolist() == [0, 1, 2] and (w == 0).all()


def test_route_unaligned_rows_and_given_outputs():
    from layer_mhc_seam_amd.seam import route
    for dt in DTYPES:
        buf = torch.randn(7 * 37 + 3).to(dt).cuda()
        l = buf[3:].view(7, 37)
        w, ids = (torch.full((7 * 5 + 16,), 9, dtype=t, device="cuda") for t in (torch.float32, torch.int32))
        route(l, 5, out=(w[:35].view(7, 5), ids[:35].view(7, 5)))
        want = ref.route(l.cpu(), 5, "softmax", None, 1, 1, 1, True, 1.0)
        assert torch.equal(ids[:35].view(7, 5).cpu(), want[1])
        assert (w[35:] == 9).all() and (ids[35:] == 9).all()


def test_route_many_tokens():
    g = torch.Generator().manual_seed(4)
    l = torch.randn(4160, 256, generator=g)
    check(l, 8, "sigmoid", 0.05 * torch.randn(256, generator=g), 8, 4, 2, scale=2.5)


def test_route_stream_graph_and_empty():
    from layer_mhc_seam_amd.seam import route
    l = torch.randn(65, 256, device="cuda")
    b = 0.1 * torch.randn(256, device="cuda")
    kw = dict(scoring="sigmoid", bias=b, groups=8, topk_groups=4, group_top=2)
    want = route(l, 8, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = tuple(torch.empty_like(t) for t in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        route(l, 8, **kw, out=out, stream=s)
    for _ in range(3):
        for t in out:
            t.zero_()
        route(l, 8, **kw)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    w, ids = route(torch.empty(0, 8, device="cuda"), 2)
    assert w.shape == (0, 2) and ids.shape == (0, 2)


def test_route_refusals():
    from layer_mhc_seam_amd.seam import SeamError, route
    l = torch.randn(4, 16, device="cuda")
    for call in (lambda: route(l.t(), 2), lambda: route(l.double(), 2), lambda: route(l[0], 2),
                 lambda: route(l, 2, bias=torch.zeros(8, device="cuda")),
                 lambda: route(l, 2, bias=torch.zeros(16)), lambda: route(l, 2, scoring="tanh"),
                 lambda: route(l, 2, out=(torch.empty(4, 2, device="cuda"),) * 2)):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(k=17), dict(k=0), dict(k=2, groups=3), dict(k=2, groups=4, topk_groups=5),
               dict(k=2, groups=16, group_top=2), dict(k=9, groups=4, topk_groups=2)):
        with pytest.raises(SeamError):
            route(l, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_logits_that_scores_cannot_tell(scoring):
    """Without a bias the order is the logits': where scores saturate or
    vanish in binary64, and beside zero."""
    l = torch.tensor([[40.0, 41, 42, 43, 44, 45, 46, 47], [-800, -801, -900, -790, -795, -1000, -799, -2000],
                      [0.0, 1e-30, -1e-30, 1e-38, -0.0, 2e-30, 0.0, -5.0]])
    _, ids = check(l, 4, scoring)
    assert ids[0].tolist() == [7, 6, 5, 4] and ids[1].tolist() == [3, 4, 6, 0] and ids[2].tolist() == [5, 1, 3, 0]
    check(l, 4, scoring, None, 2, 1, 1)
    check(l, 4, scoring, None, 4, 2, 2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep", [(256, 8, 4), (192, 16, 5), (96, 2, 1), (160, 4, 3), (512, 8, 3)])
def test_route_equal_and_near_group_sums(scoring, E, groups, keep):
    """Groups that hold the same experts' scores: equal sums on both sides of
    the border, and sums a few units of binary32's last place apart."""
    g = torch.Generator().manual_seed(E)
    base = torch.randn(30, 1, E // groups, generator=g)
    l = base.expand(30, groups, E // groups).contiguous()
    l[10:20] = (l[10:20].view(torch.int32) + torch.randint(-2, 3, l[10:20].shape, generator=g).int()).view(torch.float32)
    l[20:, 1::2] += 1e-6
    l = l.view(30, E)
    for dt in DTYPES:
        for bias in (None, torch.zeros(E), 0.25 * torch.ones(E)):
            for top in (1, 2):
                check(l.to(dt), 4, scoring, bias, groups, keep, top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_biases_of_every_size(scoring):
    """A bias far above the scores, which they hardly show beside, far below,
    of both signs, one expert out by -inf, all out."""
    g = torch.Generator().manual_seed(7)
    l = torch.randn(20, 256, generator=g)
    for b in (100 * torch.randn(256, generator=g), 1e6 + torch.zeros(256), 1e-9 * torch.randn(256, generator=g),
              1e30 * torch.randn(256, generator=g), torch.zeros(256).index_fill(0, torch.arange(0, 256, 3), -math.inf),
              torch.full((256,), -math.inf)):
        check(l, 8, scoring, b)
        check(l, 8, scoring, b, 8, 4, 2)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 4161])
def test_route_rows_beside_each_other(T):
    """Rows that need the binary64 choice among rows that do not, at every
    place of four, and a last wave that is not full."""
    g = torch.Generator().manual_seed(T)
    l = torch.randn(T, 64, generator=g)
    l[::3] = 0.5
    l[1::7, 5:] = -math.inf
    for E, k in ((64, 8), (63, 16)):
        check(l[:, :E].contiguous(), k, "sigmoid", 0.1 * torch.randn(E, generator=g))
        check(l[:, :E].contiguous(), k, "softmax")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm,scale", [(True, 1.0), (False, -2.5)])
def test_route_rows_of_masked_experts_only(dt, scoring, renorm, scale):
    """A padded batch's rows, with every expert masked, at every place of
    four, beside rows with one expert left, and one that holds a NaN too."""
    g = torch.Generator().manual_seed(12)
    for T, E, k, groups, keep, top in ((37, 160, 6, 1, 1, 1), (41, 64, 16, 8, 4, 2), (7, 512, 3, 16, 2, 1)):
        l = torch.randn(T, E, generator=g).to(dt)
        l[torch.rand(T, generator=g) < 0.6] = -math.inf
        l[3] = -math.inf
        l[4] = -math.inf
        l[4, E - 1] = 1.0
        l[5] = -math.inf
        l[5, E // 2] = math.nan
        for b in (None, 0.1 * torch.randn(E, generator=g)):
            w, ids = check(l, k, scoring, b, groups, keep, top, renorm, scale)
            assert (ids[3] == -1).all() and (w[3] == 0).all()
            assert ids[4].tolist() == [E - 1] + [-1] * (k - 1)
            assert (ids[5] == -1).all() and w[5].isnan().all()


@pytest.mark.parametrize("groups", [3, 5, 6, 7, 9, 11, 12, 13, 15])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_groups_that_do_not_divide_a_row(groups, scoring):
    """Groups with lanes of a row to spare: few experts and many, masked
    groups, equal and near sums, one group kept and all but one."""
    g = torch.Generator().manual_seed(groups)
    for size in (2, 5, 17, 31):
        E = groups * size
        l = torch.randn(24, E, generator=g)
        l[::5] = l[::5].masked_fill(torch.rand(5, E, generator=g) < 0.7, -math.inf)
        l[1, :E - size] = -math.inf
        l[2] = l[2, :size].repeat(groups)
        l[3] = (l[2].view(torch.int32) + torch.randint(-2, 3, (E,), generator=g).int()).view(torch.float32)
        l[4] = -math.inf
        for dt in DTYPES:
            for bias in (None, 0.1 * torch.randn(E, generator=g)):
                for keep, top in ((1, 1), (1, 2), (groups - 1, 1), (groups - 1, 2), (groups, 1)):
                    check(l.to(dt), min(2, size), scoring, bias, groups, keep, top)


@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_route_borders_in_every_wave(scoring, renorm):
    """Close experts and close groups at every place of four, with a bias
    that is not the same for all."""
    g = torch.Generator().manual_seed(21)
    E, groups = 128, 8
    b = 0.1 * torch.randn(E // groups, generator=g).repeat(groups)
    for step in (0.0, 2e-7, 1e-6, 1e-4):
        l = torch.randn(50, 1, E // groups, generator=g) + step * torch.randn(50, groups, 1, generator=g)
        l = l.expand(50, groups, E // groups).reshape(50, E)
        for top in (1, 2):
            check(l, 6, scoring, b, groups, 3, top, renorm)
        check(l, 6, scoring, b, 1, 1, 1, renorm)


def test_route_more_tokens_than_a_grid_line_holds():
    from layer_mhc_seam_amd.seam import route
    T = 270_000_003
    l = torch.zeros(T, 2, dtype=torch.float16, device="cuda")
    at = torch.tensor([0, 1, 33554431, 33554432, 268435455, 268435456, T - 2, T - 1], device="cuda")
    l[at, 1] = 1.0
    w, ids = route(l, 1)
    assert int(ids.sum()) == len(at) and (ids[at] == 1).all() and bool((w == 1).all())


def random_case(rng):
    E = rng.choice((rng.randint(1, 1024), rng.randint(1, 300), 8 * rng.randint(1, 64), 16 * rng.randint(1, 32)))
    groups = rng.choice([1] + [n for n in range(1, 65) if E % n == 0])
    size = E // groups
    keep = rng.randint(1, groups)
    top = rng.choice((1, 2)) if groups > 1 and size > 1 else 1
    k = rng.randint(1, min(rng.choice((8, 8, 16, 64)), keep * size))
    return dict(E=E, k=k, groups=groups, keep=keep, top=top, dt=rng.choice(DTYPES),
                scoring=rng.choice(("softmax", "sigmoid")), renorm=rng.random() < 0.7,
                scale=rng.choice((1.0, 2.5, -0.5)), bias=rng.choice((0.0, 0.05, 1.0, "masked")),
                mask=rng.choice(("none", "none", "some", "groups", "low", "lowest", "odd")),
                spread=rng.choice((1.5, 1.5, 0.05, 10.0, "few")))


@pytest.mark.parametrize("seed", range(48))
def test_route_many_rows_of_random_layouts(seed):
    """Thousands of rows of drawn layouts, types, biases and masks, so that
    experts and groups come as close as they do in a batch: every id equal to
    the binary64 choice.  Masks by -inf, by whole groups, by a large finite
    value or the type's lowest, NaN and infinities strewn in."""
    from layer_mhc_seam_amd.seam import route
    c = random_case(random.Random(seed))
    E, groups = c["E"], c["groups"]
    T = min(6000, (1 << 20) // E)
    g = torch.Generator().manual_seed(seed)
    # few values, and no x beside -x, whose sigmoids add up to 1 for every x
    l = 0.3 + torch.randint(-6, 7, (T, E), generator=g) / 8 if c["spread"] == "few" else \
        c["spread"] * torch.randn(T, E, generator=g)
    hit = torch.rand(T, E, generator=g) < 0.6 * torch.rand(T, 1, generator=g)
    if c["mask"] == "groups":
        hit = (torch.rand(T, groups, 1, generator=g) < 0.4).expand(T, groups, E // groups).reshape(T, E)
    if c["mask"] in ("some", "groups"):
        l = l.masked_fill(hit, -math.inf)
    elif c["mask"] == "low":
        l = l.masked_fill(hit, -1e4)
    elif c["mask"] == "lowest":
        l = l.masked_fill(hit, torch.finfo(c["dt"]).min)
    elif c["mask"] == "odd":
        for v in (math.nan, math.inf, -math.inf):
            l = l.masked_fill(torch.rand(T, E, generator=g) < 0.3 / E, v)
    l = l.to(c["dt"]).cuda()
    bias = None
    if c["bias"]:
        bias = 0.1 * torch.randn(E, generator=g)
        if c["bias"] == "masked":
            bias = bias.masked_fill(torch.rand(E, generator=g) < 0.2, -math.inf)
        else:
            bias = c["bias"] * bias
        bias = bias.cuda()
    w, ids = route(l, c["k"], scoring=c["scoring"], bias=bias, groups=groups, topk_groups=c["keep"],
                   group_top=c["top"], renormalize=c["renorm"], scale=c["scale"])
    want_w, want = ref.route_rows(l, c["k"], c["scoring"], bias, groups, c["keep"], c["top"], c["renorm"],
                                  c["scale"])
    bad = (ids != want).any(1).nonzero()
    assert not len(bad), f"{c}: {len(bad)} rows, first {bad[0].item()}: {ids[bad[0]]} for {want[bad[0]]}"
    nan = want_w.isnan()
    assert torch.equal(w.isnan(), nan)
    err = (w.double() - want_w).abs()[~nan]
    assert (err <= (2.0 ** -24 + 2.0 ** -40) * want_w.abs()[~nan] + 2.0 ** -149).all(), c

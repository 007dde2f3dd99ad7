"""The int8 product on the GPU, bit for bit: its sums are exact integers and
every step after them is a binary32 operation rounded once, so the plain
definition on the CPU (sums in binary64, exact) gives the same bits."""
import math

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gemm(*a, **kw):
    from layer_mhc_seam_amd.seam import int8_gemm
    a = [t.cuda() if torch.is_tensor(t) else t for t in a]
    out = int8_gemm(*a, **kw)
    torch.cuda.synchronize()
    return out.cpu()


def operands(T, N, K, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int32).to(torch.int8)
    b = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8)
    sa = 0.01 * torch.exp(torch.randn(T, generator=g))
    sb = 0.01 * torch.exp(torch.randn(N, generator=g))
    return a, sa, b, sb, (torch.randn(N, generator=g) if bias else None)


def check(got, a, sa, b, sb, bias, dt):
    want = ref.int8_gemm(a, sa, b, sb, bias, DTYPES[dt])
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    bad = ((got != want) & ~nan).nonzero()
    assert not len(bad), f"{len(bad)} differ, first {[(i, got[tuple(i)], want[tuple(i)]) for i in bad[:3].tolist()]}"


# T: one to a few rows, either side of 16, 32, 64, 128 and 256 rows and of
# the launch's changes of shape; N: odd, one, either side of the tiles;
# K: one piece, every remainder of a step, the deepest
SHAPES = [(1, 1, 16), (1, 16, 64), (1, 5120, 512), (2, 17, 48), (3, 33, 80), (4, 5120, 5120), (7, 100, 112),
          (8, 130, 8192), (15, 64, 144), (16, 512, 1024), (17, 31, 176), (31, 1000, 208), (32, 65, 240),
          (33, 129, 272), (64, 256, 5120), (65, 250, 304), (100, 1027, 1040), (127, 63, 128), (128, 128, 2048),
          (129, 255, 160), (200, 2000, 96), (255, 257, 192), (256, 4100, 224), (300, 300, 131056),
          (384, 5117, 336), (513, 2049, 400), (1000, 1111, 528), (1030, 4100, 128), (2100, 2000, 256),
          (4096, 517, 640), (4160, 256, 1024), (4097, 4099, 144)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_int8_gemm_matches_definition(T, N, K):
    c = operands(T, N, K, seed=T + N + K)
    for i, dt in enumerate(DTYPES):
        if T * N * K > 1 << 30 and i != (T + N) % 3:
            continue
        check(gemm(*c, out_dtype=dt), *c, dt)
    check(gemm(*c[:4]), *c[:4], None, "bf16")


@pytest.mark.parametrize("T,N,K", [(16384, 2048, 256), (16000, 2044, 272), (8191, 4111, 400), (4100, 5110, 1040)])
def test_int8_gemm_large_sampled(T, N, K):
    """Many blocks, ragged last ones: sampled rows, the first and last among
    them."""
    a, sa, b, sb, bias = operands(T, N, K, seed=T)
    got = gemm(a, sa, b, sb, bias)
    g = torch.Generator().manual_seed(T)
    at = torch.cat([torch.arange(4), torch.arange(252, 260), torch.arange(T - 12, T),
                    torch.randint(0, T, (60,), generator=g)])
    check(got[at], a[at], sa[at], b, sb, bias, "bf16")


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_int8_gemm_extreme_codes(T):
    """All codes -128 at the deepest K: the largest sum there is; and a
    different sign in each row."""
    K = 131056
    a = torch.full((T, K), -128, dtype=torch.int8)
    b = torch.full((24, K), -128, dtype=torch.int8)
    b[1::2] = 127
    one = torch.ones
    c = (a, one(T), b, one(24), None)
    got = gemm(*c, out_dtype="f32")
    check(got, *c, "f32")
    assert got[0, 0] == 128.0 * 128 * K


def test_int8_gemm_selects_columns():
    """One-hot weights pick codes out of the rows, wherever K they stand:
    every byte of both operands meets its own K."""
    T, K = 40, 400
    a = torch.randint(-128, 128, (T, K), dtype=torch.int32).to(torch.int8)
    b = torch.eye(K, dtype=torch.int8)
    for t in (T, 5):
        got = gemm(a[:t].contiguous(), torch.ones(t), b, torch.ones(K), out_dtype="f32")
        assert torch.equal(got, a[:t].float())


@pytest.mark.parametrize("T,N", [(3, 40), (50, 70), (300, 600)])
def test_int8_gemm_special_scales(T, N):
    """NaN, infinite, zero and negative scales, over zero codes too."""
    a, sa, b, sb, bias = operands(T, N, 96, seed=4)
    a[1] = 0
    sa[1] = math.nan
    sb[2] = math.nan
    sa[2] = math.inf
    sb[3] = -0.5
    sb[4] = 0.0
    got = gemm(a, sa, b, sb, bias, out_dtype="f32")
    check(got, a, sa, b, sb, bias, "f32")
    assert got[1].isnan().all() and got[:, 2].isnan().all()


def test_int8_gemm_f16_overflow():
    a, sa, b, sb, _ = operands(20, 20, 512, seed=6, bias=False)
    got = gemm(a, sa * 1e4, b, sb * 1e4, out_dtype="f16")
    check(got, a, sa * 1e4, b, sb * 1e4, None, "f16")
    assert got.isinf().any()


@pytest.mark.parametrize("T,N,K", [(5, 37, 80), (64, 67, 208), (130, 131, 144), (520, 4099, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_int8_gemm_writes_nothing_else(T, N, K, dt):
    c = [t.cuda() for t in operands(T, N, K, seed=7)]
    buf = torch.full((T * N + 512,), 7.0, dtype=DTYPES[dt], device="cuda")
    gemm(*c, out_dtype=dt, out=buf[:T * N].view(T, N))
    assert (buf[T * N:] == 7).all()


def test_int8_gemm_offsets_past_32_bits():
    """Weights, and then activations and results, beyond 2^31 bytes."""
    K, N = 65536, 40000
    b = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    at = [0, 32767, 32768, N - 1]
    g = torch.Generator().manual_seed(9)
    rows = torch.randint(-128, 128, (len(at), K), generator=g, dtype=torch.int32).to(torch.int8)
    b[at] = rows.cuda()
    a = torch.randint(-128, 128, (2, K), generator=g, dtype=torch.int32).to(torch.int8)
    got = gemm(a, torch.ones(2), b, torch.ones(N), out_dtype="f32")
    check(got[:, at], a, torch.ones(2), rows, torch.ones(len(at)), None, "f32")
    got = gemm(b, torch.ones(N), a, torch.ones(2), out_dtype="f32")
    check(got[at], rows, torch.ones(len(at)), a, torch.ones(2), None, "f32")
    del b
    T, N, K = 300000, 4100, 16
    a = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int32).to(torch.int8)
    b = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8)
    from layer_mhc_seam_amd.seam import int8_gemm
    got = int8_gemm(a.cuda(), torch.ones(T, device="cuda"), b.cuda(), torch.ones(N, device="cuda"))
    at = torch.tensor([0, 1, 261000, 262000, 299999])
    check(got[at.cuda()].cpu(), a[at], torch.ones(5), b, torch.ones(N), None, "bf16")


def test_int8_gemm_stream_graph_and_empty():
    from layer_mhc_seam_amd.seam import int8_gemm
    s = torch.cuda.Stream()
    cases = []
    for T, N, K in ((1, 512, 1024), (40, 300, 640), (600, 2000, 256)):
        c = [t.cuda() for t in operands(T, N, K, seed=T)]
        want = int8_gemm(*c)
        cases.append((c, want, torch.empty_like(want)))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for c, _, out in cases:
            int8_gemm(*c, out=out, stream=s)
    for _ in range(3):
        for c, _, out in cases:
            out.zero_()
            int8_gemm(*c)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for _, want, out in cases:
            assert torch.equal(out, want)
    e = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    b = torch.zeros(5, 64, dtype=torch.int8, device="cuda")
    assert int8_gemm(e, torch.empty(0, device="cuda"), b, torch.ones(5, device="cuda")).shape == (0, 5)


def test_int8_gemm_refusals():
    from layer_mhc_seam_amd.seam import SeamError, int8_gemm
    a, sa, b, sb, bias = [t.cuda() for t in operands(4, 8, 64, seed=1)]
    for call in (lambda: int8_gemm(a, sa[:3], b, sb), lambda: int8_gemm(a, sa, b[:, :48], sb),
                 lambda: int8_gemm(a, sa, b, sb.double()), lambda: int8_gemm(a.float(), sa, b, sb),
                 lambda: int8_gemm(a, sa, b.view(torch.uint8), sb), lambda: int8_gemm(a, sa.cpu(), b, sb),
                 lambda: int8_gemm(a, sa, b, sb, bias[:4]), lambda: int8_gemm(a.t(), sa, b, sb),
                 lambda: int8_gemm(a, sa, b, sb, out=torch.empty(4, 8, device="cuda")),
                 lambda: int8_gemm(a, sa, b, sb, out_dtype="i32")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(SeamError):
        int8_gemm(a[:, :24].contiguous(), sa, b[:, :24].contiguous(), sb)


# one shape, or more, for each of the launch's blocks: whole and ragged rows
# and columns, K of one step, of several, and ending inside one
BLOCK_SHAPES = [(16, 320, 512), (9, 333, 1040), (16, 5120, 512), (7, 5003, 1552), (30, 5120, 256),
                (27, 5100, 784), (90, 4000, 512), (70, 5099, 1296), (180, 5120, 256), (150, 4001, 528), (250, 5120, 768), (270, 4999, 272),
                (380, 5120, 512), (300, 5111, 800), (700, 5120, 256), (600, 5117, 400), (1000, 5120, 128),
                (900, 5101, 656), (1500, 5120, 384), (1300, 5110, 144), (2000, 5120, 256), (1900, 5109, 304),
                (2500, 5120, 128), (2400, 5103, 272), (5000, 5120, 640), (6100, 5099, 16)]


def test_block_shapes_cover_every_block():
    from layer_mhc_seam_amd.seam import int8_gemm_blocks
    seen = {}
    for T, N, _ in BLOCK_SHAPES:
        seen.setdefault(int8_gemm_blocks(T, N, 256), []).append((T, N))
    assert len(seen) == 12 and all(len(v) >= 2 for v in seen.values()), seen


@pytest.mark.parametrize("T,N,K", BLOCK_SHAPES)
@pytest.mark.parametrize("dt", list(DTYPES))
def test_int8_gemm_blocks_match_definition(T, N, K, dt):
    c = operands(T, N, K, seed=T + K)
    got = gemm(*c, out_dtype=dt)
    if T * N * K > 1 << 31:
        g = torch.Generator().manual_seed(K)
        at = torch.cat([torch.arange(3), torch.arange(T - 3, T), torch.randint(0, T, (200,), generator=g)])
        check(got[at], c[0][at], c[1][at], *c[2:], dt)
    else:
        check(got, *c, dt)

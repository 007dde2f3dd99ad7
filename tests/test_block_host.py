"""Host-side argument rules of the block norm, int8 quantiser and product and
expert routing (no GPU): every refusal comes before any device call, so the
pointers are fake addresses.  And pins of the plain definitions the GPU tests
compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_reference as ref
from layer_mhc_seam_amd import seam as S

BASE = 0x7f0000000000


def slot(k):
    return BASE + (k << 32)


def norm_args(T=4, H=512, **kw):
    a = S.BlockNormArgs(T, H, 0, 0, 0, 1e-6, 1.0, 1.0, 0)
    a.x, a.y, a.gamma, a.residual_out, a.norm = (slot(k) for k in range(5))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def block_norm(**kw):
    return S.lib().mhc_block_norm(ctypes.byref(norm_args(**kw)), None)


def message():
    return S.lib().mhc_seam_last_error().decode()


def test_struct_layouts():
    assert ctypes.sizeof(S.BlockNormArgs) == 8 + 4 * 4 + 3 * 4 + 4 + 9 * 8
    assert ctypes.sizeof(S.RouteArgs) == 8 + 8 * 4 + 4 + 4 + 4 * 8


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=32769), dict(H=32753), dict(H=32767), dict(T=1 << 30, H=1024),
    dict(dtype=2), dict(dtype=-1), dict(x_dtype=1), dict(x_dtype=3), dict(gate_kind=4),
    dict(gate_kind=-1), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=2.0),
    dict(residual_scale=math.inf), dict(branch_scale=math.nan), dict(reserved=1),
    dict(x=None), dict(y=None), dict(residual_out=None), dict(gamma=None), dict(norm=None),
    dict(gate=slot(6)), dict(gate_kind=1), dict(codes=slot(7)), dict(scales=slot(8)),
    dict(x=slot(0) + 8), dict(gamma=slot(2) + 2), dict(norm=slot(4) + 4),
    dict(codes=slot(7), scales=slot(8) + 2),
    dict(norm=slot(0)), dict(residual_out=slot(0) + 16), dict(norm=slot(1) + 64),
    dict(residual_out=slot(4)), dict(codes=slot(0), scales=slot(8)),
    dict(gate_kind=3, gate=slot(4) + 1024), dict(gate_kind=1, gate=slot(4)),
    dict(gamma_post=slot(3)),
])
def test_block_norm_refuses(kw):
    assert block_norm(**kw) == S.INVALID_ARG
    assert message()


def test_block_norm_without_a_branch_takes_no_branch_arguments():
    for kw in (dict(gamma_post=slot(5)), dict(gate_kind=1, gate=slot(5)), dict(residual_scale=0.5),
               dict(branch_scale=2.0), dict(residual_out=slot(3))):
        assert block_norm(y=None, **{"residual_out": None, **kw}) == S.INVALID_ARG
    assert block_norm(y=None, gamma=None, residual_out=None, norm=None) == S.INVALID_ARG
    assert block_norm(T=0, x=None, y=None, gamma=None) == S.OK


@pytest.mark.parametrize("rows,H,dtype,off", [(-1, 64, 0, 0), (1 << 31, 64, 0, 0), (4, 0, 0, 0),
                                              (4, 40000, 0, 0), (4, 32759, 0, 0), (4, 64, 2, 0), (4, 64, 0, 8),
                                              (1 << 30, 1024, 0, 0)])
def test_int8_quantize_refuses(rows, H, dtype, off):
    assert S.lib().mhc_int8_quantize(slot(0) + off, dtype, rows, H, slot(1), slot(2), None) == 1


def test_int8_quantize_pointer_rules():
    q = S.lib().mhc_int8_quantize
    assert q(None, 0, 4, 64, slot(1), slot(2), None) == 1
    assert q(slot(0), 0, 4, 64, None, slot(2), None) == 1
    assert q(slot(0), 0, 4, 64, slot(1), None, None) == 1
    assert q(slot(0), 0, 4, 64, slot(1), slot(2) + 1, None) == 1
    assert q(slot(0), 0, 4, 64, slot(0) + 256, slot(2), None) == 1       # codes inside src
    assert q(slot(0), 0, 4, 64, slot(1), slot(1) + 252, None) == 1       # scales inside codes
    assert q(None, 0, 0, 64, None, None, None) == 0


def gemm(a=slot(0), sa=slot(1), b=slot(2), sb=slot(3), bias=None, T=4, N=64, K=128, dt=0,
         out=slot(5)):
    return S.lib().mhc_int8_gemm(a, sa, b, sb, bias, T, N, K, dt, out, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(N=0), dict(N=-4), dict(K=0), dict(K=24), dict(K=131072),
    dict(dt=3), dict(dt=-1), dict(T=1 << 30, K=2048), dict(T=1 << 30, N=2048),
    dict(N=(1 << 31) - 1, K=1024), dict(a=None), dict(sa=None), dict(b=None), dict(sb=None),
    dict(out=None), dict(a=slot(0) + 8), dict(b=slot(2) + 4), dict(out=slot(5) + 2),
    dict(sa=slot(1) + 2), dict(sb=slot(3) + 1), dict(bias=slot(4) + 2),
    dict(out=slot(0) + 64), dict(out=slot(2)), dict(bias=slot(5) + 16)])
def test_int8_gemm_refuses(kw):
    assert gemm(**kw) == S.INVALID_ARG
    assert message()


def test_int8_gemm_nothing_to_do():
    assert gemm(T=0, a=None, out=None) == S.OK


def route_args(T=4, E=64, k=4, **kw):
    a = S.RouteArgs(T, E, k, 2, 0, 1, 1, 1, 1, 1.0, 0, slot(0), None, slot(1), slot(2))
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def route(**kw):
    return S.lib().mhc_route(ctypes.byref(route_args(**kw)), None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025), dict(T=1 << 30, E=1024), dict(dtype=3),
    dict(scoring=2), dict(groups=0), dict(groups=3), dict(E=1024, groups=128), dict(topk_groups=2),
    dict(topk_groups=0), dict(groups=8, topk_groups=9), dict(group_top=2), dict(group_top=0),
    dict(groups=4, group_top=3), dict(groups=64, group_top=2, topk_groups=8), dict(k=0),
    dict(k=65, E=128), dict(k=64, E=32), dict(groups=8, topk_groups=2, k=17),
    dict(renormalize=2), dict(scale=math.nan), dict(reserved=1), dict(logits=None),
    dict(weights=None), dict(ids=None), dict(logits=slot(0) + 2), dict(bias=slot(3) + 2),
    dict(weights=slot(1) + 1), dict(ids=slot(2) + 2), dict(ids=slot(1) + 16),
    dict(weights=slot(0) + 512), dict(bias=slot(2) + 32)])
def test_route_refuses(kw):
    assert route(**kw) == S.INVALID_ARG
    assert message()


def test_route_nothing_to_do():
    assert route(T=0, logits=None, weights=None, ids=None) == S.OK


def test_null_argument_structs():
    assert S.lib().mhc_block_norm(None, None) == S.INVALID_ARG
    assert S.lib().mhc_route(None, None) == S.INVALID_ARG


# The binding's own checks come before the library is asked for anything.

def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    g = torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: S.block_norm(x, g), lambda: S.int8_quantize(x),
                 lambda: S.int8_gemm(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4)),
                 lambda: S.route(torch.zeros(4, 8), 2)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    for call in (lambda: S.block_norm(x), lambda: S.block_norm(x[0], g),
                 lambda: S.block_norm(x, g.float()), lambda: S.int8_quantize(x.float()),
                 lambda: S.int8_quantize(x[0]), lambda: S.route(torch.zeros(8), 2),
                 lambda: S.route(torch.zeros(4, 8), 2, scoring="relu"),
                 lambda: S.route(torch.zeros(4, 8, dtype=torch.int32), 2),
                 lambda: S.int8_gemm(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4),
                                     out_dtype="f64")):
        with pytest.raises(ValueError):
            call()


# ----------------------------------------------- pins of the definitions --

def test_quantize_definition():
    """A row's largest value has code 127; ties go to even; a zero row, a row
    below the floor and rows holding an infinity or NaN."""
    v = torch.tensor([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5], [0.0] * 6, [2.0 ** -130] + [0.0] * 5,
                      [math.inf, 1, 2, 3, 4, 5], [1, math.nan, 2, 3, 4, 5]])
    codes, scales = ref.quantize(v)
    assert codes[0].tolist() == [127, -127, 0, 2, 2, 0] and scales[0] == 1.0
    assert codes[1:3].abs().max() == 0 and (scales[1:3] == np.float32(2.0 ** -119) / np.float32(127)).all()
    assert codes[3:].abs().max() == 0 and scales[3:].isnan().all()


def test_block_norm_definition():
    """Unit root mean square; the scales; a gate of zero leaves the stream."""
    g = torch.Generator().manual_seed(0)
    x, y = torch.randn(3, 64, generator=g), torch.randn(3, 64, generator=g).bfloat16()
    one = torch.ones(64, dtype=torch.bfloat16)
    r, n = ref.block_norm(x, one, y, None, torch.zeros(3, 1), 0.5, 3.0)
    assert torch.equal(r, 0.5 * x)
    assert (n.double().square().mean(1) - 1).abs().max() < 0.01
    r, _ = ref.block_norm(torch.zeros(3, 64), one, y, one, None, 1.0, 2.0, 0.0)
    assert (r.double().square().mean(1) - 4).abs().max() < 1e-5


def test_route_definition():
    """Closed forms: ties to the lowest index, groups, masks, NaN."""
    l = torch.tensor([[0.0, 2.0, 2.0, 1.0]])
    w, ids = ref.route(l, 2, "softmax", None, 1, 1, 1, True, 2.0)
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[1.0, 1.0]]
    w, ids = ref.route(l, 2, "sigmoid", torch.tensor([5.0, 0, 0, 0]), 1, 1, 1, False, 1.0)
    assert ids.tolist() == [[0, 1]] and abs(w[0, 0] - 0.5) < 1e-15       # the bias is not a weight
    w, ids = ref.route(l, 2, "sigmoid", None, 2, 1, 2, True, 1.0)
    assert ids.tolist() == [[2, 3]]                                      # 2 + 1 above 0 + 2
    w, ids = ref.route(torch.tensor([[-math.inf, 3.0], [-math.inf] * 2, [math.nan, 1.0]]), 2, "softmax",
                       None, 1, 1, 1, True, 1.0)
    assert ids.tolist() == [[1, -1], [-1, -1], [1, -1]]
    assert w[:2].tolist() == [[1.0, 0.0], [0.0, 0.0]] and w[2].isnan().all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_definitions_agree(scoring):
    """Many tokens at once choose as one token and one choice at a time."""
    g = torch.Generator().manual_seed(3)
    for E, k, groups, keep, top, renorm in ((1, 1, 1, 1, 1, True), (40, 6, 1, 1, 1, False), (64, 8, 8, 3, 1, True),
                                            (63, 9, 7, 2, 2, True), (96, 40, 48, 20, 2, False)):
        l = torch.randint(-8, 9, (60, E), generator=g) / 4
        l[::2] = torch.randn(30, E, generator=g)
        l = l.masked_fill(torch.rand(60, E, generator=g) < torch.linspace(0, 1.2, 60)[:, None], -math.inf)
        l[5, 0], l[6, E - 1] = math.nan, math.inf
        b = 0.1 * torch.randn(E, generator=g)
        b[E // 3] = -math.inf
        for bias in (None, b):
            w, ids = ref.route(l, k, scoring, bias, groups, keep, top, renorm, 1.5)
            w2, ids2 = ref.route_rows(l, k, scoring, bias, groups, keep, top, renorm, 1.5)
            assert torch.equal(ids, ids2) and torch.equal(w.isnan(), w2.isnan())
            # two evaluations in binary64: sums of up to 96 terms and k weights
            assert ((w - w2).abs().nan_to_num(0) <= 2.0 ** -44 * w.abs().nan_to_num(0)).all()


# ------------------------------------------- blocks of the int8 product --

def test_int8_gemm_blocks_by_token_count():
    """The launch's blocks at N = 5120 on 256 CUs over every change of shape
    (the shapes measured fastest there), and where one is chosen for filling
    the last round."""
    want = {1: (16, 32), 16: (16, 32), 17: (32, 32), 32: (32, 32), 33: (32, 64), 96: (32, 64),
            97: (64, 64), 192: (64, 64), 193: (96, 64), 288: (96, 64), 289: (128, 64), 384: (128, 64),
            385: (128, 128), 768: (128, 128), 769: (128, 192), 1024: (128, 192), 1280: (128, 256),
            1536: (128, 256), 2048: (192, 256), 2560: (256, 256), 4160: (192, 256), 6144: (256, 256),
            16384: (256, 256)}
    for T, shape in want.items():
        assert S.int8_gemm_blocks(T, 5120, 256) == shape, T
    assert S.int8_gemm_blocks(4160, 256, 256) == (96, 64)
    assert S.int8_gemm_blocks(1, 4096, 256) == (16, 16) and S.int8_gemm_blocks(1, 4097, 256) == (16, 32)
    assert S.int8_gemm_blocks(128, 256, 256) == (16, 16) and S.int8_gemm_blocks(384, 256, 256) == (16, 32)
    assert S.int8_gemm_blocks(128, 5120, 128) != S.int8_gemm_blocks(128, 5120, 256)


@pytest.mark.parametrize("T,N,cus", [(0, 5120, 256), (4, 0, 256), (4, 5120, 0), (1 << 31, 5120, 256)])
def test_int8_gemm_blocks_refuses(T, N, cus):
    with pytest.raises(S.SeamError):
        S.int8_gemm_blocks(T, N, cus)


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    """The launch is made with the tensors' device current and on its stream,
    and with no switch where it is current already."""
    import contextlib
    seen = []

    @contextlib.contextmanager
    def switched(index):
        seen.append(("to", index))
        yield
        seen.append(("back", index))

    def call(a, handle):
        seen.append((a, handle))
        return S.OK

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", switched)
    S._enqueue(1, call, "x")
    assert seen == [("to", 1), ("x", 101), ("back", 1)]
    seen.clear()
    S._enqueue(0, call, "x")
    assert seen == [("x", 100)]


def test_calls_on_a_stream(monkeypatch):
    """With the stream current, on its device only; what the call was given is
    recorded as used there."""
    import contextlib
    seen = []

    @contextlib.contextmanager
    def current(stream):
        seen.append("in")
        yield
        seen.append("out")

    class Stream:
        device = torch.device("cpu")

    def op(*args, **kw):
        seen.append((args, kw))
        return 5

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(t.item()))
    x, b, o1, o2 = (torch.tensor(i) for i in range(4))
    assert S._on_stream(Stream, op, x, 8, bias=b, gate=None, out=(o1, o2)) == 5
    assert seen[0] == "in" and seen[1][0][1] == 8 and seen[2:] == ["out", 0, 1, 2, 3]
    seen.clear()
    S._on_stream(Stream, op, x, None, out={"a": o1})
    assert seen[2:] == ["out", 0, 2]
    Stream.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="stream is on"):
        S._on_stream(Stream, op, x)


def test_calls_on_a_stream_keep_outputs_given_in_any_form(monkeypatch):
    """int8_quantize and route write to any pair, block_norm to any mapping:
    the tensors given are recorded as used on the stream whatever holds them,
    and each once."""
    import contextlib
    import types
    seen = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(t.item()))

    class Stream:
        device = torch.device("cpu")

    def pair(*args, out):
        first, second = out
        return first, second

    def named(*args, out):
        return dict(out)

    def one(*args, out):
        return out

    x, o1, o2 = (torch.tensor(i) for i in range(3))
    for op, out in ((pair, [o1, o2]), (pair, iter((o1, o2))), (pair, {o1: 0, o2: 0}.keys()),
                    (pair, (o1, o2)), (named, types.MappingProxyType({"a": o1, "b": o2})),
                    (named, [("a", o1), ("b", o2)]), (named, {"a": o1, "b": o2})):
        seen.clear()
        S._on_stream(Stream, op, x, out=out)
        assert sorted(seen) == [0, 1, 2], (op.__name__, type(out))
    seen.clear()
    assert S._on_stream(Stream, one, x, out=o1) is o1
    assert sorted(seen) == [0, 1]


def test_sizes_past_32_bits_are_refused():
    """ctypes would cut them to ones that the library takes."""
    S._fits(1 | 2 ** 31 - 1)
    for bad in (2 ** 31, 64 | 2 ** 32 + 64, 8 | -(2 ** 32) + 8):
        with pytest.raises(ValueError, match="out of range"):
            S._fits(bad)
    with pytest.raises(ValueError, match="out of range"):
        S.route(torch.zeros(2, 8), 2 ** 32 + 2)
    with pytest.raises(ValueError, match="out of range"):
        S.int8_gemm_blocks(16, 2 ** 32 + 16)

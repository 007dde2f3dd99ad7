"""Host-side rules of the rotary positions, the 4-bit cache and the attention
over it (no GPU): refusals of the C entries, which come before any device
call, so the pointers are fake addresses, and of the binding; the cache's
addresses, walked on the CPU with bad slots and pages; pins of the plain
definitions that the GPU tests compare with."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import cache_reference as ref
from layer_mhc_seam_amd import seam as S

HERE = os.path.dirname(os.path.abspath(__file__))
BASE = 0x7f0000000000
INF, NAN = math.inf, math.nan


def slot(k):
    return BASE + (k << 36)


def message():
    return S.lib().mhc_seam_last_error().decode()


def test_struct_layouts():
    assert ctypes.sizeof(S.RopeArgs) == 8 + 10 * 4 + 9 * 8 + 7 * 8
    assert ctypes.sizeof(S.CacheArgs) == 2 * 8 + 6 * 4 + 4 * 8 + 4 * 8
    assert ctypes.sizeof(S.CacheAttentionArgs) == 6 * 8 + 12 * 4 + 8 * 8 + 8


# ------------------------------------------------------------- addresses --

def test_layout_addresses(tmp_path):
    """Every slot and tile inside memory of the exact size, bad ones refused."""
    exe = tmp_path / "layout"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined",
                    os.path.join(HERE, "cache_layout_check.cpp"), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert got.returncode == 0 and got.stdout == "ok\n", got.stdout + got.stderr


def test_checks_do_not_overflow(tmp_path):
    """Sizes and strides at the ends of their types are refused before they are multiplied."""
    exe = tmp_path / "checks"
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    trap = [f for x in ("-fsanitize=signed-integer-overflow", "-fsanitize-trap=signed-integer-overflow")
            for f in ("-Xarch_host", x)]
    subprocess.run([hipcc, "--offload-arch=gfx950", "-std=c++17", "-O1", *trap, "-x", "hip",
                    os.path.join(HERE, "cache_arguments_check.cpp"), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert got.returncode == 0 and got.stdout == "ok\n", got.stdout + got.stderr


# ------------------------------------------------------------------ rope --

def rope_args(T=4, Hq=8, Hk=2, D=128, R=128, **kw):
    a = S.RopeArgs(T, Hq, Hk, D, R, 0, 4, 1, 0, 0, 1.0, T, Hq * D, D, Hk * D, D, Hq * D, D, Hk * D, D,
                   slot(0), slot(1), slot(2), slot(3), None, slot(4), slot(5))
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def rope(**kw):
    return S.lib().mhc_rope(ctypes.byref(rope_args(**kw)), None)


AXES = (ctypes.c_uint8 * 64)(*[i % 3 for i in range(64)])


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(D=1), dict(D=514), dict(R=0), dict(R=130), dict(R=63), dict(Hq=0),
    dict(Hq=4097), dict(Hk=-1), dict(Hk=4097), dict(dtype=2), dict(dtype=-1), dict(position_bytes=2),
    dict(position_bytes=0), dict(axes=0), dict(axes=5), dict(interleaved=2), dict(inverse=-1),
    dict(scale=INF), dict(scale=NAN), dict(q=None), dict(k=None), dict(positions=None), dict(inv_freq=None),
    dict(q_out=None), dict(k_out=None), dict(Hk=0), dict(axes=2, position_axis=3),
    dict(axes=2, position_axis=1 << 40), dict(axes=2, pair_axis=ctypes.addressof(AXES), position_axis=4),
    dict(q=slot(0) + 1), dict(k_out=slot(5) + 1), dict(positions=slot(2) + 2), dict(inv_freq=slot(3) + 2),
    dict(position_bytes=8, positions=slot(2) + 4),
    dict(q_token=0), dict(q_head=-128), dict(q_token=1023), dict(q_head=127), dict(k_out_token=255),
    dict(q_token=1 << 40), dict(T=1 << 30, q_token=1 << 12),
    dict(q_out=slot(0) + 2), dict(k_out=slot(0)), dict(q_out=slot(1)), dict(k_out=slot(4) + 64),
    dict(q_out=slot(2)), dict(k_out=slot(3)), dict(q_out=slot(0), q_out_token=2048),
    # side by side in wider rows, but one head too near
    dict(q_token=1280, k_token=1280, k=slot(0) + 2 * 896, q_out=slot(0), q_out_token=1280, k_out=slot(0) + 2 * 896,
         k_out_token=1280),
])
def test_rope_refuses(kw):
    assert rope(**kw) == S.INVALID_ARG
    assert message()


def test_rope_nothing_to_do():
    assert rope(T=0, q=None, k=None, positions=None) == S.OK


# ----------------------------------------------------------------- cache --

def cache_args(T=4, pages=8, ps=64, H=2, D=128, **kw):
    a = S.CacheArgs(T, pages, ps, H, D, 0, 8, 0, H * D, D, H * D, D, slot(0), slot(1), slot(2), slot(3))
    for n, v in kw.items():
        setattr(a, n, v)
    return a


PAGE = 64 * 136


@pytest.mark.parametrize("call", ["mhc_cache_write", "mhc_cache_read"])
@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(D=32), dict(D=96), dict(D=512), dict(ps=0), dict(ps=8), dict(ps=24),
    dict(ps=528), dict(ps=-16), dict(H=0), dict(H=4097), dict(pages=0), dict(pages=1 << 34), dict(dtype=2),
    dict(slot_bytes=2), dict(reserved=1), dict(cache=None), dict(slots=None), dict(cache=slot(0) + 8),
    dict(k=slot(2) + 8), dict(v=slot(3) + 2), dict(slots=slot(1) + 4), dict(slot_bytes=4, slots=slot(1) + 2),
    dict(k_token=0), dict(k_token=252), dict(v_head=64), dict(v_head=132), dict(k_token=1 << 40),
    dict(k=slot(0)), dict(v=slot(0) + 16 * PAGE - 16), dict(k=None, v=None), dict(slots=slot(0) + PAGE),
])
def test_cache_refuses(call, kw):
    if call == "mhc_cache_read" and "slots" in kw and kw["slots"] == slot(0) + PAGE:
        kw = dict(slots=slot(2))          # a reader's slots may lie anywhere but in what it writes
    assert getattr(S.lib(), call)(ctypes.byref(cache_args(**kw)), None) == S.INVALID_ARG
    assert message()


def test_cache_pointer_rules():
    w, r = S.lib().mhc_cache_write, S.lib().mhc_cache_read
    assert w(None, None) == 1 and r(None, None) == 1
    assert w(ctypes.byref(cache_args(k=None)), None) == 1 and w(ctypes.byref(cache_args(v=None)), None) == 1
    assert r(ctypes.byref(cache_args(v=slot(2))), None) == 1        # one over the other
    for call in (w, r):
        assert call(ctypes.byref(cache_args(T=0, cache=None, slots=None, k=None, v=None)), None) == 0


# ------------------------------------------------------------- attention --

def attention_args(T=4, B=4, Hq=8, Hk=2, D=128, ps=64, pages=8, width=4, **kw):
    a = S.CacheAttentionArgs(T, 0, pages, Hq * D, D, width, B, Hq, Hk, D, ps, width, 0, 1, 0, 0.1, 0.0, 0,
                             *(slot(k) for k in range(4)), None, slot(5), None, slot(7), 1 << 30)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(B=-1), dict(B=65536), dict(Hq=0), dict(Hq=7), dict(Hk=0), dict(Hq=1),
    dict(Hq=8192), dict(T=1 << 29, q_starts=slot(4)), dict(T=(1 << 31) - (1 << 22), Hq=2, q_starts=slot(4), B=65535), dict(D=80), dict(D=512), dict(dtype=2), dict(ps=8), dict(ps=100), dict(ps=1024), dict(pages=0),
    dict(pages=1 << 31), dict(width=0), dict(width=1 << 26), dict(max_len=-1), dict(window=-1), dict(causal=2),
    dict(scale=INF), dict(scale=NAN), dict(softcap=-1.0), dict(softcap=NAN), dict(softcap=INF), dict(scale=1e30, softcap=1e-30),
    dict(reserved=3),
    dict(T=5), dict(q=None), dict(cache=None), dict(tables=None), dict(lens=None), dict(out=None),
    dict(q=slot(0) + 8), dict(cache=slot(1) + 4), dict(out=slot(5) + 2), dict(tables=slot(2) + 2),
    dict(lens=slot(3) + 1), dict(q_starts=slot(4) + 2), dict(lse=slot(6) + 2), dict(workspace=slot(7) + 4),
    dict(q_token=1020), dict(q_token=0), dict(q_head=132), dict(table_stride=3), dict(table_stride=1 << 40),
])
def test_attention_refuses(kw):
    assert S.lib().mhc_cache_attention(ctypes.byref(attention_args(**kw)), None) == S.INVALID_ARG
    assert message()


@pytest.mark.parametrize("kw", [
    dict(out=slot(0)), dict(out=slot(0) + 4 * 2048 - 16), dict(out=slot(1) + 16 * PAGE - 16), dict(out=slot(2)),
    dict(out=slot(3)), dict(out=slot(3) - 4 * 2048 + 16), dict(q_starts=slot(4), out=slot(4)),
    dict(q_starts=slot(4), lse=slot(4) + 16), dict(lse=slot(0)), dict(lse=slot(1) + 16 * PAGE - 4),
    dict(lse=slot(2) + 60), dict(lse=slot(3) + 12), dict(lse=slot(5) + 4 * 2048 - 4), dict(lse=slot(5) - 124),
])
def test_attention_refuses_overlaps(kw):
    """out, 4 rows of 8 heads of 128 channels, and lse over the inputs and each other, by an element."""
    assert S.lib().mhc_cache_attention(ctypes.byref(attention_args(**kw)), None) == S.INVALID_ARG
    assert "overlaps" in message()


def test_attention_nothing_to_do():
    call = S.lib().mhc_cache_attention
    assert call(ctypes.byref(attention_args(T=0, B=0, q=None, out=None)), None) == S.OK
    assert call(ctypes.byref(attention_args(T=0, q_starts=slot(4), q=None)), None) == S.OK
    assert call(None, None) == S.INVALID_ARG


def test_attention_workspace():
    assert S.cache_attention_workspace(1, 1, 8, 2, 128) > 0
    assert S.cache_attention_workspace(0, 0, 8, 2, 128) == 0
    for bad in ((-1, 1, 8, 2, 128), (1, 1, 8, 3, 128), (1, 1, 8, 2, 96), (1, 1, 8, 0, 128), (1, -1, 8, 2, 128)):
        with pytest.raises(S.SeamError):
            S.cache_attention_workspace(*bad)
    for bad in (dict(cu_count=0), dict(cu_count=5000), dict(max_len=-1), dict(max_len=(1 << 30) + 1)):
        with pytest.raises(S.SeamError):
            S.cache_attention_workspace(1, 1, 8, 2, 128, **bad)
    for rows, B in ((1, 1), (64, 64), (300, 2), (5, 5)):       # not falling with the longest length
        sizes = [S.cache_attention_workspace(rows, B, 8, 2, 128, 256, n) for n in (0, 100, 1024, 4096, 1 << 20, 1 << 30)]
        assert sizes == sorted(sizes) and sizes[0] == 0
    with pytest.raises(ValueError, match="out of range"):
        S.cache_attention_workspace(1, 2 ** 32 + 1, 8, 2, 128)


def test_attention_workspace_never_falls_with_the_longest_length():
    """What suffices for a length suffices for shorter ones: so a workspace may be had once, for the longest."""
    import random
    r = random.Random(1)
    cases = [(64, 64, 40, 8, 128, 256), (1, 1, 8, 2, 128, 256), (300, 4, 16, 2, 256, 256)]
    for _ in range(300):
        kv, B = r.choice((1, 2, 4, 5, 8, 16, 40)), round(math.exp(r.uniform(0, 8)))
        cases.append((B * r.choice((1, 1, 2, 5, 40, 300, 1000)), B, kv * r.choice((1, 2, 4, 5, 8, 16)), kv,
                      r.choice((64, 128, 256)), r.choice((256, 256, 304, 64))))
    lens = sorted([1 << k for k in range(31)] + [(1 << k) + 1 for k in range(30)]
                  + [round(math.exp(r.uniform(4, 14))) for _ in range(60)])
    for case in cases:
        sizes = [S.cache_attention_workspace(*case, n) for n in lens]
        assert sizes == sorted(sizes), case
    assert S.cache_attention_workspace(64, 64, 40, 8, 128) == S.cache_attention_workspace(64, 64, 40, 8, 128, 256, 8192)


# --------------------------------------------------------------- binding --

def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("call,text", [
    (lambda: S.rope(bf(4, 2), None, torch.arange(4), torch.ones(1)), "must be \\[T, heads, D\\]"),
    (lambda: S.rope(torch.zeros(4, 2, 64), None, torch.arange(4), torch.ones(32)), "bfloat16 or float16"),
    (lambda: S.rope(bf(4, 2, 64), None, torch.arange(4), torch.ones(32)), "device tensor"),
    (lambda: S.rope(bf(4, 2, 64), bf(4, 64), torch.arange(4), torch.ones(32)), "must be \\[T, heads, D\\]"),
    (lambda: S.cache_write(bf(1, 1), bf(4, 64), bf(4, 64), torch.arange(4)), "T, heads, D"),
    (lambda: S.cache_write(bf(1, 1, 1), bf(4, 1, 64), bf(4, 1, 64), torch.arange(4)), "device tensor"),
    (lambda: S.cache_write(bf(1, 1, 1), bf(4, 1, 64).float(), bf(4, 1, 64), torch.arange(4)), "bfloat16 or float16"),
    (lambda: S.cache_read(torch.zeros(2, 1, 68 * 16, dtype=torch.uint8), torch.arange(4), 64), "device tensor"),
    (lambda: S.cache_read(torch.zeros(2, 1, 68 * 16 + 1, dtype=torch.uint8), torch.arange(4), 64), "does not hold"),
    (lambda: S.cache_read(torch.zeros(2, 1, 68 * 16, dtype=torch.uint8), torch.arange(4), 64, dtype="f32"), "bf16 or"),
    (lambda: S.cache_read(torch.zeros(2, 68 * 16, dtype=torch.uint8), torch.arange(4), 64), "cache"),
    (lambda: S.cache_attention(bf(4, 64), bf(1, 1, 1), bf(4, 1), bf(4)), "q must be"),
    (lambda: S.cache_attention(torch.zeros(4, 2, 64), bf(1, 1, 1), bf(4, 1), bf(4)), "bfloat16 or float16"),
    (lambda: S.cache_attention(bf(4, 2, 64), bf(1, 1, 1), bf(4, 1), bf(4)), "device tensor"),
    (lambda: S.cache_attention(bf(4, 2, 64), bf(1, 1, 1), bf(4, 1), bf(4), window=2 ** 32), "out of range"),
    (lambda: S.kv_cache(4, 2, 96, device="cpu"), "head_dim"),
    (lambda: S.kv_cache(4, 2, 64, 40, device="cpu"), "page_size"),
])
def test_binding_refuses(call, text):
    with pytest.raises(ValueError, match=text):
        call()


def test_pair_axes():
    assert list(S._pair_axes((0, 1, 2, 0), 4, 3)) == [0, 1, 2, 0]
    for bad in ((0, 1, 2), (0, 1, 3, 0), (0, -1, 0, 0), (0, 0.0, 0, 0)):
        with pytest.raises(ValueError):
            S._pair_axes(bad, 4, 3)


def test_head_strides_of_slices():
    """Axes of one and slices of wider rows (the device apart)."""
    rows = bf(5, 12 * 64)
    for t, want in ((rows[:, :512].view(5, 8, 64), (768, 64)), (rows[:1, :512].view(1, 8, 64), (512, 64)),
                    (rows[:, 64:128].view(5, 1, 64), (768, 64)), (bf(8, 5, 64).transpose(0, 1), (64, 320))):
        class Fake:
            dtype, shape, is_cuda = t.dtype, t.shape, True
            get_device, stride = staticmethod(lambda: 0), staticmethod(t.stride)
        assert S._head_strides("x", Fake, t.dtype, t.shape, 0) == want
    t = bf(5, 64, 8).transpose(1, 2)

    class Fake:
        dtype, shape, is_cuda = t.dtype, t.shape, True
        get_device, stride = staticmethod(lambda: 0), staticmethod(t.stride)
    with pytest.raises(ValueError, match="dense"):
        S._head_strides("x", Fake, t.dtype, t.shape, 0)


def test_kv_cache():
    c = S.kv_cache(3, 2, 128, 48, device="cpu")
    assert c.shape == (3, 2, 48 * 136) and c.dtype == torch.uint8 and not c.any()
    assert S._cache_sizes.__name__ and 48 * 136 % (128 + 8) == 0


def test_pages_of_a_cache():
    for pages, H, D, ps in ((3, 2, 128, 48), (1, 1, 64, 16), (7, 5, 256, 512)):
        shape = S.kv_cache(pages, H, D, ps, device="cpu").shape
        assert S._pages_of(shape, H, D) == (pages, ps)
        for bad in ((shape, H + 1, D), (shape[:2], H, D), ((pages, H, shape[2] + 1), H, D), ((pages, H, 0), H, D),
                    ((pages, H, shape[2] + D + D // 16), H, D), (shape, H, 0)):
            with pytest.raises(ValueError, match="cache"):
                S._pages_of(*bad)


# ------------------------------------------------------ plain definitions --

def test_groups():
    v = torch.zeros(32, dtype=torch.float64)
    assert ref.groups(v, -125, 125) == ([0] * 32, 2)
    v[0] = 6.0
    assert ref.groups(v, -125, 125)[1] == 127 and ref.groups(v, -125, 125)[0][0] == 7
    v[0] = 6.0001
    assert ref.groups(v, -125, 125)[1] == 128
    v[:9] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0])     # ties, to the even code
    assert ref.groups(v, -125, 125)[0][:9] == [7, 0, 2, 2, 4, 4, 6, 6, 14]
    v[3] = NAN
    assert ref.groups(v, -125, 125) == ([0] * 32, 255)


def test_quantized_definitions_agree():
    g = torch.Generator().manual_seed(1)
    for dt in (torch.bfloat16, torch.float16):
        x = (torch.randn(40, 64, generator=g) * torch.exp2(torch.randint(-30, 16, (40, 1), generator=g))).to(dt)
        x = torch.where(x.isfinite(), x, torch.zeros_like(x))
        x[3] = 0
        x[4, :32] = torch.arange(32).to(dt) / 4
        assert torch.equal(ref.quantized(x), ref.quantized_fast(x))
        assert torch.equal(ref.quantized(x).to(dt).to(torch.float64), ref.quantized(x))     # exact in the type


def test_cache_definition_and_packing_agree():
    g = torch.Generator().manual_seed(2)
    k, v = torch.randn(40, 2, 64, generator=g).bfloat16(), torch.randn(40, 2, 64, generator=g).bfloat16()
    order = torch.randperm(96, generator=g)[:40]
    c = ref.Cache(2, 2, 64, 48)
    for t, s in enumerate(order.tolist()):
        c.write(s, 0, k[t])
        c.write(s, 1, v[t])
    made, hk, hv = ref.packed(k, v, order, 2, 48)
    used = torch.from_numpy(c.bytes)
    assert torch.equal(used, made)
    for t, s in enumerate(order.tolist()):
        assert torch.equal(c.read(s, 0), hk[t]) and torch.equal(c.read(s, 1), hv[t])
    assert not c.read(-1, 0).any() and not c.read(96, 1).any()


def test_rope_definition():
    x = torch.randn(3, 2, 8).bfloat16()
    pos = torch.tensor([0, 1, 5])
    f = torch.tensor([1.0, 0.5, 0.25])
    y = ref.rope(x, pos, f)
    assert torch.equal(y[0], x[0].double()) and torch.equal(y[..., 6:], x[..., 6:].double())
    z = torch.complex(x[..., :3].double(), x[..., 3:6].double()) * torch.exp(1j * pos[:, None, None] * f.double())
    assert torch.allclose(y[..., :3], z.real, atol=1e-12) and torch.allclose(y[..., 3:6], z.imag, atol=1e-12)
    back = ref.rope(y, pos, f, inverse=True)
    assert torch.allclose(back, x.double(), atol=1e-12)


def test_attention_definition():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3, 4, 64, generator=g).bfloat16()
    K, V = torch.randn(5, 2, 64, generator=g).double(), torch.randn(5, 2, 64, generator=g).double()
    out, lse, bound, _ = ref.attention(q, [K], [V], [5], [0, 3])
    x = q[1].double()                       # token 3 of 5: sees tokens 0 .. 3
    for h in range(4):
        s = K[:4, h // 2] @ x[h] / 8
        assert torch.allclose(out[1, h], torch.softmax(s, 0) @ V[:4, h // 2])
        assert torch.allclose(lse[1, h], torch.logsumexp(s, 0))
    assert (bound > 0).all() and (bound < 0.1).all()
    out, lse, _, _ = ref.attention(q, [K], [V], [2], [0, 3])       # more rows than tokens: the first sees none
    assert not out[0].any() and (lse[0] == -INF).all() and out[1].any()
    out, _, _, _ = ref.attention(q, [K], [V], [5], [0, 3], window=1)
    assert torch.allclose(out[2], V[4].repeat_interleave(2, 0))

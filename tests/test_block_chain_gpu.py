"""The block operators run together as a layer does: the block norm's int8
operand into a projection, its result into the next block norm, that one's
operand into the experts' logits, and the logits into the router; and the
four-stream seam's norm through the quantiser into the product."""
import pytest
import torch

import block_reference as ref
from seam_harness import dev_inputs, host_case, make_seam

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def weights(N, K, g):
    w = torch.randn(N, K, generator=g) / K ** 0.5
    return ref.quantize(w.to(torch.bfloat16))


def layer(S, d, out=None):
    """One boundary, a projection, the next boundary, the router."""
    o = out or {}
    a = S.block_norm(d["x"], d["g1"], d["y"], gamma_post=d["gp"], branch_scale=0.5, int8=True, out=o.get("a"))
    y = S.int8_gemm(a["codes"], a["scales"], *d["w"], out=o.get("y"))
    b = S.block_norm(a["residual_out"], d["g2"], y, int8=True, norm=False, out=o.get("b"))
    l = S.int8_gemm(b["codes"], b["scales"], *d["wr"], out_dtype="f32", out=o.get("l"))
    r = S.route(l, 4, scoring="sigmoid", bias=d["bias"], groups=4, topk_groups=2, group_top=2, scale=2.5,
                out=o.get("r"))
    return {"a": a, "y": y, "b": b, "l": l, "r": r}


def reference(c):
    x, n = ref.block_norm(c["x"], c["g1"], c["y"], c["gp"], None, 1.0, 0.5)
    y = ref.int8_gemm(*ref.quantize(n), *c["w"], None, torch.bfloat16)
    x, n = ref.block_norm(x, c["g2"], y, None, None, 1.0, 1.0)
    l = ref.int8_gemm(*ref.quantize(n), *c["wr"], None, torch.float32)
    return x, y, l, ref.route(l, 4, "sigmoid", c["bias"], 4, 2, 2, True, 2.5)


@pytest.mark.parametrize("T,H,E", [(1, 512, 64), (37, 1040, 96), (300, 2048, 256)])
def test_layer_chain(T, H, E):
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(T)
    bf = torch.bfloat16
    c = dict(x=torch.randn(T, H, generator=g).to(bf), y=torch.randn(T, H, generator=g).to(bf),
             g1=(1 + 0.1 * torch.randn(H, generator=g)).to(bf), g2=(1 + 0.1 * torch.randn(H, generator=g)).to(bf),
             gp=(1 + 0.1 * torch.randn(H, generator=g)).to(bf), w=weights(H, H, g), wr=weights(E, H, g),
             bias=0.05 * torch.randn(E, generator=g))
    d = {k: tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda() for k, v in c.items()}
    got = layer(S, d)
    x, y, l, (w, ids) = reference(c)
    assert torch.equal(got["y"].cpu(), y)
    assert torch.equal(got["b"]["residual_out"].cpu(), x)
    assert torch.equal(got["l"].cpu(), l)
    assert torch.equal(got["r"][1].cpu(), ids)
    assert ((got["r"][0].cpu() - w).abs() <= 2.0 ** -23 * w.abs()).all()
    # captured as a whole, replayed on new inputs, with eager runs between
    torch.cuda.synchronize()
    out = layer(S, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer(S, d, out)
    for k in range(3):
        d["y"].copy_(torch.randn(T, H, generator=g).to(bf))
        eager = layer(S, d)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["l"], eager["l"]) and torch.equal(out["r"][1], eager["r"][1])
        assert torch.equal(out["r"][0], eager["r"][0])


def test_two_streams_at_once():
    """Nothing is shared between calls: two streams, interleaved."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(9)
    T, H, E = 64, 1024, 64
    bf = torch.bfloat16
    ds = []
    for _ in range(2):
        c = dict(x=torch.randn(T, H, generator=g).to(bf), y=torch.randn(T, H, generator=g).to(bf),
                 g1=torch.ones(H).to(bf), g2=torch.ones(H).to(bf), gp=torch.ones(H).to(bf), w=weights(H, H, g),
                 wr=weights(E, H, g), bias=torch.zeros(E))
        ds.append({k: tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda() for k, v in c.items()})
    want = [layer(S, d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(S, ds[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o["l"], want[i]["l"]) and torch.equal(o["r"][1], want[i]["r"][1])


def test_outputs_made_on_a_stream_of_their_own():
    """A call on another stream than the current one: its outputs' memory is
    that stream's (what the current one frees and fills meanwhile is not
    theirs), and inputs dropped at once stay until it is done with them."""
    from layer_mhc_seam_amd import seam as S
    g = torch.Generator().manual_seed(10)
    T, H = 2048, 5120
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    gamma = torch.ones(H).bfloat16().cuda()
    w, ws = weights(H, H, g)
    w, ws = w.cuda(), ws.cuda()
    want = S.int8_gemm(*S.int8_quantize(x), w, ws)
    want_norm = S.block_norm(x, gamma)["norm"]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        mine = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        n = S.block_norm(mine, gamma, stream=s)["norm"]
        codes, scales = S.int8_quantize(mine, stream=s)
        del mine
        got = S.int8_gemm(codes, scales, w, ws, stream=s)
        del codes, scales
        for _ in range(4):   # takes what was freed on the current stream, if anything
            torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(n, want_norm)


def test_seam_norm_through_the_int8_product():
    """The four-stream seam's norm is an operand like any other."""
    from layer_mhc_seam_amd import seam as S
    T, H, N = 24, 512, 200
    c = host_case(T, H, seed=90)
    s = make_seam(c, T)
    norm = s.run(**dev_inputs(c))["norm"]
    w = weights(N, H, torch.Generator().manual_seed(2))
    out = S.int8_gemm(*S.int8_quantize(norm), *(t.cuda() for t in w))
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), ref.int8_gemm(*ref.quantize(norm.cpu()), *w, None, torch.bfloat16))
    s.close()

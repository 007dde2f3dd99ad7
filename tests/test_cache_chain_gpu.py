"""The operators of an attention layer run together as serving does: the block norm's int8 operand into the qkv
product, rotary positions in place on its slices, keys and values into the 4-bit cache, attention over it, its output
quantised into the projection, and the next block norm.  A prefill of ragged prompts, then steps of one token; each
stage is held against its definition, given the stage before."""
import pytest
import torch

import block_reference as block
import cache_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F64, I32 = torch.bfloat16, torch.float16, torch.float64, torch.int32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def weights(N, K, g):
    return tuple(t.cuda() for t in block.quantize((torch.randn(N, K, generator=g) / K ** 0.5).to(BF)))


class Model:
    """One layer, its cache and its sequences' pages."""

    def __init__(self, B, Hq, Hk, D, ps, width, dt, seed=0):
        from layer_mhc_seam_amd import seam as S
        g = torch.Generator().manual_seed(seed)
        self.g, self.B, self.Hq, self.Hk, self.D, self.ps, self.dt = g, B, Hq, Hk, D, ps, dt
        self.H = H = 256
        self.g1, self.g2 = ((1 + 0.1 * torch.randn(H, generator=g)).to(dt).cuda() for _ in range(2))
        self.wqkv = weights((Hq + 2 * Hk) * D, H, g)
        self.wo = weights(H, Hq * D, g)
        self.freq = (10000.0 ** (-torch.arange(0, D, 2) / D)).float().cuda()
        self.cache = S.kv_cache(B * width + 1, Hk, D, ps)
        self.cache.fill_(0)
        self.tables = torch.randperm(B * width + 1, generator=g)[:B * width].view(B, width).to(I32).cuda()

    def inputs(self, lens, rows, padding=0):
        """A step whose last rows[b] tokens of lens[b] are new, and rows of padding behind them."""
        pos = torch.cat([torch.arange(n - r, n) for n, r in zip(lens, rows)] + [torch.zeros(padding).long()])
        of = torch.cat([torch.full((r,), b) for b, r in enumerate(rows)] + [torch.zeros(padding).long()])
        slots = self.tables.cpu()[of, pos // self.ps].long() * self.ps + pos % self.ps
        slots[len(slots) - padding:] = -1
        starts = torch.tensor([0] + list(rows)).cumsum(0).to(I32)
        return dict(x=torch.randn(len(pos), self.H, generator=self.g).to(self.dt).cuda(), positions=pos.cuda(),
                    slots=slots.cuda(), lens=torch.tensor(lens, dtype=I32).cuda(), starts=starts.cuda())

    def layer(self, d, cache=None, out=None, **kw):
        from layer_mhc_seam_amd import seam as S
        cache = self.cache if cache is None else cache
        Hq, Hk, D, o = self.Hq, self.Hk, self.D, out or {}
        kind = "bf16" if self.dt is BF else "f16"
        a = S.block_norm(d["x"], self.g1, int8=True, norm=False, out=o.get("a"))
        qkv = S.int8_gemm(a["codes"], a["scales"], *self.wqkv, out_dtype=kind, out=o.get("qkv"))
        product = qkv.clone()
        q, k, v = qkv.view(-1, Hq + 2 * Hk, D).split((Hq, Hk, Hk), 1)
        S.rope(q, k, d["positions"], self.freq, out=(q, k))
        S.cache_write(cache, k, v, d["slots"])
        made = o.get("heads")
        if made is None:
            made = (torch.zeros(q.shape, dtype=self.dt, device="cuda"),
                    torch.zeros(q.shape[:2], device="cuda"))
        heads = S.cache_attention(q, cache, self.tables, d["lens"], q_starts=d.get("starts"), lse=True, out=made, **kw)
        c = S.int8_quantize(heads[0].view(-1, Hq * D), out=o.get("c"))
        y = S.int8_gemm(*c, *self.wo, out_dtype=kind, out=o.get("y"))
        b = S.block_norm(d["x"], self.g2, y, out=o.get("b"))
        return {"a": a, "product": product, "qkv": qkv, "heads": heads, "c": c, "y": y, "b": b}

    def check(self, d, got, lens, rows):
        """Each stage given the one before."""
        Hq, Hk, D, n = self.Hq, self.Hk, self.D, sum(rows)
        host = lambda w: tuple(t.cpu() for t in w)   # noqa: E731
        _, norm = block.block_norm(d["x"].cpu(), self.g1.cpu(), None, None, None, 1.0, 1.0)
        product = block.int8_gemm(*block.quantize(norm), *host(self.wqkv), None, self.dt)
        assert torch.equal(got["product"].cpu(), product)
        q0, k0, v0 = product.view(-1, Hq + 2 * Hk, D).split((Hq, Hk, Hk), 1)
        q, k, v = got["qkv"].cpu().view(-1, Hq + 2 * Hk, D).split((Hq, Hk, Hk), 1)
        assert torch.equal(v, v0)
        for x, x0 in ((q, q0), (k, k0)):
            want = ref.rope(x0, d["positions"].cpu(), self.freq.cpu())
            pair = torch.hypot(*x0.to(F64).chunk(2, -1)).repeat(1, 1, 2)
            # half a step, and sine, cosine and two products of 24 bits
            bound = torch.finfo(self.dt).eps / 2 * want.abs() + 2.0 ** -21 * pair + torch.finfo(self.dt).tiny
            assert ((x.to(F64) - want).abs() <= bound).all()
        self.keys = getattr(self, "keys", None) or [torch.zeros(0, Hk, D, dtype=F64)] * self.B
        self.values = getattr(self, "values", None) or [torch.zeros(0, Hk, D, dtype=F64)] * self.B
        at = 0
        for b, r in enumerate(rows):
            self.keys[b] = torch.cat((self.keys[b], ref.quantized_fast(k[at:at + r])))
            self.values[b] = torch.cat((self.values[b], ref.quantized_fast(v[at:at + r])))
            at += r
        out, lse, bound, lse_bound = ref.attention(q[:n], self.keys, self.values, lens,
                                                   [0] + torch.tensor(rows).cumsum(0).tolist())
        heads, sums = (t.cpu().to(F64) for t in got["heads"])
        assert ((heads[:n] - out).abs() <= bound).all()
        assert ((sums[:n] - lse).abs() <= lse_bound).all()
        assert (heads[n:] == 0).all()                # padding, left as it was
        y = block.int8_gemm(*block.quantize(got["heads"][0].cpu().view(-1, Hq * D)), *host(self.wo), None, self.dt)
        assert torch.equal(got["y"].cpu(), y)
        _, norm = block.block_norm(d["x"].cpu(), self.g2.cpu(), y, None, None, 1.0, 1.0)
        assert torch.equal(got["b"]["norm"].cpu(), norm)


def check_layer(lens, Hq, Hk, D, ps, dt, padding=0):
    m = Model(len(lens), Hq, Hk, D, ps, -(-(max(lens) + 8) // ps), dt)
    d = m.inputs(lens, lens, padding)
    m.check(d, m.layer(d), lens, lens)
    for step in range(2):                            # a token each, then two of a draft
        rows = [step + 1] * len(lens)
        lens = [n + step + 1 for n in lens]
        d = m.inputs(lens, rows, padding)
        m.check(d, m.layer(d), lens, rows)
    return m, lens


@pytest.mark.parametrize("lens,Hq,Hk,D,ps,dt,padding", [
    ([5], 4, 1, 64, 16, BF, 0), ([37, 1, 130], 8, 2, 128, 16, BF, 3), ([200, 90], 6, 6, 64, 48, F16, 5),
    ([70, 3, 16, 64], 4, 2, 256, 64, F16, 0)])
def test_prefill_and_steps(lens, Hq, Hk, D, ps, dt, padding):
    check_layer(lens, Hq, Hk, D, ps, dt, padding)


def clone(d):
    return {k: tuple(x.clone() for x in v) if isinstance(v, tuple) else clone(v) if isinstance(v, dict) else v.clone()
            for k, v in d.items()}


@pytest.mark.parametrize("lens,width", [([40, 7, 100], 16), ([3000, 1, 900], 300)])
def test_captured_step(lens, width):
    """A step captured with its workspace, replayed as the sequences grow, with eager runs of the same step between.
    Behind tables for 4800 tokens the work is split and joined."""
    m = Model(len(lens), 8, 2, 128, 16, width, BF)
    d = m.inputs(lens, lens)
    m.layer(d)
    step = m.inputs([n + 1 for n in lens], [1] * len(lens))
    del step["starts"]
    rows = torch.arange(len(lens)).cuda()
    m.layer(step)
    torch.cuda.synchronize()
    out = m.layer(step)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.layer(step, out=out)
    for _ in range(4):
        step["lens"].add_(1)
        step["positions"].add_(1)
        page = m.tables[rows, step["positions"] // m.ps].long()
        step["slots"].copy_(page * m.ps + step["positions"] % m.ps)
        step["x"].copy_(torch.randn(step["x"].shape, generator=m.g).to(BF))
        cache = m.cache.clone()
        eager = m.layer(step, cache=cache)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache, m.cache)
        for name in ("qkv", "y"):
            assert torch.equal(out[name], eager[name])
        for a, b in zip(out["heads"], eager["heads"]):
            assert torch.equal(a, b)
        assert torch.equal(out["b"]["norm"], eager["b"]["norm"])


def test_two_captured_steps_at_once():
    """Two graphs of split attention, replayed on two streams: each has its own workspace."""
    ms = [Model(2, 8, 2, 128, 16, 300, BF, seed=i) for i in range(2)]
    steps, wants, outs, graphs, streams = [], [], [], [], []
    for m in ms:
        m.layer(m.inputs([4000, 2500], [4000, 2500]))
        steps.append(m.inputs([4001, 2501], [1, 1]))
        wants.append(m.layer(steps[-1]))
        outs.append(clone(wants[-1]))
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        streams.append(torch.cuda.Stream())
        streams[-1].wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graphs[-1], stream=streams[-1]):
            m.layer(steps[-1], out=outs[-1])
    for _ in range(4):
        for o in outs:
            o["heads"][0].zero_(), o["y"].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert torch.equal(o["heads"][0], w["heads"][0]) and torch.equal(o["heads"][1], w["heads"][1])
            assert torch.equal(o["y"], w["y"])


@pytest.mark.parametrize("lens,rows", [([4000, 2500], [1, 1]), ([300, 500], [300, 500]), ([3000, 2200], [150, 60])])
def test_two_streams_at_once(lens, rows):
    """Nothing is shared between calls: two streams, interleaved, and calls made for a stream of their own."""
    from layer_mhc_seam_amd import seam as S
    ms = [Model(2, 8, 2, 128, 16, 260, BF, seed=i) for i in range(2)]
    steps, wants = [], []
    for m in ms:
        m.layer(m.inputs(lens, lens))
        steps.append(m.inputs(lens, rows))
        wants.append(m.layer(steps[-1]))
    qs = [w["qkv"].view(-1, 12, 128)[:, :8].clone() for w in wants]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    got, own = [[], []], [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ms[i].layer(steps[i]))
    torch.cuda.synchronize()
    for _ in range(6):
        for i, s in enumerate(streams):
            d, q = steps[i], qs[i].clone()
            s.wait_stream(torch.cuda.current_stream())     # which made q, and drops it at once
            own[i].append(S.cache_attention(q, ms[i].cache, ms[i].tables, d["lens"], q_starts=d["starts"], stream=s))
            del q
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o["heads"][0], wants[i]["heads"][0])
            assert torch.equal(o["b"]["norm"], wants[i]["b"]["norm"])
        for o in own[i]:
            assert torch.equal(o, wants[i]["heads"][0])

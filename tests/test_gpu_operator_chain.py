"""The operators together, as a MoE block uses them: norm -> router -> route ->
expert GEMM -> combine, the shared expert on 8-bit rows beside it; MXFP4
experts through the same routing; the chain in a replayed HIP graph, and on
a stream other than the current one."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


class Block:
    def __init__(self, lib, T=48, E=16, k=4, K=256, N=256, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")        # noqa: E731
        self.lib, self.T, self.E, self.k, self.K = lib, T, E, k, K
        self.x, self.res = (rn(T, K).to(torch.bfloat16) for _ in range(2))
        self.norm_w = (1 + 0.1 * rn(K)).to(torch.bfloat16)
        self.router = 0.1 * rn(K, E)
        self.bias = 0.1 * rn(E)
        self.gate = lib.Gate(k, score=lib.SCORE_SIGMOID, n_group=4, topk_group=2, scale=2.5)
        self.up = lib.pack_weights(0.05 * rn(E, N, K))
        self.down = lib.pack_weights(0.05 * rn(E, K, N // 2))
        self.mx_up = lib.mx_quantize(0.05 * rn(E, N, K))
        self.sh_up = lib.mx_quantize(0.05 * rn(N, K))
        self.sh_down = lib.mx_quantize(0.05 * rn(K, N // 2))

    def run(self, n_rows=None, stream=None):
        m, s = self.lib, stream
        y, res, q = m.rmsnorm(self.x, self.norm_w, residual=self.res, rows=m.ROWS_MXFP8, stream=s)
        logits = (y.float().unsqueeze(2) * self.router).sum(dim=1)
        ids, w = m.gate_topk(logits, self.gate, bias=self.bias, n_rows=n_rows, stream=s)
        off, perm, inv = m.route(ids, self.E, self.k, stream=s)
        h = m.grouped_spgemm_gather(y, perm, self.k, off, self.up, m.EPI_SWIGLU, stream=s)
        d = m.grouped_spgemm(h, off, self.down, stream=s)
        out = m.unpermute(d, inv, w, self.T, self.k, stream=s)
        hx = m.mx_gemm(q, self.mx_up, off, perm=perm, k=self.k, epilogue=m.EPI_SWIGLU, stream=s)
        sh = m.mx_gemm(q, self.sh_up, epilogue=m.EPI_SWIGLU, stream=s)
        shared = m.mx_gemm(m.mx_quantize(sh, m.ROWS_MXFP8, stream=s), self.sh_down, stream=s)
        return dict(y=y, res=res, logits=logits, ids=ids, w=w, off=off, perm=perm, inv=inv, out=out, hx=hx,
                    sh=sh, shared=shared)


def test_chain_against_the_oracle(lib):
    b = Block(lib)
    o = {n: t.cpu() for n, t in b.run().items()}
    ids, w = oracle.gate_topk(o["logits"].numpy(), b.k, score="sigmoid", bias=b.bias.cpu().numpy(), n_group=4,
                              topk_group=2, scale=2.5)
    assert np.array_equal(o["ids"].numpy(), ids)
    off, perm, inv = oracle.route(ids, b.E)
    assert np.array_equal(o["off"].numpy(), off) and np.array_equal(o["perm"].numpy(), perm)
    y = o["y"].double().numpy()
    dec = [[lib.decode_weights(p, e).double().cpu().numpy() * p.global_scale[e].item() for e in range(b.E)]
           for p in (b.up, b.down)]
    _, _, _, ref = oracle.moe_chain(y, off, perm, inv, b.k, lambda e: dec[0][e], lambda e: dec[1][e], w)
    got = o["out"].double().numpy()
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
    # the shared expert from its own quantized rows
    wv = [oracle.mx_decode(t.codes.cpu().numpy(), t.scales.cpu().numpy(), "mxfp4") for t in (b.sh_up, b.sh_down)]
    xq = oracle.mx_decode(*oracle.mx_quantize(y, "mxfp8"), "mxfp8")
    h = oracle.swiglu(oracle.mx_gemm(xq, wv[0]))
    assert np.linalg.norm(o["sh"].double().numpy() - h) <= 2.0 ** -8 * np.linalg.norm(h)
    hq = oracle.mx_decode(*oracle.mx_quantize(o["sh"].double().numpy(), "mxfp8"), "mxfp8")
    ref = oracle.mx_gemm(hq, wv[1])
    assert np.linalg.norm(o["shared"].double().numpy() - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    # MXFP4 experts
    ev = oracle.mx_decode(b.mx_up.codes.cpu().numpy(), b.mx_up.scales.cpu().numpy(), "mxfp4")
    for e in range(b.E):
        r = np.arange(off[e], off[e + 1])
        if len(r):
            ref = oracle.swiglu(oracle.mx_gemm(xq[perm[r] // b.k], ev[e]))
            assert np.linalg.norm(o["hx"].double().numpy()[r] - ref) <= 2.0 ** -8 * np.linalg.norm(ref)


def test_padded_batch(lib):
    """With n_rows, the live rows come out as without it and the padding adds
    nothing."""
    b = Block(lib, T=20, seed=1)
    n = torch.tensor([13], dtype=torch.int32, device="cuda")
    full, part = b.run(), b.run(n)
    assert torch.equal(part["out"][:13], full["out"][:13]) and (part["out"][13:] == 0).all()
    assert int(part["off"][-1]) == 13 * b.k


@pytest.mark.parametrize("T", [1, 48])
def test_graph(lib, T):
    """Captured once and replayed with other inputs in the same buffers and
    another n_rows: every replay gives the eager results."""
    b = Block(lib, T=T, seed=2)
    other = Block(lib, T=T, seed=3)
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    b.run(n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b.run(n)
    keep = (b.x.clone(), b.res.clone())
    for rep in range(4):
        src = (other.x, other.res) if rep % 2 else keep
        b.x.copy_(src[0])
        b.res.copy_(src[1])
        n.fill_(T if rep < 2 else (T + 1) // 2)
        want = b.run(n)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        live = int(want["off"][-1])
        for name in want:
            u, v = got[name], want[name]
            if name in ("perm", "hx"):
                u, v = u[:live], v[:live]
            assert torch.equal(u, v), (rep, name)


def test_two_graphs_and_a_side_stream(lib):
    """Two captured chains replayed on two streams at once share nothing."""
    blocks = [Block(lib, T=40, seed=s) for s in (4, 5)]
    want = [b.run() for b in blocks]
    torch.cuda.synchronize()
    graphs, got = [], []
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(b.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        for name in v:
            assert torch.equal(u[name], v[name]), name


def test_stream_argument(lib):
    """A call given a stream runs there: ordered behind that stream's work."""
    s = torch.cuda.Stream()
    x = torch.zeros(4096, 2048, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            x.add_(1.0)
    y, _, q = lib.rmsnorm(x, w, 0.0, rows=lib.ROWS_MXFP4, stream=s)
    v = lib.mx_decode(q, stream=s)
    torch.cuda.synchronize()
    assert (y == 1).all() and (v == 1).all()


def test_results_of_a_side_stream_spare_pending_reads(lib):
    """A block that the current stream has freed but still reads must not become
    the result of a call on another stream."""
    s = torch.cuda.Stream()
    x = torch.randn(4096, 2048, device="cuda").to(torch.bfloat16)
    w = torch.ones(2048, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(4096, 128, device="cuda")
    mxw = lib.mx_quantize(torch.randn(2048, 2048, device="cuda"))
    mxx = lib.mx_quantize(x)
    gate = lib.Gate(8)
    calls = (lambda: lib.mx_quantize(x, stream=s), lambda: lib.mx_decode(mxx, stream=s),
             lambda: lib.rmsnorm(x, w, rows=lib.ROWS_MXFP8, stream=s),
             lambda: lib.gate_topk(logits, gate, stream=s), lambda: lib.mx_gemm(mxx, mxw, stream=s))
    torch.cuda.synchronize()
    for i, call in enumerate(calls):
        blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda")
                  for n in (4096 * 4096, 4096 * 2048, 4096 * 1024, 4096 * 64, 4096 * 32) for _ in range(2)]
        torch.cuda._sleep(20_000_000)
        copies = [b.clone() for b in blocks]
        del blocks
        kept = call()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies), i
        del kept, copies


def test_results_of_a_raw_stream_handle(lib):
    """A stream given as its handle: results are allocated there too, and the
    call is ordered behind that stream's work; 0 is the default stream."""
    s = torch.cuda.Stream()
    x = torch.randn(4096, 2048, device="cuda").to(torch.bfloat16)
    w = torch.ones(2048, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(4096, 128, device="cuda")
    mxw = lib.mx_quantize(torch.randn(2048, 2048, device="cuda"))
    mxx = lib.mx_quantize(x)
    gate = lib.Gate(8)
    calls = (lambda h: [(q := lib.mx_quantize(x, stream=h)).codes, q.scales], lambda h: [lib.mx_decode(mxx, stream=h)],
             lambda h: [(r := lib.rmsnorm(x, w, rows=lib.ROWS_MXFP8, stream=h))[0], r[2].codes, r[2].scales],
             lambda h: list(lib.gate_topk(logits, gate, stream=h)), lambda h: [lib.mx_gemm(mxx, mxw, stream=h)])
    torch.cuda.synchronize()
    for i, call in enumerate(calls):
        want = call(None)
        blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda")
                  for n in (4096 * 4096, 4096 * 2048, 4096 * 1024, 4096 * 64, 4096 * 32) for _ in range(2)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        copies = [b.clone() for b in blocks]
        del blocks
        got = call(s.cuda_stream)
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies), i
        for u, v, d in zip(got, want, call(0)):
            assert torch.equal(u, v) and torch.equal(d, v), i
        del got, copies


def test_rows_beyond_4_gib(lib):
    """The last rows of buffers over 4 GiB are what a call on them alone gives."""
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = 37
    T, K = (1 << 20) + tail, 2080
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-tail:] = torch.randn(tail, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(K, generator=g, device="cuda").to(torch.bfloat16)
    end = x[-tail:].clone()
    for rows in (lib.ROWS_MXFP8, lib.ROWS_NVFP4):
        y, _, q = lib.rmsnorm(x, w, rows=rows)
        ye, _, qe = lib.rmsnorm(end, w, rows=rows)
        assert torch.equal(y[-tail:], ye)
        assert torch.equal(q.codes[-tail:], qe.codes) and torch.equal(q.scales[-tail:], qe.scales)
        del y, q
    q, qe = lib.mx_quantize(x, lib.ROWS_MXFP8), lib.mx_quantize(end, lib.ROWS_MXFP8)
    assert torch.equal(q.codes[-tail:], qe.codes) and torch.equal(q.scales[-tail:], qe.scales)
    assert torch.equal(lib.mx_decode(q)[-tail:], lib.mx_decode(qe))
    del x, q
    # a product whose sums are exact in fp32 (64 products of E2M1 by two scales each)
    N, K = 2080, 64
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    mw = lib.mx_quantize(torch.randn(N, K, generator=g, device="cuda"))
    y = lib.mx_gemm(lib.mx_quantize(x), mw)
    assert torch.equal(y[-tail:], lib.mx_gemm(lib.mx_quantize(x[-tail:].clone()), mw))
    del x, y
    T, E = (1 << 20) + tail, 1024
    l = torch.zeros(T, E, device="cuda")
    l[-tail:] = torch.randn(tail, E, generator=g, device="cuda")
    gate = lib.Gate(8, score=lib.SCORE_SIGMOID, n_group=8, topk_group=4)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    for got, alone in zip(lib.gate_topk(l, gate, bias), lib.gate_topk(l[-tail:].clone(), gate, bias)):
        assert torch.equal(got.view(T, 8)[-tail:], alone.view(tail, 8))

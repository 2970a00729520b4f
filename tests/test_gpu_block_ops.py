"""The stand-alone operators together, as a program uses them: the residual MoE block with 4-bit experts for a few
tokens (norm, routing, sort, gated product, product, back with gates), eagerly and as a replayed CUDA graph,
and a training step of a block with a program's own experts."""
import ctypes
import math
import threading

import pytest
import torch

import oracle
from tests import ops64, parity
from tests.test_gpu_w4 import pack, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixture_experts_softmax_b200 as m
    return m


class Block4:
    """u = RMSNorm(h) gain;  out = sum_j gate_j * (gelu(u W) * (u Wv)) W1, 8 experts and 2 picks, 4-bit weights."""

    def __init__(self, m, T, d, ffn, group, seed=0):
        self.m, self.T, self.d, self.ffn, self.group = m, T, d, ffn, group
        g = torch.Generator().manual_seed(seed)
        self.host = dict(wl=weights(8, d, ffn, group, seed + 1), wv=weights(8, d, ffn, group, seed + 2),
                         w1=weights(8, ffn, d, group, seed + 3))
        self.p = {k: pack(m, *v, group) for k, v in self.host.items()}
        self.router = torch.randn((d, 8), generator=g) / math.sqrt(d)
        self.gain = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
        i32, bf, dev = torch.int32, torch.bfloat16, "cuda"
        self.rw, self.gd = self.router.cuda(), self.gain.cuda()
        self.h = torch.zeros((T, d), dtype=bf, device=dev)
        self.u, self.out = torch.empty_like(self.h), torch.empty_like(self.h)
        self.idx, self.slot = (torch.empty((T, 2), dtype=i32, device=dev) for _ in range(2))
        self.gate = torch.empty((T, 2), device=dev)
        self.offsets, self.off2 = (torch.empty(9, dtype=i32, device=dev) for _ in range(2))
        self.perm, self.perm2 = (torch.empty(2 * T, dtype=i32, device=dev) for _ in range(2))
        self.rows = torch.empty((2 * T, d), dtype=bf, device=dev)
        self.mid = torch.empty((2 * T, ffn), dtype=bf, device=dev)
        self.y = torch.empty((2 * T, d), device=dev)

    def run(self, stream=None):
        self.route(stream)
        self.experts(stream)

    def route(self, stream=None):
        m, T, d = self.m, self.T, self.d
        m.check(m.moe_norm_forward(m.MOE_NORM_RMS, m.MOE_BF16, T, d, self.h, self.gd, None, 1e-5, self.u, None, stream))
        m.check(m.moe_route_noalloc(T, d, self.u, self.rw, None, self.idx, self.gate, self.off2, self.perm2, stream))

    def experts(self, stream=None):
        m, T, d, G = self.m, self.T, self.d, self.group
        m.check(m.moe_sort_rows(m.MOE_BF16, T, 2, 8, d, self.u, self.idx, self.offsets, self.perm, self.slot, self.rows, stream))
        m.check(m.moe_w4_matvec(m.MOE_BF16, m.MOE_BF16, 8, d, self.ffn, G, 2 * T, self.rows, self.offsets, self.p["wl"],
                                self.p["wv"], self.mid, stream))
        m.check(m.moe_w4_matvec(m.MOE_BF16, m.MOE_F32, 8, self.ffn, d, G, 2 * T, self.mid, self.offsets, self.p["w1"], None,
                                self.y, stream))
        m.check(m.moe_unsort_rows(m.MOE_F32, m.MOE_BF16, T, 2, d, self.y, self.slot, self.gate, self.out, stream))

    def check(self, h):
        """Every step against its 64-bit form on the step's own inputs, and the whole against the whole."""
        c = {k: getattr(self, k).cpu() for k in ("u", "idx", "gate", "offsets", "perm", "slot", "rows", "mid", "y", "out")}
        assert torch.equal(self.offsets, self.off2) and torch.equal(self.perm, self.perm2)
        u, _, tol, _ = ops64.norm(h, self.gain, None, float(torch.tensor(1e-5)), False, torch.bfloat16)
        ops64.assert_close(c["u"], u, tol, "u")
        near = parity.check_routing(_Routing(c), oracle.route(c["u"], self.router), 8)
        assert near.sum() <= 1
        assert torch.equal(c["rows"], c["u"][c["perm"].long() // 2])
        mid, tol = ops64.w4(c["rows"], c["offsets"], [self.host["wl"], self.host["wv"]], self.group, torch.bfloat16)
        ops64.assert_close(c["mid"], mid, tol, "mid")
        y, tol = ops64.w4(c["mid"], c["offsets"], [self.host["w1"]], self.group, torch.float32)
        ops64.assert_close(c["y"], y, tol, "y")
        out, tol = ops64.unsort(c["y"], c["slot"], c["gate"], torch.bfloat16)
        ops64.assert_close(c["out"], out, tol, "out")
        whole = ops64.unsort(ops64.w4(mid, c["offsets"], [self.host["w1"]], self.group, torch.float32)[0], c["slot"], c["gate"],
                             torch.bfloat16)[0]
        assert (c["out"].double() - whole).abs().max() <= parity.OUT_RTOL * whole.abs().max()


class _Routing:
    def __init__(self, c):
        self.idx_h, self.gate_h = c["idx"].numpy(), c["gate"].numpy()
        self.offsets_h, self.perm_h = c["offsets"].numpy(), c["perm"].numpy()


def tokens(T, d, seed):
    return torch.randn((T, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("T,d,ffn,group", [(1, 256, 512, 128), (8, 512, 1024, 64), (33, 264, 328, 32)])
def test_decode_block(m, T, d, ffn, group):
    blk = Block4(m, T, d, ffn, group)
    h = tokens(T, d, T)
    blk.h.copy_(h)
    blk.run()
    torch.cuda.synchronize()
    blk.check(h)


def test_decode_block_on_a_side_stream_and_in_two_graphs(m):
    """The block on a stream of its own, then its expert part captured twice (two batches of buffers) and both
    graphs replayed together on two streams with new tokens: nothing is shared between the calls.  (The routing
    stays outside: calls of moe_route_noalloc share one scratch array and must not overlap.)"""
    blks = [Block4(m, 8, 256, 512, 64, seed=s) for s in (0, 10)]
    streams = [torch.cuda.Stream() for _ in blks]
    graphs = []
    for blk, s in zip(blks, streams):
        h = tokens(8, 256, 3)
        blk.h.copy_(h)
        torch.cuda.synchronize()
        blk.run(s)
        s.synchronize()
        blk.check(h)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            blk.experts()   # the capture's current stream
        graphs.append(g)
    for turn in range(3):
        hs = [tokens(8, 256, 20 + 2 * turn + i) for i in range(2)]
        for blk, h in zip(blks, hs):
            blk.h.copy_(h)
            blk.route()
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for blk, h in zip(blks, hs):
            blk.check(h)


class Train:
    """A training step's calls around a program's own experts (here: one fp32 product per expert)."""

    def __init__(self, m, kind, T, k, E, d):
        self.m, self.kind, self.T, self.k, self.E, self.d = m, kind, T, k, E, d
        n, dev = T * k, "cuda"
        f = lambda *s: torch.zeros(s, device=dev)
        i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
        self.u, self.stats, self.offsets, self.perm, self.slot = f(T, d), f(T, 2), i(E + 1), i(n), i(T, k)
        self.rows, self.y, self.out = f(n, d), f(n, d), f(T, d)
        self.dy, self.dgate, self.drows, self.du, self.dx = f(n, d), f(T, k), f(n, d), f(T, d), f(T, d)
        self.dgain, self.dbias = f(d), f(d)
        self.ws = torch.empty(m.moe_norm_workspace(T, d), dtype=torch.uint8, device=dev)

    def forward(self, x, gain, bias, idx, gate):
        m, F = self.m, self.m.MOE_F32
        m.check(m.moe_norm_forward(self.kind, F, self.T, self.d, x, gain, bias, 1e-5, self.u, self.stats))
        m.check(m.moe_sort_rows(F, self.T, self.k, self.E, self.d, self.u, idx, self.offsets, self.perm, self.slot, self.rows))

    def back(self, gate):
        m, F = self.m, self.m.MOE_F32
        m.check(m.moe_unsort_rows(F, F, self.T, self.k, self.d, self.y, self.slot, gate, self.out))

    def backward_rows(self, dout, gate):
        m, F = self.m, self.m.MOE_F32
        m.check(m.moe_unsort_rows_backward(F, F, self.T, self.k, self.d, dout, self.y, self.slot, gate, self.dy, self.dgate))

    def backward_x(self, x, gain, has_bias):
        m, F = self.m, self.m.MOE_F32
        m.check(m.moe_unsort_rows(F, F, self.T, self.k, self.d, self.drows, self.slot, None, self.du))
        m.check(m.moe_norm_backward(self.kind, F, self.T, self.d, x, gain, self.stats, self.du, self.dx, self.dgain,
                                    self.dbias if has_bias else None, self.ws))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("T,k,E,d", [(40, 2, 8, 96), (700, 3, 5, 50)])
def test_training_step(m, kind, T, k, E, d):
    g = torch.Generator().manual_seed(T + kind)
    x, dout = (torch.randn((T, d), generator=g) for _ in range(2))
    gain, bias = 1 + 0.2 * torch.randn(d, generator=g), (0.1 * torch.randn(d, generator=g) if kind else None)
    idx = torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32).contiguous()
    idx[torch.rand((T, k), generator=g) < 0.1] = -1
    gate = torch.rand((T, k), generator=g)
    w = torch.randn((E, d, d), generator=g) / math.sqrt(d)

    # the whole in 64 bits, by differentiation
    leaves = [t.double().requires_grad_() for t in (x, gain, gate, w)] + ([bias.double().requires_grad_()] if kind else [])
    x8, gain8, gate8, w8 = leaves[:4]
    c = x8 - x8.mean(1, keepdim=True) if kind else x8
    u8 = c * (c.square().mean(1, keepdim=True) + float(torch.tensor(1e-5))).rsqrt() * gain8 + (leaves[4] if kind else 0)
    each = torch.einsum("td,edf->tef", u8, w8)
    hit = torch.nn.functional.one_hot(idx.clamp_min(0).long(), E).double() * (idx >= 0)[..., None]
    out8 = torch.einsum("tke,tk,tef->tf", hit, gate8, each)
    want = torch.autograd.grad((out8 * dout.double()).sum(), leaves)

    st = Train(m, kind, T, k, E, d)
    dev = [t.cuda() for t in (x, gain, idx, gate, w, dout)]
    xd, gd, idxd, gated, wd, doutd = dev
    bd = bias.cuda() if kind else None
    st.forward(xd, gd, bd, idxd, gated)
    off = st.offsets.tolist()
    dw = torch.zeros((E, d, d), dtype=torch.float64)
    rows = st.rows.double()
    for e in range(E):   # the experts' products in 64 bits: only the operators' own arithmetic is measured
        st.y[off[e]:off[e + 1]] = (rows[off[e]:off[e + 1]] @ wd[e].double()).float()
    st.back(gated)
    st.backward_rows(doutd, gated)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        dw[e] = (rows[r].T @ st.dy[r].double()).cpu()
        st.drows[r] = (st.dy[r].double() @ wd[e].double().T).float()
    st.backward_x(xd, gd, bool(kind))
    torch.cuda.synchronize()
    got = [st.dx, st.dgain, st.dgate, dw] + ([st.dbias] if kind else [])
    ops64.assert_close(st.out.cpu(), out8.detach(), 400 * ops64.U * (out8.detach().abs().max() + torch.zeros_like(out8)))
    # each value passes at most 400 fp32 roundings on the largest terms of its kind (84 + 84 in the norm's two
    # directions, T / 64 + 100 in the columns' sums, a few in each other step), each term at most the largest size
    sizes = [(want[0].abs().max(), 4), (dout.abs().sum(0).max() * x8.abs().max() * 4, 1), (want[2].abs().max(), 4),
             (want[3].abs().max(), 4), (want[0].abs().max() * T, 1)]
    for a, b, (size, f) in zip(got, want, sizes):
        ops64.assert_close(a.cpu(), b, 400 * ops64.U * f * float(size.detach()) + torch.zeros_like(b))


def test_training_calls_in_a_graph(m):
    """Forward and backward calls captured into one graph and replayed on new tokens give the eager bits, with
    an unrelated autograd graph of the same leaves alive."""
    T, k, E, d = 300, 2, 8, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    f = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, gain, dout, gate = f(T, d), f(d), f(T, d), f(T, k)
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    leaf = gain.requires_grad_()
    alive = (leaf * 2).sum()
    eager, cap = Train(m, 1, T, k, E, d), Train(m, 1, T, k, E, d)

    def step(st):
        st.forward(x, gain.detach(), None, idx, gate)
        st.y.copy_(st.rows)
        st.back(gate)
        st.backward_rows(dout, gate)
        st.drows.copy_(st.dy)
        st.backward_x(x, gain.detach(), True)
    step(cap)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for _ in range(3):
        x.copy_(f(T, d))
        idx.copy_(torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32))
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for name in ("out", "dx", "dgain", "dbias", "dgate", "slot", "perm", "offsets"):
            assert torch.equal(getattr(eager, name), getattr(cap, name)), name
    alive.backward()
    assert (leaf.grad == 2).all()


def test_binding_refuses_tensors_it_would_misread(m):
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    bad = [(x.t(), y), (x[:, ::2], y), (x.float(), y), (x, y[:4]), (x.cpu(), y), (x, torch.empty((8, 64), device="cuda"))]
    for a, b in bad:
        with pytest.raises(ValueError):
            m.moe_norm_forward(m.MOE_NORM_RMS, m.MOE_BF16, 8, 64, a, None, None, 1e-5, b)
    # a view that begins off a 16-byte boundary is the library's to refuse
    flat = torch.zeros(8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 64)
    assert m.moe_norm_forward(m.MOE_NORM_RMS, m.MOE_BF16, 8, 64, flat, None, None, 1e-5, y) == m.MOE_EINVAL


def test_calls_right_behind_one_another(m):
    """Launches may be scheduled before their predecessors on the stream have ended: chains of calls that reuse every
    buffer (rows, workspace, order) with new inputs each turn give the bits of the same chain with waits."""
    T, k, E, d = 2000, 2, 16, 768
    g = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn((T, d), generator=g, device="cuda") for _ in range(4)]
    idxs = [torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous() for _ in range(4)]
    gain, gate = torch.randn(d, generator=g, device="cuda"), torch.rand((T, k), generator=g, device="cuda")
    blk = Block4(m, 8, 256, 512, 64)

    def chain(wait):
        st, out = Train(m, 1, T, k, E, d), []
        pause = torch.cuda.synchronize if wait else (lambda: None)
        for turn in range(8):
            x, idx = xs[turn % 4], idxs[turn * 3 % 4]
            st.forward(x, gain, None, idx, gate)
            pause()
            m.check(m.moe_unsort_rows(m.MOE_F32, m.MOE_F32, T, k, d, st.rows, st.slot, gate, st.out))
            pause()
            m.check(m.moe_unsort_rows_backward(m.MOE_F32, m.MOE_F32, T, k, d, st.out, st.rows, st.slot, gate, st.dy, st.dgate))
            pause()
            m.check(m.moe_unsort_rows(m.MOE_F32, m.MOE_F32, T, k, d, st.dy, st.slot, None, st.du))
            pause()
            m.check(m.moe_norm_backward(1, m.MOE_F32, T, d, x, gain, st.stats, st.du, st.dx, st.dgain, st.dbias, st.ws))
            pause()
            out += [t.clone() for t in (st.out, st.dx, st.dgain, st.dbias, st.dgate, st.perm, st.slot)]
        h = tokens(8, 256, 1).cuda()
        for _ in range(6):   # the block on its own output, routing and experts in a row
            blk.h.copy_(h)
            blk.run()
            pause()
            h = blk.out.clone()
        return out + [h]
    want = chain(True)
    for _ in range(3):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)


def test_a_refused_call_leaves_no_error_behind(m):
    """A call that the runtime refuses (on the legacy stream while another stream is being captured) returns MOE_ECUDA and is
    over with it: the next call of any entry point does not report it again."""
    cu = ctypes.CDLL("libcuda.so.1")
    s, graph = ctypes.c_void_p(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert cu.cuStreamCreate(ctypes.byref(s), 0) == 0   # a stream that the legacy stream waits for
    T, d = 64, 64
    i32 = dict(dtype=torch.int32, device="cuda")
    x, w = torch.ones((T, d), dtype=torch.bfloat16, device="cuda"), torch.ones((d, 8), device="cuda")
    idx, offsets, perm, gate = (torch.empty((T, 2), **i32), torch.empty(9, **i32), torch.empty(2 * T, **i32),
                                torch.empty((T, 2), device="cuda"))
    g = torch.ones(d, device="cuda")
    calls = {"sort": lambda: m.moe_sort_rows(0, 0, 2, 8, d, None, None, offsets, None, None, None, 0),
             "norm": lambda: m.moe_norm_backward(0, 0, 0, d, None, None, None, None, None, g, None, None, 0)}
    m.check(m.moe_route_noalloc(T, d, x, w, None, idx, gate, offsets, perm))
    for name, call in calls.items():
        torch.cuda.synchronize()
        assert cu.cuStreamBeginCapture_v2(s, 0) == 0   # 0: the mode that forbids this everywhere
        try:
            assert call() == m.MOE_ECUDA, name
        finally:
            assert cu.cuStreamEndCapture(s, ctypes.byref(graph)) != 0   # the call ended the capture
        assert m.moe_route_noalloc(T, d, x, w, None, idx, gate, offsets, perm) == m.MOE_OK, name
        torch.cuda.synchronize()
    assert cu.cuStreamDestroy_v2(s) == 0


def test_blocks_of_several_host_threads(m):
    """Blocks of different sizes run by a host thread each, on streams of their own, give the bits of a block run alone."""
    blks = [Block4(m, T, d, ffn, group, seed=T) for T, d, ffn, group in ((1, 256, 512, 128), (8, 512, 1024, 64), (33, 264, 328, 32))]
    streams, want, failed = [torch.cuda.Stream() for _ in blks], [], []
    for blk in blks:
        blk.h.copy_(tokens(blk.T, blk.d, blk.T))
        blk.run()
        torch.cuda.synchronize()
        want.append([getattr(blk, k).clone() for k in ("rows", "mid", "y", "out")])
    torch.cuda.synchronize()

    def work(blk, stream):
        try:
            for _ in range(300):
                blk.experts(stream.cuda_stream)   # the routing stays outside: it shares a scratch array
        except Exception as e:   # noqa: BLE001 -- the test's own thread reports it
            failed.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(blks, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for blk, ref in zip(blks, want):
        for got, r in zip((blk.rows, blk.mid, blk.y, blk.out), ref):
            assert torch.equal(got, r)

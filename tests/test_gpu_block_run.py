"""The operators around the layer as they are used together: the norms between
two blocks, routing, dispatch, a caller's own experts, combine, and the way
back; the stack whose blocks carry norms; CUDA graphs; streams.

The forward run is compared with a 64-bit run of the same routing, the
backward run with 64-bit autograd of that. Tolerances: relative to the 2-norm,
1e-5 in fp32 (each operator adds at most some hundred steps of 2^-24 to its
magnitudes, five of them follow one another, and the matrix products of the
experts in between are torch's fp32)."""
import pytest

torch = pytest.importorskip("torch")

import synth  # noqa: E402
from tests import block_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def rel(a, b):
    a, b = ref.d(a), ref.d(b)
    return float((a - b).norm() / b.norm())


class Moe:
    """A block with a caller's own experts (one matrix each) between its norms, and its gradient, by the library."""

    def __init__(self, coli, dev, T, H, E, K, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g).to(dev)  # noqa: E731
        self.coli, self.T, self.H, self.E, self.K = coli, T, H, E, K
        self.wr, self.bias = r(E, H) / H ** 0.5, r(E)
        self.experts = r(E, H, H) / H ** 0.5
        self.first = coli.Block(pre_gain=1 + 0.2 * r(H))
        self.end = dict(post_norm=True, post_gain=1 + 0.2 * r(H), gate=r(H), x_scale=0.9, y_scale=1.1)
        self.prev = coli.Block(**self.end)
        self.next = coli.Block(pre_gain=1 + 0.2 * r(H))
        z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
        i32 = torch.int32
        self.x, self.c1, self.c2, self.u = r(T, H), r(T, H), r(T, H), torch.rand(T, generator=g).to(dev)
        self.n0, self.y, self.xo, self.n1 = z(T, H), z(T, H), z(T, H), z(T, H)
        self.ids, self.w = z(T, K, dtype=i32), z(T, K)
        self.counts, self.offsets = z(E, dtype=i32), z(E + 1, dtype=i32)
        self.pos, self.slot = z(T, K, dtype=i32), z(T * K, dtype=i32)
        self.rows, self.out, self.dout, self.drows = (z(T * K, H) for _ in range(4))
        self.dxo, self.dy, self.dn0, self.dn0r, self.dx = (z(T, H) for _ in range(5))
        self.dw, self.dl = z(T, K), z(T, K)
        self.dwr, self.db, self.dpost, self.dgate, self.dpre, self.dpre0 = z(E, H), z(E), z(H), z(H), z(H), z(H)
        self.du = z(T)
        need = max(coli.dispatch_workspace(T, K, E), coli.block_norm_workspace(T, H),
                   coli.route_backward_workspace(T, K, E, H), 16)
        self.work = torch.empty(need, dtype=torch.uint8, device=dev)

    def forward(self):
        c = self.coli
        c.block_norm(None, self.first, self.x, n=self.n0)
        c.route_noalloc(self.wr, self.bias, self.E, self.H, self.K, self.n0, self.ids, self.w)
        c.dispatch(self.ids, self.n0, self.E, self.counts, self.offsets, self.pos, self.slot, self.rows, self.work)
        self.which = torch.gather(self.ids.reshape(-1), 0, self.slot.long())  # expert of each row
        self.out.copy_(torch.bmm(self.rows.unsqueeze(1), self.experts[self.which.long()]).squeeze(1))
        c.combine(self.pos, self.w, self.out, self.y, self.n0)
        c.block_norm(self.prev, self.next, self.x, self.y, self.xo, self.n1, self.u)

    def backward(self):
        """Gradients of <c1, x_out> + <c2, n1>."""
        c = self.coli
        c.block_norm_backward(self.prev, self.next, self.xo, self.y, self.c1, self.c2, self.dxo, self.dy,
                              dpre_gain=self.dpre, dpost_gain=self.dpost, dgate=self.dgate, token_gate=self.u,
                              dtoken_gate=self.du, work=self.work)
        c.combine_backward(self.pos, self.w, self.dy, self.out, self.dout, self.dw)
        self.drows.copy_(torch.bmm(self.dout.unsqueeze(1), self.experts[self.which.long()].transpose(1, 2)).squeeze(1))
        c.route_backward(self.wr, self.n0, self.ids, self.w, self.dw, self.offsets, self.slot, self.dl, self.dn0r,
                         self.dwr, self.db, self.work)
        self.dn0r.add_(self.dy)  # the combine's base was n0
        c.dispatch_backward(self.pos, self.drows, self.dn0, self.dn0r)
        c.block_norm_backward(None, self.first, self.x, dx_out=self.dxo, dn=self.dn0, dx=self.dx, dpre_gain=self.dpre0,
                              work=self.work)

    GRADS = ("dx", "dwr", "db", "dpost", "dgate", "dpre", "dpre0", "du")

    def reference(self):
        """The same in 64 bits with the routing's ids, and autograd's gradients."""
        D = torch.float64
        leaf = {k: v.detach().to(D).requires_grad_() for k, v in dict(
            dx=self.x, dwr=self.wr, db=self.bias, dpost=self.prev.tensors[1], dgate=self.prev.tensors[2],
            dpre=self.next.tensors[0], dpre0=self.first.tensors[0], du=self.u).items()}
        norm = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
        n0 = norm(leaf["dx"]) * leaf["dpre0"]
        ids = self.ids.long()
        w = torch.softmax((n0 @ leaf["dwr"].t() + leaf["db"]).gather(1, ids), 1)
        y = n0
        for k in range(self.K):
            o = torch.bmm(n0.unsqueeze(1), self.experts.to(D)[ids[:, k]]).squeeze(1)
            y = y + w[:, k:k + 1] * o
        s = self.end["x_scale"] * leaf["dx"] + self.end["y_scale"] * leaf["du"].unsqueeze(1) * leaf["dgate"] * \
            leaf["dpost"] * norm(y)
        n1 = norm(s) * leaf["dpre"]
        ((s * self.c1.to(D)).sum() + (n1 * self.c2.to(D)).sum()).backward()
        return s, n1, {k: v.grad for k, v in leaf.items()}


@pytest.mark.parametrize("T,H,E,K", [(1, 128, 4, 2), (33, 256, 16, 4), (60, 384, 8, 8)])
def test_block_and_its_gradient(gpu, coli, T, H, E, K):
    m = Moe(coli, gpu, T, H, E, K)
    m.forward()
    m.backward()
    s, n1, grads = m.reference()
    assert rel(m.xo, s) < 1e-5 and rel(m.n1, n1) < 1e-5
    for k in m.GRADS:
        assert rel(getattr(m, k), grads[k]) < 1e-5, k


def test_captured_and_replayed(gpu, coli):
    """Forward and backward in CUDA graphs, two of them with one workspace on one stream, replayed on new inputs."""
    m = Moe(coli, gpu, 60, 256, 16, 4)
    m.forward()  # route_noalloc looks its scratch up outside a capture
    m.backward()
    torch.cuda.synchronize()
    fwd, bwd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(fwd):
        m.forward()
    with torch.cuda.graph(bwd):
        m.backward()
    for seed in (1, 2):
        m.x.copy_(torch.randn(m.x.shape, generator=torch.Generator().manual_seed(seed)))
        for name in m.GRADS + ("xo", "n1"):
            getattr(m, name).fill_(float("nan"))
        fwd.replay()
        bwd.replay()
        torch.cuda.synchronize()
        got = {k: getattr(m, k).clone() for k in m.GRADS + ("xo", "n1")}
        m.forward()
        m.backward()
        for k, v in got.items():
            assert torch.equal(v, getattr(m, k)), k


@pytest.mark.parametrize("T", [7, 1500, 17000])
def test_large_plan_captured(gpu, coli, T):
    """The sort's several launches in a graph, back to back with another call's on the same workspace."""
    K, E, H = 8, 64, 128
    g = torch.Generator().manual_seed(3)
    ids = [torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32) for _ in range(3)]
    dev_ids = torch.zeros((T, K), dtype=torch.int32, device=gpu)
    x = torch.randn((T, H), device=gpu)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=gpu)  # noqa: E731
    a = [(z(E), z(E + 1), z(T, K), z(T * K), torch.zeros((T * K, H), device=gpu)) for _ in range(2)]
    work = torch.empty(max(16, coli.dispatch_workspace(T, K, E)), dtype=torch.uint8, device=gpu)
    other = ids[2].to(gpu)

    def both():
        coli.dispatch(dev_ids, x, E, *a[0], work)
        coli.dispatch(other, x, E, *a[1], work)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in (0, 1):
        dev_ids.copy_(ids[i])
        graph.replay()
        torch.cuda.synchronize()
        for got, src in ((a[0], ids[i]), (a[1], ids[2])):
            want = ref.plan(src, E)
            for v, w in zip(got, want):
                assert torch.equal(v.cpu(), w)
            n = int(want[1][-1])
            assert torch.equal(got[4][:n], x[(want[3][:n] // K).long().to(gpu)])


def test_on_another_stream(gpu, coli):
    """Calls on a side stream, given or current, wait for that stream's work alone."""
    T, H = 2048, 1024
    side = torch.cuda.Stream()
    x = torch.zeros((T, H), device=gpu)
    n, n2 = torch.empty_like(x), torch.empty_like(x)
    b = coli.Block()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            x.add_(1.0)
        coli.block_norm(None, b, x, n=n)
    coli.block_norm(None, b, x, n=n2, stream=side)
    side.synchronize()
    assert torch.allclose(n, torch.ones_like(n)) and torch.equal(n, n2)


def layers_of(coli, n, T, cached=False):
    H, I, E, K = 512, 256, 16, 2
    out = []
    for l in range(n):
        experts = [synth.expert(5, l, e, H, I) for e in range(E)]
        import numpy as np
        out.append(coli.Layer(coli.make_config(H, I, E, K, 0, T), synth.router(5, l, E, H), None,
                              np.concatenate([e[0] for e in experts]), np.concatenate([e[1] for e in experts]),
                              resident=E if cached else None))
    return out


@pytest.mark.parametrize("T", [1, 5, 96])
@pytest.mark.parametrize("cached", [False, True])
def test_block_stack(gpu, coli, T, cached):
    """The stack with norms against its layers called one by one with 64-bit norms between them."""
    H = 512
    layers = layers_of(coli, 3, T, cached)
    g = torch.Generator().manual_seed(12)
    v = lambda: (1 + 0.2 * torch.randn(H, generator=g)).to(gpu)  # noqa: E731
    par = [dict(pre_gain=v(), post_norm=True, post_gain=v(), gate=v(), x_scale=0.9, y_scale=0.7, eps=1e-5),
           dict(), dict(post_norm=True, gate=v(), eps=1e-6)]
    x0 = torch.from_numpy(synth.x_f32(5, 0, T, H)).to(gpu)
    x, work = x0.clone(), torch.empty_like(x0)
    counts = [l.launch_count() for l in layers]
    coli.block_stack_forward(layers, [coli.Block(**p) for p in par], x, work)
    assert all(l.launch_count() > c for l, c in zip(layers, counts))
    want = x0.double()
    for l, p in zip(layers, par):
        r = ref.Norm(p, p)
        n = r.n(want.cpu()).float().to(gpu)
        y = torch.empty_like(n)
        l.forward(n, y)
        want = r.x_out(want.cpu(), ref.d(y))[0].to(gpu)
    # a norm input off by 28 steps of 2^-24 moves the layer's 15-bit block-floating codes by one of their
    # steps at most, 2^-15 of a group's largest value, in few of them
    assert float((x.double() - want).abs().max() / want.abs().max()) < 1e-3
    if T > 1:  # the first rows alone
        part, before = x0.clone(), x0[T - 1].clone()
        coli.block_stack_forward(layers, [coli.Block(**p) for p in par], part, work, n_tokens=T - 1)
        assert torch.equal(part[T - 1], before) and not torch.equal(part[:T - 1], x0[:T - 1])
        assert float((part[:T - 1] - x[:T - 1]).abs().max() / x.abs().max()) < 1e-3
    # unit parameters: the plain stack
    a, b = x0.clone(), x0.clone()
    coli.stack_forward(layers, a)
    coli.block_stack_forward(layers, [coli.Block() for _ in layers], b, work)
    assert float((a - b).abs().max() / a.abs().max()) < 1e-3
    for l in layers:
        l.close()


def test_block_stack_refuses(gpu, coli):
    layers = layers_of(coli, 1, 4)
    x = torch.zeros((4, 512), device=gpu)
    w = torch.zeros_like(x)
    with pytest.raises(ValueError):
        coli.block_stack_forward(layers, [], x, w)
    with pytest.raises(ValueError):
        coli.block_stack_forward(layers, [coli.Block(gate=torch.ones(256, device=gpu))], x, w)
    with pytest.raises(TypeError):
        coli.block_stack_forward(layers, [coli.Block()], x.double(), w)
    with pytest.raises(coli.ColiError, match="overlap"):
        coli.block_stack_forward(layers, [coli.Block()], x, x)
    big = torch.zeros((9, 512), device=gpu)
    with pytest.raises(coli.ColiError, match="max_tokens"):
        coli.block_stack_forward(layers, [coli.Block()], big, torch.zeros_like(big))
    layers[0].close()
    with pytest.raises(ValueError):
        coli.block_stack_forward(layers, [coli.Block()], x, w)

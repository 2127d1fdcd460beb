"""What the operators around the layer refuse of torch tensors, and calls that
the documentation allows at the edges: views, broadcast rows, wrong plans."""
import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402
from tests.test_gpu_dispatch import make_ids  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def bad_calls(coli, dev):
    T, K, E, H = 4, 2, 8, 64
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
    i32 = torch.int32
    ids, pos, slot = z(T, K, dtype=i32), z(T, K, dtype=i32), z(T * K, dtype=i32)
    counts, offsets = z(E, dtype=i32), z(E + 1, dtype=i32)
    x, rows, w = z(T, H), z(T * K, H), z(T, K)
    d = lambda **kw: coli.dispatch(*{**dict(ids=ids, x=x, E=E, counts=counts, offsets=offsets, pos=pos, slot=slot,  # noqa: E731
                                            rows=rows), **kw}.values())
    c = lambda **kw: coli.combine(*{**dict(pos=pos, w=w, rows=rows, y=z(T, H), base=None), **kw}.values())  # noqa: E731
    n = lambda **kw: coli.block_norm(*{**dict(prev=coli.Block(), next=coli.Block(), x=x, y=z(T, H), xo=z(T, H),  # noqa: E731
                                              n=z(T, H), u=None), **kw}.values())
    V, Ty = ValueError, TypeError
    return [
        (V, "shape", lambda: d(ids=ids[0])), (Ty, "int32", lambda: d(ids=ids.long())), (V, "shape", lambda: d(E=7)),
        (V, "contiguous", lambda: d(pos=z(K, T, dtype=i32).t())), (V, "shape", lambda: d(rows=z(T * K, H + 1))),
        (coli.ColiError, "n_rows", lambda: d(rows=z(T * K - 1, H))), (Ty, "bfloat16", lambda: d(x=x.half())),
        (V, "CUDA", lambda: d(x=x.cpu())), (V, "contiguous rows", lambda: d(x=z(H, T).t())),
        (V, "out of range", lambda: d(E=-1)), (Ty, "integer", lambda: d(E="8")), (Ty, "tensor", lambda: d(counts=[1])),
        (V, "out of range", lambda: d(E=1 << 40, counts=None)), (coli.ColiError, "counts", lambda: d(counts=None)),
        (Ty, "tensor", lambda: c(rows=None)), (Ty, "dtype", lambda: c(base=z(T, H, dtype=torch.bfloat16))),
        (V, "shape", lambda: c(w=z(T, K + 1))), (coli.ColiError, "overlap", lambda: c(y=rows[:T])),
        (coli.ColiError, "stride", lambda: c(y=z(1, H).expand(T, H))), (V, "negated", lambda: c(base=torch._neg_view(x))),
        (Ty, "stream", lambda: coli.combine(pos, w, rows, z(T, H), None, "s")),
        (Ty, "Block", lambda: n(prev=1)), (V, "arrays", lambda: n(prev=coli.Block(gate=z(H + 1)))),
        (Ty, "dtype", lambda: n(xo=z(T, H, dtype=torch.bfloat16))), (V, "shape", lambda: n(u=z(T + 1))),
        (coli.ColiError, "overlap", lambda: n(n=x)), (V, "matrix", lambda: n(x=z(H))),
        (coli.ColiError, "work", lambda: coli.block_norm_backward(coli.Block(), coli.Block(), x, x.clone(), None, x.clone(),
                                                                  dpre_gain=z(H))),
        (V, "dweights needs rows", lambda: coli.combine_backward(pos, w, x, None, rows, z(T, K))),
        (coli.ColiError, "offsets and slot", lambda: coli.route_backward(z(E, H), x, ids, w, w.clone(), None, None, z(T, K),
                                                                         None, z(E, H), None, z(1 << 16))),
    ]


def test_bad_tensors(gpu, coli):
    for exc, msg, call in bad_calls(coli, gpu):
        with pytest.raises(exc, match=msg):
            call()
    torch.cuda.synchronize()


def test_columns_of_one_wider_matrix(gpu, coli):
    """Inputs and outputs that are columns of one buffer do not overlap."""
    T, K, H = 9, 3, 64
    buf = torch.randn((T * K, 3 * H), device=gpu)
    want = buf[:, H:2 * H].clone()
    pos = torch.arange(T * K, dtype=torch.int32, device=gpu).reshape(T, K)
    y = torch.empty((T, H), device=gpu)
    coli.dispatch_backward(pos, buf[:, H:2 * H], y)
    assert torch.allclose(y, want.reshape(T, K, H).sum(1), atol=1e-5)
    coli.combine_backward(pos, torch.full((T, K), 2.0, device=gpu), y, buf[:, :H], buf[:, 2 * H:])
    assert torch.equal(buf[:, 2 * H:], (2 * y).repeat_interleave(K, 0))
    one = torch.randn((1, H), device=gpu)
    coli.dispatch_backward(torch.zeros((1, 2), dtype=torch.int32, device=gpu), one.expand(1, H), y[:1], one)
    assert torch.equal(y[0], (one + one + one)[0])


@pytest.mark.parametrize("T,E", [(3, 64), (50, 64)])
def test_absent_slots_of_the_router(gpu, coli, T, E):
    """A slot of weight 0 leaves out its router row and its token, whatever they hold."""
    K, H = 2, 128
    ids = torch.stack([torch.arange(T) % 8, torch.full((T,), E - 1)], 1).int().to(gpu)
    w = torch.tensor([[1.0, 0.0]], device=gpu).repeat(T, 1)
    dw = torch.ones((T, K), device=gpu)
    dw[:, 1] = float("nan")
    wr = torch.randn((E, H), device=gpu)
    wr[E - 1] = float("inf")
    x = torch.randn((T, H), device=gpu)
    counts, offsets, pos, slot = (t.to(gpu) for t in ref.plan(ids.cpu(), E))
    z = lambda *s: torch.full(s, 7.0, device=gpu)  # noqa: E731
    dl, dx, dwr, db = z(T, K), z(T, H), z(E, H), z(E)
    work = torch.empty(coli.route_backward_workspace(T, K, E, H), dtype=torch.uint8, device=gpu)
    coli.route_backward(wr, x, ids, w, dw, offsets, slot, dl, dx, dwr, db, work)
    for t in (dl, dx, dwr, db):  # with one slot left its weight is 1 whatever the logits are: no gradient
        assert (t == 0).all()


def test_a_plan_of_another_routing_stays_in_bounds(gpu, coli):
    """offsets and slot that do not belong to the ids: drouter_w means nothing then, the rest is right."""
    T, K, E, H = 900, 8, 32, 136
    g = torch.Generator().manual_seed(5)
    ids, other = make_ids(T, K, E, "random", 1), make_ids(T, K, E, "one", 2)
    w, dw = torch.softmax(torch.randn((T, K), generator=g), 1).to(gpu), torch.randn((T, K), generator=g).to(gpu)
    wr, x = torch.randn((E, H), generator=g).to(gpu), torch.randn((T, H), generator=g).to(gpu)
    outs = []
    for plan_of in (ids, other):
        counts, offsets, pos, slot = (t.to(gpu) for t in ref.plan(plan_of, E))
        if plan_of is other:
            offsets = offsets + torch.arange(E + 1, device=gpu, dtype=torch.int32) * 1000 - 500
        dl, dx = torch.empty((T, K), device=gpu), torch.empty((T, H), device=gpu)
        dwr, db = torch.empty((E, H), device=gpu), torch.empty((E,), device=gpu)
        work = torch.full((coli.route_backward_workspace(T, K, E, H),), 0x7F, dtype=torch.uint8, device=gpu)
        coli.route_backward(wr, x, ids.to(gpu), w, dw, offsets, slot, dl, dx, dwr, db, work)
        outs.append((dl, dx))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_two_streams_with_workspaces_of_their_own(gpu, coli):
    """Calls that overlap on the GPU, each with its own outputs and workspace."""
    T, H = 600, 512
    streams = [torch.cuda.Stream() for _ in range(2)]
    g = torch.Generator().manual_seed(6)
    s, y, o, n = (torch.randn((T, H), generator=g).to(gpu) for _ in range(4))
    prev, nxt = coli.Block(post_norm=True), coli.Block()
    res = []
    for _ in range(2):
        res.append(dict(dx=torch.empty_like(s), dy=torch.empty_like(s), dq=torch.empty(H, device=gpu),
                        dp=torch.empty(H, device=gpu),
                        work=torch.empty(coli.block_norm_workspace(T, H), dtype=torch.uint8, device=gpu)))
    torch.cuda.synchronize()
    for _ in range(10):
        for st, r in zip(streams, res):
            coli.block_norm_backward(prev, nxt, s, y, o, n, r["dx"], r["dy"], dpre_gain=r["dq"], dpost_gain=r["dp"],
                                     work=r["work"], stream=st)
    torch.cuda.synchronize()
    for k in ("dx", "dy", "dq", "dp"):
        assert torch.equal(res[0][k], res[1][k])


def test_calls_of_several_threads(gpu, coli):
    """Calls of one kernel with different amounts of shared memory, made at the same time."""
    from concurrent.futures import ThreadPoolExecutor

    def work(i):
        E, T, K, H = (4, 16, 300, 1024)[i], (700, 4000, 1500, 900)[i], (3, 8, 4, 2)[i], (1024, 4096, 512, 2048)[i]
        g = torch.Generator().manual_seed(i)
        ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int32).to(gpu)
        x, y, o = (torch.randn((T, H), generator=g).to(gpu) for _ in range(3))
        w, dw = (torch.randn((T, K), generator=g).to(gpu) for _ in range(2))
        wr = torch.randn((E, H), generator=g).to(gpu)
        st, first = torch.cuda.Stream(gpu), None
        i32 = dict(dtype=torch.int32, device=gpu)
        bufs = [torch.zeros(n, **i32) for n in (E, E + 1, (T, K), T * K)]
        dl, dx, dwr, db = (torch.zeros(n, device=gpu) for n in ((T, K), (T, H), (E, H), (E,)))
        xo, n, gx, gy = (torch.zeros_like(x) for _ in range(4))
        dwork = torch.zeros(coli.dispatch_workspace(T, K, E), dtype=torch.uint8, device=gpu)
        rwork = torch.zeros(coli.route_backward_workspace(T, K, E, H), dtype=torch.uint8, device=gpu)
        torch.cuda.synchronize()
        for _ in range(200):
            counts, offsets, pos, slot = bufs
            coli.dispatch(ids, None, E, counts, offsets, pos, slot, None, dwork, stream=st)
            coli.route_backward(wr, x, ids, w, dw, offsets, slot, dl, dx, dwr, db, rwork, stream=st)
            coli.block_norm(coli.Block(), coli.Block(), x, y, xo, n, stream=st)
            coli.block_norm_backward(coli.Block(), coli.Block(), x, y, o, x, gx, gy, stream=st)
            st.synchronize()
            if first is None:
                first = [t.clone() for t in (*bufs, dl, dx, dwr, db, xo, n, gx, gy)]
                torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip(first, (*bufs, dl, dx, dwr, db, xo, n, gx, gy)))

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(4)))

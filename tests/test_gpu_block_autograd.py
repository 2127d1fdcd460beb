"""The operators around the layer write the caller's tensors and record no
gradient. Their writes move the tensors' versions, as torch's own in-place
operations do, so that autograd notices a saved tensor that was overwritten."""
import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def calls(coli, dev):
    """(name, call, tensors that it writes, tensors that it reads)"""
    T, K, E, H = 6, 2, 8, 64
    f = lambda *s: torch.rand(s, device=dev)  # noqa: E731
    ids = (torch.arange(T * K, device=dev, dtype=torch.int32) % E).reshape(T, K)
    counts, offsets, pos, slot = (t.to(dev) for t in ref.plan(ids.cpu(), E))
    x, y, dy, w, dw, dl, wr, dwr, db = f(T, H), f(T, H), f(T, H), f(T, K), f(T, K), f(T, K), f(E, H), f(E, H), f(E)
    rows, drows, dx, base = f(T * K, H), f(T * K, H), f(T, H), f(T, H)
    xo, n, gx, gy, u, du = f(T, H), f(T, H), f(T, H), f(T, H), f(T), f(T)
    dq, dp, dg = f(H), f(H), f(H)
    rwork = torch.empty(coli.route_backward_workspace(T, K, E, H), dtype=torch.uint8, device=dev)
    nwork = torch.empty(coli.block_norm_workspace(T, H), dtype=torch.uint8, device=dev)
    a, b = coli.Block(post_norm=True), coli.Block()
    return [
        ("dispatch", lambda: coli.dispatch(ids, x, E, counts, offsets, pos, slot, rows), (counts, offsets, pos, slot, rows),
         (ids, x)),
        ("plan", lambda: coli.dispatch(ids, None, E, counts, offsets, pos, slot, None), (counts, offsets, pos, slot),
         (ids, rows)),
        ("dispatch_backward", lambda: coli.dispatch_backward(pos, drows, dx, base), (dx,), (pos, drows, base)),
        ("combine", lambda: coli.combine(pos, w, rows, y, base), (y,), (pos, w, rows, base)),
        ("combine_backward", lambda: coli.combine_backward(pos, w, dy, rows, drows, dw), (drows, dw), (pos, w, dy, rows)),
        ("route_backward", lambda: coli.route_backward(wr, x, ids, w, dw, offsets, slot, dl, dx, dwr, db, rwork),
         (dl, dx, dwr, db, rwork), (wr, x, ids, w, dw, offsets, slot)),
        ("block_norm", lambda: coli.block_norm(a, b, x, y, xo, n, u), (xo, n), (x, y, u)),
        ("block_norm_backward",
         lambda: coli.block_norm_backward(a, b, xo, y, dy, n, gx, gy, dq, dp, dg, u, du, nwork),
         (gx, gy, dq, dp, dg, du, nwork), (xo, y, dy, n, u)),
    ]


def test_versions(gpu, coli):
    for name, call, written, read in calls(coli, gpu):
        before = [t._version for t in written], [t._version for t in read]
        call()
        assert all(t._version > v for t, v in zip(written, before[0])), name
        assert all(t._version == v for t, v in zip(read, before[1])), name


def test_autograd_notices_overwritten_rows(gpu, coli):
    """The experts of a training step, whose saved inputs a second dispatch overwrites."""
    name, call, (counts, offsets, pos, slot, rows), _ = calls(coli, gpu)[0]
    call()
    expert = torch.randn((64, 64), device=gpu, requires_grad=True)
    loss = (rows @ expert).sum()
    call()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    loss = (rows @ expert).sum()
    loss.backward()
    assert torch.isfinite(expert.grad).all()


def test_a_refused_call_moves_no_version(gpu, coli):
    T, K, H = 4, 2, 64
    pos, w = torch.zeros((T, K), dtype=torch.int32, device=gpu), torch.zeros((T, K), device=gpu)
    rows = torch.zeros((T * K, H), device=gpu)
    y = rows[:T]
    v = rows._version
    with pytest.raises(coli.ColiError, match="overlap"):
        coli.combine(pos, w, rows, y)
    assert rows._version == v


def test_inference_tensors(gpu, coli):
    """They have no version; inside and outside of inference mode they can be written as before."""
    x = torch.randn((3, 64), device=gpu)
    want = torch.empty_like(x)
    coli.block_norm(None, coli.Block(), x, n=want)
    with torch.inference_mode():
        n = torch.zeros((3, 64), device=gpu)
        coli.block_norm(None, coli.Block(), x, n=n)
        assert torch.equal(n, want)
        n.zero_()
    coli.block_norm(None, coli.Block(), x, n=n)
    assert torch.equal(n, want)


def test_block_stack_moves_versions(gpu, coli):
    import numpy as np
    import synth
    H, I, E, K, T = 512, 256, 16, 2, 4
    experts = [synth.expert(5, 0, e, H, I) for e in range(E)]
    layer = coli.Layer(coli.make_config(H, I, E, K, 0, T), synth.router(5, 0, E, H), None,
                       np.concatenate([e[0] for e in experts]), np.concatenate([e[1] for e in experts]))
    x = torch.from_numpy(synth.x_f32(5, 0, T, H)).to(gpu)
    work = torch.empty_like(x)
    before = x._version, work._version
    coli.block_stack_forward([layer], [coli.Block()], x, work)
    assert x._version > before[0] and work._version > before[1]
    with torch.inference_mode():
        xi, wi = x.clone(), work.clone()
    coli.block_stack_forward([layer], [coli.Block()], xi, wi)
    layer.close()

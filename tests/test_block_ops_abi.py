"""The operators around the layer refuse bad arguments before any CUDA call
(these run on the CPU: the pointers are never read)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def coli():
    import __graft_entry__  # noqa: F401
    import os
    from int4_expert_ffn_router_b200 import build as b
    if not os.path.exists(b.SO):
        b.build()
    import int4_expert_ffn_router_b200 as m
    return m


@pytest.fixture(scope="module", autouse=True)
def _argtypes(coli):
    L, vp, i, q = coli.lib, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.coli_moe_dispatch.argtypes = [vp, i, i, i, vp, i, q, i, vp, vp, vp, vp, vp, i, q, q, vp, q, i, vp]
    L.coli_moe_combine.argtypes = [vp, vp, i, i, vp, i, q, q, i, vp, q, vp, i, q, i, vp]
    L.coli_moe_combine_backward.argtypes = [vp, vp, i, i, vp, i, q, i, vp, i, q, q, vp, q, vp, i, vp]
    L.coli_moe_route_backward.argtypes = [vp, i, i, i, vp, i, q, i, vp, vp, vp, vp, vp, vp, vp, q, vp, vp, vp, q, i, vp]
    L.coli_block_norm.argtypes = [vp, vp, vp, i, q, vp, i, q, vp, vp, q, vp, i, q, i, i, i, vp]
    L.coli_block_norm_backward.argtypes = [vp, vp, vp, i, q, vp, i, q, vp, vp, q, vp, i, q, vp, q, vp, q, vp, vp, vp, vp, vp,
                                           q, i, i, i, vp]


# addresses far apart, 16-byte aligned, never dereferenced
P = [0x10_0000_0000 * (i + 1) for i in range(16)]


def _status(coli, st):
    return st, coli.lib.coli_last_error().decode()


def _dispatch(coli, **kw):
    a = dict(ids=P[0], T=4, K=2, E=16, x=P[1], xt=F32, xs=64, H=64, counts=P[2], offsets=P[3], pos=P[4], slot=P[5],
             rows=P[6], rt=F32, rs=64, n_rows=8, work=None, nw=0, dev=0)
    a.update(kw)
    return _status(coli, coli.lib.coli_moe_dispatch(
        a["ids"], a["T"], a["K"], a["E"], a["x"], a["xt"], a["xs"], a["H"], a["counts"], a["offsets"], a["pos"],
        a["slot"], a["rows"], a["rt"], a["rs"], a["n_rows"], a["work"], a["nw"], a["dev"], None))


@pytest.mark.parametrize("kw,msg", [
    (dict(T=-1), "n_tokens"), (dict(T=(1 << 20) + 1), "n_tokens"), (dict(K=0), "top_k"), (dict(K=33), "top_k"),
    (dict(T=1 << 20, K=17), "2^24"), (dict(E=0), "n_experts"), (dict(E=1025), "n_experts"), (dict(ids=None), "ids"),
    (dict(counts=None), "counts"), (dict(offsets=None), "offsets"), (dict(pos=None), "pos"), (dict(slot=None), "slot"),
    (dict(rows=None), "both or neither"), (dict(x=None), "both or neither"), (dict(H=0), "hidden"),
    (dict(H=65537, xs=65537, rs=65537), "hidden"), (dict(xt=2), "dtype"), (dict(rt=-1), "dtype"),
    (dict(xs=63), "x_stride"), (dict(rs=0), "rows_stride"), (dict(n_rows=7), "n_rows"), (dict(x=P[1] + 2), "aligned"),
    (dict(rows=P[6] + 1), "aligned"), (dict(ids=P[0] + 2), "4-byte"), (dict(rows=P[1] + 64), "overlap"),
    (dict(pos=P[0]), "overlap"), (dict(counts=P[3] + 4), "overlap"), (dict(slot=P[1] + 16), "overlap"),
    (dict(dev=-1), "device"), (dict(T=40000, K=8, n_rows=1 << 19), "work"),
    (dict(T=40000, K=8, n_rows=1 << 19, work=P[7], nw=511), "work"),
    (dict(T=40000, K=8, n_rows=1 << 19, work=P[7] + 8, nw=1 << 20), "16-byte"),
])
def test_dispatch_refuses(coli, kw, msg):
    st, err = _dispatch(coli, **kw)
    assert st == coli.COLI_EINVAL and msg in err, err


def test_workspaces(coli):
    assert coli.dispatch_workspace(0, 8, 256) == 0
    assert coli.block_norm_workspace(0, 64) == 0 and coli.block_norm_workspace(1, 64) >= 2 * 64 * 4
    for f, a in ((coli.dispatch_workspace, (-1, 8, 256)), (coli.dispatch_workspace, (1, 8, 2000)),
                 (coli.block_norm_workspace, (1, 0)), (coli.route_backward_workspace, (1, 8, 256, 1 << 20))):
        with pytest.raises(ValueError):
            f(*a)


def _combine(coli, **kw):
    a = dict(pos=P[0], w=P[1], T=4, K=2, rows=P[2], rt=F32, rs=64, n_rows=8, H=64, base=None, bs=64, y=P[3], yt=F32,
             ys=64, dev=0)
    a.update(kw)
    return _status(coli, coli.lib.coli_moe_combine(
        a["pos"], a["w"], a["T"], a["K"], a["rows"], a["rt"], a["rs"], a["n_rows"], a["H"], a["base"], a["bs"], a["y"],
        a["yt"], a["ys"], a["dev"], None))


@pytest.mark.parametrize("kw,msg", [
    (dict(T=-1), "n_tokens"), (dict(K=40), "top_k"), (dict(pos=None), "pos"), (dict(w=None), "weights"),
    (dict(rows=None), "rows"), (dict(y=None), "output"), (dict(n_rows=-1), "n_rows"), (dict(H=0), "hidden"),
    (dict(rs=60), "rows_stride"), (dict(ys=60), "stride"), (dict(base=P[4], bs=60), "base_stride"),
    (dict(base=P[3] + 16), "base"), (dict(y=P[2]), "overlap"), (dict(y=P[0]), "overlap"), (dict(y=P[1]), "overlap"),
    (dict(yt=7), "dtype"), (dict(rt=7), "dtype"), (dict(w=P[1] + 1), "aligned"), (dict(dev=-2), "device"),
])
def test_combine_refuses(coli, kw, msg):
    st, err = _combine(coli, **kw)
    assert st == coli.COLI_EINVAL and msg in err, err


def _combine_backward(coli, **kw):
    a = dict(pos=P[0], w=P[1], T=4, K=2, dy=P[2], dt=F32, ds=64, H=64, rows=P[3], rt=F32, rs=64, n_rows=8, drows=P[4],
             drs=64, dw=P[5], dev=0)
    a.update(kw)
    return _status(coli, coli.lib.coli_moe_combine_backward(
        a["pos"], a["w"], a["T"], a["K"], a["dy"], a["dt"], a["ds"], a["H"], a["rows"], a["rt"], a["rs"], a["n_rows"],
        a["drows"], a["drs"], a["dw"], a["dev"], None))


@pytest.mark.parametrize("kw,msg", [
    (dict(w=None), "weights"), (dict(dy=None), "dy"), (dict(rows=None), "rows"), (dict(drs=2), "drows_stride"),
    (dict(drows=P[2]), "overlap"), (dict(drows=P[3] + 16), "overlap"), (dict(dw=P[3]), "overlap"),
    (dict(dw=P[4]), "overlap"), (dict(drows=P[0]), "overlap"), (dict(dt=3), "dtype"), (dict(dw=P[5] + 2), "aligned"),
])
def test_combine_backward_refuses(coli, kw, msg):
    st, err = _combine_backward(coli, **kw)
    assert st == coli.COLI_EINVAL and msg in err, err


def _route_backward(coli, **kw):
    a = dict(wr=P[0], E=16, H=64, K=2, x=P[1], t=F32, xs=64, T=4, ids=P[2], w=P[3], dw=P[4], off=P[5], slot=P[6],
             dl=P[7], dx=P[8], dxs=64, dwr=P[9], db=P[10], work=P[11], nw=1 << 32, dev=0)
    a.update(kw)
    return _status(coli, coli.lib.coli_moe_route_backward(
        a["wr"], a["E"], a["H"], a["K"], a["x"], a["t"], a["xs"], a["T"], a["ids"], a["w"], a["dw"], a["off"], a["slot"],
        a["dl"], a["dx"], a["dxs"], a["dwr"], a["db"], a["work"], a["nw"], a["dev"], None))


@pytest.mark.parametrize("kw,msg", [
    (dict(T=-1), "n_tokens"), (dict(E=0), "n_experts"), (dict(H=0), "hidden"), (dict(K=33), "top_k"),
    (dict(t=2), "dtype"), (dict(wr=None), "router_w"), (dict(x=None), "x"), (dict(ids=None), "ids"),
    (dict(w=None), "weights"), (dict(dl=None), "dlogits"), (dict(off=None), "offsets"), (dict(slot=None), "slot"),
    (dict(dx=P[1]), "overlap"), (dict(dwr=P[0]), "overlap"), (dict(db=P[9]), "overlap"), (dict(dl=P[3]), "overlap"),
    (dict(xs=3), "x_stride"), (dict(dxs=3), "dx_stride"), (dict(dw=P[4] + 1), "aligned"), (dict(work=P[11] + 4), "work"),
])
def test_route_backward_refuses(coli, kw, msg):
    st, err = _route_backward(coli, **kw)
    assert st == coli.COLI_EINVAL and msg in err, err


def _norm(coli, prev=(), next=(), **kw):
    a = dict(x=P[0], xt=F32, xs=64, y=P[1], yt=F32, ys=64, tg=None, xo=P[2], xos=64, n=P[3], nt=F32, ns=64, T=4, H=64,
             dev=0)
    a.update(kw)
    bp = coli.Block(**dict(prev)) if prev is not None else None
    bn = coli.Block(**dict(next)) if next is not None else None
    for b, key in ((bp, "prev_set"), (bn, "next_set")):
        for f, v in kw.get(key, {}).items():
            setattr(b, f, v)
    return _status(coli, coli.lib.coli_block_norm(
        bp.address if bp is not None else None, bn.address if bn is not None else None, a["x"], a["xt"], a["xs"], a["y"],
        a["yt"], a["ys"], a["tg"], a["xo"], a["xos"], a["n"], a["nt"], a["ns"], a["T"], a["H"], a["dev"], None))


@pytest.mark.parametrize("kw,msg", [
    (dict(prev=None, next=None), "both NULL"), (dict(prev=None), "need prev"), (dict(next=None), "n needs next"),
    (dict(T=-1), "n_tokens"), (dict(H=0), "hidden"), (dict(x=None), "x is NULL"), (dict(y=None), "y is NULL"),
    (dict(xo=None), "x_out is NULL"), (dict(n=None), "n is NULL"), (dict(xs=8), "x_stride"), (dict(yt=9), "dtype"),
    (dict(prev=dict(eps=-1.0)), "eps"), (dict(prev_set=dict(eps=float("nan"))), "eps"),
    (dict(prev_set=dict(post_norm=2)), "post_norm"), (dict(prev_set=dict(post_gain=P[5])), "post_norm"),
    (dict(next_set=dict(pre_gain=P[5] + 2)), "aligned"), (dict(next_set=dict(pre_gain=P[3] + 16)), "overlap"),
    (dict(xo=P[0] + 16), "overlap"), (dict(xo=P[1]), "overlap"), (dict(n=P[0]), "overlap"), (dict(n=P[2]), "overlap"),
    (dict(n=P[1], nt=BF16), "overlap"), (dict(tg=P[2] + 32), "overlap"), (dict(dev=-1), "device"),
])
def test_block_norm_refuses(coli, kw, msg):
    st, err = _norm(coli, **kw)
    assert st == coli.COLI_EINVAL and msg in err, err


def _norm_backward(coli, prev=(("post_norm", True),), next=(), **kw):
    a = dict(s=P[0], xt=F32, y=P[1], yt=F32, tg=None, dxo=P[2], dn=P[3], nt=F32, dx=P[4], dy=P[5], dq=P[6], dp=P[7],
             dg=P[8], dt=P[9], work=P[10], nw=1 << 30, T=4, H=64, st=64)
    a.update(kw)
    bp = coli.Block(**dict(prev)) if prev is not None else None
    bn = coli.Block(**dict(next)) if next is not None else None
    s = a["st"]
    return _status(coli, coli.lib.coli_block_norm_backward(
        bp.address if bp is not None else None, bn.address if bn is not None else None, a["s"], a["xt"], s, a["y"],
        a["yt"], s, a["tg"], a["dxo"], s, a["dn"], a["nt"], s, a["dx"], s, a["dy"], s, a["dq"], a["dp"], a["dg"], a["dt"],
        a["work"], a["nw"], a["T"], a["H"], 0, None))


@pytest.mark.parametrize("kw,msg", [
    (dict(prev=None), "need prev"), (dict(next=None), "need next"), (dict(prev=()), "dpost_gain needs post_norm"),
    (dict(s=None), "x_out is NULL"), (dict(y=None), "y is NULL"), (dict(dn=None), "dn is NULL"), (dict(st=8), "stride"),
    (dict(work=None), "work"), (dict(nw=16), "work"), (dict(work=P[10] + 4), "16-byte"), (dict(dx=P[1]), "dx overlaps"),
    (dict(dy=P[0]), "dy overlaps"), (dict(dx=P[4], dy=P[4]), "overlap"), (dict(dq=P[7]), "overlap"),
    (dict(dg=P[0]), "overlap"), (dict(dt=P[4]), "overlap"), (dict(dq=P[6] + 1), "aligned"), (dict(xt=5), "dtype"),
])
def test_block_norm_backward_refuses(coli, kw, msg):
    st, err = _norm_backward(coli, **kw)
    assert st == coli.COLI_EINVAL and msg in err, err


def test_block_stack_refuses_null(coli):
    L = coli.lib
    assert L.coli_moe_block_stack_forward(None, None, 1, None, None, 1, None) == coli.COLI_EINVAL
    h = (ctypes.c_void_p * 1)()
    b = coli.Block()
    assert L.coli_moe_block_stack_forward(ctypes.cast(h, ctypes.c_void_p), b.address, 1, P[0], P[1], 1, None) == \
        coli.COLI_EINVAL  # a NULL layer
    assert L.coli_moe_block_stack_forward(ctypes.cast(h, ctypes.c_void_p), b.address, -1, P[0], P[1], 1, None) == \
        coli.COLI_EINVAL


def test_python_checks_tensors(coli):
    i32 = torch.int32
    ids = torch.zeros((2, 2), dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        coli.dispatch(ids, None, 4, None, None, None, None, None)
    with pytest.raises(TypeError):
        coli.dispatch(None, None, 4, None, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        coli.Block(pre_gain=torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        coli.block_norm(None, coli.Block(), torch.zeros(2, 8), n=torch.zeros(2, 8))
    with pytest.raises(TypeError):
        coli.block_norm(None, coli.Block(), None)
    with pytest.raises(TypeError):
        coli.Block(gate=[1.0])
    with pytest.raises(TypeError):
        coli.Block(gate=torch.ones(8, dtype=torch.float64))

"""The norms around a block with gates and scales, and their gradients, against
a plain form in 64 bits.

Tolerances, in steps U = 2^-24 of the magnitudes that block_ref adds up:
- a sum of squares over a row: a thread adds at most 16 columns and 10 tree
  levels follow (wider rows are summed in fp64), 26 steps and 2 of the mean and
  eps; the reciprocal root halves them and adds 2 ulp (4 U): 18 at most. 25 is used.
- x_out: the branch has the norm's 25 and 6 products, the fma one: 32.
- n: 25 and 2 products: 28, of x_out as stored.
- ds: the mean of s q dn has 26 steps and two scales (2 x 25), 8 products: 100.
- dy: a second mean over ds, the same again: 200.
- sums over tokens: 200 for each value and one step for each of a block's rows
  (T / 148 + 1 at most) and for the blocks (1184 / 16 + 16 = 90): 300 + T / 148.
Then one rounding to the output's type.
"""
import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402
from tests.test_gpu_dispatch import DT, SENTINEL, view  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def params(H, dev, gen, post=True, gains=True, gate=True, x_scale=0.75, y_scale=1.25, eps=1e-5):
    v = lambda: (1 + 0.3 * torch.randn(H, generator=gen)).to(dev)  # noqa: E731
    return dict(pre_gain=v() if gains else None, post_gain=v() if gains and post else None, gate=v() if gate else None,
                post_norm=post, x_scale=x_scale, y_scale=y_scale, eps=eps)


def both(coli, p):
    return None if p is None else coli.Block(**p)


# T, H, layout
SHAPES = [(1, 6144, "dense"), (1, 1, "dense"), (3, 7, "odd"), (5, 64, "apart"), (2, 8192, "dense"), (3, 8200, "dense"),
          (2, 16384, "apart"), (2, 16392, "dense"), (2, 1537, "dense"), (3, 8190, "odd"), (2, 8193, "dense"),
          (300, 136, "dense"), (1, 65536, "dense"), (700, 40, "odd"), (160, 516, "four"), (3, 2052, "four")]
TYPES = [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"), ("bf16", "f32", "f32")]


@pytest.mark.parametrize("xt,yt,nt", TYPES)
@pytest.mark.parametrize("T,H,layout", SHAPES)
def test_forward(gpu, coli, T, H, layout, xt, yt, nt):
    gen = torch.Generator().manual_seed(5)
    x, y = view((T, H), DT[xt], gpu, layout, gen), view((T, H), DT[yt], gpu, layout, gen)
    for post, gains, gate, token in ((True, True, True, True), (True, False, False, False), (False, True, True, False)):
        a, b = params(H, gpu, gen, post, gains, gate), params(H, gpu, gen, gains=gains, eps=1e-6)
        u = torch.rand(T, generator=gen).to(gpu) if token else None
        xo = view((T, H), DT[xt], gpu, layout, fill=SENTINEL)
        n = view((T, H), DT[nt], gpu, layout, fill=SENTINEL)
        coli.block_norm(both(coli, a), both(coli, b), x, y, xo, n, u)
        r = ref.Norm(a, b, u)
        want, mag = r.x_out(ref.d(x), ref.d(y))
        ref.assert_near(xo, want, mag, 32, "x_out", DT[xt])
        wn = r.n(ref.d(xo))
        ref.assert_near(n, wn, wn.abs(), 28, "n", DT[nt])
        # the ends of a stack: the norm alone, and the residual alone (the same bits)
        n2 = torch.empty((T, H), dtype=DT[nt], device=gpu)
        coli.block_norm(None, both(coli, b), xo, n=n2)
        assert torch.equal(n2, n)
        xo2 = torch.empty((T, H), dtype=DT[xt], device=gpu)
        coli.block_norm(both(coli, a), None, x, y, xo2, token_gate=u)
        assert torch.equal(xo2, xo)
    # in place: x_out over x, n over y where the types agree
    want_n = n.clone()
    coli.block_norm(both(coli, a), both(coli, b), x, y, x, y if nt == yt else n, u)
    assert torch.equal(x, xo) and torch.equal(y if nt == yt else n, want_n)


def run_backward(coli, a, b, s, y, dxo, dn, u, xt, yt, dx=None, dy=None):
    T, H = s.shape
    dev = s.device
    out = dict(dx=torch.full((T, H), SENTINEL, device=dev).to(DT[xt]) if dx is None else dx)
    f = lambda n: torch.full((n,), SENTINEL, device=dev)  # noqa: E731
    kw = {}
    if a is not None:
        out["dy"] = torch.full((T, H), SENTINEL, device=dev).to(DT[yt]) if dy is None else dy
        out.update(dgate=f(H), dtoken=f(T))
        kw.update(dy=out["dy"], dgate=out["dgate"], dtoken_gate=out["dtoken"], token_gate=u)
        if a["post_norm"]:
            out["dpost"] = f(H)
            kw["dpost_gain"] = out["dpost"]
    if b is not None:
        out["dpre"] = f(H)
        kw["dpre_gain"] = out["dpre"]
    work = torch.full((coli.block_norm_workspace(T, H),), 0xFF, dtype=torch.uint8, device=dev)
    coli.block_norm_backward(both(coli, a), both(coli, b), s, y, dxo, dn, dx=out["dx"], work=work, **kw)
    return out


def check_backward(out, want, T, xt, yt):
    coeff = dict(dx=100, dy=200, dtoken=200)
    for name, got in out.items():
        value, mag = want[name]
        ref.assert_near(got, value, mag, coeff.get(name, 300 + T / 148), name,
                        DT[xt] if name == "dx" else DT[yt] if name == "dy" else torch.float32)


@pytest.mark.parametrize("xt,yt,nt", TYPES)
@pytest.mark.parametrize("T,H,layout", SHAPES)
def test_backward(gpu, coli, T, H, layout, xt, yt, nt):
    gen = torch.Generator().manual_seed(6)
    s, y = view((T, H), DT[xt], gpu, layout, gen), view((T, H), DT[yt], gpu, layout, gen)
    dxo, dn = view((T, H), DT[xt], gpu, layout, gen), view((T, H), DT[nt], gpu, layout, gen)
    for post, gains, gate, token, with_dxo in ((True, True, True, True, True), (True, False, False, False, False),
                                               (False, True, True, False, True)):
        a, b = params(H, gpu, gen, post, gains, gate), params(H, gpu, gen, gains=gains, eps=1e-6)
        u = torch.rand(T, generator=gen).to(gpu) if token else None
        o = dxo if with_dxo else None
        out = run_backward(coli, a, b, s, y, o, dn, u, xt, yt)
        r = ref.Norm(a, b, u)
        check_backward(out, r.backward(ref.d(s), ref.d(y), ref.d(o), ref.d(dn)), T, xt, yt)
        again = run_backward(coli, a, b, s, y, o, dn, u, xt, yt)
        for k in out:
            assert torch.equal(out[k], again[k]), k  # fixed orders of summation
        first = run_backward(coli, None, b, s, None, o, dn, None, xt, yt)
        check_backward(first, ref.Norm(None, b).backward(ref.d(s), None, ref.d(o), ref.d(dn)), T, xt, yt)
        last = run_backward(coli, a, None, s, y, dxo, None, u, xt, yt)
        check_backward(last, ref.Norm(a, None, u).backward(ref.d(s), ref.d(y), ref.d(dxo), None), T, xt, yt)
    # in place: dx over x_out, dy over dn; dx over dx_out, dy over y
    want = run_backward(coli, a, b, s, y, dxo, dn, u, xt, yt)
    s2, dn2 = s.clone(), dn.clone()
    got = run_backward(coli, a, b, s2, y, dxo, dn2, u, xt, yt, dx=s2, dy=dn2 if nt == yt else None)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    got = run_backward(coli, a, b, s, y, dxo, dn, u, xt, yt, dx=dxo, dy=y)
    for k in want:
        assert torch.equal(want[k], got[k]), k


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(2048, 512), (1500, 1000), (449, 6144), (400, 8192), (700, 3001), (3000, 64)])
def test_many_rows(gpu, coli, T, H, t):
    """Blocks that take several rows each, with rings of one to four rows (8192 columns of fp32 leave room for
    one row in the gradient), both ways; a block without post norm and without gate has one sum a row."""
    gen = torch.Generator().manual_seed(7)
    s, y, dxo, dn = (torch.randn((T, H), generator=gen).to(gpu).to(DT[t]) for _ in range(4))
    u = torch.rand(T, generator=gen).to(gpu)
    for post in (True, False):
        a, b = params(H, gpu, gen, post=post, gate=post), params(H, gpu, gen)
        r = ref.Norm(a, b, u)
        out = run_backward(coli, a, b, s, y, dxo, dn, u, t, t)
        check_backward(out, r.backward(ref.d(s), ref.d(y), ref.d(dxo), ref.d(dn)), T, t, t)
        xo, n = torch.empty_like(s), torch.empty_like(s)
        coli.block_norm(both(coli, a), both(coli, b), s, y, xo, n, u)
        want, mag = r.x_out(ref.d(s), ref.d(y))
        ref.assert_near(xo, want, mag, 32, "x_out", DT[t])
        wn = r.n(ref.d(xo))
        ref.assert_near(n, wn, wn.abs(), 28, "n", DT[t])
        for prev, nxt, kw in ((None, b, dict(n=torch.empty_like(s))), (a, None, dict(x_out=torch.empty_like(s)))):
            first = dict(x=xo) if prev is None else dict(x=s, y=y, token_gate=u)
            coli.block_norm(both(coli, prev), both(coli, nxt), **first, **kw)
            assert torch.equal(kw.get("n", n), n) and torch.equal(kw.get("x_out", xo), xo)


def test_arrays_off_16_bytes(gpu, coli):
    """Gains and gate that start on 4 bytes (the columns are then read one by one)."""
    T, H = 5, 256
    gen = torch.Generator().manual_seed(13)
    x, y = torch.randn((T, H), generator=gen).to(gpu), torch.randn((T, H), generator=gen).to(gpu)
    a, b = params(H, gpu, gen), params(H, gpu, gen)
    off = lambda v: torch.cat([v.new_zeros(1), v])[1:]  # noqa: E731
    res = []
    for f in (lambda v: v, off):
        aa = {k: f(v) if torch.is_tensor(v) else v for k, v in a.items()}
        bb = {k: f(v) if torch.is_tensor(v) else v for k, v in b.items()}
        xo, n = torch.empty_like(x), torch.empty_like(x)
        coli.block_norm(both(coli, aa), both(coli, bb), x, y, xo, n)
        res.append((xo, n, ref.Norm(aa, bb)))
    for xo, n, r in res:
        want, mag = r.x_out(ref.d(x), ref.d(y))
        ref.assert_near(xo, want, mag, 32, "x_out")
        wn = r.n(ref.d(xo))
        ref.assert_near(n, wn, wn.abs(), 28, "n")


@pytest.mark.parametrize("H", [512, 1001, 20000])
@pytest.mark.parametrize("scale,eps", [(1e25, 1e-6), (1e-25, 0.0), (3e-20, 1e-30)])
def test_rows_beyond_the_range_of_fp32_squares(gpu, coli, H, scale, eps):
    """Squares that overflow or vanish in fp32: the sums are taken again in fp64."""
    gen = torch.Generator().manual_seed(8)
    x, y = torch.randn((3, H), generator=gen) * scale, torch.randn((3, H), generator=gen) * scale
    x[1] = torch.randn(H, generator=gen)  # an ordinary row between them
    a, b = dict(post_norm=True, eps=eps), dict(eps=eps)
    a2 = dict(post_norm=True, eps=eps, x_scale=1.0, y_scale=1.0)
    xo, n = torch.empty((3, H), device=gpu), torch.empty((3, H), device=gpu)
    coli.block_norm(both(coli, a), both(coli, b), x.to(gpu), y.to(gpu), xo, n)
    r = ref.Norm(a2, b)
    want, mag = r.x_out(ref.d(x), ref.d(y))
    ref.assert_near(xo, want, mag, 32, "x_out")
    wn = r.n(ref.d(xo))
    ref.assert_near(n, wn, wn.abs(), 28, "n")
    s = x.to(gpu)
    dn = torch.randn((3, H), generator=gen)
    out = dict(dx=torch.empty((3, H), device=gpu))
    coli.block_norm_backward(None, both(coli, b), s, dn=dn.to(gpu), dx=out["dx"])
    w = ref.Norm(None, b).backward(ref.d(x), None, None, ref.d(dn))
    ref.assert_near(out["dx"], w["dx"][0], w["dx"][1], 100, "dx")


def test_zero_and_non_finite_rows(gpu, coli):
    H = 640
    x = torch.randn((5, H), device=gpu)
    x[1] = 0.0
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    n = torch.empty_like(x)
    coli.block_norm(None, coli.Block(eps=1e-6), x, n=n)
    assert torch.equal(n[1], torch.zeros(H, device=gpu))
    assert torch.isnan(n[2, 7]) and (n[2, torch.arange(H, device=gpu) != 7] == 0).all()
    assert torch.isnan(n[3]).all()
    for t in (0, 4):
        want = ref.Norm(None, dict(eps=1e-6)).n(ref.d(x[t:t + 1]))
        ref.assert_near(n[t:t + 1], want, want.abs(), 28, "n")
    coli.block_norm(None, coli.Block(eps=0.0), x, n=n)
    assert torch.isnan(n[1]).all()  # 0 / 0, as the formula says


def test_no_tokens(gpu, coli):
    x = torch.empty((0, 64), device=gpu)
    coli.block_norm(coli.Block(), coli.Block(), x, x.clone(), x.clone(), x.clone())
    dq = torch.full((64,), SENTINEL, device=gpu)
    coli.block_norm_backward(coli.Block(), coli.Block(), x, x.clone(), None, x.clone(), dpre_gain=dq)
    assert (dq == 0).all()


@pytest.mark.parametrize("post,token", [(True, True), (False, False)])
def test_gradients_against_differences(gpu, coli, post, token):
    """<grad, direction> against a fourth-order difference of the 64-bit forward along that direction."""
    gen = torch.Generator().manual_seed(9)
    T, H = 6, 200
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, y, c1, c2 = r(T, H), r(T, H), r(T, H), r(T, H)
    a = dict(post_norm=post, post_gain=1 + 0.3 * r(H) if post else None, gate=r(H), x_scale=0.75, y_scale=1.25, eps=1e-5)
    b = dict(pre_gain=1 + 0.3 * r(H), eps=1e-5)
    u = torch.rand(T, generator=gen) if token else torch.ones(T)
    leaves = dict(x=x, y=y, gate=a["gate"], dpre=b["pre_gain"], token=u)
    if post:
        leaves["post"] = a["post_gain"]
    v = {k: torch.randn(t.shape, generator=gen, dtype=torch.float64) for k, t in leaves.items()}

    def loss(h):
        at = {k: t.double() + h * v[k] for k, t in leaves.items()}
        n = ref.Norm(dict(a, gate=at["gate"], post_gain=at.get("post")), dict(b, pre_gain=at["dpre"]), at["token"])
        s, _ = n.x_out(at["x"], at["y"])
        return (s * c1.double()).sum() + (n.n(s) * c2.double()).sum()

    h = 2.0 ** -9
    diff = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    dev = lambda p: {k: t.to(gpu) if torch.is_tensor(t) else t for k, t in p.items()}  # noqa: E731
    da, db = dev(a), dev(b)
    xo, n = torch.empty((T, H), device=gpu), torch.empty((T, H), device=gpu)
    coli.block_norm(both(coli, da), both(coli, db), x.to(gpu), y.to(gpu), xo, n, u.to(gpu))
    g = run_backward(coli, da, db, xo, y.to(gpu), c1.to(gpu), c2.to(gpu), u.to(gpu), "f32", "f32")
    names = dict(x="dx", y="dy", gate="dgate", dpre="dpre", token="dtoken", post="dpost")
    dot = sum((ref.d(g[names[k]]) * v[k]).sum() for k in leaves)
    want = ref.Norm(a, b, u).backward(*(ref.d(t) for t in (xo, y, c1, c2)))
    mag = sum((want[names[k]][1] * v[k].abs()).sum() for k in leaves)
    # 300 steps of each gradient's magnitude (x_out's own rounding, 32 steps, moves ds by as little), and
    # h^4 of the difference's remainder: h^4 = 2^-36
    assert abs(dot - diff) <= 340 * ref.U * mag + 2.0 ** -36 * mag

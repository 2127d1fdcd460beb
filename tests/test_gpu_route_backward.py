"""The router's gradient against a plain form in 64 bits.

Tolerances in steps U = 2^-24: dlogits has the sum over K (5 tree levels, K
products) and two products: 10 of w (|dw| + sum w |dw|). dx adds K products:
K + 12 of the magnitudes. drouter_w adds an expert's slots one after another
in parts (at most n steps for n slots, 12 for the factor, 40 for the parts).
"""
import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402
from tests.test_gpu_dispatch import DT, SENTINEL, make_ids, view  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def formula(wr, x, ids, w, dw):
    """(value, magnitude) of dlogits, dx, drouter_w, dbias in 64 bits."""
    T, K = ids.shape
    E, H = wr.shape
    wr, x, w, dw = (ref.d(t) for t in (wr, x, w, dw))
    on = (ids >= 0) & (ids < E) & (w != 0)
    w, dw = torch.where(on, w, torch.zeros_like(w)), torch.where(on, dw, torch.zeros_like(dw))
    dl = w * (dw - (w * dw).sum(1, keepdim=True))
    Dl = w.abs() * (dw.abs() + (w * dw).abs().sum(1, keepdim=True))
    z = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    dx, Dx, dwr, Dwr, db, Db = z(T, H), z(T, H), z(E, H), z(E, H), z(E), z(E)
    e = torch.where(on, ids, torch.zeros_like(ids)).long()  # a slot that is off has dl and Dl 0
    for k in range(K):
        d, D = dl[:, k:k + 1], Dl[:, k:k + 1]
        dx += d * wr[e[:, k]]
        Dx += D * wr[e[:, k]].abs()
        dwr.index_add_(0, e[:, k], d * x)
        Dwr.index_add_(0, e[:, k], D * x.abs())
        db.index_add_(0, e[:, k], dl[:, k])
        Db.index_add_(0, e[:, k], Dl[:, k])
    return dict(dlogits=(dl, Dl), dx=(dx, Dx), dwr=(dwr, Dwr), dbias=(db, Db))


def run(coli, wr, x, ids, w, dw, dev, layout="dense", only=("dx", "dwr", "dbias")):
    T, K = ids.shape
    E, H = wr.shape
    counts, offsets, pos, slot = (t.to(dev) for t in ref.plan(ids, E))
    out = dict(dlogits=torch.full((T, K), SENTINEL, device=dev))
    out["dx"] = view((T, H), x.dtype, dev, layout, fill=SENTINEL)
    out["dwr"], out["dbias"] = torch.full((E, H), SENTINEL, device=dev), torch.full((E,), SENTINEL, device=dev)
    n = coli.route_backward_workspace(T, K, E, H)
    work = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) if n else None
    keep = {k: (out[k] if k in only else None) for k in ("dx", "dwr", "dbias")}
    coli.route_backward(wr, x, ids.to(dev), w.to(dev), dw.to(dev), offsets, slot, out["dlogits"], keep["dx"],
                        keep["dwr"], keep["dbias"], work)
    return out


CASES = [(1, 1, 1, 1, "random", "dense"), (1, 8, 256, 6144, "random", "dense"), (64, 2, 16, 512, "random", "dense"),
         (33, 4, 7, 130, "holes", "odd"), (50, 32, 40, 264, "holes", "apart"), (300, 8, 64, 72, "holes", "dense"),
         (700, 3, 2, 100, "one", "dense"), (20, 4, 9, 64, "none", "dense"), (1200, 8, 256, 256, "random", "dense"),
         (5, 2, 1024, 2056, "random", "dense"),
         # chunks that fill a block's shared memory; several chunks to a split
         (690, 8, 256, 19072, "random", "dense"), (2048, 8, 256, 6144, "holes", "dense"), (400, 32, 1024, 6100, "holes", "dense"),
         (3000, 8, 32, 19000, "random", "dense"), (130, 1, 400, 128, "random", "four"), (2000, 16, 801, 256, "random", "dense")]


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,E,H,kind,layout", CASES)
def test_route_backward(gpu, coli, T, K, E, H, kind, layout, xt):
    gen = torch.Generator().manual_seed(10)
    ids = make_ids(T, K, E, kind)
    w = torch.softmax(torch.randn((T, K), generator=gen), 1)
    if kind == "holes":  # slots that expert top-p dropped: slot 0's id again, weight 0, no gradient
        w[::3, K - 1] = 0.0
        ids[::3, K - 1] = ids[::3, 0]
    dw = torch.randn((T, K), generator=gen)
    absent = (w == 0) | (ids < 0) | (ids >= E)
    dw[absent] = float("nan")
    x = view((T, H), DT[xt], gpu, layout, gen)
    wr = torch.randn((E, H), generator=gen).to(gpu)
    out = run(coli, wr, x, ids, w, dw, gpu, layout)
    want = formula(wr, x, ids, w, dw)
    n = int(ref.plan(ids, E)[0].max()) if T else 0
    ref.assert_near(out["dlogits"], *want["dlogits"], 10, "dlogits")
    ref.assert_near(out["dx"], *want["dx"], K + 12, "dx", DT[xt])
    ref.assert_near(out["dwr"], *want["dwr"], n + 52, "drouter_w")
    ref.assert_near(out["dbias"], *want["dbias"], n + 52, "dbias")
    assert (out["dlogits"].cpu()[absent] == 0).all()
    again = run(coli, wr, x, ids, w, dw, gpu, layout)
    for k in out:
        assert torch.equal(out[k], again[k]), k
    for only in ("dx", "dwr", "dbias"):
        one = run(coli, wr, x, ids, w, dw, gpu, layout, (only,))
        assert torch.equal(one[only], out[only]), only


def test_no_tokens(gpu, coli):
    out = run(coli, torch.randn((4, 64), device=gpu), torch.empty((0, 64), device=gpu),
              torch.zeros((0, 2), dtype=torch.int32), torch.zeros((0, 2)), torch.zeros((0, 2)), gpu)
    assert (out["dwr"] == 0).all() and (out["dbias"] == 0).all()


def test_gradient_against_differences(gpu, coli):
    """The weights of coli_moe_route's rule (softmax over the selected logits) along a direction of router and input."""
    gen = torch.Generator().manual_seed(11)
    T, K, E, H = 40, 4, 16, 96
    wr, x = torch.randn((E, H), generator=gen) / H ** 0.5, torch.randn((T, H), generator=gen)
    bias = torch.randn(E, generator=gen)
    dw = torch.randn((T, K), generator=gen)
    top, ids = torch.topk(x.double() @ wr.double().t() + bias, K, dim=1)
    w = torch.softmax(top, 1).float()
    vw, vx, vb = (torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in (wr, x, bias))

    def loss(h):  # the selection stays
        l = ((x + h * vx) @ (wr + h * vw).t() + bias + h * vb).gather(1, ids)
        return (torch.softmax(l, 1) * dw.double()).sum()

    h = 2.0 ** -9
    diff = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    out = run(coli, wr.to(gpu), x.to(gpu), ids.int(), w, dw, gpu)
    want = formula(wr, x, ids, w, dw)
    dot = (ref.d(out["dx"]) * vx).sum() + (ref.d(out["dwr"]) * vw).sum() + (ref.d(out["dbias"]) * vb).sum()
    mag = (want["dx"][1] * vx.abs()).sum() + (want["dwr"][1] * vw.abs()).sum() + (want["dbias"][1] * vb.abs()).sum()
    # the weights' own rounding (1 step, in products), T + 52 steps at most, h^4 of the difference
    assert abs(dot - diff) <= (T + 56) * ref.U * mag + 2.0 ** -30 * mag

"""Tokens sorted by expert and back, with their gradients, against plain forms
in 64 bits.

Tolerances. A sum of K products in fp32 (one fma each, after the base): every
step is off by at most U = 2^-24 of its value, so K + 1 steps by (K + 1) U of
the sum of magnitudes, then one rounding to the output's type. A dot of H
products over a block: a thread adds at most max(8, H / 32 + 8) of them, ten
tree levels follow, so H / 32 + 20 steps. A product w dy is one rounding in
fp32 and one to the rows' type. Moved rows are rounded once: equal to the bit.
"""
import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SENTINEL = -12345.0


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def make_ids(T, K, E, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":          # every slot names one expert: the same expert many times in a token
        return torch.full((T, K), E - 1, dtype=torch.int32)
    if kind == "none":         # nothing is held here
        return torch.full((T, K), -1, dtype=torch.int32)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    if kind == "holes":        # ids outside [0, E) in some slots, whole tokens without one
        bad = torch.tensor([-1, -7, E, E + 1000, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
        hit = torch.rand((T, K), generator=g) < 0.4
        ids = torch.where(hit, bad[torch.randint(0, len(bad), (T, K), generator=g)], ids)
        if T > 2:
            ids[1] = -1
    return ids


def run_plan(coli, ids, E, dev, x=None, rows=None):
    T, K = ids.shape
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(counts=torch.full((E,), -9, **i32), offsets=torch.full((E + 1,), -9, **i32),
               pos=torch.full((T, K), -9, **i32), slot=torch.full((T * K,), -9, **i32))
    n = coli.dispatch_workspace(T, K, E)
    work = torch.full((n,), 0xA5, dtype=torch.uint8, device=dev) if n else None
    coli.dispatch(ids.to(dev), x, E, out["counts"], out["offsets"], out["pos"], out["slot"], rows, work)
    return out


PLANS = [(1, 1, 1, "random"), (1, 8, 256, "random"), (3, 2, 16, "holes"), (5, 32, 32, "random"), (64, 8, 256, "random"),
         (127, 8, 256, "one"), (33, 4, 7, "none"), (256, 8, 256, "holes"), (257, 8, 256, "random"), (1000, 6, 64, "holes"),
         (2048, 8, 256, "random"), (2049, 8, 1024, "holes"), (5000, 8, 300, "one"), (70000, 3, 1024, "random"), (16385, 8, 64, "holes")]


@pytest.mark.parametrize("T,K,E,kind", PLANS)
def test_plan(gpu, coli, T, K, E, kind):
    ids = make_ids(T, K, E, kind)
    got = run_plan(coli, ids, E, gpu)
    want = ref.plan(ids, E)
    for name, w in zip(("counts", "offsets", "pos", "slot"), want):
        assert torch.equal(got[name].cpu(), w), name


def test_plan_of_no_tokens(gpu, coli):
    got = run_plan(coli, torch.zeros((0, 8), dtype=torch.int32), 5, gpu)
    assert got["counts"].tolist() == [0] * 5 and got["offsets"].tolist() == [0] * 6


def test_plan_matches_the_layers(gpu, coli):
    """The plan of a layer's routing equals the layer's own batch-union plan."""
    import synth
    H, E, K, T = 512, 16, 2, 96
    layer = coli.Layer(coli.make_config(H, 256, E, K, 0, T), synth.router(3, 0, E, H))
    x = torch.from_numpy(synth.x_f32(3, 0, T, H)).to(gpu)
    y = torch.empty_like(x)
    layer.forward(x, y)
    p = layer.plan(T)
    got = run_plan(coli, torch.from_numpy(p["ids"]), E, gpu)
    assert (got["counts"].cpu().numpy() == p["cnt"]).all() and (got["offsets"].cpu().numpy() == p["off"]).all()
    assert (got["pos"].cpu().numpy() == p["pos"]).all() and (got["slot"].cpu().numpy() // K == p["tok"]).all()
    layer.close()


def view(shape, dtype, dev, layout, gen=None, fill=None):
    """A matrix [rows][H]: dense, rows further apart (16-byte starts kept), or starting off 16 bytes."""
    r, H = shape
    if layout == "dense":
        m = torch.empty((r, H), dtype=dtype, device=dev)
    elif layout == "four":  # rows that start on 8 bytes (bf16) or 16 (fp32)
        m = torch.full((r, H + 8), SENTINEL, device=dev).to(dtype)[:, 4:4 + H]
    elif layout == "apart":
        m = torch.full((r, H + 24), SENTINEL, device=dev).to(dtype)[:, 8:8 + H]
    else:
        m = torch.full((r, H + 5), SENTINEL, device=dev).to(dtype)[:, 1:1 + H]
    m.copy_(torch.randn((r, H), generator=gen) if fill is None else torch.full((r, H), fill))
    return m


# T, K, E, H, kind, layout
ROWS = [(1, 8, 256, 6144, "random", "dense"), (1, 1, 1, 1, "random", "dense"), (3, 2, 4, 7, "holes", "odd"),
        (17, 8, 32, 256, "holes", "apart"), (64, 8, 256, 2056, "random", "dense"), (40, 32, 64, 136, "holes", "odd"),
        (300, 8, 256, 264, "holes", "dense"), (33, 4, 7, 64, "none", "dense"), (20, 9, 3, 1000, "one", "apart"),
        (2, 3, 5, 40000, "random", "dense"), (600, 4, 8, 1030, "holes", "dense"), (650, 3, 8, 516, "holes", "four"),
        (7, 8, 16, 1028, "random", "four")]


@pytest.mark.parametrize("xt,rt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,K,E,H,kind,layout", ROWS)
def test_dispatch_rows(gpu, coli, T, K, E, H, kind, layout, xt, rt):
    gen = torch.Generator().manual_seed(1)
    ids = make_ids(T, K, E, kind)
    x = view((T, H), DT[xt], gpu, layout, gen)
    rows = view((T * K + 2, H), DT[rt], gpu, layout, fill=SENTINEL)
    got = run_plan(coli, ids, E, gpu, x, rows)
    counts, offsets, pos, slot = ref.plan(ids, E)
    assert torch.equal(got["pos"].cpu(), pos) and torch.equal(got["slot"].cpu(), slot)
    want = torch.full((T * K + 2, H), SENTINEL).to(DT[rt])
    n = int(offsets[-1])
    if n:
        want[:n] = x.cpu()[(slot[:n] // K).long()].to(DT[rt])
    assert torch.equal(rows.cpu(), want)
    if layout != "dense":  # nothing beside the columns is written
        whole = rows._base
        assert (whole[:, -4:] == torch.tensor(SENTINEL).to(DT[rt]).to(gpu)).all()


@pytest.mark.parametrize("rt,yt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,K,E,H,kind,layout", ROWS)
def test_combine_and_dispatch_backward(gpu, coli, T, K, E, H, kind, layout, rt, yt):
    gen = torch.Generator().manual_seed(2)
    pos = ref.plan(make_ids(T, K, E, kind), E)[2]
    rows = view((T * K, H), DT[rt], gpu, layout, gen)
    unused = torch.ones(T * K, dtype=torch.bool)
    unused[pos[pos >= 0].long()] = False
    rows[unused.to(gpu)] = float("nan")  # rows that no slot names are never read
    w = torch.rand((T, K), generator=gen)
    w[pos < 0] = float("nan")           # nor is an empty slot's weight used
    base = view((T, H), DT[yt], gpu, layout, gen)
    for use_base in (False, True):
        y = view((T, H), DT[yt], gpu, layout, fill=SENTINEL)
        coli.combine(pos.to(gpu), w.to(gpu), rows, y, base if use_base else None)
        want, mag = ref.gather_sum(pos, w, rows.cpu(), base if use_base else None, H)
        ref.assert_near(y, want, mag, K + 1, "y", DT[yt])
        dx = view((T, H), DT[yt], gpu, layout, fill=SENTINEL)
        coli.dispatch_backward(pos.to(gpu), rows, dx, base if use_base else None)
        want, mag = ref.gather_sum(pos, None, rows.cpu(), base if use_base else None, H)
        ref.assert_near(dx, want, mag, K + 1, "dx", DT[yt])
    coli.combine(pos.to(gpu), w.to(gpu), rows, base, base)  # in place
    assert torch.equal(base, y)


@pytest.mark.parametrize("rt,yt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,K,E,H,kind,layout", ROWS)
def test_combine_backward(gpu, coli, T, K, E, H, kind, layout, rt, yt):
    gen = torch.Generator().manual_seed(3)
    pos = ref.plan(make_ids(T, K, E, kind), E)[2]
    rows = view((T * K, H), DT[rt], gpu, layout, gen)
    dy = view((T, H), DT[yt], gpu, layout, gen)
    w = torch.rand((T, K), generator=gen)
    drows = view((T * K, H), DT[rt], gpu, layout, fill=SENTINEL)
    dw = torch.full((T, K), SENTINEL, device=gpu)
    coli.combine_backward(pos.to(gpu), w.to(gpu), dy, rows, drows, dw)
    want = torch.full((T * K, H), SENTINEL).to(DT[rt]).double()
    dots, mags = torch.zeros((T, K), dtype=torch.float64), torch.zeros((T, K), dtype=torch.float64)
    mag = torch.zeros_like(want)
    dyd, rd = ref.d(dy), ref.d(rows)
    for t in range(T):
        for k in range(K):
            q = int(pos[t, k])
            if q >= 0:
                want[q] = float(w[t, k]) * dyd[t]
                mag[q] = want[q].abs()
                dots[t, k] = (dyd[t] * rd[q]).sum()
                mags[t, k] = (dyd[t] * rd[q]).abs().sum()
    ref.assert_near(drows, want, mag, 1, "drows", DT[rt])
    ref.assert_near(dw, dots, mags, H / 32 + 20, "dweights")
    # each output alone gives the same bits; the rows' gradient may take the rows' place
    dw2 = torch.empty_like(dw)
    coli.combine_backward(pos.to(gpu), w.to(gpu), dy, rows, None, dw2)
    assert torch.equal(dw2, dw)
    only = view((T * K, H), DT[rt], gpu, layout, fill=SENTINEL)
    coli.combine_backward(pos.to(gpu), w.to(gpu), dy, None, only)
    assert torch.equal(only, drows)
    coli.combine_backward(pos.to(gpu), w.to(gpu), dy, rows, rows, dw2)
    held = torch.zeros(T * K, dtype=torch.bool)
    held[pos[pos >= 0].long()] = True
    assert torch.equal(rows[held.to(gpu)], drows[held.to(gpu)]) and torch.equal(dw2, dw)


def test_positions_outside_the_rows_add_nothing(gpu, coli):
    pos = torch.tensor([[0, 5, 99], [-3, 2 ** 31 - 1, 2]], dtype=torch.int32, device=gpu)
    rows = torch.randn((3, 64), device=gpu)
    y = torch.empty((2, 64), device=gpu)
    w = torch.full((2, 3), 2.0, device=gpu)
    coli.combine(pos, w, rows, y)
    assert torch.equal(y, 2 * rows[[0, 2]])
    dw = torch.empty((2, 3), device=gpu)
    drows = torch.full((3, 64), 7.0, device=gpu)
    coli.combine_backward(pos, w, y, rows, drows, dw)
    assert dw[0, 1:].tolist() == [0, 0] and dw[1, :2].tolist() == [0, 0]
    assert torch.equal(drows[1], torch.full((64,), 7.0, device=gpu)) and torch.equal(drows[0], 2 * y[0])


def test_infinite_and_nan_rows_stay_in_their_tokens(gpu, coli):
    ids = torch.tensor([[0, 1], [1, 0], [0, 1]], dtype=torch.int32)
    pos = ref.plan(ids, 2)[2].to(gpu)
    rows = torch.ones((6, 128), device=gpu)
    rows[pos[1, 0]] = float("inf")
    rows[pos[1, 1]] = float("nan")
    y = torch.empty((3, 128), device=gpu)
    coli.combine(pos, torch.full((3, 2), 0.5, device=gpu), rows, y)
    assert torch.equal(y[0], torch.ones(128, device=gpu)) and torch.equal(y[2], torch.ones(128, device=gpu))
    assert torch.isnan(y[1]).all()


@pytest.mark.parametrize("T,K,H", [(2, 8, 6144), (700, 8, 6144)])
def test_gradients_against_differences(gpu, coli, T, K, H):
    """<grad, direction> of the combine against the change of its 64-bit form along that direction.
    The form is linear in the rows and in the weights, so the difference is exact but for rounding."""
    gen = torch.Generator().manual_seed(4)
    E = 32
    pos = ref.plan(make_ids(T, K, E, "random"), E)[2]
    rows, w, dy = torch.randn((T * K, H), generator=gen), torch.rand((T, K), generator=gen), torch.randn((T, H), generator=gen)
    drows, dw = torch.empty((T * K, H), device=gpu), torch.empty((T, K), device=gpu)
    coli.combine_backward(pos.to(gpu), w.to(gpu), dy.to(gpu), rows.to(gpu), drows, dw)
    vr, vw = torch.randn((T * K, H), generator=gen).double(), torch.randn((T, K), generator=gen).double()

    def loss(r, ww):
        return ((r[pos.long()] * ww.unsqueeze(-1)).sum(1) * dy.double()).sum()

    h = 2.0 ** -10
    for grad, direction, up, dn in ((drows, vr, (rows + h * vr, w.double()), (rows - h * vr, w.double())),
                                    (dw, vw, (rows.double(), w + h * vw), (rows.double(), w - h * vw))):
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        dot, mag = (ref.d(grad) * direction).sum(), (ref.d(grad) * direction).abs().sum()
        # rounding of each gradient value (at most H / 32 + 20 steps of its magnitude; dots of random signs
        # have magnitudes sqrt(H) above their values) and of the difference in 64 bits
        assert abs(dot - diff) <= (H / 32 + 20) * ref.U * mag * H ** 0.5 + 1e-9 * mag


def test_offsets_beyond_32_bits(gpu, coli):
    """2^31 elements and more of rows: 43700 tokens of 8 slots, 6144 wide, in bf16."""
    T, K, E, H = 43700, 8, 256, 6144
    ids = make_ids(T, K, E, "random")
    x = torch.empty((T, H), dtype=torch.bfloat16, device=gpu)
    x.copy_((torch.arange(T, device=gpu) % 251).unsqueeze(1).expand(T, H))
    x[:, 1] = (torch.arange(T, device=gpu) // 251).to(torch.bfloat16)
    rows = torch.empty((T * K, H), dtype=torch.bfloat16, device=gpu)
    got = run_plan(coli, ids, E, gpu, x, rows)
    tok = (got["slot"] // K).long()
    at = torch.tensor([0, 1, 2, H - 1], device=gpu)
    assert torch.equal(rows[:, at], x[tok][:, at])
    w = torch.zeros((T, K), device=gpu)
    w[:, 3] = 1.0
    y = torch.empty_like(x)
    coli.combine(got["pos"], w, rows, y)
    assert torch.equal(y, x)
    dw = torch.empty((T, K), device=gpu)
    dy = torch.zeros_like(x)
    dy[:, H - 1] = 1.0
    coli.combine_backward(got["pos"], w, dy, rows, None, dw)
    assert torch.equal(dw, x[:, H - 1:].float().expand(T, K))
    del rows, y, dy
    torch.cuda.empty_cache()

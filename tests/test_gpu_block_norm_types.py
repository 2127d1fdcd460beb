"""The norms over all combinations of the three types, with one matrix alone
off 16 bytes, and rows beyond the range of fp32 squares with a block before
them. Tolerances as in test_gpu_block_norm.

Calls that take the same number of columns at a time give the same bits with
and without the other block; which that is goes by the types and starts of all
matrices of the call, so between other calls only the tolerance holds."""
import itertools

import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402
from tests.test_gpu_block_norm import both, check_backward, params, run_backward  # noqa: E402
from tests.test_gpu_dispatch import DT, SENTINEL, view  # noqa: E402

pytestmark = pytest.mark.gpu

TRIPLES = list(itertools.product(("f32", "bf16"), repeat=3))


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def forward(coli, a, b, x, y, u, xt, nt):
    xo = torch.full(tuple(x.shape), SENTINEL, device=x.device).to(DT[xt])
    n = torch.full(tuple(x.shape), SENTINEL, device=x.device).to(DT[nt])
    coli.block_norm(both(coli, a), both(coli, b), x, y, xo, n, u)
    r = ref.Norm(a, b, u)
    want, mag = r.x_out(ref.d(x), ref.d(y))
    ref.assert_near(xo, want, mag, 32, "x_out", DT[xt])
    wn = r.n(ref.d(xo))
    ref.assert_near(n, wn, wn.abs(), 28, "n", DT[nt])
    return xo, n


@pytest.mark.parametrize("xt,yt,nt", TRIPLES)
@pytest.mark.parametrize("T,H", [(1, 6144), (3, 64), (200, 264), (350, 1028), (160, 77), (2, 8192), (2, 9000)])
def test_types(gpu, coli, T, H, xt, yt, nt):
    gen = torch.Generator().manual_seed(31)
    x, y = view((T, H), DT[xt], gpu, "dense", gen), view((T, H), DT[yt], gpu, "dense", gen)
    a, b = params(H, gpu, gen), params(H, gpu, gen, eps=1e-6)
    u = torch.rand(T, generator=gen).to(gpu)
    xo, _ = forward(coli, a, b, x, y, u, xt, nt)
    # the ends of a stack, within the tolerance
    n2 = torch.empty((T, H), dtype=DT[nt], device=gpu)
    coli.block_norm(None, both(coli, b), xo, n=n2)
    wn = ref.Norm(None, b).n(ref.d(xo))
    ref.assert_near(n2, wn, wn.abs(), 28, "n alone", DT[nt])
    xo2 = torch.empty((T, H), dtype=DT[xt], device=gpu)
    coli.block_norm(both(coli, a), None, x, y, xo2, token_gate=u)
    want, mag = ref.Norm(a, b, u).x_out(ref.d(x), ref.d(y))
    ref.assert_near(xo2, want, mag, 32, "x_out alone", DT[xt])
    s, dxo, dn = (view((T, H), DT[t], gpu, "dense", gen) for t in (xt, xt, nt))
    out = run_backward(coli, a, b, s, y, dxo, dn, u, xt, yt)
    check_backward(out, ref.Norm(a, b, u).backward(ref.d(s), ref.d(y), ref.d(dxo), ref.d(dn)), T, xt, yt)


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(2, 512), (300, 264)])
def test_one_matrix_off_16_bytes(gpu, coli, T, H, t, which):
    gen = torch.Generator().manual_seed(32)
    m = [view((T, H), DT[t], gpu, "odd" if i == which else "dense", gen) for i in range(4)]
    s, y, dxo, dn = m
    a, b = params(H, gpu, gen), params(H, gpu, gen)
    u = torch.rand(T, generator=gen).to(gpu)
    out = run_backward(coli, a, b, s, y, dxo, dn, u, t, t)
    check_backward(out, ref.Norm(a, b, u).backward(*(ref.d(v) for v in m)), T, t, t)
    if which < 2:
        forward(coli, a, b, s, y, u, t, t)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("H", [512, 1001, 6001, 20000])
@pytest.mark.parametrize("sx,sy", [(1e25, 1.0), (1.0, 1e25), (1e25, 1e25), (1e-25, 1.0), (1.0, 1e-25), (1e-16, 1e-16)])
def test_gradient_of_rows_beyond_the_range_of_fp32_squares(gpu, coli, H, sx, sy, post):
    """Squares of x_out, of y or of both that overflow or (eps 0) vanish in fp32, with all gradients."""
    gen = torch.Generator().manual_seed(33)
    s, y, dxo, dn = (torch.randn((4, H), generator=gen) for _ in range(4))
    s[::2] *= sx  # ordinary rows between them
    y[::2] *= sy
    s, y, dxo, dn = (v.to(gpu) for v in (s, y, dxo, dn))
    eps = 0.0 if min(sx, sy) < 1 else 1e-6
    a, b = params(H, gpu, gen, post=post, eps=eps), params(H, gpu, gen, eps=eps)
    u = torch.rand(4, generator=gen).to(gpu)
    out = run_backward(coli, a, b, s, y, dxo, dn, u, "f32", "f32")
    check_backward(out, ref.Norm(a, b, u).backward(*(ref.d(v) for v in (s, y, dxo, dn))), 4, "f32", "f32")

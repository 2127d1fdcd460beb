"""Rows too wide for registers: their sums of squares hold as many bits as the
narrow rows' (the tolerances of test_gpu_block_norm)."""
import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


@pytest.mark.parametrize("run", [1, 512, 1024])
@pytest.mark.parametrize("H", [8193, 16384, 65536])
def test_small_squares_behind_large_ones(gpu, coli, H, run):
    """Runs of columns of 1 at the row's start, then columns whose squares are just under half a step of 1: a
    sum that adds them to the large ones one at a time in fp32 loses every one of them."""
    x = torch.full((2, H), 0.99 * 2.0 ** -12)
    x[:, :run] = 1.0
    x[1] = x[1].flip(0)
    n, xo = torch.empty((2, H), device=gpu), torch.empty((2, H), device=gpu)
    xd = x.to(gpu)
    b, a = dict(eps=1e-6), dict(post_norm=True, x_scale=0.0, eps=1e-6)
    coli.block_norm(None, coli.Block(**b), xd, n=n)
    want = ref.Norm(None, b).n(ref.d(x))
    ref.assert_near(n, want, want.abs(), 28, "n")
    coli.block_norm(coli.Block(**a), coli.Block(**b), xd, xd.clone(), xo, n)
    r = ref.Norm(a, b)
    want, mag = r.x_out(ref.d(x), ref.d(x))
    ref.assert_near(xo, want, mag, 32, "x_out")
    want = r.n(ref.d(xo))
    ref.assert_near(n, want, want.abs(), 28, "n of x_out")

"""The norms' gradient where an input does not enter it: without `next` no
output depends on x_out, and without a post norm dy does not depend on y, so
infinities and NaN there must not show, at any width.

Tolerances as in test_gpu_block_norm."""
import pytest

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402
from tests.test_gpu_block_norm import both, check_backward, params, run_backward  # noqa: E402
from tests.test_gpu_dispatch import DT, view  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def poisoned(t):
    """Every second row holds an infinity or NaN in some columns, one row nothing else."""
    t = t.clone()
    H = t.shape[1]
    for row in range(0, t.shape[0], 2):
        t[row, row % H] = float("inf") if row % 4 else float("nan")
        t[row, H - 1] = -float("inf")
    t[t.shape[0] - 1] = float("nan")
    return t


# widths: vector accesses and a ring; single columns, loaded ahead (1001) or not (6001); too wide for registers
WIDTHS = [64, 516, 1001, 6001, 8192, 8193, 16384]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("T", [3, 400])
@pytest.mark.parametrize("H", WIDTHS)
def test_last_block_does_not_depend_on_x_out(gpu, coli, H, T, post, t):
    gen = torch.Generator().manual_seed(21)
    s, y, dxo = (view((T, H), DT[t], gpu, "dense", gen) for _ in range(3))
    a = params(H, gpu, gen, post=post)
    u = torch.rand(T, generator=gen).to(gpu)
    want = run_backward(coli, a, None, s, y, dxo, None, u, t, t)
    got = run_backward(coli, a, None, poisoned(s), y, dxo, None, u, t, t)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    if T == 3:
        check_backward(got, ref.Norm(a, None, u).backward(ref.d(s), ref.d(y), ref.d(dxo), None), T, t, t)
    nothing = run_backward(coli, a, None, poisoned(s), y, None, None, u, t, t)  # no gradient comes in: none goes out
    assert all((v == 0).all() for v in nothing.values())


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("with_next", [True, False])
@pytest.mark.parametrize("T", [3, 400])
@pytest.mark.parametrize("H", WIDTHS)
def test_dy_without_post_norm_does_not_depend_on_y(gpu, coli, H, T, with_next, t):
    gen = torch.Generator().manual_seed(22)
    s, y, dxo, dn = (view((T, H), DT[t], gpu, "dense", gen) for _ in range(4))
    a, b = params(H, gpu, gen, post=False), params(H, gpu, gen) if with_next else None
    u = torch.rand(T, generator=gen).to(gpu)
    n = dn if with_next else None
    got = run_backward(coli, a, b, s, poisoned(y), dxo, n, u, t, t)
    r = ref.Norm(a, b, u)
    want = r.backward(ref.d(s), torch.zeros((T, H), dtype=ref.D), ref.d(dxo), None if n is None else ref.d(n))
    same = {k: got[k] for k in ("dx", "dy", "dpre") if k in got}
    check_backward(same, want, T, t, t)
    bad = torch.zeros(T, dtype=torch.bool, device=gpu)
    bad[::2] = True
    bad[T - 1] = True
    # the sums over the columns of y do hold what y holds
    assert not torch.isfinite(got["dtoken"][bad]).any() and torch.isfinite(got["dtoken"][~bad]).all()

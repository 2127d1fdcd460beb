"""Workspaces of the operators around the layer: what their size functions say
for a number of tokens is enough for fewer tokens too (on the CPU: a call with
enough scratch memory fails for want of a device, not of memory; the pointers
are never read)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests.test_block_ops_abi import P, _argtypes, _dispatch, _route_backward, coli  # noqa: E402, F401


@pytest.mark.parametrize("K,E", [(1, 1), (8, 64), (3, 1000), (32, 256)])
def test_dispatch_workspace_holds_fewer_tokens(coli, K, E):  # noqa: F811
    top = min(1 << 20, (1 << 24) // K)
    sizes = {T: coli.dispatch_workspace(T, K, E) for T in range(0, 70000)}
    sizes.update({T: coli.dispatch_workspace(T, K, E) for T in range(70000, top + 1, 997)})
    last = 0
    for T in sorted(sizes):
        assert sizes[T] >= last, T
        last = sizes[T]
    if torch.cuda.is_available():  # the rest would launch
        return
    for T in (1, 16384 // K + 1, 131072 // K, 131072 // K + 1, 50000):
        most = max(T, 131072 // K + 7)
        st, err = _dispatch(coli, T=T, K=K, E=E, x=None, rows=None, work=P[7], nw=coli.dispatch_workspace(most, K, E))
        assert st != coli.COLI_OK and "work" not in err, (T, err)


@pytest.mark.parametrize("E,H,K", [(16, 128, 2), (1, 1, 1), (256, 6144, 8), (1024, 100, 32), (64, 1000, 3)])
def test_route_backward_workspace_holds_fewer_tokens(coli, E, H, K):  # noqa: F811
    top = min(1 << 20, (1 << 24) // K)
    steps = list(range(0, 30000)) + list(range(30000, top + 1, 991))
    last = 0
    for T in steps:
        n = coli.route_backward_workspace(T, K, E, H)
        assert n >= last, T
        last = n
    if torch.cuda.is_available():
        return
    for T in (1, 127, 128, 129, 18944, 20000, 29999):
        st, err = _route_backward(coli, E=E, H=H, xs=H, dxs=H, K=K, T=T, nw=coli.route_backward_workspace(T + 1, K, E, H))
        assert st != coli.COLI_OK and "work" not in err, (T, err)

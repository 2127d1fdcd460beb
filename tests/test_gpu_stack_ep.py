"""Expert-parallel layers in the stacks. Such a layer's forward writes this
rank's part of the output, which the caller sums over the ranks; a stack would
go on with the part alone, so the stacks refuse it where more follows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import synth  # noqa: E402

pytestmark = pytest.mark.gpu

H, I, E, K, T = 512, 256, 16, 2, 4


@pytest.fixture(scope="module")
def coli():
    import int4_expert_ffn_router_b200 as m
    return m


def layer(coli, l, ep=None):
    experts = [synth.expert(5, l, e, H, I) for e in range(E)]
    return coli.Layer(coli.make_config(H, I, E, K, 0, T), synth.router(5, l, E, H), None,
                      np.concatenate([e[0] for e in experts]), np.concatenate([e[1] for e in experts]), ep=ep)


@pytest.mark.parametrize("where", [0, 1])
@pytest.mark.parametrize("rank", [0, 1])
@pytest.mark.parametrize("post", [True, False])
def test_block_stack_refuses_a_part_of_the_experts(gpu, coli, where, rank, post):
    layers = [layer(coli, l, (rank, 2) if l == where else None) for l in range(2)]
    x = torch.from_numpy(synth.x_f32(5, 0, T, H)).to(gpu)
    before, work = x.clone(), torch.full_like(x, 3.0)
    with pytest.raises(coli.ColiError, match="experts"):
        coli.block_stack_forward(layers, [coli.Block(post_norm=post) for _ in layers], x, work)
    torch.cuda.synchronize()
    assert torch.equal(x, before) and (work == 3.0).all()  # refused before any launch
    for l in layers:
        l.close()


def test_block_stack_of_one_rank_that_holds_all(gpu, coli):
    """One rank of one holds every expert: the same layer as without ranks."""
    full, one = layer(coli, 0), layer(coli, 0, (0, 1))
    x = torch.from_numpy(synth.x_f32(5, 0, T, H)).to(gpu)
    a, b, work = x.clone(), x.clone(), torch.empty_like(x)
    coli.block_stack_forward([full], [coli.Block(post_norm=True)], a, work)
    coli.block_stack_forward([one], [coli.Block(post_norm=True)], b, work)
    assert torch.equal(a, b) and not torch.equal(a, x)
    full.close()
    one.close()


@pytest.mark.parametrize("rank", [0, 1])
def test_stack_refuses_a_part_of_the_experts_before_another_layer(gpu, coli, rank):
    layers = [layer(coli, 0, (rank, 2)), layer(coli, 1)]
    x = torch.from_numpy(synth.x_f32(5, 0, T, H)).to(gpu)
    before = x.clone()
    with pytest.raises(coli.ColiError, match="experts"):
        coli.stack_forward(layers, x)
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    for l in layers:
        l.close()


def test_stack_that_ends_in_a_part_of_the_experts(gpu, coli):
    """The last layer adds its part to x: over the ranks, the parts sum to the whole layer's output (1e-5 of the
    largest value, as in test_gpu_ep: the order of the fp32 additions)."""
    first, full = layer(coli, 0), layer(coli, 1)
    ranks = [layer(coli, 1, (r, 2)) for r in range(2)]
    x = torch.from_numpy(synth.x_f32(5, 0, T, H)).to(gpu)
    runs = []
    for last in (full, *ranks):
        runs.append(x.clone())
        coli.stack_forward([first, last], runs[-1])
    mid = x.clone()
    coli.stack_forward([first], mid)
    whole, a, b, mid = (r.double() for r in (*runs, mid))
    assert float((a + b - mid - whole).abs().max()) <= 1e-5 * float(whole.abs().max())
    for l in (first, full, *ranks):
        l.close()

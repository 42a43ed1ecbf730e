"""The linear attention blocks of examples/recurrent_layers.py: the operators together, as they are used.

Tolerances, relative 2-norm. A block rounds to bf16 six times in a row (the norm, the projection, the
attention with one or two roundings inside, the head norm, the projection, the stream and its norm), each
1.7e-3 of the norm: two blocks 1.7e-3 sqrt(14) = 6.4e-3, with room for what the norms amplify 1.5e-2;
gradients pass the chain twice: 3e-2. Some gradients keep less: the head norm's divides by |o|, and a row's
first step has o = (q . k) v, of which the rounding of q and k to bf16 leaves 2^-9 |q| |k| out, whatever q . k is;
steps with a small q . k are those with the largest gradients. So the definition is also evaluated in float64
with nothing but the intermediate tensors rounded to bf16 where a layer in bf16 holds them, and where that
alone moves a gradient by more, twice what it moves is allowed (the second time for the gradients' own
roundings on the way back). A prompt continued token by token differs from a whole one by the
roundings inside the attention of both blocks and what they move: 1e-2."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_reference as K  # noqa: E402
import layer_reference as R  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    import recurrent_layers
    return recurrent_layers


def _x(*shape, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("T", [70, 300])
def test_tokens_continue_a_prompt(ex, T):
    layer = ex.LinearAttentionBlocks()
    x = _x(3, T, 512)
    whole, _ = layer.forward(x)
    assert R.rel(ex.continued(layer, x, 5), whole) <= 1e-2


def _blocks64(layer, lens, x, w_first, held=lambda t: t, **w):
    n = held(R.norm(x, 1, w_first, None, None, "none", 1e-5, False))
    for i in range(len(layer.blocks)):
        q, k, v, z = layer._split(held(n @ w[f"W_in{i}"].t()))
        o, _ = K.linattn(q, k, v, layer.g.double(), None, lens)
        m = held(R.norm(held(o).flatten(-2), layer.Hv, w[f"w_head{i}"], None, z, "silu", 1e-5, False))
        h = held(m @ w[f"W_out{i}"].t())
        x, n = (held(t) for t in K.resnorm(x, h, None, w[f"scale{i}"], w[f"w_post{i}"], w[f"w_pre{i}"], True, True, "none", 1e-5))
    return n


def _in_bf16(t):
    return t + (t.to(torch.bfloat16).double() - t).detach()


@pytest.mark.parametrize("ragged", [False, True])
def test_blocks_train(ex, ragged):
    """The blocks' output and gradients against float64."""
    layer = ex.LinearAttentionBlocks(width=128)
    T = 150
    x, dy = _x(3, T, 128, seed=1), _x(3, T, 128, seed=2)
    lens = torch.tensor([T, 0, 77], dtype=torch.int32, device="cuda") if ragged else None
    y, saved = layer.forward(x, train=True, lens=lens)
    got = layer.backward(saved, dy)
    leaves = {"x": x.double(), "w_first": layer.w_first.double()}
    mine = {"x": got["dx"], "w_first": got["dw_first"]}
    for i, b in enumerate(layer.blocks):
        leaves.update({n + str(i): t.double() for n, t in b.items()})
        mine.update({n + str(i): got["blocks"][i][n] for n in b})
    (y64,), g = R.with_grads(lambda **k: _blocks64(layer, lens, **k), leaves, (dy.double(),))
    _, rounded = R.with_grads(lambda **k: _blocks64(layer, lens, held=_in_bf16, **k), leaves, (dy.double(),))
    assert R.rel(y, y64) <= 1.5e-2
    for n, r in g.items():
        assert R.rel(mine[n], r) <= max(3e-2, 2 * R.rel(rounded[n], r)), (n, R.rel(mine[n], r), R.rel(rounded[n], r))


def test_a_training_step_replayed_from_a_graph(ex):
    """Forward and backward captured once and replayed on other inputs: the bits of the eager step."""
    layer = ex.LinearAttentionBlocks(width=256)
    flat = lambda y, g: [y, g["dx"], g["dw_first"]] + [t for b in g["blocks"] for t in b.values()]  # noqa: E731

    def step(x, dy):
        y, saved = layer.forward(x, train=True)
        return flat(y, layer.backward(saved, dy))

    live, dy = _x(2, 200, 256, seed=3), _x(2, 200, 256, seed=4)
    other = _x(2, 200, 256, seed=5)
    want = step(other, dy)
    step(live, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(live, dy)
    live.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))

"""Layers whose weights come out of a gather that goes on: what is gathered next into
the same memory changes nothing in a layer until it is loaded."""
import numpy as np
import pytest
import torch

from test_gpu_moe import choices
from test_gpu_moe_layer import bf16, mlp, moe, mx, setting  # noqa: F401  (mx, mlp, moe: fixtures)

pytestmark = pytest.mark.gpu


def steps(moe, mlp):  # noqa: F811
    """For either layer: (a maker of layers, its weights as views of one flat parameter, that
    parameter, a forward pass, a backward pass of what that kept, to lists of tensors)."""
    rng = np.random.default_rng(4)
    T, k, E, K, F = 50, 2, 3, 64, 96
    gate_up, down, norm, x, res, ids, w = setting(rng, T, k, E, K, F)
    dy = bf16(rng, T, K, scale=1e-3)
    flat = torch.cat((gate_up.flatten(), down.flatten(), norm))
    dense = torch.cat((gate_up[0].flatten(), down[0].flatten(), norm))
    n = 2 * F * K

    def expert_back(layer, kept):
        dx, dw = layer.backward(dy, kept)
        return [dx, dw, layer.d_gate_up, layer.d_down, layer.d_norm]

    def dense_back(layer, kept):
        return [layer.backward(dy, kept), layer.d_gate_up, layer.d_down, layer.d_norm]

    return {"experts": (moe.ExpertMLP, moe.gathered(flat, E, K, F), flat,
                        lambda layer: layer.forward(x, ids, w, residual=res), expert_back),
            "dense": (lambda a, b, c: mlp.GatedMLP(a, b, norm=c), (dense[:n].view(2 * F, K), dense[n:n + n // 2].view(K, F), dense[n + n // 2:]),
                      dense, lambda layer: layer.forward(x, residual=res), dense_back)}


@pytest.mark.parametrize("which", ["experts", "dense"])
def test_the_next_gather_changes_nothing(moe, mlp, which):  # noqa: F811
    make, views, flat, forward, backward = steps(moe, mlp)[which]
    apart = make(*(v.clone() for v in views))
    y, kept = forward(apart)
    want = [y] + backward(apart, kept)
    layer = make(*views)
    flat.mul_(-2)
    y, kept = forward(layer)
    flat.mul_(-2)
    got = [y] + backward(layer, kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_layers_of_one_codec(moe):  # noqa: F811
    """Two layers gathered one after the other by the same codec, into the same memory."""
    from lossless_bf16_exponent_codec_gb300.codec import Codec
    E, K, F, W = 4, 96, 64, 4
    n = 3 * E * F * K + K
    rng = np.random.default_rng(6)
    x, ids = bf16(rng, 33, K), torch.from_numpy(choices(rng, 33, 2, E)).cuda()
    w = torch.full((33, 2), 0.5, device="cuda")
    codec, made, alone = Codec(n, W), [], []
    for gain in (1.0, 3.0):
        shards = bf16(rng, n, scale=0.02)
        shards[-K:] = gain
        codec.stats(shards)
        codec.encode_code3(shards)
        made.append(moe.ExpertMLP(*moe.gathered(codec.gather_decode(*codec.exchange()), E, K, F)))
        alone.append(moe.ExpertMLP(*moe.gathered(shards, E, K, F)))
    assert codec.status_word() == 0
    for a, b in zip(made, alone):
        assert torch.equal(a.forward(x, ids, w)[0], b.forward(x, ids, w)[0])


@pytest.mark.parametrize("which", ["experts", "dense"])
def test_a_captured_pass_runs_with_what_was_loaded_last(moe, mlp, which):  # noqa: F811
    make, views, flat, forward, backward = steps(moe, mlp)[which]
    layer = make(*views)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        backward(layer, forward(layer)[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, kept = forward(layer)
        outs = [y] + backward(layer, kept)
    sums = [layer.d_gate_up, layer.d_down, layer.d_norm]
    for factor in (0.5, -3.0):
        flat.mul_(factor)
        layer.load(*views)
        other = [torch.full_like(t, 255) for s in (layer.w1, layer.w1t, layer.w2, layer.w2t) for t in (s.codes, s.scales)]
        for s in sums:
            s.zero_()
        graph.replay()
        got = [t.clone() for t in outs]
        fresh = make(*views)
        y, kept = forward(fresh)
        want = [y] + backward(fresh, kept)
        assert len(other) == 8 and all(torch.equal(a, b) for a, b in zip(got, want))
    assert layer.status_word() == 0

"""What the layers hold of the weights that they are given, without a GPU: the
quantisation, which needs one, is left out."""
import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32
E, F, K = 3, 64, 96


@pytest.fixture(scope="module")
def layers():
    from lossless_bf16_exponent_codec_gb300 import build
    build.build()
    from lossless_bf16_exponent_codec_gb300 import mlp, moe, mx
    return mlp, moe, mx


@pytest.fixture(params=["dense", "experts"])
def made(request, layers, monkeypatch):
    """(a maker of layers from (gate_up, down, norm), the gathered parameter's views, its values)"""
    mlp, moe, mx = layers
    monkeypatch.setattr(mx, "quantize", lambda *a, **kw: None)
    if request.param == "dense":
        flat = torch.randn(3 * F * K + K).to(BF16)
        views = (flat[:2 * F * K].view(2 * F, K), flat[2 * F * K:3 * F * K].view(K, F), flat[3 * F * K:])
        return (lambda a, b, n=None: mlp.GatedMLP(a, b, norm=n)), views, flat
    flat = torch.randn(3 * E * F * K + K).to(BF16)
    return moe.ExpertMLP, moe.gathered(flat, E, K, F), flat


def test_the_norm_is_a_copy(made):
    """A gather into the same memory changes nothing in a layer until it is loaded."""
    make, (gate_up, down, norm), flat = made
    layer = make(gate_up, down, norm)
    first, mine = norm.clone(), layer.norm
    flat.fill_(7.0)
    assert torch.equal(layer.norm, first)
    layer.load(gate_up, down, norm)
    assert layer.norm is mine and torch.equal(mine, norm)        # the same memory: captured graphs read it
    assert torch.equal(mine, torch.full((K,), 7.0, dtype=BF16))


def test_a_norm_that_requires_grad_still_does(made):
    make, (gate_up, down, norm), _ = made
    layer = make(gate_up, down, norm.clone().requires_grad_())
    assert layer.norm.requires_grad and layer.norm.is_leaf
    layer.load(gate_up, down, norm.clone().requires_grad_())
    assert layer.norm.requires_grad
    layer.load(gate_up, down, norm)
    assert not layer.norm.requires_grad and torch.equal(layer.norm, norm)


def test_norms_of_other_sizes_and_types_are_refused(made):
    make, (gate_up, down, norm), _ = made
    layer = make(gate_up, down, norm)
    for bad in (norm[:-1], norm.float(), norm.to("meta")):
        with pytest.raises(ValueError, match="norm"):
            make(gate_up, down, bad)
        with pytest.raises(ValueError, match="norm"):
            layer.load(gate_up, down, bad)
    assert torch.equal(layer.norm, norm)


def test_a_load_neither_drops_nor_adds_a_norm(made):
    """Its gradient's sum is there or not from the start; a refused load changes nothing."""
    make, (gate_up, down, norm), _ = made
    with_norm, without = make(gate_up, down, norm), make(gate_up, down)
    held, was = with_norm.w1, without.w1
    with pytest.raises(ValueError, match="norm"):
        with_norm.load(gate_up, down)
    with pytest.raises(ValueError, match="norm"):
        without.load(gate_up, down, norm)
    assert torch.equal(with_norm.norm, norm) and with_norm.d_norm is not None and with_norm.w1 is held
    assert without.norm is None and without.d_norm is None and without.w1 is was
    without.load(gate_up, down)
    with_norm.load(gate_up, down, norm)


def forms_of(layer):
    return [t for s in (layer.w1, layer.w1t, layer.w2, layer.w2t) for t in (s.codes, s.scales)]


def test_a_load_goes_into_the_same_forms(made):
    """A captured pass holds the forms' addresses: a load fills these, and makes no new ones."""
    make, (gate_up, down, norm), _ = made
    layer = make(gate_up, down, norm)
    before = [(t.data_ptr(), t.nbytes) for t in forms_of(layer)]
    held = forms_of(layer)
    layer.load(gate_up, down, norm)
    assert [(t.data_ptr(), t.nbytes) for t in forms_of(layer)] == before and len(held) == 8


def test_weights_of_other_shapes_are_not_loaded(made):
    make, (gate_up, down, norm), _ = made
    layer = make(gate_up, down, norm)
    was = layer.norm.clone()
    norm.add_(1)
    for a, b in ((gate_up[..., :-1], down), (gate_up, down[..., :-1]), (gate_up[..., :F, :], down[..., :F // 2])):
        with pytest.raises(ValueError, match="gate_up"):
            layer.load(a, b, norm)
    assert torch.equal(layer.norm, was)


def test_made_in_inference_mode_and_loaded_outside(made):
    make, (gate_up, down, norm), _ = made
    with torch.inference_mode():
        layer = make(gate_up, down, norm)
    norm.add_(1)
    layer.load(gate_up, down, norm)
    assert torch.equal(layer.norm, norm)
    with torch.inference_mode():
        norm.add_(1)
        layer.load(gate_up, down, norm)
        assert torch.equal(layer.norm, norm)

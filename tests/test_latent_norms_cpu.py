"""The norm checks of latent attention's gradients (tests/latent_ref.py) without a GPU: outputs with the library's roundings
pass them at the expected size, and outputs with a planted mistake do not."""
import pytest
import torch

from latent_ref import (check_norms, latent_inputs, latent_norms, latent_reference, norm_parts,
                        norm_ratios, rounded_latent)

FAULTS = ("no D behind the middle", "16 keys dropped", "dS off by 1 %", "one head's k_rope", "no gradient", "negated")


@pytest.mark.parametrize("shape", [(1, 129, 2, 64, 32, 64), (2, 300, 2, 32, 16, 48), (1, 700, 2, 128, 64, 128),
                                   (1, 1000, 1, 64, 32, 64)], ids=str)
def test_rounded_outputs_have_the_expected_norms(shape):
    scale = (shape[3] + shape[4]) ** -0.5
    x = latent_inputs(*shape, seed=shape[1], device="cpu")
    norms = latent_norms(x, scale)
    got = rounded_latent(x, scale)
    check_norms(got, shape[3], norms, str(shape))
    for name, (block, whole) in norm_ratios(got, shape[3], norms).items():
        assert whole >= 0.6, (name, whole)              # the model is not loose


@pytest.mark.parametrize("fault", FAULTS)
@pytest.mark.parametrize("S", [700, 1500])
def test_planted_mistakes_are_seen(S, fault):
    shape = (1, S, 2, 128, 64, 128)
    scale = 192 ** -0.5
    x = latent_inputs(*shape, seed=S, device="cpu")
    ratios = norm_ratios(rounded_latent(x, scale, fault), 128, latent_norms(x, scale))
    assert any(max(r) > 1.0 for r in ratios.values()), ratios


@pytest.mark.parametrize("shape", [(1, 700, 2, 128, 64, 128), (1, 1500, 4, 64, 32, 64)], ids=str)
def test_a_rounding_more_is_seen(shape):
    """dS from the bf16 P instead of the fp32 one."""
    scale = (shape[3] + shape[4]) ** -0.5
    x = latent_inputs(*shape, seed=shape[1], device="cpu")
    ratios = norm_ratios(rounded_latent(x, scale, "dS of bf16 P"), shape[3], latent_norms(x, scale))
    assert all(max(ratios[n]) > 1.0 for n in ("dq", "dq rope", "dk", "dk_rope")), ratios


def test_the_elementwise_bounds_and_the_norms_have_one_definition():
    x = latent_inputs(1, 70, 2, 32, 16, 48, seed=1, device="cpu")
    ref = latent_reference(x, 0.1)
    for name, val in norm_parts({n: ref[n][0] for n in ("o", "dq", "dkv", "dk_rope")}, 32).items():
        assert torch.allclose(val, latent_norms(x, 0.1)[name][0], rtol=1e-12, atol=1e-14), name

"""Latent attention's expanded form: error norms by head and block of 128 rows against what the roundings lead one to expect
(tests/latent_ref.py), where elementwise bounds grow too wide to see a mistake; heads of fewer than 64 numbers over several
tiles and units; gradients against differences along themselves."""
import math

import pytest
import torch

from latent_ref import check_norms, latent_inputs, latent_norms, latent_reference
from window_ref import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bwd_xattn_fwd_gb300 import xattn  # noqa: F401  (fails loudly if not built)


def _run(x, scale):
    from bwd_xattn_fwd_gb300 import xattn
    q, kv, rope, dO = (x[n] for n in ("q", "kv", "k_rope", "dO"))
    o, lse = xattn.attention_latent_fwd(q, kv, rope, scale)
    dq, dkv, drope = xattn.attention_latent_bwd(q, kv, rope, o, dO, lse, scale)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    return {"o": o, "lse": lse, "dq": dq, "dkv": dkv, "dk_rope": drope}


# (B, S, nh, dn, dr, dv); dn, dv <= 64 and not both 64: kernels of their own
SMALL = [(2, 129, 3, 32, 16, 48), (2, 513, 3, 32, 16, 48), (1, 1030, 4, 64, 32, 48), (1, 385, 2, 16, 64, 64), (1, 640, 2, 48, 48, 16),
         (40, 200, 8, 48, 16, 32), (1, 1500, 2, 16, 16, 16)]
SHAPES = SMALL + [(2, 1100, 3, 64, 32, 64), (30, 385, 8, 64, 32, 64), (1, 3001, 2, 64, 64, 64), (1, 700, 4, 128, 64, 128),
                  (2, 1500, 2, 128, 64, 128), (9, 300, 12, 128, 64, 128), (1, 3001, 2, 128, 64, 128), (1, 1030, 4, 96, 32, 64),
                  (1, 900, 3, 80, 48, 112), (1, 1200, 2, 128, 32, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_expanded_norms(shape):
    x = latent_inputs(*shape, seed=shape[1])
    scale = (shape[3] + shape[4]) ** -0.5
    got = _run(x, scale)
    check(got, latent_reference(x, scale), str(shape))
    check_norms(got, shape[3], latent_norms(x, scale), str(shape))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5, 1e-30])
@pytest.mark.parametrize("dims", [(64, 32, 64), (32, 16, 48)], ids=str)
def test_scales(dims, scale):
    x = latent_inputs(1, 300, 2, *dims, seed=3)
    check(_run(x, scale), latent_reference(x, scale), f"scale {scale}")


@pytest.mark.parametrize("dims", [(64, 32, 64), (32, 16, 48)], ids=str)
@pytest.mark.parametrize("scale", [0.3, -0.3])
def test_growing_scores(dims, scale):
    """Row maxima that grow by more than 2^8 from tile to tile, and ones that the first tile holds."""
    x = latent_inputs(1, 900, 2, *dims, seed=5)
    up = torch.linspace(0.05, 1.0, 900, device="cuda")
    for ramp in (up, up.flip(0)):
        y = dict(x)
        y["kv"] = x["kv"].clone()
        y["kv"][..., :dims[0]] = (x["kv"][..., :dims[0]].float() * ramp[None, :, None, None] * 8).bfloat16()
        y["q"] = (x["q"].float() * 4).bfloat16()
        check(_run(y, scale), latent_reference(y, scale), "ramp")


def test_many_units_of_small_heads_repeat():
    for shape in ((30, 385, 8, 48, 16, 32), (4, 1100, 16, 64, 32, 48)):
        x = latent_inputs(*shape, seed=7)
        first = _run(x, 0.1)
        for _ in range(4):
            again = _run(x, 0.1)
            assert all(torch.equal(first[n], again[n]) for n in first)


@pytest.mark.parametrize("shape", [(1, 150, 3, 64, 32, 64), (1, 300, 2, 128, 64, 128), (2, 270, 2, 32, 16, 48)], ids=str)
def test_gradients_against_differences_along_them(shape):
    """Differences of L = sum(dO * o), in 64 bits of the definition, along the exact gradient (d = grad / |grad|, so that the slope is
    |grad|) against <got, d>. The two differ by at most |got - grad|, of which the norms' check says how large it may be, and by
    the difference's own O(h^2) error, some 1e-6 of the slope. A gradient of zero, or of the other sign, is off by |grad| or more."""
    scale = (shape[3] + shape[4]) ** -0.5
    dn = shape[3]
    x = latent_inputs(*shape, seed=9)
    got, norms = _run(x, scale), latent_norms(x, scale)

    def loss(y):
        return float((x["dO"].double() * latent_reference({**x, **y}, scale)["o"][0]).sum())

    heads = lambda *parts: torch.cat([norms[p][0] for p in parts], 3).transpose(1, 2)
    for name, parts in (("q", ("dq", "dq rope")), ("kv", ("dk", "dv")), ("k_rope", ("dk_rope",))):
        grad = heads(*parts).reshape(x[name].shape)
        d = grad / grad.norm()
        h = 1e-4
        slope = (loss({name: x[name].double() + h * d}) - loss({name: x[name].double() - h * d})) / (2 * h)
        room = math.sqrt(sum(float(norms[p][1][-1].sum()) for p in parts)) + 1e-5 * abs(slope)
        along = float((got["d" + name].double() * d).sum())
        assert abs(along - slope) <= room, (name, along, slope, room)
        assert room <= 0.02 * abs(slope), (name, room, slope)          # so that neither 0 nor the negated gradient passes

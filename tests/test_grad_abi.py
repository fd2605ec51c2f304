"""any4_linear_lora_grad asks for what its outputs need and for no more (CPU
only: every call is stopped by a workspace that is too small)."""
import ctypes

import pytest

import learned_bit_lut_b200 as a4

P, Z = ctypes.c_void_p(4096), ctypes.c_void_p(0)
NEEDS = {"dx": ("dy", "packed", "a", "b", "s"), "da": ("dy", "x", "b", "s"), "db": ("dy", "u")}


def grad(outputs, dy=Z, x=Z, u=Z, packed=Z, a=Z, b=Z, s=Z):
    dx, da, db = (P if o in outputs else Z for o in ("dx", "da", "db"))
    return a4.lib.any4_linear_lora_grad(4, dy, x, Z, Z, 0, u, packed, 4, 64, 128, 64, a, b, s, Z, 2, 16, dx, da, db, P, 0,
                                        None)


@pytest.mark.parametrize("outputs", [("dx",), ("da",), ("db",), ("dx", "db"), ("da", "db"), ("dx", "da", "db")], ids=str)
def test_needs_of_the_outputs(outputs):
    needed = {name for o in outputs for name in NEEDS[o]}
    assert grad(outputs, **{name: P for name in needed}) == a4.ANY4_EWORKSPACE
    for name in needed:
        assert grad(outputs, **{other: P for other in needed - {name}}) == a4.ANY4_EINVAL, name

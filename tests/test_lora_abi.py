"""Adapter and checkpoint entry points: sizes, and refusals on the host before
anything is launched (CPU only)."""
import ctypes

import pytest
import torch

import learned_bit_lut_b200 as a4

P, Z, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(0), ctypes.c_void_p(4104)
BIG = 1 << 40


def lora(bits=4, x=P, packed=P, m=4, n=64, k=128, g=64, a=P, b=P, s=P, ids=P, L=2, r=16, y=P, u=P, ws=P, size=BIG):
    return a4.lib.any4_linear_lora(bits, x, packed, m, n, k, g, a, b, s, ids, L, r, y, u, ws, size, None)


def grad(bits=4, dy=P, x=P, codes=Z, steps=Z, xg=0, u=P, packed=P, m=4, n=64, k=128, g=64, a=P, b=P, s=P, ids=P,
         L=2, r=16, dx=P, da=P, db=P, ws=P, size=BIG):
    return a4.lib.any4_linear_lora_grad(bits, dy, x, codes, steps, xg, u, packed, m, n, k, g, a, b, s, ids, L, r, dx,
                                        da, db, ws, size, None)


@pytest.mark.parametrize("bad", [dict(bits=5), dict(bits=1), dict(m=0), dict(m=-1), dict(m=(1 << 20) + 1), dict(n=0),
                                 dict(n=24), dict(k=96), dict(k=0), dict(g=32), dict(g=256), dict(L=0), dict(L=-3),
                                 dict(L=65537), dict(r=0), dict(r=4), dict(r=12), dict(r=136), dict(r=-8)])
def test_shapes_outside_the_accepted_set(bad):
    assert lora(**bad) == a4.ANY4_ESHAPE
    assert grad(**bad) == a4.ANY4_ESHAPE
    full = dict(bits=4, m=4, n=64, k=128, g=64, L=2, r=16) | bad
    args = [full[i] for i in ("bits", "m", "n", "k", "g", "L", "r")]
    assert a4.lib.any4_lora_workspace_bytes(*args) == 0
    assert a4.lib.any4_lora_grad_workspace_bytes(*args) == 0


def test_null_pointers():
    for name in ("x", "packed", "a", "b", "s", "y", "ws"):
        assert lora(**{name: Z}) == a4.ANY4_EINVAL, name
    for name in ("dy", "x", "u", "packed", "a", "b", "s", "ws"):
        assert grad(**{name: Z}) == a4.ANY4_EINVAL, name
    assert grad(dx=Z, da=Z, db=Z) == a4.ANY4_EINVAL
    assert grad(codes=P, steps=P, xg=64) == a4.ANY4_EINVAL          # two forms of x
    assert grad(x=Z, codes=P, steps=Z, xg=64) == a4.ANY4_EINVAL     # half a checkpoint
    assert grad(x=Z, codes=Z, steps=P, xg=64) == a4.ANY4_EINVAL


def test_alignment_and_checkpoint_groups():
    for name in ("x", "packed", "a", "b", "u", "ws"):
        assert lora(**{name: ODD}) == a4.ANY4_EALIGN, name
    assert lora(y=ctypes.c_void_p(4098)) == a4.ANY4_EALIGN
    assert lora(s=ctypes.c_void_p(4098)) == a4.ANY4_EALIGN
    assert lora(ids=ctypes.c_void_p(4098)) == a4.ANY4_EALIGN
    for name in ("dy", "x", "u", "packed", "a", "b", "dx", "da", "db", "ws"):
        assert grad(**{name: ODD}) == a4.ANY4_EALIGN, name
    assert grad(x=Z, codes=ODD, steps=P, xg=64) == a4.ANY4_EALIGN
    assert grad(x=Z, codes=P, steps=ctypes.c_void_p(4097), xg=64) == a4.ANY4_EALIGN
    for group in (0, 32, 96, 256, -64):
        assert grad(x=Z, codes=P, steps=P, xg=group) == a4.ANY4_ESHAPE


def test_workspaces_too_small():
    assert grad(size=0) == a4.ANY4_EWORKSPACE
    assert grad(size=a4.lib.any4_lora_grad_workspace_bytes(4, 4, 64, 128, 64, 2, 16) - 1) in (a4.ANY4_EWORKSPACE,
                                                                                           a4.ANY4_ECUDA)
    assert a4.lib.any4_lora_header_bytes() == 65536 * 4 + 256


def test_checkpoint_refusals():
    pack, unpack = a4.lib.any4_act_pack, a4.lib.any4_act_unpack
    assert pack(Z, 4, 128, 64, P, P, None) == a4.ANY4_EINVAL
    assert pack(P, 4, 128, 64, Z, P, None) == a4.ANY4_EINVAL
    assert unpack(P, Z, 4, 128, 64, P, None) == a4.ANY4_EINVAL
    for m, k, g in ((0, 128, 64), (4, 0, 64), (4, 100, 64), (4, 128, 256), (4, 128, 32), (4, (1 << 20) + 64, 64),
                    ((1 << 20) + 1, 64, 64)):
        assert pack(P, m, k, g, P, P, None) == a4.ANY4_ESHAPE
        assert unpack(P, P, m, k, g, P, None) == a4.ANY4_ESHAPE
    assert pack(ODD, 4, 128, 64, P, P, None) == a4.ANY4_EALIGN
    assert pack(P, 4, 128, 64, ODD, P, None) == a4.ANY4_EALIGN
    assert unpack(P, P, 4, 128, 64, ODD, None) == a4.ANY4_EALIGN
    assert unpack(P, ctypes.c_void_p(4097), 4, 128, 64, P, None) == a4.ANY4_EALIGN


def test_checkpoint_refuses_overlapping_buffers():
    x, codes, steps, near = (ctypes.c_void_p(v) for v in (1 << 20, 2 << 20, 3 << 20, (1 << 20) + 4 * 128 * 2 - 16))
    pack, unpack = a4.lib.any4_act_pack, a4.lib.any4_act_unpack
    for c, s in ((x, steps), (near, steps), (codes, near), (codes, codes)):
        assert pack(x, 4, 128, 64, c, s, None) == a4.ANY4_EINVAL
    for c, s in ((x, steps), (near, steps), (codes, near)):
        assert unpack(c, s, 4, 128, 64, x, None) == a4.ANY4_EINVAL


def test_binding_refuses_tensors_of_the_host():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        a4.any4_linear_lora(x, x, 64, 128, 64, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        a4.any4_linear_lora_grad(x, x, x, x, 64, 128, 64, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        a4.any4_act_pack(x, 64)
    with pytest.raises(ValueError, match="CUDA"):
        a4.any4_act_unpack(x, x, 64)

"""Edges of the adapter operators that the tables of shapes in test_gpu_lora.py
do not reach, against the same float64 references and derived bounds
(lora_util)."""
import pytest
import torch

import learned_bit_lut_b200 as a4
from gpu_util import require_gpu
from lora_util import Case, check

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)


def forward(c: Case, **kw):
    return a4.any4_linear_lora(c.x, c.packed(), *c.shape(), c.a, c.b, c.scale, c.ids, bits=c.bits, **kw)


def inner(c: Case):
    return c.u_ref()[0].to(torch.bfloat16)


def grads(c: Case, kept=None, u=None, **kw):
    kept = c.x if kept is None else kept
    u = inner(c) if u is None else u
    return a4.any4_linear_lora_grad(c.dy, kept, u, c.packed(), *c.shape(), c.a, c.b, c.scale, c.ids, bits=c.bits, **kw)


def status(ws):
    at = 65536 * 4
    return int(ws[at:at + 4].view(torch.int32).item())


# ---- non-finite adapter values in many short tiles in a row: the tiles that are
# patched ahead of the epilogue must not share a flag with the tile it is at

def spread(t, every, offset=0):
    """Infinities of both signs and NaN over the rows of t (rows x ranks)."""
    rows = torch.arange(offset, t.shape[0], every, device=t.device)
    for i, v in enumerate((INF, -INF, NAN)):
        t[rows[i::3], i % t.shape[1]] = v


@pytest.mark.parametrize("every", [128, 300, 1111])
def test_short_tiles_of_dx_with_spoilt_adapters(every):
    """One chunk and one adapter stage a tile, about seven tiles a pair of blocks."""
    c = Case(8192, 64, 4096, 64, 4, 1, 8, "holes", seed=61)
    spread(c.a[0].T, every)
    need = a4.any4_lora_grad_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    u = torch.zeros(c.m, c.rank, dtype=torch.bfloat16, device="cuda")
    for _ in range(5):
        dx = grads(c, u=u, outputs=("dx",), workspace=ws)[0]
        assert status(ws) == 0
        check(dx, *c.grad_ref(c.x, u)[0], "dx")


@pytest.mark.parametrize("m,n", [(8192, 4096), (512, 65536)], ids=["pairs", "fused"])
def test_short_tiles_of_the_forward_with_spoilt_adapters(m, n):
    """K = 64. In the fused kernel the first token tile has no adapter, so its
    tiles take one stage and the others' patching is further ahead."""
    c = Case(m, n, 64, 64, 4, 1, 8, "holes", seed=62)
    if m == 512:
        c.ids[:256] = -1
        c.tokens = [torch.nonzero(c.ids == 0).flatten()]
    spread(c.b[0], 300)
    ws = torch.zeros(a4.any4_lora_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        y = forward(c, workspace=ws)
        assert status(ws) == 0
        check(y, *c.y_ref(), "y")


# ---- decoding tokens without an adapter: their clusters have nothing to sum, so
# their blocks exchange at once, while others of the cluster may not have started

@pytest.mark.parametrize("order", ["nobody", "holes"])
def test_decode_tokens_without_an_adapter_in_a_row(order):
    c = Case(16, 4096, 1024, 128, 4, 3, 128, order, seed=63)
    packed = c.packed()
    ref = c.y_ref()
    outs = [a4.any4_linear_lora(c.x, packed, *c.shape(), c.a, c.b, c.scale, c.ids) for _ in range(200)]
    check(outs[0], *ref, "y")
    assert all(torch.equal(y, outs[0]) for y in outs)


# ---- the dequantized weight right behind whatever wrote the packed one

@pytest.mark.parametrize("bits", [4, 3, 2])
def test_dequantization_follows_a_copy_of_the_weight(bits):
    one, two = (Case(8, 1024, 1024, 128, bits, 1, 8, "null", seed=s).packed() for s in (64, 65))
    wants = [a4.any4_dequant_bits(bits, p, 1024, 1024, 128) for p in (one, two)]
    x = torch.randn(600, 1024, device="cuda").to(torch.bfloat16)
    ys = [a4.any4_linear_bits(bits, x, p, 1024, 1024, 128) for p in (one, two)]
    torch.cuda.synchronize()
    packed, outs = one.clone(), []
    for i in range(60):
        packed.copy_((one, two)[i % 2])
        outs.append((a4.any4_dequant_bits(bits, packed, 1024, 1024, 128) if i % 4 < 2 else
                     a4.any4_linear_bits(bits, x, packed, 1024, 1024, 128)))
    for i, out in enumerate(outs):
        assert torch.equal(out, (wants if i % 4 < 2 else ys)[i % 2])


# ---- host threads

def test_two_threads_on_one_stream():
    """Threads share the default stream, and each gets its own results."""
    import threading
    cases = [Case(40, 272, 512, 128, 4, 3, 16, "mixed", seed=66), Case(700, 528, 1088, 64, 3, 6, 40, "holes", seed=67),
             Case(9, 528, 1024, 128, 4, 2, 24, "mixed", seed=68)]
    packed, us = [c.packed() for c in cases], [inner(c) for c in cases]

    def step(i):
        c = cases[i]
        args = (packed[i], *c.shape(), c.a, c.b, c.scale, c.ids)
        return (a4.any4_linear_lora(c.x, *args, bits=c.bits), a4.any4_linear_bits(c.bits, c.x, packed[i], *c.shape()),
                *a4.any4_linear_lora_grad(c.dy, c.x, us[i], *args, bits=c.bits))

    wants = [step(i) for i in range(len(cases))]
    torch.cuda.synchronize()
    outs = [[] for _ in cases]

    def job(i):
        torch.cuda.set_device(0)
        outs[i] = [step(i) for _ in range(40)]

    threads = [threading.Thread(target=job, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert len(got) == 40
        assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for one in got for p, q in zip(one, want))

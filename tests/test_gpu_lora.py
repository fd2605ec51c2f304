"""Low-rank adapters beside an any4 weight, forward and gradients, against
plain float64 references (lora_util) with derived bounds: token counts around
every tile and kernel border, ragged rows and columns, ranks that end inside a
tile, adapters in any order, tokens without one, values that must not leak
from one request into another, streams, graphs, repeated calls and buffers."""
import pytest
import torch

import learned_bit_lut_b200 as a4
from gpu_util import require_gpu
from lora_util import Case, check, guarded

pytestmark = pytest.mark.gpu
STATUS_OFFSET = 65536 * 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)


def forward(c: Case, u=None, **kw):
    return a4.any4_linear_lora(c.x, c.packed(), *c.shape(), c.a, c.b, c.scale, c.ids, bits=c.bits, u=u, **kw)


def inner(c: Case):
    return c.u_ref()[0].to(torch.bfloat16)


def grads(c: Case, kept=None, u=None, **kw):
    kept = c.x if kept is None else kept
    u = inner(c) if u is None else u
    return a4.any4_linear_lora_grad(c.dy, kept, u, c.packed(), *c.shape(), c.a, c.b, c.scale, c.ids, bits=c.bits, **kw)


# (m, n, k, g, bits, adapters, rank, ids)
SHAPES = [
    (1, 16, 64, 64, 4, 1, 8, "null"),
    (1, 1024, 4096, 128, 4, 8, 16, "mixed"),
    (2, 48, 192, 64, 4, 3, 24, "holes"),
    (4, 272, 1024, 128, 3, 5, 128, "mixed"),
    (5, 4096, 512, 256, 4, 70, 16, "mixed"),
    (8, 160, 320, 64, 2, 2, 40, "runs"),
    (9, 96, 1088, 64, 4, 4, 72, "holes"),
    (16, 4096, 4096, 128, 4, 32, 16, "mixed"),
    (16, 80, 2048, 1024, 4, 16, 64, "nobody"),
    (17, 16, 64, 64, 4, 2, 8, "mixed"),
    (33, 144, 192, 64, 4, 7, 24, "holes"),
    (64, 272, 320, 64, 4, 3, 16, "runs"),
    (65, 48, 1024, 512, 4, 65, 8, "mixed"),
    (127, 256, 512, 128, 4, 2, 120, "mixed"),
    (129, 400, 1088, 64, 4, 40, 128, "mixed"),
    (190, 1040, 1024, 128, 4, 24, 32, "holes"),
    (256, 128, 512, 128, 3, 9, 56, "runs"),
    (257, 1024, 768, 256, 4, 300, 16, "mixed"),
    (300, 272, 320, 64, 2, 6, 64, "last"),
    (512, 512, 512, 128, 4, 3, 96, "nobody"),
    (513, 304, 1024, 128, 4, 12, 40, "holes"),
    (700, 1024, 2048, 128, 4, 1, 64, "null"),
    (1100, 528, 1088, 64, 4, 130, 16, "mixed"),
    (2011, 272, 576, 64, 4, 4, 16, "runs"),
]
NAMES = ["m%d_n%d_k%d_g%d_b%d_L%d_r%d_%s" % s for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=NAMES)
def test_forward(shape):
    c = Case(*shape)
    y, y_ok = guarded((c.m, c.n))
    u, u_ok = guarded((c.m, c.rank))
    ws = torch.zeros(a4.any4_lora_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank, bits=c.bits),
                     dtype=torch.uint8, device="cuda")
    forward(c, u=u, out=y, workspace=ws)
    torch.cuda.synchronize()
    check(u, *c.u_ref(), "u")
    check(y, *c.y_ref(), "y")
    assert y_ok() and u_ok()
    assert not bool(ws[:a4.lib.any4_lora_header_bytes()].any())   # counters and status word left zero
    first = y.clone()
    forward(c, out=y, workspace=ws)   # without u, on the used workspace
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("kept", ["bf16", "8bit"])
@pytest.mark.parametrize("shape", SHAPES, ids=NAMES)
def test_gradients(shape, kept):
    c = Case(*shape)
    x, stored = c.x, c.x
    if kept == "8bit":
        group = max(g for g in (64, 128, 256, 512, 1024) if c.k % g == 0)
        stored = a4.any4_act_pack(c.x, group)
        x = a4.any4_act_unpack(*stored, group)
    u = inner(c)
    outs = {"dx": (c.m, c.k), "da": (c.adapters, c.rank, c.k), "db": (c.adapters, c.n, c.rank)}
    bufs = {name: guarded(s) for name, s in outs.items()}
    ws = torch.zeros(a4.any4_lora_grad_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank, bits=c.bits),
                     dtype=torch.uint8, device="cuda")
    got = grads(c, stored, u, workspace=ws, **{name: b[0] for name, b in bufs.items()})
    torch.cuda.synchronize()
    for name, g, ref in zip(("dx", "da", "db"), got, c.grad_ref(x, u)):
        check(g, *ref, name)
    assert all(ok() for _, ok in bufs.values())
    assert not bool(ws[:a4.lib.any4_lora_header_bytes()].any())
    again = grads(c, stored, u, workspace=ws)
    torch.cuda.synchronize()
    for one, two in zip(got, again):
        assert torch.equal(one.view(torch.int16), two.view(torch.int16))
    if kept == "8bit":   # a checkpoint's gradients are those of its values, bit for bit
        plain = grads(c, x, u)
        for one, two in zip(got, plain):
            assert torch.equal(one.view(torch.int16), two.view(torch.int16))


@pytest.mark.parametrize("shape", [(1300, 1024, 8192, 128, 4, 1, 16, "null"), (5000, 2048, 4096, 128, 4, 2, 24, "holes"),
                                   (5000, 4096, 2048, 256, 4, 1, 64, "null"), (2300, 2064, 4160, 64, 3, 1, 40, "holes")],
                         ids=str)
def test_longer_steps(shape):
    """More tiles than SMs, several shares of every sum, ragged last waves."""
    c = Case(*shape, seed=14)
    u = torch.empty(c.m, c.rank, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(a4.any4_lora_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank, bits=c.bits),
                     dtype=torch.uint8, device="cuda")
    y = forward(c, u=u, workspace=ws)
    check(u, *c.u_ref(), "u")
    check(y, *c.y_ref(), "y")
    assert not bool(ws[:a4.lib.any4_lora_header_bytes()].any())
    del ws
    ws = torch.zeros(a4.any4_lora_grad_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank, bits=c.bits),
                     dtype=torch.uint8, device="cuda")
    got = grads(c, u=u, workspace=ws)
    for name, g, ref in zip(("dx", "da", "db"), got, c.grad_ref(c.x, u)):
        check(g, *ref, name)
    assert not bool(ws[:a4.lib.any4_lora_header_bytes()].any())
    again = forward(c, u=u), *grads(c, u=u)
    assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip((y, *got), again))


@pytest.mark.parametrize("outputs", [("dx",), ("da",), ("db",), ("da", "db"), ("dx", "db")])
def test_some_outputs_equal_all(outputs):
    c = Case(77, 272, 320, 64, 4, 3, 24, "holes")
    every = dict(zip(("dx", "da", "db"), grads(c)))
    some = dict(zip(("dx", "da", "db"), grads(c, outputs=outputs)))
    for name in every:
        if name in outputs:
            assert torch.equal(every[name].view(torch.int16), some[name].view(torch.int16))
        else:
            assert some[name] is None


@pytest.mark.parametrize("m", [13, 150, 600])
def test_nothing_leaks_between_requests(m):
    """An adapter with infinities or NaN spoils its own tokens only; a padding
    token with them spoils no gradient but its own dx."""
    c = Case(m, 272, 320, 64, 4, 4, 24, "holes", seed=3)
    c.a[1, 3, 17] = float("nan")
    c.b[2, 5, 7] = float("inf")
    c.b[2, 200, 1] = float("-inf")
    c.b[2, 201, 2] = float("nan")
    c.scale[3] = float("inf")
    y = forward(c)
    check(y, *c.y_ref(), "y")
    clean = ~torch.isin(c.ids, torch.tensor([1, 2, 3], device="cuda", dtype=torch.int32))
    assert bool(torch.isfinite(y[clean].float()).all())

    c = Case(m, 272, 320, 64, 4, 4, 24, "holes", seed=4)
    nobody = torch.nonzero((c.ids < 0) | (c.ids >= 4)).flatten()
    c.x[nobody[0]] = float("nan")
    c.x[nobody[1], 3] = float("inf")
    c.dy[nobody[0], 11] = float("nan")
    c.dy[nobody[2]] = float("inf")
    t = c.tokens[2][0]
    c.x[t, 100] = float("inf")
    c.x[t, 101] = float("nan")
    c.dy[t, 9] = float("-inf")
    u = inner(c)
    for stored in (c.x, a4.any4_act_pack(c.x, 64)):
        x = c.x if stored is c.x else a4.any4_act_unpack(*stored, 64)
        got = grads(c, stored, u)
        for name, g, ref in zip(("dx", "da", "db"), got, c.grad_ref(x, u)):
            check(g, *ref, name)
        for l in (0, 1, 3):
            assert bool(torch.isfinite(got[1][l].float()).all()) and bool(torch.isfinite(got[2][l].float()).all())


def test_gradients_agree_with_differences():
    """dx, dA and dB against central differences of the float64 layer that the
    forward is tested against, along random directions."""
    c = Case(40, 96, 192, 64, 4, 2, 16, "mixed", seed=5)
    w, dy = c.weight(), c.dy.double()
    x, a, b, scale = c.x.double(), c.a.double(), c.b.double(), c.scale.double()

    def loss(x, a, b):
        y = x @ w.T
        for l, t in enumerate(c.tokens):
            y[t] += scale[l] * (x[t] @ a[l].T) @ b[l].T
        return (y * dy).sum()

    dx, da, db = (g.double() for g in grads(c))
    refs = c.grad_ref(c.x, inner(c))
    gen = torch.Generator(device="cuda").manual_seed(1)
    for which, (grad, (ref, bound)) in enumerate(zip((dx, da, db), refs)):
        d = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-3
        args = [x, a, b]
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + h * d, args[which] - h * d
        slope = (loss(*up) - loss(*down)) / (2 * h)   # the loss is linear in each argument alone
        # each gradient element is off by its bound and half a step of its value; dB's u was rounded too
        room = ((bound + 2.0 ** -8 * (ref.abs() + bound)) * d.abs()).sum()
        if which == 2:
            u = c.u_ref()[0].abs()
            for l, t in enumerate(c.tokens):
                room += 2.0 ** -8 * ((dy[t].abs().T @ u[t]) * d[l].abs()).sum()
        assert abs(float((grad * d).sum() - slope)) <= float(room)


def test_order_of_tokens_does_not_matter():
    c = Case(333, 272, 512, 128, 4, 6, 40, "mixed", seed=6)
    y = forward(c)
    perm = torch.randperm(c.m, device="cuda")
    c.x, c.ids = c.x[perm].contiguous(), c.ids[perm].contiguous()
    assert torch.equal(forward(c).view(torch.int16), y[perm].view(torch.int16))


def test_zero_adapters_leave_the_projection():
    """With B = 0 the decode layer is any4_linear bit for bit."""
    for m in (1, 3, 7, 16):
        c = Case(m, 1024, 1024, 128, 4, 3, 16, "mixed", seed=7)
        c.b.zero_()
        base = a4.any4_linear(c.x, c.packed(), *c.shape())
        y = forward(c)
        assert bool((y == base).all())


@pytest.mark.parametrize("m", [40, 100, 200, 700])
def test_zero_adapters_leave_the_prefill(m):
    """With B = 0 the prefill layer is any4_linear bit for bit too."""
    c = Case(m, 1024, 1024, 128, 4, 3, 16, "mixed", seed=7)
    c.b.zero_()
    base = a4.any4_linear(c.x, c.packed(), *c.shape())
    assert bool((forward(c) == base).all())


@pytest.mark.parametrize("m", [1, 16, 60, 600])
def test_streams_graphs_and_two_calls_at_once(m):
    c = Case(m, 528, 1024, 128, 4, 5, 16, "mixed", seed=8)
    d = Case(m + 3, 272, 512, 128, 4, 3, 24, "holes", seed=9)
    want_c, want_d = forward(c), forward(d)
    gc, gd = grads(c), grads(d)
    pc, pd = c.packed(), d.packed()
    uc, ud = inner(c), inner(d)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(3):
        for stream, z, p, u in ((one, c, pc, uc), (two, d, pd, ud)):
            with torch.cuda.stream(stream):
                y = a4.any4_linear_lora(z.x, p, *z.shape(), z.a, z.b, z.scale, z.ids)
                g = a4.any4_linear_lora_grad(z.dy, z.x, u, p, *z.shape(), z.a, z.b, z.scale, z.ids)
                outs.append((y, g))
    torch.cuda.synchronize()
    for i, (y, g) in enumerate(outs):
        want, wg = (want_c, gc) if i % 2 == 0 else (want_d, gd)
        assert torch.equal(y, want)
        assert all(torch.equal(p, q) for p, q in zip(g, wg))

    # two graphs, captured one after the other, replayed in turn and at once
    graphs, results = [], []
    for z, p, u in ((c, pc, uc), (d, pd, ud)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = a4.any4_linear_lora(z.x, p, *z.shape(), z.a, z.b, z.scale, z.ids)
            gr = a4.any4_linear_lora_grad(z.dy, z.x, u, p, *z.shape(), z.a, z.b, z.scale, z.ids)
        graphs.append(g)
        results.append((y, *gr))
    for _ in range(3):
        for r in results:
            for t in r:
                t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            graphs[0].replay()
        with torch.cuda.stream(two):
            graphs[1].replay()
        torch.cuda.synchronize()
        for got, want in zip(results, ((want_c, *gc), (want_d, *gd))):
            assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("m,order", [(24, "mixed"), (400, "runs")])
def test_a_training_step_as_it_is_used(m, order):
    """Checkpoint, forward, gradients and update together: two stacked layers,
    the gradients against the float64 formulas on the kept values, and the next
    forward on the updated adapters."""
    c1 = Case(m, 256, 320, 64, 4, 3, 16, order, seed=10)
    c2 = Case(m, 272, 256, 64, 4, 3, 16, order, seed=11)
    c2.ids, c2.tokens = c1.ids, c1.tokens
    u1 = torch.empty(m, 16, dtype=torch.bfloat16, device="cuda")
    u2 = torch.empty_like(u1)
    kept1 = a4.any4_act_pack(c1.x, 64)
    c2.x = forward(c1, u=u1)
    kept2 = a4.any4_act_pack(c2.x, 64)
    forward(c2, u=u2)
    g2 = grads(c2, kept2, u2)
    c1.dy = g2[0]
    g1 = grads(c1, kept1, u1)
    for c, kept, u, g in ((c1, kept1, u1, g1), (c2, kept2, u2, g2)):
        check(u, *c.u_ref(), "u")
        for name, got, ref in zip(("dx", "da", "db"), g, c.grad_ref(a4.any4_act_unpack(*kept, 64), u)):
            check(got, *ref, name)
        c.a -= 0.05 * g[1]
        c.b -= 0.05 * g[2]
    check(forward(c1), *c1.y_ref(), "y after the update")


def test_adapters_at_far_offsets():
    """Adapter tables past 2^31 elements and 4 GiB."""
    n, k, rank = 4096, 4096, 128
    adapters = 4200   # 4200 * 128 * 4096 = 2.2e9 elements of A
    c = Case(5, n, k, 128, 4, 1, 8, "null", seed=12)
    a = torch.zeros(adapters, rank, k, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(adapters, n, rank, dtype=torch.bfloat16, device="cuda")
    for l in (0, adapters - 1):
        a[l].normal_(std=k ** -0.5)
        b[l].normal_(std=0.05)
    for m in (5, 140):
        c = Case(m, n, k, 128, 4, 1, 8, "null", seed=12)
        c.rank, c.adapters = rank, adapters
        c.a, c.b, c.scale = a, b, torch.full((adapters,), 0.5, device="cuda")
        c.ids = torch.full((m,), adapters - 1, dtype=torch.int32, device="cuda")
        c.ids[1::2] = 0
        c.tokens = [torch.empty(0, dtype=torch.int64, device="cuda")] * adapters
        c.tokens[0] = torch.arange(1, m, 2, device="cuda")
        c.tokens[-1] = torch.arange(0, m, 2, device="cuda")
        check(forward(c), *c.y_ref(), "y")
        dx = grads(c, outputs=("dx",))[0]
        v, vb = c.v_ref()
        w, dy = c.weight(), c.dy.double()
        ref, bound = dy @ w, (n + 2 * rank + 8) * 2.0 ** -23 * (dy.abs() @ w.abs())
        for l in (0, adapters - 1):
            t = c.tokens[l]
            ref[t] += v[t] @ a[l].double()
            bound[t] += (vb[t] + 2.0 ** -14 * v[t].abs()) @ a[l].double().abs()
        check(dx, ref, bound, "dx")


@pytest.mark.parametrize("m,n,k", [(1, 1024, 4096), (3, 4096, 4096), (7, 4096, 4096), (16, 272, 1024), (16, 14336, 1024)])
def test_decode_reads_what_the_kernel_before_it_wrote(m, n, k):
    """Back-to-back calls whose inputs the kernel right before each call
    overwrites: the decode kernel runs beside the adapters' kernel and may not
    read its inputs early."""
    c = Case(m, n, k, 128, 4, 6, 16, "mixed", seed=13)
    packed = c.packed()
    xs = [torch.randn(m, k, device="cuda").to(torch.bfloat16) for _ in range(8)]
    ids = [torch.randint(0, 6, (m,), device="cuda", dtype=torch.int32) for _ in range(8)]
    want = [a4.any4_linear_lora(x, packed, *c.shape(), c.a, c.b, c.scale, i) for x, i in zip(xs, ids)]
    torch.cuda.synchronize()
    x, i, outs = xs[0].clone(), ids[0].clone(), []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            for xv, iv in zip(xs, ids):
                torch.mul(xv, 1.0, out=x)
                torch.add(iv, 0, out=i)
                outs.append(a4.any4_linear_lora(x, packed, *c.shape(), c.a, c.b, c.scale, i))
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[j % 8]) for j, o in enumerate(outs))


# more than 148 tiles of 128 x 256, so two blocks share each: an odd number of
# row tiles forward (19) and backward (17), a last tile whose second block has
# no tokens (2600 = 10 x 256 + 40) and one whose second block has no rows
@pytest.mark.parametrize("shape", [(2600, 2320, 2112, 64, 4, 5, 24, "holes"), (2600, 2320, 2112, 64, 3, 3, 72, "runs"),
                                   (2600, 2320, 2112, 64, 4, 1, 128, "null"), (5200, 1040, 1088, 64, 2, 40, 16, "mixed")],
                         ids=["holes", "runs", "null", "many"])
def test_tiles_shared_by_two_blocks(shape):
    c = Case(*shape, seed=21)
    if c.adapters == 5:   # spoilt adapters must not reach the tokens that share their tiles
        c.a[1, 3, 17] = float("nan")
        c.b[2, 5, 7] = float("inf")
        c.b[2, 2319, 1] = float("-inf")
        c.a[3, 0, 2111] = float("inf")
    y, y_ok = guarded((c.m, c.n))
    forward(c, out=y)
    check(y, *c.y_ref(), "y")
    u = inner(c)
    dx, dx_ok = guarded((c.m, c.k))
    got = grads(c, u=u, dx=dx)
    for name, g, ref in zip(("dx", "da", "db"), got, c.grad_ref(c.x, u)):
        check(g, *ref, name)
    assert y_ok() and dx_ok()
    if c.adapters == 5:
        clean = ~torch.isin(c.ids, torch.tensor([1, 2, 3], device="cuda", dtype=torch.int32))
        assert bool(torch.isfinite(y[clean].float()).all()) and bool(torch.isfinite(dx[clean].float()).all())


@pytest.mark.parametrize("m,n,k,bits", [(2600, 2320, 2112, 4), (5200, 1040, 1088, 3)])
def test_plain_tiles_shared_by_two_blocks(m, n, k, bits):
    """any4_linear itself: with B = 0 the reference is its own, and so are the bits."""
    c = Case(m, n, k, 64, bits, 2, 16, "mixed", seed=22)
    c.b.zero_()
    y, y_ok = guarded((m, n))
    a4.any4_linear_bits(bits, c.x, c.packed(), n, k, 64, out=y)
    check(y, *c.y_ref(), "y")
    assert y_ok() and bool((forward(c) == y).all())


def test_calls_in_a_row_share_a_workspace():
    """Kernels of one call run beside each other; calls still follow each other:
    every order of short and long calls, forward and backward, on one stream
    and one workspace, gives what each gives alone."""
    cases = [Case(40, 272, 512, 128, 4, 3, 16, "mixed", seed=31), Case(700, 1040, 1088, 64, 3, 6, 40, "holes", seed=32),
             Case(333, 1024, 2048, 128, 4, 5, 8, "mixed", seed=33), Case(2011, 2112, 1024, 64, 4, 1, 16, "null", seed=34),
             Case(3, 528, 1024, 128, 4, 2, 24, "mixed", seed=35)]
    packed, us = [c.packed() for c in cases], [inner(c) for c in cases]

    def step(i, ws):
        c = cases[i]
        args = (packed[i], *c.shape(), c.a, c.b, c.scale, c.ids)
        y = a4.any4_linear_lora(c.x, *args, bits=c.bits, workspace=ws)
        return y, *a4.any4_linear_lora_grad(c.dy, c.x, us[i], *args, bits=c.bits, workspace=ws)

    def space(c, size):
        return size(c.m, *c.shape(), c.adapters, c.rank, bits=c.bits)

    need = max(max(space(c, a4.any4_lora_workspace_bytes), space(c, a4.any4_lora_grad_workspace_bytes)) for c in cases)
    alone = []
    for i in range(len(cases)):
        alone.append(step(i, torch.zeros(need, dtype=torch.uint8, device="cuda")))
        torch.cuda.synchronize()
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    order = [i for a in range(len(cases)) for b in range(len(cases)) for i in (a, b)]
    outs = [step(i, ws) for i in order]
    torch.cuda.synchronize()
    for i, out in zip(order, outs):
        assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(out, alone[i]))
    assert not bool(ws[:a4.lib.any4_lora_header_bytes()].any())


@pytest.mark.parametrize("shape", [(7, 272, 1024, 128, 4, 3, 64, "mixed"), (190, 1040, 1024, 128, 4, 24, 32, "mixed"),
                                   (700, 1040, 1088, 64, 3, 6, 40, "holes"), (2011, 2112, 2048, 128, 4, 1, 16, "null"),
                                   (333, 1024, 4096, 128, 4, 5, 8, "mixed")], ids=str)
def test_what_follows_on_the_stream_may_overwrite_everything(shape):
    """The kernels of a call run beside each other, and the call is over for
    whatever follows it on its stream: inputs, weight and workspace change
    right behind it, and the results are those of the inputs before."""
    c = Case(*shape, seed=41)
    packed, u = c.packed(), inner(c)
    args = (packed, *c.shape(), c.a, c.b, c.scale, c.ids)
    need = max(f(c.m, *c.shape(), c.adapters, c.rank, bits=c.bits)
               for f in (a4.any4_lora_workspace_bytes, a4.any4_lora_grad_workspace_bytes))
    header = a4.lib.any4_lora_header_bytes()
    want = (forward(c), *grads(c, u=u))
    inputs = [t for t in (c.x, c.dy, u, packed, c.a, c.b, c.scale, c.ids) if t is not None]
    kept = [t.clone() for t in inputs]
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def spoil():
        for t in inputs:
            t.view(torch.uint8).fill_(0xFF)
        ws[header:] = 0xFF

    torch.cuda.synchronize()
    for _ in range(4):
        y = a4.any4_linear_lora(c.x, *args, bits=c.bits, workspace=ws)
        spoil()
        for t, k in zip(inputs, kept):
            t.copy_(k)
        got = a4.any4_linear_lora_grad(c.dy, c.x, u, *args, bits=c.bits, workspace=ws)
        spoil()
        for t, k in zip(inputs, kept):
            t.copy_(k)
        torch.cuda.synchronize()
        assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip((y, *got), want))


def test_overlapping_buffers_are_refused():
    c = Case(40, 128, 128, 64, 4, 2, 16, "mixed", seed=42)   # N = K: dx fits where dy lies
    u = inner(c)
    ws = torch.zeros(a4.any4_lora_grad_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank), dtype=torch.uint8,
                     device="cuda")

    def refused(call):
        with pytest.raises(a4.Any4Error) as e:
            call()
        assert e.value.status == a4.ANY4_EINVAL

    inside = ws[-2 * c.m * c.n:].view(torch.bfloat16).view(c.m, c.n)   # in the workspace
    for bad in (dict(dx=c.dy), dict(dx=c.x), dict(da=c.a), dict(db=c.b), dict(dx=inside)):
        refused(lambda: grads(c, u=u, workspace=ws, **bad))
    refused(lambda: forward(c, out=c.x))
    own = torch.zeros(a4.any4_lora_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank), dtype=torch.uint8, device="cuda")
    refused(lambda: forward(c, out=own[-2 * c.m * c.n:].view(torch.bfloat16).view(c.m, c.n), workspace=own))
    refused(lambda: forward(c, u=c.x[:, :16].contiguous(), out=c.x))
    # what the call does not read may be written: x without dA
    want = grads(c, u=u)
    x = c.x.clone()
    dx, da, db = grads(c, kept=x, u=u, dx=x, outputs=("dx", "db"))
    assert da is None and torch.equal(dx, want[0]) and torch.equal(db, want[2])


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import learned_bit_lut_b200 as a4
from lora_util import Case
c = Case({m}, 528, 1024, 128, 4, 3, 16, "mixed", seed=51)
p, args = c.packed(), (*c.shape(), c.a, c.b, c.scale, c.ids)
u = torch.empty(c.m, c.rank, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = a4.any4_linear_lora(c.x, p, *args, u=u)
    kept = a4.any4_act_pack(c.x, 128)
    x = a4.any4_act_unpack(*kept, 128)
    g = a4.any4_linear_lora_grad(c.dy, kept, u, p, *args)
graph.replay()
torch.cuda.synchronize()
again = a4.any4_linear_lora(c.x, p, *args), x, *a4.any4_linear_lora_grad(c.dy, x, u, p, *args)
assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip((y, x, *g), again))
print("captured")
"""


@pytest.mark.parametrize("m", [2, 100, 700])
def test_first_call_of_a_process_is_captured(m):
    """What a call asks the driver once (sizes, how many clusters fit) may be
    asked while a graph is being captured."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests, m=m)
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]

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


# ---- infinities and NaN where one adapter fills a tile, where several share it,
# and in every order of the tokens: the formulas' values

def same(p, q):
    return torch.equal(p.nan_to_num(7.0, 8.0, 9.0), q.nan_to_num(7.0, 8.0, 9.0)) and torch.equal(p.isnan(), q.isnan())


def non_finite(t):
    """One of each kind, far apart, in the first and the last adapter."""
    for l in {0, t.shape[0] - 1}:
        rows, cols = t[l].shape
        t[l, 0, cols // 3], t[l, rows - 1, cols // 2], t[l, rows // 2, 1] = INF, -INF, NAN


ORDERS = ["null", "runs", "last", "holes"]
# fused and dequantized prefill, splits, pairs of blocks; ranks inside, at and over a stage's halves
SPOILT = [(40, 272, 320, 64, 4, 8), (150, 528, 1024, 128, 4, 16), (300, 272, 320, 64, 3, 24), (600, 272, 576, 64, 4, 72),
          (2600, 2320, 2112, 64, 4, 40), (1100, 1040, 4096, 128, 4, 16)]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("m,n,k,g,bits,rank", SPOILT, ids=["m%d_r%d" % (s[0], s[5]) for s in SPOILT])
def test_infinite_adapters(m, n, k, g, bits, rank, order):
    """B in y, A in dx: their products with u and v are +-infinity, not NaN."""
    c = Case(m, n, k, g, bits, 1 if order == "null" else 3, rank, order, seed=71)
    non_finite(c.b)
    y = forward(c)
    check(y, *c.y_ref(), "y")
    assert bool(y.isinf().any())
    if c.ids is not None:   # and the same next to other tokens
        perm = torch.randperm(m, device="cuda")
        other = a4.any4_linear_lora(c.x[perm].contiguous(), c.packed(), *c.shape(), c.a, c.b, c.scale,
                                    c.ids[perm].contiguous(), bits=bits)
        assert same(other, y[perm])
    c = Case(m, n, k, g, bits, c.adapters, rank, order, seed=72)
    non_finite(c.a)
    u = torch.zeros(m, rank, dtype=torch.bfloat16, device="cuda")
    dx = grads(c, u=u, outputs=("dx",))[0]
    check(dx, *c.grad_ref(c.x, u)[0], "dx")
    assert bool(dx.isinf().any())
    if c.ids is not None:
        other = a4.any4_linear_lora_grad(c.dy[perm].contiguous(), None, None, c.packed(), *c.shape(), c.a, c.b, c.scale,
                                         c.ids[perm].contiguous(), bits=bits, outputs=("dx",))[0]
        assert same(other, dx[perm])


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("m,n,k,g,bits,rank", SPOILT, ids=["m%d_r%d" % (s[0], s[5]) for s in SPOILT])
def test_infinite_inputs_of_the_adapters_gradients(m, n, k, g, bits, rank, order):
    """An infinite x[t][k] makes column k of its adapter's dA infinite with the
    signs of v[t], or NaN where two tokens' signs differ; u the same in dB."""
    c = Case(m, n, k, g, bits, 1 if order == "null" else 3, rank, order, seed=73)
    u = inner(c)
    for i, v in enumerate((INF, -INF, INF, NAN)):
        for t in (min(i, m - 1), m - 1 - i):
            c.x[t, 5 + 7 * i] = v
    c.x[m // 2, k - 1] = INF
    u[m // 2, rank - 1], u[m // 3, 0] = -INF, NAN
    got = grads(c, u=u)
    refs = c.grad_ref(c.x, u)
    for name, g_, ref in zip(("dx", "da", "db"), got, refs):
        check(g_, *ref, name)


def test_pairs_of_any_size_meet_an_infinity():
    """u from 2^-140 to 2^120, powers of two (whose bf16 form is exact) among
    them, times an infinite B, in tiles of one adapter and of several."""
    for order in ("null", "holes"):
        c = Case(64, 16, 64, 64, 4, 1, 8, order, seed=74)
        c.x.zero_(), c.a.zero_(), c.b.zero_()
        size = torch.linspace(-132, 120, 64, device="cuda").round()
        c.x[:, 0] = torch.exp2(size.double()).to(torch.bfloat16)
        c.x[1::2, 0] *= -1.0
        c.x[2::4, 0] *= 1.5
        c.a[0, 0, 0], c.a[0, 1, 0] = 1.0, 2.0 ** -8
        c.scale.fill_(1.0)
        c.b[0, 3, 0], c.b[0, 4, 0], c.b[0, 5, 1] = INF, -INF, INF
        y = forward(c)
        x, t = c.x.double(), c.tokens[0]
        assert bool((x[t, 0] != 0).all())
        assert torch.equal(y[t, 3].double(), torch.copysign(torch.full_like(x[t, 0], INF), x[t, 0]))
        assert torch.equal(y[t, 4].double(), torch.copysign(torch.full_like(x[t, 0], INF), -x[t, 0]))
        big = t[x[t, 0].abs() > 2.0 ** -118]   # u = 2^-8 x is a normal number
        assert torch.equal(y[big, 5].double(), torch.copysign(torch.full_like(x[big, 0], INF), x[big, 0]))


# ranks that end inside 16 columns: an infinite input meets A's and B's missing ranks

@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("m,n,k,g,bits,rank", [(40, 272, 320, 64, 4, 8), (40, 272, 320, 64, 4, 16), (300, 272, 320, 64, 3, 24),
                                               (600, 272, 4096, 64, 4, 72), (2600, 2320, 2112, 64, 4, 40)], ids=str)
def test_infinite_inputs_of_the_layer(m, n, k, g, bits, rank, order):
    """x in y and u, dy in dx and (over v) dA: signs by the formulas. A and B
    are made positive, so that u and v of such a token are +-infinity."""
    c = Case(m, n, k, g, bits, 1 if order == "null" else 3, rank, order, seed=75)
    c.a, c.b = c.a.abs() + 2.0 ** -9, c.b.abs() + 2.0 ** -9
    c.a, c.b = c.a.to(torch.bfloat16), c.b.to(torch.bfloat16)
    c.x[0, 3], c.x[m // 2, k - 1], c.x[m - 1, 64], c.x[m - 2, 1] = INF, -INF, INF, NAN
    u = torch.empty(m, rank, dtype=torch.bfloat16, device="cuda")
    y = forward(c, u=u)
    check(u, *c.u_ref(), "u")
    check(y, *c.y_ref(), "y")
    c = Case(m, n, k, g, bits, c.adapters, rank, order, seed=76)
    c.a, c.b = (c.a.abs() + 2.0 ** -9).to(torch.bfloat16), (c.b.abs() + 2.0 ** -9).to(torch.bfloat16)
    c.dy[0, 3], c.dy[m // 2, n - 1], c.dy[m - 1, 15], c.dy[m - 2, 1] = INF, -INF, INF, NAN
    u = inner(c)
    for name, g_, ref in zip(("dx", "da", "db"), grads(c, u=u), c.grad_ref(c.x, u)):
        check(g_, *ref, name)


@pytest.mark.parametrize("m", [13, 40, 300, 600, 2600])
@pytest.mark.parametrize("order", ["null", "holes", "runs"])
def test_infinite_input_and_infinite_adapter_meet(m, order):
    """u (v) and B (A) infinite at the same rank: their product is an infinity
    of their signs, whoever else shares the tile."""
    shape = (2320, 2112, 64) if m == 2600 else (272, 320, 64)
    c = Case(m, *shape, 4, 1 if order == "null" else 3, 24, order, seed=77)
    c.a, c.b = (c.a.abs() + 2.0 ** -9).to(torch.bfloat16), (c.b.abs() + 2.0 ** -9).to(torch.bfloat16)
    c.x[0, 3], c.x[m // 2, 7], c.x[m - 1, 64] = INF, -INF, INF
    c.b[:, 5, 2], c.b[:, 6, 20], c.b[:, 7, 9] = INF, -INF, NAN
    y = forward(c)
    check(y, *c.y_ref(), "y")
    if c.ids is not None:
        perm = torch.randperm(m, device="cuda")
        assert same(a4.any4_linear_lora(c.x[perm].contiguous(), c.packed(), *c.shape(), c.a, c.b, c.scale,
                                        c.ids[perm].contiguous()), y[perm])
    c = Case(m, *shape, 4, c.adapters, 24, order, seed=78)
    c.a, c.b = (c.a.abs() + 2.0 ** -9).to(torch.bfloat16), (c.b.abs() + 2.0 ** -9).to(torch.bfloat16)
    c.dy[0, 3], c.dy[m // 2, 7], c.dy[m - 1, 64] = INF, -INF, INF
    c.a[:, 2, 5], c.a[:, 20, 6], c.a[:, 9, 7] = INF, -INF, NAN
    u = torch.zeros(m, 24, dtype=torch.bfloat16, device="cuda")
    check(grads(c, u=u, outputs=("dx",))[0], *c.grad_ref(c.x, u)[0], "dx")


# ---- checkpoints whose finite steps stand for values that round to infinity

@pytest.mark.parametrize("order", ["mixed", "runs", "null"])
@pytest.mark.parametrize("m", [13, 150, 600])
def test_values_beyond_bf16_of_one_request_reach_no_other(m, order):
    c = Case(m, 272, 320, 64, 4, 1 if order == "null" else 3, 24, order, seed=79)
    top = torch.finfo(torch.bfloat16).max
    spoilt = c.tokens[c.adapters - 1][:2]
    c.x[spoilt[0], 64:70] = torch.tensor([top, -top, top / 2, 1e38, -1e30, 1.0], device="cuda")
    c.x[spoilt[1], 200] = -top
    kept = a4.any4_act_pack(c.x, 64)
    x = a4.any4_act_unpack(*kept, 64)
    assert bool(torch.isfinite(kept[1].float()).all()) and int(x.isinf().sum()) == 3
    u = inner(c)
    got = grads(c, kept, u)
    for name, g, ref in zip(("dx", "da", "db"), got, c.grad_ref(x, u)):
        check(g, *ref, name)
    assert bool(torch.isfinite(got[1][:-1].float()).all())
    # the same from the values, and with every code as the host may hand them over
    plain = grads(c, x, u)
    assert all(same(p, q) for p, q in zip(got, plain))
    codes, steps = kept[0].clone(), kept[1].clone()
    codes[spoilt[0], :64] = torch.arange(-128, -64, dtype=torch.int8, device="cuda")
    steps[spoilt[0], 0] = 2.0 ** 121
    steps[spoilt[1], 1] = -2.0 ** 123
    x = a4.any4_act_unpack(codes, steps, 64)
    assert bool(x.isinf().any())
    got = grads(c, (codes, steps), u, outputs=("da",))
    check(got[1], *c.grad_ref(x, u)[1], "da")


# ---- graphs

@pytest.mark.parametrize("m,n,k", [(1, 1024, 4096), (4, 4096, 2048), (16, 4096, 4096), (40, 1024, 4096), (700, 1024, 4096)])
def test_graphs_of_the_plain_layer_share_no_workspace(m, n, k):
    """Captured without a call before, replayed in another order than captured,
    at the same time, and beside eager calls on the stream of the capture."""
    cases = [Case(m, n, k, 128, 4, 1, 8, "null", seed=s) for s in (81, 82)]
    packed = [c.packed() for c in cases]
    side, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in cases]
    graphs, outs = [], []
    for c, p in zip(cases, packed):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append([a4.any4_linear(c.x, p, *c.shape()) for _ in range(4)])
        graphs.append(g)
    graphs[1].replay()   # the second one first
    torch.cuda.synchronize()
    wants = [a4.any4_linear(c.x, p, *c.shape()) for c, p in zip(cases, packed)]
    assert all(torch.equal(y, wants[1]) for y in outs[1])
    for _ in range(10):
        for ys in outs:
            for y in ys:
                y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, others):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(side):
            eager = [a4.any4_linear(cases[0].x, packed[0], *cases[0].shape()) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for ys, w in zip(outs, wants) for y in ys)
        assert all(torch.equal(y, wants[0]) for y in eager)


def test_one_graph_of_many_calls_clears_one_workspace():
    """Calls of all kinds in one graph, the workspace growing on the way."""
    cases = [Case(3, 528, 1024, 128, 4, 2, 24, "mixed", seed=83), Case(40, 272, 512, 128, 4, 3, 16, "mixed", seed=84),
             Case(700, 1040, 1088, 64, 3, 6, 40, "holes", seed=85), Case(2, 528, 1024, 128, 4, 2, 24, "mixed", seed=86)]
    packed, us = [c.packed() for c in cases], [inner(c) for c in cases]

    def step(i):
        c = cases[i]
        args = (packed[i], *c.shape(), c.a, c.b, c.scale, c.ids)
        return (a4.any4_linear_lora(c.x, *args, bits=c.bits), a4.any4_linear_bits(c.bits, c.x, packed[i], *c.shape()),
                *a4.any4_linear_lora_grad(c.dy, c.x, us[i], *args, bits=c.bits))

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [step(i) for i in (0, 1, 2, 3, 1, 0)]
    wants = [step(i) for i in (0, 1, 2, 3, 1, 0)]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, wants):
            assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(got, want))


def test_status_of_the_kept_workspaces():
    c = Case(700, 528, 1088, 64, 3, 6, 40, "holes", seed=87)
    want = forward(c)
    a4.any4_linear(c.x[:4].contiguous(), Case(4, 528, 1088, 64, 4, 1, 8, "null").packed(), *c.shape())
    assert a4.workspace_status() == 0
    a4.reset_workspaces()
    assert torch.equal(forward(c), want) and a4.workspace_status(torch.device("cuda")) == 0


def test_db_alone_needs_neither_b_nor_scale():
    c = Case(150, 272, 320, 64, 4, 3, 24, "holes", seed=88)
    u = inner(c)
    want = grads(c, u=u, outputs=("db",))[2]
    db, ws = torch.empty_like(want), torch.zeros(
        a4.any4_lora_grad_workspace_bytes(c.m, *c.shape(), c.adapters, c.rank), dtype=torch.uint8, device="cuda")
    assert a4.lib.any4_linear_lora_grad(4, c.dy.data_ptr(), None, None, None, 0, u.data_ptr(), None, c.m, *c.shape(), None,
                                        None, None, c.ids.data_ptr(), c.adapters, c.rank, None, None, db.data_ptr(),
                                        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == a4.ANY4_OK
    assert torch.equal(db, want)
    # b is not read, so it may be what is written
    assert torch.equal(grads(c, u=u, outputs=("db",), db=c.b)[2], want)


# ---- the trailing parts of u and v: with W_hat = 0 and factors that cancel the
# leading parts, y, dx and dA are made of what rounding u and v to bf16 loses

def nothing_of_the_weight(c: Case):
    c.q.alpha[:], c.q.beta[:] = 0, 0
    c._w = None
    return c


def limit_of(ref, bound):
    return bound + 2.0 ** -8 * (ref.abs() + bound) + 1e-37


def without_trailing_part(ref, bound, planted):
    """The planted mistake (u or v rounded to bf16) is well outside the bound."""
    assert float(((planted - ref).abs() > limit_of(ref, bound)).double().mean()) > 0.5


@pytest.mark.parametrize("order", ["null", "mixed"])
@pytest.mark.parametrize("m,rank", [(40, 16), (40, 72), (300, 8), (600, 40)])
def test_trailing_parts_in_y(m, rank, order):
    c = nothing_of_the_weight(Case(m, 272, 64, 64, 4, 1 if order == "null" else 3, rank, order, seed=91))
    c.scale.fill_(1.0)
    c.a[:, 1::2] = c.a[:, 0::2]
    c.a[:, 1::2, 3] += 2.0 ** -6
    c.b[:, :, 1::2] = -c.b[:, :, 0::2]
    ref, bound = c.y_ref()
    u, planted = c.u_ref()[0].to(torch.bfloat16).double(), torch.zeros_like(ref)
    for l, t in enumerate(c.tokens):
        planted[t] = u[t] @ c.b[l].double().T
    without_trailing_part(ref, bound, planted)
    check(forward(c), ref, bound, "y")


@pytest.mark.parametrize("order", ["null", "mixed"])
@pytest.mark.parametrize("m,rank", [(40, 16), (40, 72), (300, 8), (600, 40)])
def test_trailing_parts_in_dx(m, rank, order):
    c = nothing_of_the_weight(Case(m, 64, 320, 64, 4, 1 if order == "null" else 3, rank, order, seed=92))
    c.scale.fill_(1.0)
    c.b[:, :, 1::2] = c.b[:, :, 0::2]
    c.b[:, 3, 1::2] += 2.0 ** -8
    c.a[:, 1::2] = -c.a[:, 0::2]
    u = torch.zeros(m, rank, dtype=torch.bfloat16, device="cuda")
    ref, bound = c.grad_ref(c.x, u)[0]
    v, planted = c.v_ref()[0].to(torch.bfloat16).double(), torch.zeros_like(ref)
    for l, t in enumerate(c.tokens):
        planted[t] = v[t] @ c.a[l].double()
    without_trailing_part(ref, bound, planted)
    check(grads(c, u=u, outputs=("dx",))[0], ref, bound, "dx")


@pytest.mark.parametrize("kept", ["bf16", "8bit"])
@pytest.mark.parametrize("m,adapters,rank", [(8, 1, 16), (40, 10, 16), (600, 150, 8), (130, 33, 72)])
def test_trailing_parts_in_da(m, adapters, rank, kept):
    c = Case(m, 64, 320, 64, 4, adapters, rank, "mixed", seed=93)
    c.scale.fill_(1.0)
    c.ids = torch.arange(m, device="cuda", dtype=torch.int32) // 4 % adapters   # two such pairs of tokens an adapter
    c.tokens = [torch.nonzero(c.ids == l).flatten() for l in range(adapters)]
    c.dy[1::2] = c.dy[0::2]
    c.dy[1::2, 3] += 2.0 ** -9
    c.x[1::2] = -c.x[0::2]
    stored, x = c.x, c.x
    if kept == "8bit":
        stored = a4.any4_act_pack(c.x, 64)
        x = a4.any4_act_unpack(*stored, 64)
    u = torch.zeros(m, rank, dtype=torch.bfloat16, device="cuda")
    ref, bound = c.grad_ref(x, u)[1]
    v, planted = c.v_ref()[0].to(torch.bfloat16).double(), torch.zeros_like(ref)
    for l, t in enumerate(c.tokens):
        planted[l] = v[t].T @ x[t].double()
    without_trailing_part(ref, bound, planted)
    check(grads(c, stored, u, outputs=("da",))[1], ref, bound, "da")


@pytest.mark.parametrize("m", [1, 8, 16, 40])
def test_the_layer_right_behind_its_pack(m):
    from gpu_util import to_dev
    cases = [Case(m, 1024, 2048, 64, 4, 1, 8, "null", seed=s) for s in (94, 95)]
    raw = [tuple(to_dev(t) for t in (c.q.idx_nib, c.q.lut, c.q.alpha, c.q.beta)) for c in cases]
    wants = [a4.any4_linear(cases[0].x, c.packed(), *c.shape()) for c in cases]
    packed, outs = torch.empty_like(cases[0].packed()), []
    for i in range(60):
        a4.any4_pack(*raw[i % 2], 64, packed)
        outs.append(a4.any4_linear(cases[0].x, packed, *cases[0].shape()))
    assert all(torch.equal(y, wants[i % 2]) for i, y in enumerate(outs))


# ---- addresses and sizes at the borders of what is accepted

def at_offset(t, count):
    """A copy of t that starts `count` elements into a buffer."""
    buf = torch.empty(t.numel() + count + 64, dtype=t.dtype, device=t.device)
    view = buf[count:count + t.numel()].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("m,n,k,bits,rank", [(1, 1024, 2048, 4, 16), (7, 272, 1024, 4, 24), (16, 4096, 1024, 4, 8),
                                             (40, 272, 1024, 4, 16), (300, 1040, 512, 4, 72), (600, 272, 320, 3, 8),
                                             (2600, 2320, 2112, 4, 40)])
def test_least_alignment(m, n, k, bits, rank):
    """y on 4 bytes, scales and ids on 4, everything else on 16."""
    c = Case(m, n, k, 64, bits, 3, rank, "holes", seed=96)
    u0 = inner(c)
    want, wants = forward(c), grads(c, u=u0)
    packed = at_offset(c.packed(), 16)
    y = at_offset(torch.zeros_like(want), 2)
    assert y.data_ptr() % 16 == 4
    x, dy, a, b, u = (at_offset(t, 8) for t in (c.x, c.dy, c.a, c.b, u0))
    scale, ids = at_offset(c.scale, 1), at_offset(c.ids, 3)
    size = max(f(m, n, k, 64, 3, rank, bits=bits) for f in (a4.any4_lora_workspace_bytes, a4.any4_lora_grad_workspace_bytes))
    ws = at_offset(torch.zeros(size, dtype=torch.uint8, device="cuda"), 16)
    assert {t.data_ptr() % 32 for t in (x, dy, a, b, u, packed, ws)} == {16}
    got_u = at_offset(torch.zeros_like(u0), 8)
    a4.any4_linear_lora(x, packed, n, k, 64, a, b, scale, ids, bits=bits, out=y, u=got_u, workspace=ws)
    assert torch.equal(y, want)
    outs = {"dx": at_offset(wants[0], 8), "da": at_offset(wants[1], 8), "db": at_offset(wants[2], 8)}
    for t in outs.values():
        t.zero_()
    got = a4.any4_linear_lora_grad(dy, x, u, packed, n, k, 64, a, b, scale, ids, bits=bits, workspace=ws, **outs)
    assert all(torch.equal(p, q) for p, q in zip(got, wants))
    assert status(ws) == 0


def test_as_many_tokens_as_are_accepted():
    m = 1 << 20
    c = Case(m, 16, 64, 64, 4, 5, 8, "holes", seed=97)
    u = torch.empty(m, 8, dtype=torch.bfloat16, device="cuda")
    check(forward(c, u=u), *c.y_ref(), "y")
    check(u, *c.u_ref(), "u")
    for kept in (c.x, a4.any4_act_pack(c.x, 64)):
        x = c.x if kept is c.x else a4.any4_act_unpack(*kept, 64)
        for name, g, ref in zip(("dx", "da", "db"), grads(c, kept, u), c.grad_ref(x, u)):
            check(g, *ref, name)


@pytest.mark.parametrize("m", [5, 300, 1100])
def test_as_many_adapters_as_are_accepted(m):
    """65536 adapters, of which a few have tokens, the first and the last among them."""
    few = Case(m, 48, 64, 64, 4, 4, 8, "mixed", seed=98)
    places = torch.tensor([0, 257, 32768, 65535], device="cuda")
    many = {t: torch.randn(65536, *s, device="cuda").to(d) for t, s, d in (
        ("a", (8, 64), torch.bfloat16), ("b", (48, 8), torch.bfloat16), ("scale", (), torch.float32))}
    for name, t in many.items():
        t[places] = getattr(few, name)
    ids = places[few.ids.long()].to(torch.int32)
    packed, u = few.packed(), inner(few)
    y = a4.any4_linear_lora(few.x, packed, *few.shape(), many["a"], many["b"], many["scale"], ids)
    check(y, *few.y_ref(), "y")
    dx, da, db = a4.any4_linear_lora_grad(few.dy, few.x, u, packed, *few.shape(), many["a"], many["b"], many["scale"], ids)
    for name, g, ref in zip(("dx", "da", "db"), (dx, da[places], db[places]), few.grad_ref(few.x, u)):
        check(g, *ref, name)
    others = torch.ones(65536, dtype=torch.bool, device="cuda")
    others[places] = False
    assert not bool(da[others].any()) and not bool(db[others].any())


# ---- infinities and NaN cost their own sums a little, and no other

@pytest.mark.parametrize("kept", ["bf16", "8bit"])
def test_a_column_of_nan_takes_no_longer_than_its_tokens(kept):
    """2^20 tokens of 2048 mixed adapters: going through all tokens again for
    each adapter and column took half a minute."""
    tokens, adapters, rank, cols, n = 1 << 20, 2048, 64, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(tokens, cols, device="cuda", generator=gen).to(torch.bfloat16)
    x[:, 5] = NAN
    x[7, 9], x[9, 9], x[adapters + 9, 9] = INF, INF, -INF
    dy = torch.randn(tokens, n, device="cuda", generator=gen).to(torch.bfloat16)
    a = torch.zeros(adapters, rank, cols, dtype=torch.bfloat16, device="cuda")
    b = torch.randn(adapters, n, rank, device="cuda", generator=gen).to(torch.bfloat16)
    scale, ids = torch.ones(adapters, device="cuda"), torch.arange(tokens, device="cuda", dtype=torch.int32) % adapters
    u = torch.zeros(tokens, rank, dtype=torch.bfloat16, device="cuda")
    group = 64
    stored = a4.any4_act_pack(x, group) if kept == "8bit" else x
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

    def call():
        return a4.any4_linear_lora_grad(dy, stored, u, None, n, cols, group, a, b, scale, ids, outputs=("da",))[1]

    call()
    start.record()
    da = call()
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 1000.0 and a4.workspace_status() == 0
    xs = (a4.any4_act_unpack(*stored, group) if kept == "8bit" else x).double()
    for l in (0, 7, 9, 1000, adapters - 1):
        t = torch.arange(l, tokens, adapters, device="cuda")
        v = dy[t].double() @ b[l].double()
        ref = v.T @ xs[t]
        bound = (n + 2) * 2.0 ** -23 * (dy[t].double().abs() @ b[l].double().abs()) + 2.0 ** -16 * v.abs()
        bound = bound.T @ xs[t].abs() + (2 * len(t) + 8) * 2.0 ** -23 * (v.abs().T @ xs[t].abs())
        check(da[l], ref, bound, f"da of {l}")


@pytest.mark.parametrize("m,adapters,rank", [(40, 3, 24), (600, 3, 72), (1100, 40, 16), (3000, 5, 8)])
@pytest.mark.parametrize("order", ["mixed", "holes"])
def test_everything_not_finite(m, adapters, rank, order):
    """All of x and dy NaN or infinite for two adapters and for tokens of none."""
    c = Case(m, 272, 320, 64, 4, adapters, rank, order, seed=101)
    for l, v in ((0, NAN), (adapters - 1, INF)):
        c.x[c.tokens[l]], c.dy[c.tokens[l]] = v, v
    others = torch.nonzero((c.ids < 0) | (c.ids >= adapters)).flatten()
    c.x[others], c.dy[others] = NAN, -INF
    u = inner(c)
    for stored in (c.x, a4.any4_act_pack(c.x, 64)):
        x = c.x if stored is c.x else a4.any4_act_unpack(*stored, 64)
        for name, g, ref in zip(("dx", "da", "db"), grads(c, stored, u), c.grad_ref(x, u)):
            check(g, *ref, name)

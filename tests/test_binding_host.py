"""What the binding does on the host around a call: workspaces, locks, sizes and
errors (CPU only: host tensors that say they are on a GPU, and stand-ins for
the library's calls)."""
import threading
import time

import pytest
import torch

from learned_bit_lut_b200 import _lib

N, K, G, RANK = 64, 128, 64, 16
HEADER = _lib.lib.any4_lora_header_bytes()


class OnGpu(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class Host:
    """The state the stand-ins look at."""

    def __init__(self):
        self.stream = threading.local()
        self.capturing, self.capture = False, 0
        self.need = HEADER + 4096
        self.calls = []
        self.during = lambda name, args: None   # what happens inside a library call

    def library_call(self, name):
        def call(*args):
            self.calls.append((name, args))
            self.during(name, args)
            return 0
        return call


@pytest.fixture
def host(monkeypatch):
    h = Host()
    plain = torch.empty

    def empty(*shape, dtype=None, device=None):
        t = plain(*shape, dtype=dtype)
        t.view(torch.uint8).fill_(0xA5)   # not zero by chance
        return t.as_subclass(OnGpu)

    monkeypatch.setattr(torch, "empty", empty)
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *s, dtype=None, device=None: zeros(*s, dtype=dtype).as_subclass(OnGpu))
    monkeypatch.setattr(_lib, "_stream", lambda device: getattr(h.stream, "at", 7))
    monkeypatch.setattr(_lib, "_stream_of", lambda t: getattr(h.stream, "at", 7))
    monkeypatch.setattr(_lib, "_capturing", lambda: h.capturing)
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    for name in ("any4_lora_workspace_bytes", "any4_lora_grad_workspace_bytes", "any4_linear_workspace_bytes_bits"):
        monkeypatch.setattr(_lib.lib, name, lambda *a: h.need)
    for name in ("any4_linear_lora", "any4_linear_lora_grad", "any4_linear", "any4_linear_bits"):
        monkeypatch.setattr(_lib.lib, name, h.library_call(name))
    def capture_id(stream, out):
        out._obj.value = h.capture if h.capturing else 0
        return 0

    monkeypatch.setattr(_lib.lib, "any4_stream_capture_id", capture_id)
    for cache in ("_WORKSPACES", "_KEPT", "_GRAPH_WORKSPACES"):
        if hasattr(_lib, cache):
            monkeypatch.setattr(_lib, cache, {})
    for size in (_lib._linear_need, _lib._lora_need, _lib._grad_need):
        size.cache_clear()
    yield h
    for size in (_lib._linear_need, _lib._lora_need, _lib._grad_need):
        size.cache_clear()


@pytest.mark.parametrize("name", ["lora", "grad", "linear", "decode"])
def test_a_device_that_cannot_be_asked_is_not_a_shape(host, monkeypatch, name):
    """A size of 0 is told apart, and asked for again by the next call."""
    ask = lambda: call("linear", m=1) if name == "decode" else call(name)   # noqa: E731
    host.need = 0
    monkeypatch.setattr(_lib.lib, "any4_linear_kernel", lambda *a: _lib.ANY4_ECUDA)
    with pytest.raises(_lib.Any4Error) as e:
        ask()
    assert e.value.status == _lib.ANY4_ECUDA
    monkeypatch.setattr(_lib.lib, "any4_linear_kernel", lambda *a: _lib.ANY4_ESHAPE)
    with pytest.raises(_lib.Any4Error) as e:
        ask()
    assert e.value.status == _lib.ANY4_ESHAPE
    host.need = HEADER + 4096
    ask()
    assert len(host.calls) == 1


PACKED_BYTES = _lib.lib.any4_packed_bytes(N, K, G)


def call(name, m=40, workspace=None):
    x, packed = on_gpu(m, K), on_gpu(PACKED_BYTES, dtype=torch.uint8)
    if name == "linear":
        return _lib.any4_linear(x, packed, N, K, G, workspace=workspace)
    if name == "linear_bits":
        return _lib.any4_linear_bits(4, x, packed, N, K, G, workspace=workspace)
    a, b, scale = on_gpu(2, RANK, K), on_gpu(2, N, RANK), on_gpu(2, dtype=torch.float32)
    if name == "lora":
        return _lib.any4_linear_lora(x, packed, N, K, G, a, b, scale, workspace=workspace)
    return _lib.any4_linear_lora_grad(on_gpu(m, N), x, on_gpu(m, RANK), packed, N, K, G, a, b, scale, workspace=workspace)


def run_threads(*jobs):
    errors = []

    def guard(job):
        try:
            job()
        except BaseException as e:   # noqa: BLE001  (reported below)
            errors.append(e)

    threads = [threading.Thread(target=guard, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert not any(t.is_alive() for t in threads) and not errors, errors


@pytest.mark.parametrize("pair", [("lora", "lora"), ("lora", "grad"), ("grad", "linear"), ("linear", "linear_bits")], ids=str)
def test_calls_of_two_threads_on_one_stream_do_not_mix_their_launches(host, pair):
    """A call's kernels hand each other results in its workspace, and the
    interpreter lock is open while the library launches them."""
    inside, most = [], []

    def during(name, args):
        inside.append(name)
        most.append(len(inside))
        time.sleep(0.002)
        inside.remove(name)

    host.during = during
    run_threads(*[lambda name=name: [call(name) for _ in range(10)] for name in pair])
    assert len(host.calls) == 20 and max(most) == 1


def test_threads_on_their_own_streams_do_not_wait_for_each_other(host):
    both = threading.Barrier(2)
    host.during = lambda name, args: both.wait(10)   # each call is inside while the other is

    def job(stream):
        host.stream.at = stream
        for _ in range(5):
            call("lora")

    run_threads(lambda: job(1), lambda: job(2))


# ---- workspaces of captured calls

def test_capture_id_needs_a_place_for_it():
    assert _lib.lib.any4_stream_capture_id(None, None) == _lib.ANY4_EINVAL

WORKSPACE_AT = {"any4_linear_lora": -3, "any4_linear_lora_grad": -3, "any4_linear": -3, "any4_linear_bits": -3}


def used(host):
    """Addresses of the workspaces of the calls so far."""
    return [args[WORKSPACE_AT[name]] for name, args in host.calls]


KINDS = ["lora", "grad", "linear", "linear_bits", "decode"]


def make(name):
    return call("linear", m=4) if name == "decode" else call(name)


@pytest.mark.parametrize("warm", [False, True])
@pytest.mark.parametrize("name", KINDS)
def test_a_graph_has_a_workspace_of_its_own(host, monkeypatch, name, warm):
    """Not the stream's, which eager calls use beside a replay and which is freed
    when it grows, nor another graph's; and it is not left to eager calls,
    for which nothing has cleared it."""
    held = []   # no address is used twice by chance
    zeroed = _lib._zeroed
    monkeypatch.setattr(_lib, "_zeroed", lambda *a: held.append(zeroed(*a)) or held[-1])
    if warm:
        make(name)
    host.capturing, host.capture = True, 11
    make(name), make(name)
    host.capture = 12
    make(name)
    host.capturing = False
    make(name), make(name)
    at = used(host)[1:] if warm else used(host)
    first, again, other, eager, later = at
    assert first == again and eager == later and len({first, other, eager}) == 3
    assert not warm or used(host)[0] == eager
    assert not _lib._GRAPH_WORKSPACES   # graphs keep their memory themselves


@pytest.mark.parametrize("name", KINDS)
def test_a_graph_clears_its_workspace_before_the_first_call(host, name):
    seen = []

    def during(call_name, args):
        at = args[WORKSPACE_AT[call_name]]
        ws = next(w for _, w in _lib._GRAPH_WORKSPACES.values() if w.data_ptr() == at)
        seen.append(int(ws[:HEADER].max()))

    host.during, host.capturing, host.capture = during, True, 5
    make(name)
    host.need += 8192   # a larger call of the same graph
    for size in (_lib._linear_need, _lib._lora_need, _lib._grad_need):
        size.cache_clear()
    make(name)
    assert seen == [0, 0] and len(set(used(host))) == 2


def test_calls_of_several_kernels_share_the_stream_s_workspace(host):
    """It may hold a whole dequantized weight, once; decode calls, which take no
    lock, have a small one of their own."""
    for name in ("linear", "lora", "grad", "linear_bits", "decode", "lora"):
        make(name)
    at = used(host)
    assert len({at[i] for i in (0, 1, 2, 3, 5)}) == 1 and at[4] != at[0]
    host.stream.at = 8
    make("linear")
    assert used(host)[-1] not in at


# ---- after a wait that gave up

@pytest.mark.parametrize("name", KINDS)
def test_a_call_that_gave_up_is_seen_and_mended(host, monkeypatch, name):
    """The kernels leave the status word set and counters behind, in a workspace
    that the caller cannot see."""
    import learned_bit_lut_b200 as a4
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: None)
    dev = torch.device("cuda", 0)
    assert a4.workspace_status(dev) == 0
    make(name)
    host.stream.at = 9
    make("lora")
    assert a4.workspace_status(dev) == 0
    broken = used(host)[0]
    ws = next(w for w in _lib._workspaces_of(dev) if w.data_ptr() == broken)
    ws[65536 * 4], ws[12] = 1, 3
    assert a4.workspace_status(dev) == 1 and a4.workspace_status(torch.device("cuda", 1)) == 0
    a4.reset_workspaces(torch.device("cuda", 1))
    assert a4.workspace_status(dev) == 1
    a4.reset_workspaces(dev)
    assert a4.workspace_status(dev) == 0 and not bool(ws[:HEADER].any())
    host.stream.at = 7
    make(name)
    assert used(host)[-1] == broken


def test_workspaces_made_in_inference_mode_are_reset_outside_it(host, monkeypatch):
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: None)
    dev = torch.device("cuda", 0)
    with torch.inference_mode():
        for name in KINDS:
            make(name)
        for ws in _lib._workspaces_of(dev):
            ws[65536 * 4] = 1
    _lib.reset_workspaces(dev)
    assert _lib.workspace_status(dev) == 0
    for name in KINDS:
        make(name)

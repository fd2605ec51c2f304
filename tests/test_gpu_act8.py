"""8-bit activation checkpoints on the GPU: codes, steps and values equal the
definition's in 64 bits exactly, at every group size, for values next to the
code borders, tiny and huge groups, zeros, infinities and NaN."""
import pytest
import torch

import learned_bit_lut_b200 as a4
from gpu_util import require_gpu
from lora_util import guarded

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)


def pack_ref(x: torch.Tensor, group: int):
    """The definition in float64: (codes, steps); exact for bf16 inputs."""
    m, k = x.shape
    v = x.to(F64).view(m, k // group, group)
    finite = torch.isfinite(v).all(-1)
    top = torch.where(finite, v.abs().amax(-1), 0.0)
    # smallest bf16 no less than top / 127: 8 significant bits, or steps of 2^-133 below 2^-126
    mant, expo = torch.frexp(top / 127.0)
    unit = torch.ldexp(torch.ones_like(top), torch.clamp(expo - 8, min=-133))
    step = torch.ceil(top / 127.0 / unit) * unit
    codes = torch.where((step > 0)[..., None], torch.round(v / step.clamp_min(1e-300)[..., None]), 0.0)
    codes = torch.where(finite[..., None], codes, 0.0)
    step = torch.where(finite, step, float("nan"))
    return codes.view(m, k) + 0.0, step   # a code has one zero


def check(x, group):
    codes, steps = a4.any4_act_pack(x, group)
    back = a4.any4_act_unpack(codes, steps, group)
    c, s = pack_ref(x, group)
    assert torch.equal(steps.to(F64).nan_to_num(-1.0), s.nan_to_num(-1.0))
    assert torch.equal(codes.to(F64), c)
    want = (c.view(*s.shape, group) * s[..., None]).view_as(x).to(torch.bfloat16)
    assert torch.equal(back.view(torch.int16)[~want.isnan()], want.view(torch.int16)[~want.isnan()])
    assert torch.equal(back.isnan(), want.isnan())


@pytest.mark.parametrize("m,k,group", [(1, 64, 64), (1, 1024, 1024), (3, 192, 64), (37, 4096, 64), (5, 1280, 128),
                                       (7, 768, 256), (2, 1536, 512), (9, 5 * 1024, 1024), (129, 14336, 128),
                                       (1, 14336, 512), (611, 320, 64)])
def test_equals_the_definition(m, k, group):
    g = torch.Generator(device="cuda").manual_seed(m + k)
    x = torch.randn(m, k, generator=g, device="cuda") * torch.exp(2.0 * torch.randn(m, 1, generator=g, device="cuda"))
    check(x.to(torch.bfloat16), group)


def test_every_magnitude_and_exact_halves():
    # all finite bf16 magnitudes, each group led by its own maximum: quotients on and next to every border
    bits = torch.arange(0, 0x7F80, dtype=torch.int32, device="cuda")
    top = bits.view(-1, 1).expand(-1, 64)
    below = torch.arange(64, device="cuda", dtype=torch.int32) * 9
    x = (top - below).clamp_min(0)
    x[:, 1::2] |= 0x8000
    check(x.to(torch.int16).view(torch.bfloat16).contiguous(), 64)
    # 2 (c + 1/2) step with step = 2^-7: exact ties for every code
    ties = torch.arange(-127, 128, dtype=torch.float32, device="cuda") + 0.5
    rows = torch.zeros(4, 64, device="cuda")
    rows.view(-1)[:254] = ties[:254].clamp(-127, 127)
    rows[:, 63] = 127.0
    check((rows * 2.0 ** -7).to(torch.bfloat16), 64)


def test_zero_tiny_huge_and_non_finite_groups():
    x = torch.randn(12, 256, device="cuda")
    x[0] = 0.0
    x[1] *= 1e-38
    x[2] = 0.0
    x[2, 5] = 9.2e-41        # the smallest bf16 subnormal
    x[3] *= 1e38
    x[4, 70] = float("inf")
    x[5, 0] = float("-inf")
    x[6, 255] = float("nan")
    x[7, :64] = -0.0
    x[8] *= 2.0 ** -119      # steps around the border of the divided form
    x[9] *= 2.0 ** -126
    x[10] = 3.3895313892515355e38
    x[11, 3] = -3.3895313892515355e38
    for group in (64, 128, 256):
        check(x.to(torch.bfloat16), group)


def test_outputs_stay_within_their_buffers_and_repeat():
    x = torch.randn(33, 320, device="cuda").to(torch.bfloat16)
    codes, c_ok = guarded((33, 320), torch.int8)
    steps, s_ok = guarded((33, 5))
    out, o_ok = guarded((33, 320))
    a4.any4_act_pack(x, 64, codes, steps)
    a4.any4_act_unpack(codes, steps, 64, out)
    torch.cuda.synchronize()
    assert c_ok() and s_ok() and o_ok()
    again = a4.any4_act_pack(x, 64)
    assert torch.equal(again[0], codes) and torch.equal(again[1], steps)


def test_on_another_stream_and_in_a_graph():
    x = torch.randn(65, 512, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        codes, steps = a4.any4_act_pack(x, 128)
        back = a4.any4_act_unpack(codes, steps, 128)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c2, s2 = a4.any4_act_pack(x, 128)
        b2 = a4.any4_act_unpack(c2, s2, 128)
    x.mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c2, -codes) and torch.equal(s2, steps * 2) and torch.equal(b2, back * -2)


def test_inputs_at_odd_addresses():
    """x on a 16-byte but not a 32-byte boundary."""
    for group, k in ((64, 320), (128, 4096), (1024, 2048)):
        buf = torch.randn(700 * k + 8, device="cuda").to(torch.bfloat16)
        x = buf[8:].view(700, k)
        assert x.data_ptr() % 32 == 16
        check(x, group)


def test_every_code_at_every_magnitude_of_step():
    """Reading back: all codes, -128 among them, against every kind of step."""
    steps = torch.tensor([0x0000, 0x0001, 0x0007, 0x007F, 0x0080, 0x0133, 0x3F80, 0x3FFF, 0x7AFF, 0x7B00, 0x7BFF, 0x7F7F,
                          0x7F80, 0x7FC0], dtype=torch.int16, device="cuda").view(torch.bfloat16)
    codes = torch.arange(-128, 128, dtype=torch.int8, device="cuda").repeat(len(steps), 1).contiguous()
    got = a4.any4_act_unpack(codes, steps.view(-1, 1).repeat(1, 4).contiguous(), 64)
    want = (codes.to(F64) * steps.to(F64)[:, None]).to(torch.bfloat16)
    assert torch.equal(got.isnan(), want.isnan())
    fine = ~want.isnan()
    assert torch.equal(got[fine].to(F64), want[fine].to(F64))   # values; a zero's sign is not the format's

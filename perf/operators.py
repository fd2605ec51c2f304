"""What is measured of the adapter and checkpoint operators of the any4 linear layer.

Three operators, used together when low-rank adapters are served or trained on
top of a frozen any4 weight:

* ``lora``: the any4 projection with a low-rank adapter per token,
  y[t] = x[t] . W_hat^T + s_l (x[t] . A_l^T) . B_l^T with l = ids[t]
  (no adapter term where ids[t] < 0), and the adapters' inner activation
  u[t] = s_l (x[t] . A_l^T) that a training step keeps;
* ``grad``: the gradients of that layer for the frozen weight: the input's
  dx[t] = dy[t] . W_hat + v[t] . A_l with v[t] = s_l dy[t] . B_l, and for each
  adapter dA_l = sum_t v[t]^T x[t] and dB_l = sum_t dy[t]^T u[t] over its
  tokens; the kept input x is bf16 or an 8-bit checkpoint;
* ``act``: the 8-bit activation checkpoint itself, one bf16 scale per token
  and group of columns: packed, and read back.

``run`` computes them in plain torch operations in 32 bits (``own`` false) or
through this package's entry points (``own`` true).
"""
import math

import torch

own = False

DEV = "cuda"
GROUPS = (64, 128, 256, 512, 1024)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one request decoding through the k/v projection of an 8B model: launch and latency count
        dict(name="lora_decode_kv_m1", op="lora", m=1, n=1024, k=4096, group=128, bits=4, adapters=8, rank=16,
             order="mixed", none=0.0, keep_u=False),
        # 16 requests, each with its own adapter out of 32, through the q/o projection
        dict(name="lora_decode_qo_m16", op="lora", m=16, n=4096, k=4096, group=128, bits=4, adapters=32, rank=16,
             order="mixed", none=0.0, keep_u=False),
        # a ragged decode batch through gate/up, large rank, some requests without an adapter
        dict(name="lora_decode_gate_m7", op="lora", m=7, n=14336, k=4096, group=128, bits=4, adapters=5, rank=64,
             order="mixed", none=0.25, keep_u=False),
        # a mixed serving batch: prompts of several requests side by side and single decoding tokens
        dict(name="lora_batch_qo_m190", op="lora", m=190, n=4096, k=4096, group=128, bits=4, adapters=24, rank=32,
             order="mixed", none=0.1, keep_u=False),
        # the same for 3-bit weights and prompts that lie one after the other
        dict(name="lora_batch_any3_m700", op="lora", m=700, n=4096, k=4096, group=128, bits=3, adapters=6, rank=16,
             order="runs", none=0.1, keep_u=False),
        # forward of a training step, one adapter, the down projection
        dict(name="lora_train_down_m4096", op="lora", m=4096, n=4096, k=14336, group=128, bits=4, adapters=1, rank=64,
             order="runs", none=0.0, keep_u=True),
        # backward of a small ragged step: five adapters trained at once from 8-bit checkpoints
        dict(name="grad_kv_8bit_m333", op="grad", m=333, n=1024, k=4096, group=128, bits=4, adapters=5, rank=8,
             order="mixed", none=0.1, kept="8bit", act_group=128),
        # backward of an ordinary step, one adapter, inputs kept in bf16
        dict(name="grad_qo_bf16_m2011", op="grad", m=2011, n=4096, k=4096, group=128, bits=4, adapters=1, rank=16,
             order="runs", none=0.0, kept="bf16", act_group=128),
        # backward of a long step through gate/up from 8-bit checkpoints: the largest
        dict(name="grad_gate_8bit_m8192", op="grad", m=8192, n=14336, k=4096, group=128, bits=4, adapters=1, rank=64,
             order="runs", none=0.0, kept="8bit", act_group=128),
        # checkpoint of a short ragged batch, and of a long step's widest activation
        dict(name="act_m37", op="act", m=37, k=4096, act_group=64),
        dict(name="act_m8192", op="act", m=8192, k=14336, act_group=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: 1 .. 8192 tokens, 16 .. 14336 rows and 64 ..
    14336 columns in the steps the format allows, every group size, 1 .. 64
    adapters of rank 8 .. 128."""
    op = rng.choice(["lora", "lora", "grad", "grad", "act"])
    group = rng.choice([g for g in GROUPS for _ in range(3 if g == 128 else 1)])
    if rng.random() < 0.4:
        n, k = rng.choice([(4096, 4096), (1024, 4096), (14336, 4096), (4096, 14336)])
    else:
        n = 16 * max(1, _log_int(rng, 4, 896))
        k = group * max(1, _log_int(rng, 1, 14336 // group))
    if k % group:
        group = 128
    m = min(8192, max(1, _log_int(rng, 1, 8192)))
    act_group = rng.choice([g for g in GROUPS if k % g == 0])
    if op == "act":
        return dict(op="act", m=m, k=k, act_group=act_group)
    case = dict(op=op, m=m, n=n, k=k, group=group, bits=rng.choice([4, 4, 4, 3, 2]),
                adapters=1 if rng.random() < 0.3 else _log_int(rng, 2, 64), rank=8 * _log_int(rng, 1, 16),
                order=rng.choice(["mixed", "runs"]), none=rng.choice([0.0, 0.1, 0.5]))
    # no dearer than the largest listed case, in either form (the plain one multiplies with every adapter)
    token = 2 * n * k + 4 * case["adapters"] * case["rank"] * (n + k)
    case["m"] = max(1, min(m, int(2 * 8192 * 14336 * 4096 // token)))
    if op == "lora":
        case["keep_u"] = rng.random() < 0.5
    else:
        case["kept"] = rng.choice(["8bit", "bf16"])
        case["act_group"] = act_group
    return case


# ------------------------------------------------------------------ the inputs

def _inputs(case, seed):
    """What both sides are given, from the seed alone: canonical any4 tensors
    (the recipe of the package's synthetic layers), adapters as they are after
    some training, activations with per-channel scales, ids of the tokens."""
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 11)
    m, k = case["m"], case["k"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = dict(case=case)
    channel = torch.exp(0.5 * normal(k))
    x = (normal(m, k) * channel).to(torch.bfloat16)
    if case["op"] == "act":
        s["x"] = x
        return s
    n, group, adapters, rank = case["n"], case["group"], case["adapters"], case["rank"]
    if case["bits"] == 4:
        s["idx"] = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    else:   # indices below 2^bits, still one nibble each
        top = 1 << case["bits"]
        lo = torch.randint(0, top, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        hi = torch.randint(0, top, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["idx"] = lo | (hi << 4)
    lut = torch.rand(n, 16, generator=g, device=DEV) * 15.0 - 8.0
    s["lut"] = torch.sort(lut, dim=1).values.to(torch.bfloat16)
    s["alpha"] = (0.02 * 8.0 / 15.0 * torch.exp(0.3 * normal(n, k // group))).to(torch.bfloat16)
    s["beta"] = (0.005 * normal(n, k // group)).to(torch.bfloat16)
    s["a"] = (normal(adapters, rank, k) / math.sqrt(k)).to(torch.bfloat16)
    s["b"] = (0.02 * normal(adapters, n, rank)).to(torch.bfloat16)
    s["scale"] = (16.0 / rank) * torch.exp(0.3 * normal(adapters))
    ids = torch.randint(0, adapters, (m,), generator=g, device=DEV)
    if case["order"] == "runs":   # the tokens of one request after the other
        ids = torch.sort(ids).values
    if case["none"] > 0:
        ids = torch.where(torch.rand(m, generator=g, device=DEV) < case["none"], -1, ids)
    s["ids"] = ids.to(torch.int32)
    if case["op"] == "lora":
        s["x"] = x
        return s
    s["dy"] = (0.01 * normal(m, n) * torch.exp(0.5 * normal(m, 1))).to(torch.bfloat16)
    # what the forward kept: the adapters' inner activation and the input
    s["u"] = _select(x.float() @ s["a"].float().flatten(0, 1).T, s["ids"], s["scale"]).sum(1).to(torch.bfloat16)
    if case["kept"] == "8bit":
        s["codes"], s["steps"] = _pack8(x, case["act_group"])
    else:
        s["x"] = x
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] != "act":   # the device layout of the weight, laid out once when a model is loaded
        import learned_bit_lut_b200 as a4
        s["packed"] = a4.any4_pack_bits(case["bits"], s["idx"], s["lut"], s["alpha"], s["beta"], case["group"])
    return s


# -------------------------------------------------------------- the plain form

def _dequant(s):
    """W_hat (N x K) in fp32: fma(alpha, LUT[idx], beta) rounded to bf16. The
    product of two bf16 values is exact in fp32, so product and sum round once."""
    idx, case = s["idx"], s["case"]
    n, k = case["n"], case["k"]
    at = torch.stack((idx & 15, idx >> 4), dim=-1).view(n, k)
    w = torch.gather(s["lut"].float(), 1, at.long()).view(n, k // case["group"], case["group"])
    w = w * s["alpha"].float()[:, :, None] + s["beta"].float()[:, :, None]
    return w.to(torch.bfloat16).float().view(n, k)


def _select(every, ids, scale):
    """[M, L * R] products with all adapters -> [M, L, R], each token's own
    adapter scaled and zeros for the others."""
    adapters = scale.numel()
    mine = ids[:, None] == torch.arange(adapters, device=ids.device, dtype=ids.dtype)
    return every.view(every.shape[0], adapters, -1) * (mine * scale)[:, :, None]


def _pack8(x, group):
    """Codes -127 .. 127 and one bf16 step per token and group: the largest
    magnitude over 127, rounded up to bf16; zero steps for groups of zeros, NaN
    for groups that hold an infinity or a NaN."""
    m, k = x.shape
    v = x.float().view(m, k // group, group)
    top = v.abs().amax(-1, keepdim=True)
    step = (((top.double() / 127.0).float().view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
    step = torch.where(torch.isfinite(top), step, float("nan"))
    codes = torch.where(step > 0, torch.round(v / step), 0.0).clamp(-127, 127).to(torch.int8)
    return codes.view(m, k), step.to(torch.bfloat16).view(m, k // group)


def _unpack8(codes, steps):
    """The value a code stands for: code * step, rounded to bf16."""
    m, k = codes.shape
    v = codes.float().view(m, steps.shape[1], -1) * steps.float()[:, :, None]
    return v.view(m, k).to(torch.bfloat16)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "act":
        codes, steps = _pack8(s["x"], case["act_group"])
        return {"x": _unpack8(codes, steps), "steps": steps}
    w = _dequant(s)
    a, b = s["a"].float(), s["b"].float()
    flat_a = a.flatten(0, 1)                           # [L * R, K]
    flat_b = b.permute(0, 2, 1).flatten(0, 1)          # [L * R, N]
    if case["op"] == "lora":
        x = s["x"].float()
        u = _select(x @ flat_a.T, s["ids"], s["scale"])
        out = {"y": (x @ w.T + u.flatten(1) @ flat_b).to(torch.bfloat16)}
        if case["keep_u"]:
            out["u"] = u.sum(1).to(torch.bfloat16)
        return out
    dy = s["dy"].float()
    x = (_unpack8(s["codes"], s["steps"]) if case["kept"] == "8bit" else s["x"]).float()
    v = _select(dy @ flat_b.T, s["ids"], s["scale"]).flatten(1)
    mine = s["ids"][:, None] == torch.arange(case["adapters"], device=DEV, dtype=torch.int32)
    u = (s["u"].float()[:, None, :] * mine[:, :, None]).flatten(1)
    return {
        "dx": (dy @ w + v @ flat_a).to(torch.bfloat16),
        "da": (v.T @ x).to(torch.bfloat16).view_as(s["a"]),
        "db": (u.T @ dy).to(torch.bfloat16).view(case["adapters"], case["rank"], -1).permute(0, 2, 1).contiguous(),
    }


# ------------------------------------------------------------------- a user's calls

def _run_own(s):
    import learned_bit_lut_b200 as a4
    case = s["case"]
    if case["op"] == "act":
        codes, steps = a4.any4_act_pack(s["x"], case["act_group"])
        return {"x": a4.any4_act_unpack(codes, steps, case["act_group"]), "steps": steps}
    shape = (case["n"], case["k"], case["group"])
    if case["op"] == "lora":
        if not case["keep_u"]:
            return {"y": a4.any4_linear_lora(s["x"], s["packed"], *shape, s["a"], s["b"], s["scale"], s["ids"],
                                             bits=case["bits"])}
        u = torch.empty(case["m"], case["rank"], dtype=torch.bfloat16, device=DEV)
        y = a4.any4_linear_lora(s["x"], s["packed"], *shape, s["a"], s["b"], s["scale"], s["ids"],
                                bits=case["bits"], u=u)
        return {"y": y, "u": u}
    kept = (s["codes"], s["steps"]) if case["kept"] == "8bit" else s["x"]
    dx, da, db = a4.any4_linear_lora_grad(s["dy"], kept, s["u"], s["packed"], *shape, s["a"], s["b"], s["scale"],
                                          s["ids"], bits=case["bits"])
    return {"dx": dx, "da": da, "db": db}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work and exact values

def work(case):
    m, k = case["m"], case["k"]
    if case["op"] == "act":   # x in, codes and steps kept, the values out
        return {"bytes": m * k * 5 + m * (k // case["act_group"]) * 2, "flops": 4 * m * k}
    n, rank = case["n"], case["rank"]
    used = min(case["adapters"], m)
    weight = n * k * case["bits"] // 8 + 32 * n + 4 * n * (k // case["group"])
    adapters = used * (rank * (n + k) * 2 + 4) + 4 * m
    if case["op"] == "lora":
        kept = 2 * m * rank if case["keep_u"] else 0
        return {"bytes": weight + adapters + 2 * m * k + 2 * m * n + kept,
                "flops": 2 * m * n * k + 2 * m * rank * (n + k)}
    x = m * k + 2 * m * (k // case["act_group"]) if case["kept"] == "8bit" else 2 * m * k
    grads = case["adapters"] * rank * (n + k) * 2
    return {"bytes": weight + adapters + x + 2 * m * n + 2 * m * k + 2 * m * rank + grads,
            "flops": 2 * m * n * k + 4 * m * rank * (n + k)}


def exact(case, seed):
    """The same results from the definitions in 64 bits, adapter by adapter
    over its own tokens."""
    s = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "act":
        m, k, group = case["m"], case["k"], case["act_group"]
        x = s["x"].to(f64).reshape(m, -1, group)
        peak = x.abs().max(dim=2).values
        # the smallest bf16 number (8 significant bits) that is no less than peak / 127
        mant, expo = torch.frexp(peak / 127.0)
        step = torch.ldexp(torch.ceil(mant * 256.0) / 256.0, expo)
        code = torch.where(step[..., None] > 0, (x / step[..., None].clamp_min(1e-300)).round(), 0.0)
        return {"x": (code * step[..., None]).reshape(m, k), "steps": step}
    n, k, group = case["n"], case["k"], case["group"]
    nib = torch.empty(n, k, dtype=torch.int64, device=DEV)
    nib[:, 0::2], nib[:, 1::2] = s["idx"].long() % 16, s["idx"].long() // 16
    w = s["lut"].to(f64)[torch.arange(n, device=DEV)[:, None], nib]
    w = w * s["alpha"].to(f64).repeat_interleave(group, 1) + s["beta"].to(f64).repeat_interleave(group, 1)
    w = w.to(torch.float32).to(torch.bfloat16).to(f64)   # the format's own rounding of a weight
    del nib
    a, b, scale, ids = s["a"].to(f64), s["b"].to(f64), s["scale"].to(f64), s["ids"].long()
    if case["op"] == "lora":
        x = s["x"].to(f64)
        y = x @ w.T
        u = torch.zeros(case["m"], case["rank"], dtype=f64, device=DEV)
        for l in range(case["adapters"]):
            t = torch.nonzero(ids == l).flatten()
            u[t] = scale[l] * (x[t] @ a[l].T)
            y[t] += u[t] @ b[l].T
        return {"y": y, "u": u} if case["keep_u"] else {"y": y}
    dy = s["dy"].to(f64)
    if case["kept"] == "8bit":
        x = s["codes"].to(f64) * s["steps"].to(f64).repeat_interleave(case["act_group"], 1)
        x = x.to(torch.bfloat16).to(f64)   # the value a code stands for
    else:
        x = s["x"].to(f64)
    u = s["u"].to(f64)
    dx, da, db = dy @ w, torch.zeros_like(a), torch.zeros_like(b)
    for l in range(case["adapters"]):
        t = torch.nonzero(ids == l).flatten()
        v = scale[l] * (dy[t] @ b[l])
        dx[t] += v @ a[l]
        da[l] = v.T @ x[t]
        db[l] = dy[t].T @ u[t]
    return {"dx": dx, "da": da, "db": db}

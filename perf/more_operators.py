"""Moments in 8 bits and gradient dropout, at the sizes this library meets:
AdamW on a state that is read back and quantised again by every step, the
quantising and the reading back by themselves, and the two ends of an exchange
that sends one element of each group, chosen by a counter-based generator.

With `own` false every operator runs in its plain form (elementary torch
operations, 32 bits; the random numbers in whole numbers, a scaling by a power
of two in 64 bits where 32 would round it away); with `own` true through the
library's entry points. `exact` gives the same results from the definitions in
64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}
BLOCK = 32                                   # elements that share an exponent
TOP = {"e4m3": 15, "ue5m3": 31}              # largest exponent field of a code
LEAST = {"e4m3": 0, "ue5m3": 11}             # least exponent byte
NOT_FINITE = {"e4m3": 0x7F, "ue5m3": 0xFF}
TAG_STATE, TAG_DROPOUT = 1, 2                # the generator's streams
SHARD = 842301440                            # the 7B shape's Stage-1 shard at 8 ranks
LAYER = 202375168                            # one decoder layer of it


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the tiny shard, fp16 under a loss scale: latency
        {"name": "step tiny fp16", "op": "step", "n": 733953, "grads": "fp16", "params": "fp16", "second": "ue5m3"},
        # the 7B shape's shard, bf16 training
        {"name": "step 7B shard", "op": "step", "n": SHARD, "grads": "bf16", "params": "bf16", "second": "ue5m3"},
        # accumulated fp32 grads, a second moment of 16 bits (beta2 near 1), a length that ends inside a block
        {"name": "step fp32 ragged bf16 v", "op": "step", "n": 45088771, "grads": "fp32", "params": "bf16",
         "second": "bf16"},
        # a running fp32 first moment taken over into 8 bits, and read back
        {"name": "quantise 7B layer", "op": "quantise", "n": LAYER, "format": "e4m3", "random": True},
        # a resumed second moment, to the nearest code
        {"name": "quantise ragged nearest", "op": "quantise", "n": 45088771, "format": "ue5m3", "random": False},
        # the first moment of a small shard for a look at it
        {"name": "read back tiny", "op": "read", "n": 733953, "format": "e4m3", "to": "fp32"},
        # the shard's second moment for a checkpoint
        {"name": "read back 7B shard", "op": "read", "n": SHARD, "format": "ue5m3", "to": "fp32"},
        # small fp16 grads, one in four sent
        {"name": "compress tiny fp16", "op": "compress", "n": 733953, "x": "fp16", "values": "fp16", "ratio": 4,
         "feedback": True},
        # the shard's bf16 grads, one in sixteen sent
        {"name": "compress 7B shard", "op": "compress", "n": SHARD, "x": "bf16", "values": "bf16", "ratio": 16,
         "feedback": True},
        # fp32 grads, every other one, no feedback (unbiased by itself)
        {"name": "compress ragged no feedback", "op": "compress", "n": 45088771, "x": "fp32", "values": "fp32",
         "ratio": 2, "feedback": False},
        # eight ranks' messages into the shard's gradient
        {"name": "decompress 8 peers", "op": "decompress", "n": SHARD, "values": "bf16", "to": "fp32", "ratio": 8,
         "peers": 8, "add": False},
        # a sparse message added to an accumulator
        {"name": "decompress add ragged", "op": "decompress", "n": 45088771, "values": "fp32", "to": "fp32",
         "ratio": 64, "peers": 2, "add": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: any operator, sizes spread over their logarithm."""
    op = rng.choice(("step", "step", "quantise", "read", "compress", "decompress"))
    case = {"op": op, "n": _log(rng, 2000, 300_000_000)}
    if op == "step":
        return {**case, "grads": rng.choice(("fp16", "bf16", "fp32")), "params": rng.choice(("fp16", "bf16")),
                "second": rng.choice(("ue5m3", "ue5m3", "bf16"))}
    if op == "quantise":
        return {**case, "format": rng.choice(("e4m3", "ue5m3", "bf16")), "random": rng.random() < 0.6}
    if op == "read":
        return {**case, "format": rng.choice(("e4m3", "ue5m3", "bf16")), "to": rng.choice(("fp32", "fp32", "bf16"))}
    ratio = 2 ** rng.randint(1, 8)
    if op == "compress":
        return {**case, "x": rng.choice(("fp16", "bf16", "fp32")), "values": rng.choice(("fp16", "bf16", "fp32")),
                "ratio": ratio, "feedback": rng.random() < 0.8}
    values = rng.choice(("fp16", "bf16", "fp32"))
    to = rng.choice((values, "fp32"))
    return {**case, "values": values, "to": to, "ratio": ratio, "peers": rng.randint(1, 16),
            "add": to == "fp32" and rng.random() < 0.4}


# ------------------------------------------------------------------ random numbers

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85
LOW = 0xFFFFFFFF


def _philox(first, count, step, tag, seed):
    """The four 32-bit words of calls first .. first + count - 1 of
    Philox4x32-10, (count, 4) in 64-bit whole numbers."""
    at = torch.arange(first, first + count, dtype=torch.int64, device="cuda")
    c = [at & LOW, at >> 32, torch.full_like(at, step), torch.full_like(at, tag)]
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        p0, p1 = c[0] * M0, c[2] * M1
        c = [((p1 >> 32) & LOW) ^ c[1] ^ k0, p1 & LOW, ((p0 >> 32) & LOW) ^ c[3] ^ k1, p0 & LOW]
        k0, k1 = (k0 + W0) & LOW, (k1 + W1) & LOW
    return torch.stack(c, 1)


def _rounding_bits(n, first, s):
    """16 random bits for each of n elements from flat index `first` (a
    multiple of 8): word (f / 2) % 4 of call f / 8, its half f % 2."""
    words = _philox(first // 8, -(-n // 8), s["step"], TAG_STATE, s["seed"])
    return words.to(torch.int32).view(torch.int16).view(-1)[:n].to(torch.int32) & 0xFFFF


def _kept(n, ratio, first, s):
    """The kept element of every group of `ratio`: its place in the group."""
    j0, groups = first // ratio, -(-n // ratio)
    call = j0 // 16
    words = _philox(call, (j0 + groups - 1) // 16 - call + 1, s["step"], TAG_DROPOUT, s["seed"])
    byte = words.to(torch.int32).view(torch.uint8).view(-1)[j0 - 16 * call:][:groups]
    return byte.to(torch.int64) >> (8 - int(math.log2(ratio)))


# ------------------------------------------------------------------ the formats, plainly

def _bits(x):
    return x.view(torch.int32)


def _pow2(k):
    """2^k in 64 bits, for whole k."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _blocks(x):
    """(blocks, 32) with zeros behind the end."""
    n = x.numel()
    full = -(-n // BLOCK) * BLOCK
    if full != n:
        x = torch.cat([x, torch.zeros(full - n, dtype=x.dtype, device=x.device)])
    return x.view(-1, BLOCK)


def _quantise(x, fmt, r16):
    """(codes, exponent bytes) of fp32 x; r16: 16 random bits an element, or
    None for the nearest code."""
    n = x.numel()
    if fmt != "e4m3" and r16 is not None:
        r16 = (r16 >> 8) | ((r16 & 0xFF) << 8)
    if fmt == "bf16":
        b = _bits(x)
        mag = b & 0x7FFFFFFF
        up = r16 if r16 is not None else 0x7FFF + ((mag >> 16) & 1)
        code = torch.where(mag < 0x7F800000, (mag + up) >> 16, (mag >> 16) | ((mag & 0x7FFFFF) != 0).int() * 0x40)
        code = torch.maximum(code, (mag != 0).int())
        return (code | ((b >> 16) & 0x8000)).to(torch.int16).view(torch.bfloat16), None
    blocks = _blocks(x)
    mag = _bits(blocks.abs())
    exps = ((mag.amax(1).to(torch.int64) + 0x1FFFFF) >> 23).clamp(LEAST[fmt], 255)
    z = _bits((blocks.abs().double() * _pow2(TOP[fmt] - exps)[:, None]).float())
    up = 0x7FFFF + ((z >> 20) & 1) if r16 is None else _blocks(r16) * 16 + 8
    code = (z + up) >> 20
    bad = mag >= 0x7F800000
    if fmt == "ue5m3":
        code = torch.maximum(code, (mag != 0).int())
        bad = bad | (blocks < 0)
    code = torch.where(bad, NOT_FINITE[fmt], code)
    if fmt == "e4m3":
        code = code | ((_bits(blocks) >> 24) & 0x80)
    return code.to(torch.uint8).view(-1)[:n].contiguous(), exps.to(torch.uint8)


def _read(codes, exps, fmt):
    """fp32 values of the codes."""
    if fmt == "bf16":
        return codes.float()
    n = codes.numel()
    c = _blocks(codes).to(torch.int32)
    mag = c & NOT_FINITE[fmt]
    x = (mag << 20).view(torch.float32).double() * _pow2(exps.to(torch.int64) - TOP[fmt])[:, None]
    x = torch.where(mag == NOT_FINITE[fmt], float("nan"), x)
    if fmt == "e4m3":
        x = torch.where(c >= 128, -x, x)
    return x.float().view(-1)[:n]


# ------------------------------------------------------------------ inputs

HP = dict(lr=3e-4, beta1=0.9, eps=1e-8, weight_decay=0.1)
BETA2 = {"ue5m3": 0.95, "bf16": 0.999}
T0 = 200
LOSS_SCALE = {"fp16": 2.0 ** 10, "bf16": 1.0, "fp32": 1.0}
CLIP = 0.8125


def _f32(x):
    return float(np.float32(x))


def _constants(case):
    """The step's fp32 scalars after T0 steps."""
    b1, b2 = _f32(HP["beta1"]), _f32(BETA2[case["second"]])
    lr, wd = _f32(HP["lr"]), _f32(HP["weight_decay"])
    return dict(b1=b1, b2=b2, omb1=_f32(np.float32(1) - np.float32(b1)), omb2=_f32(np.float32(1) - np.float32(b2)),
                eps=_f32(HP["eps"]), step_size=_f32(lr / (1.0 - b1 ** (T0 + 1))),
                bc2=_f32(math.sqrt(1.0 - b2 ** (T0 + 1))), decay=_f32(1.0 - lr * wd),
                gs=_f32(CLIP / LOSS_SCALE[case["grads"]]))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(n, sigma, g):
    return torch.empty(n, device="cuda").normal_(0.0, sigma, generator=g)


def _levels(n, g):
    """A gradient size for every run of 256 elements, over twelve binades;
    some runs, as rows of an embedding that no token met, are zero."""
    runs = -(-n // 256)
    size = torch.exp2(torch.rand(runs, generator=g, device="cuda") * 12 - 18)
    size = torch.where(torch.rand(runs, generator=g, device="cuda") < 0.02, 0.0, size)
    return size[:, None].expand(runs, 256).reshape(-1)[:n]


def _moments(n, g, scale):
    """A first and a second moment as a run of steps leaves them."""
    level = _levels(n, g)
    m = _normal(n, 0.3 * scale, g).mul_(level)
    v = torch.rand(n, generator=g, device="cuda").add_(0.1).square_().mul_(level).mul_(level).mul_(scale * scale)
    return level, m, v


def _inputs(case, seed):
    """The tensors of a case, from its seed alone."""
    g = _gen(seed)
    n = case["n"]
    s = {"case": dict(case), "seed": (int(seed) * 0x9E3779B97F4A7C15 + 0x1234567) & (2 ** 63 - 1),
         "step": 1000 + int(seed) % 1000, "first": 256 * (int(seed) % 40961)}
    op = case["op"]
    if op == "step":
        level, m, v = _moments(n, g, 1.0)
        s["exp_avg"] = _quantise(m, "e4m3", None)
        s["exp_avg_sq"] = _quantise(v, case["second"], None)
        del m, v
        s["grads"] = _normal(n, LOSS_SCALE[case["grads"]], g).mul_(level).to(DTYPES[case["grads"]])
        s["master"] = _normal(n, 0.02, g)
        s["params"] = torch.zeros(n, dtype=DTYPES[case["params"]], device="cuda")
        s["read"] = [torch.empty(n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        s["k"] = _constants(case)
    elif op in ("quantise", "read"):
        _, m, v = _moments(n, g, 1.0)
        x = m if case["format"] == "e4m3" else v
        if op == "quantise":
            s["x"] = x
            s["out"] = torch.empty(n, device="cuda")
        else:
            s["codes"] = _quantise(x, case["format"], None)
            s["out"] = torch.empty(n, dtype=DTYPES[case["to"]], device="cuda")
    elif op == "compress":
        scale = LOSS_SCALE[case["x"]]
        level = _levels(n, g)
        s["scale"] = scale
        s["x"] = _normal(n, scale, g).mul_(level).to(DTYPES[case["x"]])
        s["error"] = _normal(n, 2.0, g).mul_(level) if case["feedback"] else None
        s["values"] = torch.zeros(-(-n // case["ratio"]), dtype=DTYPES[case["values"]], device="cuda")
    else:
        groups = -(-n // case["ratio"])
        s["peers"] = [_normal(groups, 1e-2, g).to(DTYPES[case["values"]]) for _ in range(case["peers"])]
        s["dst"] = _normal(n, 1e-2, g).to(DTYPES[case["to"]]) if case["add"] else torch.zeros(
            n, dtype=DTYPES[case["to"]], device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from zero_sharded_mixed_tensor_amd import zds
        s["state"] = zds.new_state()
        k = s.get("k", {})
        zds.write_scalars(s["state"], zds.StepState(
            scale=s.get("scale", 1.0), window=1000, hysteresis=1, min_scale=1.0, t=T0, steps_seen=s["step"],
            beta1_pow=k.get("b1", 0.9) ** T0, beta2_pow=k.get("b2", 0.9) ** T0))
        s["scalars"] = zds.new_scalars()
        zds.write_scalars(s["scalars"], zds.StepScalars(accum_steps=1, clip_coef=CLIP, grad_scale=k.get("gs", 1.0),
                                                        scale_used=s.get("scale", 1.0)))
        fmts = {"e4m3": zds.ZDS_STATE_E4M3, "ue5m3": zds.ZDS_STATE_UE5M3, "bf16": zds.ZDS_STATE_BF16}
        if case["op"] == "step":
            s["hp"] = zds.hparams(beta2=BETA2[case["second"]], **HP)
            s["m"] = zds.QuantisedState(fmts["e4m3"], *s["exp_avg"])
            s["v"] = zds.QuantisedState(fmts[case["second"]], *s["exp_avg_sq"])
        elif case["op"] == "quantise":
            s["q"] = zds.new_quantised_state(case["n"], fmts[case["format"]])
        elif case["op"] == "read":
            s["q"] = zds.QuantisedState(fmts[case["format"]], *s["codes"])
    return s


# ------------------------------------------------------------------ one pass

def _own_pass(s):
    from zero_sharded_mixed_tensor_amd import zds
    case, key = s["case"], (s["seed"], s["first"])
    op = case["op"]
    if op == "step":
        zds.zds_adam_step_q8(s["hp"], s["grads"], s["master"], s["m"], s["v"], s["params"], *key, s["scalars"],
                             s["state"])
        for q, out in zip((s["m"], s["v"]), s["read"]):
            zds.zds_state_dequantise(q, out)
        return s["master"], s["params"], s["read"][0], s["read"][1]
    if op == "quantise":
        rounding = zds.ZDS_ROUND_RANDOM if case["random"] else zds.ZDS_ROUND_NEAREST
        zds.zds_state_quantise(s["x"], s["q"], rounding, *key, s["state"])
        zds.zds_state_dequantise(s["q"], s["out"])
        return s["out"]
    if op == "read":
        zds.zds_state_dequantise(s["q"], s["out"])
        return s["out"]
    if op == "compress":
        zds.zds_dropout_compress(s["x"], s["error"], case["ratio"], s["values"], *key, s["state"], s["scalars"])
        return s["values"], s["error"]
    zds.zds_dropout_decompress(s["peers"], case["ratio"], s["dst"], *key, s["state"],
                               zds.ZDS_ACCUMULATE if case["add"] else zds.ZDS_OVERWRITE)
    return s["dst"]


def _plain_step(s):
    case, k, n = s["case"], s["k"], s["case"]["n"]
    g = s["grads"].float() * k["gs"]
    m = _read(*s["exp_avg"], "e4m3") * k["b1"] + g * k["omb1"]
    v = _read(*s["exp_avg_sq"], case["second"]) * k["b2"] + (g * g) * k["omb2"]
    denom = v.sqrt() / torch.full((1,), k["bc2"], device="cuda") + k["eps"]
    p = s["master"].mul_(k["decay"]).sub_((m / denom) * k["step_size"])
    s["params"].copy_(p)
    r16 = _rounding_bits(n, s["first"], s)
    for name, x, fmt, out in (("exp_avg", m, "e4m3", s["read"][0]), ("exp_avg_sq", v, case["second"], s["read"][1])):
        codes, exps = _quantise(x, fmt, r16)
        s[name][0].copy_(codes)
        if exps is not None:
            s[name][1].copy_(exps)
        out.copy_(_read(*s[name], fmt))
    return p, s["params"], s["read"][0], s["read"][1]


def _plain_compress(s):
    case, n, ratio = s["case"], s["case"]["n"], s["case"]["ratio"]
    at = torch.arange(s["values"].numel(), device="cuda") * ratio + _kept(n, ratio, s["first"], s)
    inside = at < n                                  # of a last group that is not whole, what is kept may be missing
    at = at.clamp(max=n - 1)
    x = s["x"].float()
    if s["error"] is None:
        s["values"].copy_(torch.where(inside, x[at] * float(ratio), 0.0))
        return s["values"], None
    c = x + s["error"] * s["scale"]
    sent = torch.where(inside, c[at], 0.0).to(s["values"].dtype)
    s["values"].copy_(sent)
    left = torch.where(inside & torch.isfinite(sent), c[at] - sent.float(), c[at])
    s["error"].copy_(c.index_copy_(0, at, left) * (1.0 / s["scale"]))
    return s["values"], s["error"]


def _plain_decompress(s):
    case, n, ratio = s["case"], s["case"]["n"], s["case"]["ratio"]
    total = s["peers"][0].float()
    for peer in s["peers"][1:]:
        total = total + peer.float()
    at = torch.arange(total.numel(), device="cuda") * ratio + _kept(n, ratio, s["first"], s)
    at, total = at[at < n], total[at < n]
    if case["add"]:
        s["dst"][at] += total
    else:
        s["dst"].zero_()
        s["dst"][at] = total.to(s["dst"].dtype)
    return s["dst"]


def run(s):
    if own:
        return _own_pass(s)
    case = s["case"]
    if case["op"] == "step":
        return _plain_step(s)
    if case["op"] == "quantise":
        r16 = _rounding_bits(case["n"], s["first"], s) if case["random"] else None
        return s["out"].copy_(_read(*_quantise(s["x"], case["format"], r16), case["format"]))
    if case["op"] == "read":
        return s["out"].copy_(_read(*s["codes"], case["format"]))
    return _plain_compress(s) if case["op"] == "compress" else _plain_decompress(s)


# ------------------------------------------------------------------ what it costs

def work(case):
    """Bytes: every input once, every output once, and the codes that lie
    between a quantising and its reading back written and read."""
    n = case["n"]
    size = {"e4m3": 1 + 1 / BLOCK, "ue5m3": 1 + 1 / BLOCK, "bf16": 2}
    if case["op"] == "step":
        codes = size["e4m3"] + size[case["second"]]
        return {"bytes": n * (BYTES[case["grads"]] + 8 + 2 * codes + 2 + codes + 4), "flops": 60 * n}
    if case["op"] == "quantise":
        return {"bytes": n * (4 + 2 * size[case["format"]] + 4), "flops": 12 * n}
    if case["op"] == "read":
        return {"bytes": n * (size[case["format"]] + BYTES[case["to"]]), "flops": 3 * n}
    groups = -(-n // case["ratio"])
    if case["op"] == "compress":
        x = n if case["feedback"] else groups
        return {"bytes": x * BYTES[case["x"]] + groups * BYTES[case["values"]] + (8 * n if case["feedback"] else 0),
                "flops": 4 * x}
    dst = 2 * groups * BYTES[case["to"]] if case["add"] else n * BYTES[case["to"]]
    return {"bytes": groups * BYTES[case["values"]] * case["peers"] + dst, "flops": groups * case["peers"]}


# ------------------------------------------------------------------ 64 bits

def _words(calls, step, tag, seed):
    """The generator once more, its products from 16-bit limbs: an array of
    four words for each of the given calls."""
    def times(a, m):
        """(high, low) 32 bits of a * m."""
        lo, hi = (a & 0xFFFF) * m, (a >> 16) * m         # each below 2^48
        both = lo + ((hi & 0xFFFF) << 16)
        return (hi >> 16) + (both >> 32), both & LOW

    x0, x1 = calls % 2 ** 32, torch.div(calls, 2 ** 32, rounding_mode="floor")
    x2, x3 = torch.zeros_like(calls) + step, torch.zeros_like(calls) + tag
    for r in range(10):
        key = (seed % 2 ** 32 + r * W0) % 2 ** 32, (seed // 2 ** 32 + r * W1) % 2 ** 32
        (h0, l0), (h1, l1) = times(x0, M0), times(x2, M1)
        x0, x1, x2, x3 = h1 ^ x1 ^ key[0], l1, h0 ^ x3 ^ key[1], l0
    return x0, x1, x2, x3


def _exact_bits(a, b, s):
    """The 16 random bits of elements a .. b - 1 (a a multiple of 8)."""
    f = s["first"] + a
    calls = f // 8 + torch.arange(-(-(b - a) // 8), device="cuda")
    out = []
    for w in _words(calls, s["step"], TAG_STATE, s["seed"]):
        out += [w % 65536, torch.div(w, 65536, rounding_mode="floor")]
    return torch.stack(out, 1).reshape(-1)[:b - a]


def _exact_quantised(x, fmt, r16):
    """The values that codes of x (64 bits) stand for."""
    n = x.numel()
    if r16 is not None and fmt != "e4m3":
        r16 = r16 // 256 + (r16 % 256) * 256
    mag = x.abs()
    if fmt == "bf16":
        _, e = torch.frexp(mag)
        step = torch.exp2((e - 8).clamp(min=-133).double())
        q = mag / step
        q = q.round() if r16 is None else torch.floor(q + r16 / 65536)
        return torch.sign(x) * torch.where((q == 0) & (mag > 0), step, q * step)
    rows = -(-n // BLOCK)
    mag = torch.nn.functional.pad(mag, (0, rows * BLOCK - n)).view(rows, BLOCK)
    top = mag.amax(1, keepdim=True)
    f, e = torch.frexp(top)                               # top = f 2^e, f in [0.5, 1)
    e = torch.where(f > 0.875, e, e - 1)                  # 2^e 1.75 is the largest value of the block
    e = torch.where(top == 0, torch.full_like(e, -127), e).clamp(min=LEAST[fmt] - 127)
    # the values of 8 a binade, down to where the exponent field ends
    _, own_e = torch.frexp(mag)
    low = e - TOP[fmt] + 1                                # the least binade that has its own exponent
    step = torch.exp2((torch.maximum(own_e - 1, low) - 3).double())
    q = mag / step
    if r16 is None:
        q = q.round()                                     # halves to the even code
    else:
        pad = torch.nn.functional.pad(r16, (0, rows * BLOCK - n)).view(rows, BLOCK)
        q = torch.floor(q + (16 * pad + 8) / 2 ** 20)
    if fmt == "ue5m3":
        q = torch.where(mag > 0, q.clamp(min=1.0), q)
    return torch.sign(x) * (q * step).view(-1)[:n]


def _exact_read(codes, exps, fmt):
    if fmt == "bf16":
        return codes.double()
    c = codes.to(torch.int64)
    sign = torch.where(c >= 128, -1.0, 1.0).double() if fmt == "e4m3" else 1.0
    c = c % 128 if fmt == "e4m3" else c
    field, frac = torch.div(c, 8, rounding_mode="floor"), c % 8
    e = exps.to(torch.int64).repeat_interleave(BLOCK)[:c.numel()] - 127 - TOP[fmt]
    value = torch.where(field > 0, 1.0 + frac.double() / 8, frac.double() / 4) * torch.exp2((field + e).double())
    return sign * value


def _of(codes, exps, a, b):
    """Elements a .. b - 1 (a a multiple of the block) of a quantised array."""
    return codes[a:b], None if exps is None else exps[a // BLOCK:-(-b // BLOCK)]


def _pieces(n):
    """Ranges of whole blocks."""
    size = 1 << 26
    return [(a, min(n, a + size)) for a in range(0, n, size)]


def _exact_piece(case, s, a, b):
    """Outputs of elements a .. b - 1 of a step, a quantising or a reading back."""
    x = slice(a, b)
    if case["op"] == "read":
        return (_exact_read(*_of(*s["codes"], a, b), case["format"]),)
    if case["op"] == "quantise":
        r16 = _exact_bits(a, b, s) if case["random"] else None
        return (_exact_quantised(s["x"][x].double(), case["format"], r16),)
    k = s["k"]
    g = s["grads"][x].double() * k["gs"]
    m = k["b1"] * _exact_read(*_of(*s["exp_avg"], a, b), "e4m3") + k["omb1"] * g
    v = k["b2"] * _exact_read(*_of(*s["exp_avg_sq"], a, b), case["second"]) + k["omb2"] * g ** 2
    p = k["decay"] * s["master"][x].double() - k["step_size"] * m / (v.sqrt() / k["bc2"] + k["eps"])
    r16 = _exact_bits(a, b, s)
    return p, p, _exact_quantised(m, "e4m3", r16), _exact_quantised(v, case["second"], r16)


def _exact_places(s, n, ratio):
    """Flat places of the kept elements, one a group (some past the end)."""
    j = s["first"] // ratio + torch.arange(-(-n // ratio), device="cuda")
    calls = torch.arange(int(j[0]) // 16, int(j[-1]) // 16 + 1, device="cuda")
    words = _words(calls, s["step"], TAG_DROPOUT, s["seed"])
    bytes_ = torch.stack([torch.div(w, 256 ** i, rounding_mode="floor") % 256 for w in words for i in range(4)], 1)
    byte = bytes_.view(-1)[int(j[0]) % 16:][:j.numel()]
    return (j - s["first"] // ratio) * ratio + torch.div(byte * ratio, 256, rounding_mode="floor")


def exact(case, seed):
    s = _inputs(case, seed)
    n = case["n"]
    if case["op"] in ("step", "quantise", "read"):
        outs = None
        for a, b in _pieces(n):
            got = _exact_piece(case, s, a, b)
            outs = outs or [torch.empty(n, dtype=torch.float64, device="cuda") for _ in got]
            for o, x in zip(outs, got):
                o[a:b] = x
        return tuple(outs) if case["op"] == "step" else outs[0]
    ratio = case["ratio"]
    at = _exact_places(s, n, ratio)
    inside = at < n
    if case["op"] == "compress":
        x = s["x"].double()
        if s["error"] is None:
            return torch.where(inside, x[at.clamp(max=n - 1)] * ratio, 0.0), None
        c = x + s["error"].double() * s["scale"]
        values = torch.where(inside, c[at.clamp(max=n - 1)], 0.0)
        rounded = values.to(DTYPES[case["values"]]).double()
        c[at[inside]] -= rounded[inside]
        return values, c / s["scale"]
    total = sum(p.double() for p in s["peers"])
    out = s["dst"].double() if case["add"] else torch.zeros(n, dtype=torch.float64, device="cuda")
    out[at[inside]] += total[inside]
    return out

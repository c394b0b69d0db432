"""The Muon update's operators at the sizes this library meets: the momentum
pass over a flat gradient bucket, the Newton-Schulz orthogonalisation of the
update's matrices, and the pass that applies the result to the fp32 master.

With `own` false every operator runs in its plain form (elementary torch
operations in 32 bits, rounded once at the end); with `own` true through the
library's entry points. `exact` gives the same results from the definitions in
64 bits.
"""

import math

import torch

own = False

ALIGN = 64                      # flat layout alignment (elements)
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}


# ------------------------------------------------------------------ the cases

# A matrix set is written as "COUNTxROWSxCOLS,..." in flat order.
LAYER = "4x4096x4096,2x11008x4096,1x4096x11008"
TINY = "24x16x32,16x64x64,12x96x160,8x256x128,4x200x333"


def listed():
    return [
        # the tiny shard's size: a latency-bound pass over fp16 grads under a loss scale
        {"name": "momentum tiny fp16", "op": "momentum", "n": 733953, "grads": "fp16", "update": "bf16",
         "nesterov": True},
        # one decoder layer of the 7B shape, bf16 training
        {"name": "momentum 7B layer", "op": "momentum", "n": 202375168, "grads": "bf16", "update": "bf16",
         "nesterov": True},
        # fp32 accumulated grads, an fp32 update, a length that ends inside a vector
        {"name": "momentum fp32 ragged", "op": "momentum", "n": 45088771, "grads": "fp32", "update": "fp32",
         "nesterov": False},
        # many small matrices in one call (a small model, or per-head blocks): latency
        {"name": "orthogonalise tiny set", "op": "orthogonalise", "shapes": TINY, "update": "bf16"},
        # one attention projection of the 7B shape by itself
        {"name": "orthogonalise 4096", "op": "orthogonalise", "shapes": "1x4096x4096", "update": "bf16"},
        # one decoder layer of the 7B shape: square, tall and wide matrices together
        {"name": "orthogonalise 7B layer", "op": "orthogonalise", "shapes": LAYER, "update": "bf16"},
        # the largest: one MLP projection of the 65B shape
        {"name": "orthogonalise 65B mlp", "op": "orthogonalise", "shapes": "1x8192x22016", "update": "bf16"},
        # odd and ragged sizes, thin ones among them
        {"name": "orthogonalise ragged", "op": "orthogonalise",
         "shapes": "2x1000x4096,3x777x1333,1x2752x129,2x1x513,1x1025x1023", "update": "bf16"},
        # an fp32 update kept at fp32 accuracy: the 1024-row chunks of a 7B projection
        {"name": "orthogonalise fp32", "op": "orthogonalise", "shapes": "4x1024x4096", "update": "fp32"},
        # the small set's weights
        {"name": "apply tiny set", "op": "apply", "shapes": TINY, "update": "bf16", "params": "fp16",
         "scale": "aspect"},
        # one decoder layer of the 7B shape, bf16 weights
        {"name": "apply 7B layer", "op": "apply", "shapes": LAYER, "update": "bf16", "params": "bf16",
         "scale": "rms"},
        # fp32 updates, odd sizes
        {"name": "apply fp32 ragged", "op": "apply", "shapes": "2x1000x4096,3x777x1333,1x2752x129,2x1x513,8x1025x1023",
         "update": "fp32", "params": "bf16", "scale": "rms"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: any operator, sizes spread over their logarithm."""
    op = rng.choice(("momentum", "orthogonalise", "orthogonalise", "apply"))
    if op == "momentum":
        return {"op": op, "n": _log(rng, 4096, 200_000_000), "grads": rng.choice(("fp16", "bf16", "fp32")),
                "update": rng.choice(("bf16", "bf16", "fp32")), "nesterov": rng.random() < 0.7}
    update = rng.choice(("bf16", "bf16", "fp32"))
    top = 6000 if op == "apply" or update == "bf16" else 2500
    shapes, left = [], 100_000_000 if op == "apply" else 60_000_000
    for _ in range(rng.randint(1, 4)):
        r, c = _log(rng, 16, top), _log(rng, 16, top)
        k = min(_log(rng, 1, 24), max(0, left // (r * c)))
        if k > 0:
            shapes.append("%dx%dx%d" % (k, r, c))
            left -= k * r * c
    case = {"op": op, "shapes": ",".join(shapes), "update": update}
    if op == "apply":
        case["params"] = rng.choice(("fp16", "bf16"))
        case["scale"] = rng.choice(("aspect", "rms"))
    return case


# ------------------------------------------------------------------ layout

def _groups(shapes):
    """[(count, rows, cols, first offset, offset step)] of a matrix set laid
    out matrix after matrix, each at a multiple of ALIGN; and the flat length."""
    out, pos = [], 0
    for part in shapes.split(","):
        k, r, c = (int(x) for x in part.split("x"))
        step = -(-(r * c) // ALIGN) * ALIGN
        out.append((k, r, c, pos, step))
        pos += k * step
    return out, pos


def _batch(flat, group):
    """The (count, rows, cols) view of one group's matrices in a flat buffer."""
    k, r, c, pos, step = group
    return torch.as_strided(flat, (k, r, c), (step, c, 1), flat.storage_offset() + pos)


def _scale(case, r, c):
    return math.sqrt(max(1.0, r / c)) if case["scale"] == "aspect" else 0.2 * math.sqrt(max(r, c))


# ------------------------------------------------------------------ inputs

LR, MOMENTUM, DECAY = 2e-3, 0.95, 0.1
LOSS_SCALE = {"fp16": 2.0 ** 14, "bf16": 1.0, "fp32": 1.0}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(n, sigma, g, dtype=torch.float32):
    return torch.empty(n, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=g)


def _update_like(groups, n, g, dtype):
    """A momentum buffer as training leaves it: for each matrix a part of low
    rank (the gradient's outer products) and noise over the whole spectrum."""
    flat = torch.zeros(n, dtype=dtype, device="cuda")
    for group in groups:
        k, r, c, _, _ = group
        rank = max(1, min(r, c) // 16)
        for b in _batch(flat, group):
            p = _normal(r * rank, 1.0, g).view(r, rank)
            q = _normal(rank * c, 1.0, g).view(rank, c)
            b.copy_((p @ q) * (1e-3 / math.sqrt(rank)) + _normal(r * c, 5e-4, g).view(r, c))
    return flat


def _inputs(case, seed):
    """The tensors of a case, from its seed alone."""
    g = _gen(seed)
    s = {"case": dict(case)}
    if case["op"] == "momentum":
        n = case["n"]
        scale = LOSS_SCALE[case["grads"]]
        s["grads"] = _normal(n, 2e-3 * scale, g, DTYPES[case["grads"]])
        s["momentum"] = _normal(n, 5e-4, g)
        s["update"] = torch.zeros(n, dtype=DTYPES[case["update"]], device="cuda")
        s["grad_scale"] = 0.8125 / scale   # a clip coefficient over the loss scale
        return s
    s["groups"], n = _groups(case["shapes"])
    dt = DTYPES[case["update"]]
    if case["op"] == "orthogonalise":
        s["src"] = _update_like(s["groups"], n, g, dt)
        s["dst"] = torch.zeros(n, dtype=dt, device="cuda")
        return s
    s["update"] = torch.zeros(n, dtype=dt, device="cuda")
    s["master"] = torch.zeros(n, dtype=torch.float32, device="cuda")
    s["params"] = torch.zeros(n, dtype=DTYPES[case["params"]], device="cuda")
    for group in s["groups"]:
        k, r, c, _, _ = group
        _batch(s["update"], group).copy_(_normal(k * r * c, 1.0 / math.sqrt(max(r, c)), g).view(k, r, c))
        _batch(s["master"], group).copy_(_normal(k * r * c, 0.02, g).view(k, r, c))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from zero_sharded_mixed_tensor_amd import zds
        s["scalars"] = zds.new_scalars()
        zds.write_scalars(s["scalars"], zds.StepScalars(accum_steps=1, clip_coef=1.0, scale_used=1.0,
                                                        grad_scale=s.get("grad_scale", 1.0)))
        s["hp"] = zds.muon_hparams(lr=LR, momentum=MOMENTUM, weight_decay=DECAY,
                                   nesterov=case.get("nesterov", True), scale=case.get("scale", "rms"))
        if "groups" in s:
            shapes = [(pos + i * step, r, c) for k, r, c, pos, step in s["groups"] for i in range(k)]
            s["plan"] = zds.zds_matrix_plan_create(shapes)
            if case["op"] == "orthogonalise":
                s["ws"] = zds.new_newton_schulz_workspace(s["plan"], s["src"].dtype)
    return s


# ------------------------------------------------------------------ one pass

def _own_pass(s):
    from zero_sharded_mixed_tensor_amd import zds
    op = s["case"]["op"]
    if op == "momentum":
        zds.zds_muon_momentum(s["hp"], s["grads"], s["momentum"], s["update"], s["scalars"])
        return s["momentum"], s["update"]
    if op == "orthogonalise":
        zds.zds_newton_schulz(s["plan"], s["src"], s["dst"], s["ws"])
        return s["dst"]
    zds.zds_muon_apply(s["hp"], s["plan"], s["update"], s["master"], s["params"], s["scalars"])
    return s["master"], s["params"]


def _plain_orthogonalise(x):
    """Newton-Schulz of a (count, rows, cols) batch, in 32 bits."""
    a, b, c = QUINTIC
    x = x.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.mT.contiguous()
    # the norm is a sum over the whole matrix: in 64 bits
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = x / (norm + EPS).float()
    for _ in range(STEPS):
        gram = torch.bmm(x, x.mT.contiguous())
        x = torch.baddbmm(x, torch.baddbmm(gram, gram, gram, beta=b, alpha=c), x, beta=a)
    return x.mT if tall else x


def run(s):
    if own:
        return _own_pass(s)
    case = s["case"]
    if case["op"] == "momentum":
        g = s["grads"].float() * s["grad_scale"]
        m = s["momentum"].mul_(MOMENTUM).add_(g * (1.0 - MOMENTUM))
        s["update"].copy_(g * (1.0 - MOMENTUM) + m * MOMENTUM if case["nesterov"] else m)
        return m, s["update"]
    for group in s["groups"]:
        if case["op"] == "orthogonalise":
            _batch(s["dst"], group).copy_(_plain_orthogonalise(_batch(s["src"], group)))
        else:
            _, r, c, _, _ = group
            p = _batch(s["master"], group)
            p.mul_(1.0 - LR * DECAY).sub_(_batch(s["update"], group).float() * (LR * _scale(case, r, c)))
            _batch(s["params"], group).copy_(p)
    return s["dst"] if case["op"] == "orthogonalise" else (s["master"], s["params"])


# ------------------------------------------------------------------ what it costs

def work(case):
    """Bytes: every input once, every output once. Operations of the
    orthogonalisation: with R <= C the matrix's two sizes, each step forms the
    symmetric R x R products X X^T and A A (one triangle each) and the full
    product B X."""
    if case["op"] == "momentum":
        return {"bytes": case["n"] * (BYTES[case["grads"]] + 8 + BYTES[case["update"]]), "flops": 6 * case["n"]}
    groups, _ = _groups(case["shapes"])
    elems = sum(k * r * c for k, r, c, _, _ in groups)
    if case["op"] == "apply":
        return {"bytes": elems * (BYTES[case["update"]] + 8 + BYTES[case["params"]]), "flops": 3 * elems}
    flops = 0
    for k, r, c, _, _ in groups:
        m, n = min(r, c), max(r, c)
        flops += k * STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)
    return {"bytes": 2 * elems * BYTES[case["update"]], "flops": flops}


# ------------------------------------------------------------------ 64 bits

def _exact_orthogonalise(x):
    """The same iteration through its Gram matrix: every step multiplies the
    matrix by a polynomial of W = X X^T from the left, so the product of the
    steps' polynomials is built from W alone and applied once."""
    a, b, c = QUINTIC
    x = x.double()
    rows, cols = x.shape
    x = x / (torch.linalg.vector_norm(x) + EPS)
    w = x @ x.T if rows <= cols else x.T @ x
    eye = torch.eye(w.shape[0], dtype=torch.float64, device=w.device)
    total = eye
    for _ in range(STEPS):
        q = a * eye + b * w + c * (w @ w)
        total = q @ total
        w = q @ w @ q
    return total @ x if rows <= cols else x @ total


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "momentum":
        g = s["grads"].double() * s["grad_scale"]
        m = s["momentum"].double() * MOMENTUM + g * (1.0 - MOMENTUM)
        u = m * MOMENTUM + g * (1.0 - MOMENTUM) if case["nesterov"] else m
        return m, u
    out = torch.zeros(s["update" if case["op"] == "apply" else "src"].numel(), dtype=torch.float64, device="cuda")
    for group in s["groups"]:
        _, r, c, _, _ = group
        if case["op"] == "apply":
            p = _batch(s["master"], group).double() * (1.0 - LR * DECAY)
            _batch(out, group).copy_(p - LR * _scale(case, r, c) * _batch(s["update"], group).double())
        else:
            for o, x in zip(_batch(out, group), _batch(s["src"], group)):
                o.copy_(_exact_orthogonalise(x))
    return (out, out.clone()) if case["op"] == "apply" else out

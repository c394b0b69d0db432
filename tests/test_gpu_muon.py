"""Muon's operators on the GPU against the plain definitions: the two element
passes bit for bit, the orthogonalisation against float64.

Tolerances of the orthogonalisation (2-norm of the difference over the 2-norm
of the result). bf16: the result's rounding is at most 2^-8 per element, and
the operands' fp16 roundings (at most 2^-11 each; X, A and B in 5 steps, so 15
of them, independent) are carried to the result by slopes of the step's
polynomial below 3.5 in a step and are contracted by later ones: together at
most another 2^-8 or so. Hence 2^-7. fp32: operands of 22 bits (2^-23), fp32
sums over up to K terms (sqrt(K) 2^-24), 15 of them, with the same slopes:
15 * 3.5 * sqrt(1400) * 2^-24 is 1.2e-4 if all errors added up; as they are
independent, sqrt(15) * 3.5 * sqrt(1400) * 2^-24 = 3e-5.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import muon as M  # noqa: E402
from oracle.zero_step import narrow, widen  # noqa: E402
from tests.util import to_dev, to_host  # noqa: E402
from zero_sharded_mixed_tensor_amd import zds  # noqa: E402

TOL = {"bf16": 2.0 ** -7, "fp32": 3e-5}
TDT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def scalars(grad_scale=1.0, overflow=0):
    t = zds.new_scalars()
    zds.write_scalars(t, zds.StepScalars(overflow=overflow, accum_steps=1, clip_coef=1.0, grad_scale=grad_scale,
                                         scale_used=1.0))
    return t


def bits(x, dtype):
    """fp32 values -> the dtype's host form."""
    return x.astype(np.float32) if dtype == "fp32" else narrow(x.astype(np.float32), dtype)


# ------------------------------------------------------------------ momentum

@pytest.mark.parametrize("gdt", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("udt", ["bf16", "fp32"])
@pytest.mark.parametrize("n,shift", [(1, 0), (3, 0), (4, 0), (1021, 0), (1024, 1), (70003, 0), (70003, 3)])
def test_momentum_bit_exact(gdt, udt, n, shift):
    rng = np.random.default_rng(n * 10 + shift)
    g = bits(rng.standard_normal(n + shift) * 8, gdt)
    m = (rng.standard_normal(n + shift) * 1e-3).astype(np.float32)
    for nesterov in (True, False):
        hp = zds.muon_hparams(momentum=0.95, nesterov=nesterov)
        dg, dm = to_dev(g, gdt), to_dev(m, "fp32")
        du = torch.full((n + shift + 8,), 7.0, dtype=TDT[udt], device="cuda")
        zds.zds_muon_momentum(hp, dg[shift:], dm[shift:], du[shift:shift + n], scalars(0.37))
        wm, wu = M.muon_momentum(g[shift:], gdt, m[shift:], 0.37, 0.95, nesterov, udt)
        assert np.array_equal(to_host(dm)[shift:].view(np.uint32), wm.view(np.uint32))
        assert np.array_equal(to_host(du)[shift:shift + n], wu)
        assert np.array_equal(to_host(dm)[:shift], m[:shift])  # nothing in front or behind is written
        assert (du[:shift] == 7).all() and (du[shift + n:] == 7).all()


def test_momentum_skips_on_overflow_and_takes_none():
    n = 1000
    g = torch.full((n,), float("inf"), device="cuda", dtype=torch.bfloat16)
    m = torch.ones(n, device="cuda")
    u = torch.full((n,), 3.0, device="cuda", dtype=torch.bfloat16)
    zds.zds_muon_momentum(zds.muon_hparams(), g, m, u, scalars(0.0, overflow=1))
    zds.zds_muon_momentum(zds.muon_hparams(), g, m, u, scalars(1.0), n=0)
    assert (m == 1).all() and (u == 3).all()


# ------------------------------------------------------------------ layouts

def layout(shapes, gap=0, first=0):
    """Matrices one after another, `gap` elements between them."""
    out, pos = [], first
    for r, c in shapes:
        out.append((pos, r, c))
        pos += r * c + gap
    return out, pos


def fill(mats, total, seed, dtype, kind="gauss"):
    rng = np.random.default_rng(seed)
    x = np.full(total, 5.0, np.float32)
    for o, r, c in mats:
        if kind == "gauss":
            g = rng.standard_normal((r, c))
        else:  # most of the weight in a few directions
            k = max(1, min(r, c) // 16)
            g = rng.standard_normal((r, k)) @ rng.standard_normal((k, c)) / np.sqrt(k) + 0.3 * rng.standard_normal((r, c))
        x[o:o + r * c] = (g * 1e-3).reshape(-1)
    return bits(x, dtype)


# ------------------------------------------------------------------ apply

@pytest.mark.parametrize("udt", ["bf16", "fp32"])
@pytest.mark.parametrize("pdt", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["none", "aspect", "rms"])
@pytest.mark.parametrize("gap,first", [(0, 0), (64, 0), (5, 3)])
def test_apply_bit_exact(udt, pdt, mode, gap, first):
    mats, total = layout([(16, 32), (1, 1), (7, 1), (0, 9), (65, 130), (130, 65), (1, 4099)], gap, first)
    u = fill(mats, total, 3, udt)
    rng = np.random.default_rng(4)
    p = (rng.standard_normal(total) * 0.02).astype(np.float32)
    du, dp = to_dev(u, udt), to_dev(p, "fp32")
    do = torch.full((total,), 3.0, dtype=TDT[pdt], device="cuda")
    want_p, want_o = p.copy(), to_host(do).copy()
    for o, r, c in mats:
        s = slice(o, o + r * c)
        want_p[s], want_o[s] = M.muon_apply(u[s], udt, p[s], r, c, 2e-2, 0.1, mode, pdt)
    plan = zds.zds_matrix_plan_create(mats)
    hp = zds.muon_hparams(lr=2e-2, weight_decay=0.1, scale=mode)
    zds.zds_muon_apply(hp, plan, du, dp, do, scalars(overflow=1))   # skipped
    assert np.array_equal(to_host(dp), p) and (do == 3).all()
    zds.zds_muon_apply(hp, plan, du, dp, do, scalars())
    assert np.array_equal(to_host(dp).view(np.uint32), want_p.view(np.uint32))
    assert np.array_equal(to_host(do), want_o)
    zds.zds_muon_apply(hp, plan, du, dp, None, scalars())           # no cast
    assert np.array_equal(to_host(do), want_o)
    plan.close()


# ------------------------------------------------------------------ orthogonalise

SETS = {
    "one": [(1, 1)],
    "thin": [(1, 513), (513, 1), (2, 64), (63, 3)],
    "small": [(16, 32), (64, 64), (65, 63), (63, 65), (128, 128), (129, 127)],
    "middle": [(200, 333), (333, 200), (256, 256), (257, 511)],
    "large": [(1024, 1024), (1025, 1090), (1400, 1030)],
    "mixed": [(64, 64), (0, 5), (300, 1030), (1030, 1100), (5, 0), (1, 3)],
}


def check(mats, x, y, dtype, steps=5, coef=None, tol=None):
    xs, ys = widen(x, dtype).astype(np.float64), widen(y, dtype).astype(np.float64)
    for o, r, c in mats:
        if r * c == 0:
            continue
        want = M.newton_schulz(xs[o:o + r * c].reshape(r, c), steps, coef)
        got = ys[o:o + r * c].reshape(r, c)
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= (tol or TOL[dtype]), (r, c, rel)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("kind,gap,first", [("gauss", 0, 0), ("lowrank", 3, 1)])
def test_orthogonalise(dtype, name, kind, gap, first):
    mats, total = layout(SETS[name], gap, first)
    total += 8
    x = fill(mats, total, 11, dtype, kind)
    plan = zds.zds_matrix_plan_create(mats)
    assert plan.span == max(o + r * c for o, r, c in mats)
    dx = to_dev(x, dtype)
    ws = zds.new_newton_schulz_workspace(plan, TDT[dtype])
    ws.fill_(0xFF)                                    # NaN patterns: nothing stale is read
    dy = torch.full((total,), 9.0, dtype=TDT[dtype], device="cuda")
    zds.zds_newton_schulz(plan, dx, dy, ws)
    y = to_host(dy)
    check(mats, x, y, dtype)
    inside = np.zeros(total, bool)
    for o, r, c in mats:
        inside[o:o + r * c] = True
    assert (widen(y, dtype)[~inside] == 9.0).all()
    again = torch.full((total,), 9.0, dtype=TDT[dtype], device="cuda")
    zds.zds_newton_schulz(plan, dx, again, ws)        # the same bits, on a used workspace
    assert np.array_equal(to_host(again), y)
    zds.zds_newton_schulz(plan, dx, dx, ws)           # in place
    got = to_host(dx)
    assert np.array_equal(got[inside], y[inside]) and np.array_equal(got[~inside], x[~inside])
    plan.close()


@pytest.mark.parametrize("dtype,shapes", [
    ("bf16", [(2000, 4090)]), ("fp32", [(2000, 2040)]),     # a few tiles of 256 with long sums
    ("bf16", [(128, 4096), (250, 2000), (256, 256), (100, 120)]),   # tiles of 128, deep and shallow ones
    ("fp32", [(128, 4096), (250, 2000), (256, 256), (100, 120)]),
    ("bf16", [(128, 5000)] * 3), ("fp32", [(8000, 130)]),
])
def test_orthogonalise_sums_in_pieces(dtype, shapes):
    """Sums long enough, and tiles few enough, to be cut into pieces: right, and
    the same bits in every call."""
    mats, total = layout(shapes, 3, 1)
    x = fill(mats, total, 17, dtype)
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, TDT[dtype])
    ws.fill_(0xFF)
    dx = to_dev(x, dtype)
    dy = torch.full((total,), 9.0, dtype=TDT[dtype], device="cuda")
    zds.zds_newton_schulz(plan, dx, dy, ws)
    y = to_host(dy)
    check(mats, x, y, dtype)
    for _ in range(2):
        again = torch.full((total,), 9.0, dtype=TDT[dtype], device="cuda")
        zds.zds_newton_schulz(plan, dx, again, ws)
        assert np.array_equal(to_host(again), y)
    plan.close()


def newton_schulz_64(x):
    """The default steps in 64 bits on the GPU."""
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        a = x @ x.T.contiguous()
        x = 3.4445 * x + (-4.7750 * a + 2.0315 * (a @ a)) @ x
    return x.T.contiguous() if tall else x


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shapes", [
    [(4000, 4090)],                     # tiles of 192, over a padded 4096
    [(4090, 4001)],
    [(2000, 2040)] * 8,                 # 288 tiles of 256: the last 32 in pieces
    [(1100, 1110)] * 12,                # 540 tiles of 128, in FP32 the last 28 in pieces
    [(2430, 2432)] * 3,                 # 570 tiles of 128: the last 58 in pieces
    [(1000, 1000)] * 2,                 # in FP32 all of 72 tiles in pieces
    [(700, 700)] * 21,                  # 441 tiles of 128, two to a unit
], ids=lambda s: f"{len(s)}x{s[0][0]}x{s[0][1]}")
def test_orthogonalise_tilings(dtype, shapes):
    """Sets that the tilings differ for; the first and last matrix against 64 bits."""
    mats, total = layout(shapes, 3, 1)
    dx = torch.randn(total, generator=torch.Generator().manual_seed(19)).to(TDT[dtype]).cuda()
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, TDT[dtype])
    ws.fill_(0xFF)
    dy = torch.full((total,), 9.0, dtype=TDT[dtype], device="cuda")
    zds.zds_newton_schulz(plan, dx, dy, ws)
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for o, r, c in mats:
        inside[o:o + r * c] = True
    assert (dy[~inside] == 9).all()
    for o, r, c in (mats[0], mats[-1]):
        want = newton_schulz_64(dx[o:o + r * c].double().view(r, c))
        rel = ((dy[o:o + r * c].double().view(r, c) - want).norm() / want.norm()).item()
        assert rel <= TOL[dtype], (r, c, rel)
    again = torch.full((total,), 9.0, dtype=TDT[dtype], device="cuda")
    zds.zds_newton_schulz(plan, dx, again, ws)
    assert torch.equal(again, dy)
    plan.close()


@pytest.mark.parametrize("rows,cols", [(16, 16), (16, 24), (90, 20), (32, 1000), (24, 3000), (64, 64), (64, 2000),
                                       (96, 160), (333, 200), (700, 1000)])
def test_orthogonalise_bf16_is_about_one_rounding(rows, cols):
    """The error's 2-norm against that of rounding the exact result to bf16:
    with that rounding and as much again of everything before it (independent
    of it) it is sqrt(2) of it; a margin of 5 % for the draw."""
    k = max(1, 200_000 // (rows * cols))
    mats, total = layout([(rows, cols)] * k)
    dx = torch.randn(total, generator=torch.Generator().manual_seed(20)).to(torch.bfloat16).cuda()
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, torch.bfloat16)
    dy = torch.zeros_like(dx)
    zds.zds_newton_schulz(plan, dx, dy, ws)
    err = rounding = 0.0
    for o, r, c in mats:
        want = newton_schulz_64(dx[o:o + r * c].double().view(r, c))
        err += (dy[o:o + r * c].double().view(r, c) - want).square().sum().item()
        rounding += (want.bfloat16().double() - want).square().sum().item()
    assert (err / rounding) ** 0.5 <= 1.05 * 2 ** 0.5, (err / rounding) ** 0.5
    plan.close()


@pytest.mark.parametrize("rows,cols", [(64, 64), (96, 160), (333, 200), (700, 1000), (1500, 2000)])
def test_orthogonalise_fp32_is_an_fp32_evaluation(rows, cols):
    """Operands of 22 bits or more and fp32 sums: at most the error of the steps
    in plain fp32 and half as much again, for sums of 64 or more."""
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(21)).cuda()
    plan = zds.zds_matrix_plan_create([(0, rows, cols)])
    ws = zds.new_newton_schulz_workspace(plan, torch.float32)
    y = torch.zeros_like(x)
    zds.zds_newton_schulz(plan, x.view(-1), y.view(-1), ws)
    want = newton_schulz_64(x.double())
    err, plain = ((a.double() - want).norm().item() for a in (y, newton_schulz_64(x)))
    assert err <= 1.5 * plain, (err, plain)
    plan.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("steps,coef", [(1, None), (2, None), (8, None), (3, [(1.875, -1.25, 0.375)] * 3),
                                        (4, [(3.4, -4.7, 2.0), (3.0, -4.0, 1.8), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)])])
def test_orthogonalise_steps_and_coefficients(dtype, steps, coef):
    mats, total = layout([(40, 70), (300, 180)])
    x = fill(mats, total, 5, dtype)
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, TDT[dtype])
    dy = torch.zeros(total, dtype=TDT[dtype], device="cuda")
    zds.zds_newton_schulz(plan, to_dev(x, dtype), dy, ws, steps=steps, coef=coef)
    check(mats, x, to_host(dy), dtype, steps, coef)
    plan.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_orthogonalise_extremes(dtype):
    """Infinite, NaN, zero, tiny and huge matrices next to an ordinary one."""
    shapes = [(40, 50)] * 6 + [(1050, 1100)] * 3
    mats, total = layout(shapes)
    x = widen(fill(mats, total, 6, dtype), dtype).copy()
    part = [slice(o, o + r * c) for o, r, c in mats]
    x[part[0]][7] = np.inf
    x[part[1]][9] = np.nan
    x[part[2]] = 0
    x[part[3]] *= 2.0 ** 110
    x[part[4]] *= 2.0 ** 60
    x[part[6]][12345] = -np.inf
    x[part[7]] = 0
    xb = bits(x, dtype)
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, TDT[dtype])
    dy = torch.full((total,), 9.0, dtype=TDT[dtype], device="cuda")
    zds.zds_newton_schulz(plan, to_dev(xb, dtype), dy, ws)
    y = to_host(dy)
    yf = widen(y, dtype)
    for k in (0, 1, 6):
        assert np.isnan(yf[part[k]]).all()
    for k in (2, 7):
        assert (yf[part[k]] == 0).all()
    check([mats[k] for k in (3, 4, 5, 8)], xb, y, dtype)
    plan.close()


def test_orthogonalise_small_norms_follow_the_floor():
    """A norm next to the 1e-7 floor: the floor's share shows in the result."""
    mats, total = layout([(48, 96)] * 3)
    x = widen(fill(mats, total, 8, "fp32"), "fp32").copy()
    for k, s in enumerate((1e-6, 1e-5, 1e-4)):
        x[mats[k][0]:mats[k][0] + 48 * 96] *= s
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, torch.float32)
    dy = torch.zeros(total, device="cuda")
    zds.zds_newton_schulz(plan, to_dev(x, "fp32"), dy, ws)
    check(mats, x, to_host(dy), "fp32")
    plan.close()


def test_orthogonalise_skips_on_overflow_and_takes_an_empty_plan():
    mats, total = layout([(40, 50), (200, 200), (1024, 1030)])
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, torch.bfloat16)
    src = torch.ones(total, dtype=torch.bfloat16, device="cuda")
    dst = torch.full_like(src, 9.0)
    zds.zds_newton_schulz(plan, src, dst, ws, scalars=scalars(overflow=1))
    assert (dst == 9).all()
    zds.zds_newton_schulz(plan, src, dst, ws, scalars=scalars())
    assert (dst != 9).all()
    plan.close()
    for empty in ([], [(0, 0, 7), (0, 7, 0)]):
        plan = zds.zds_matrix_plan_create(empty)
        assert plan.span == 0 and zds.zds_newton_schulz_workspace_bytes(plan, torch.bfloat16) == 0
        e = torch.empty(0, dtype=torch.bfloat16, device="cuda")
        zds.zds_newton_schulz(plan, e, e, zds.new_newton_schulz_workspace(plan, torch.bfloat16))
        zds.zds_muon_apply(zds.muon_hparams(), plan, e, torch.empty(0, device="cuda"), None, scalars())
        plan.close()


def test_refusals_with_a_plan():
    mats, total = layout([(40, 50)])
    plan = zds.zds_matrix_plan_create(mats)
    x = torch.ones(total, dtype=torch.bfloat16, device="cuda")
    ws = zds.new_newton_schulz_workspace(plan, torch.bfloat16)

    def refused(text, fn):
        with pytest.raises(zds.ZdsError) as e:
            fn()
        assert text in str(e.value), str(e.value)

    refused("workspace of", lambda: zds.zds_newton_schulz(plan, x, x, ws[:-1]))
    big = torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")
    refused("256-byte aligned", lambda: zds.zds_newton_schulz(plan, x, x, big[16:]))
    refused("src holds", lambda: zds.zds_newton_schulz(plan, x[:-1], x, ws))
    refused("dst holds", lambda: zds.zds_newton_schulz(plan, x, x[:-1], ws))
    refused("one dtype", lambda: zds.zds_newton_schulz(plan, x, x.float(), ws))
    h = x.half()
    refused("bf16 or fp32", lambda: zds.zds_newton_schulz(plan, h, h, ws))
    refused("bf16 or fp32", lambda: zds.zds_muon_apply(zds.muon_hparams(), plan, h, x.float(), None, scalars()))
    refused("fp16 or bf16", lambda: zds.zds_muon_apply(zds.muon_hparams(), plan, x, x.float(), x.float(), scalars()))
    refused("device tensor", lambda: zds.zds_newton_schulz(plan, x.cpu(), x, ws))
    torch.cuda.synchronize()
    assert (x == 1).all()
    plan.close()


def test_overlaps_are_refused():
    mats, total = layout([(40, 50), (3, 7)])
    plan = zds.zds_matrix_plan_create(mats)
    x = torch.ones(total, dtype=torch.bfloat16, device="cuda")
    ws = zds.new_newton_schulz_workspace(plan, torch.bfloat16)

    def refused(text, fn):
        with pytest.raises(zds.ZdsError) as e:
            fn()
        assert text in str(e.value), str(e.value)

    two = torch.ones(2 * total + 64, dtype=torch.bfloat16, device="cuda")
    refused("overlaps src", lambda: zds.zds_newton_schulz(plan, two[:total], two[total - 1:], ws))
    refused("overlaps src", lambda: zds.zds_newton_schulz(plan, two[8:], two, ws))
    flat = ws.view(torch.bfloat16)
    assert flat.numel() > total
    refused("workspace overlaps", lambda: zds.zds_newton_schulz(plan, flat[flat.numel() - total:], x, ws))
    refused("workspace overlaps", lambda: zds.zds_newton_schulz(plan, x, flat, ws))
    p = torch.ones(total, device="cuda")
    hp = zds.muon_hparams()
    refused("overlap", lambda: zds.zds_muon_apply(hp, plan, p, p, None, scalars()))
    refused("overlap", lambda: zds.zds_muon_apply(hp, plan, x, p, p.view(torch.bfloat16), scalars()))
    refused("overlap", lambda: zds.zds_muon_apply(hp, plan, two, p, two[1:], scalars()))
    torch.cuda.synchronize()
    assert (x == 1).all() and (two == 1).all() and (p == 1).all()
    two[:total].normal_()                             # side by side in one buffer is fine
    zds.zds_newton_schulz(plan, two[:total], two[total:], ws)
    zds.zds_newton_schulz(plan, two[:total], x, ws)
    assert torch.equal(two[total:2 * total], x)
    plan.close()


@pytest.mark.parametrize("dtype,shapes", [("fp32", [(1000, 1000)] * 2), ("bf16", [(4000, 4090)])])
def test_graph_replays_of_large_sets(dtype, shapes):
    """Captured once, replayed with refilled grads: sums in pieces, and tiles
    that hang over."""
    mats, total = layout(shapes)
    plan = zds.zds_matrix_plan_create(mats)
    ws, ws2 = (zds.new_newton_schulz_workspace(plan, TDT[dtype]) for _ in range(2))
    src = torch.randn(total, device="cuda").to(TDT[dtype])
    out, want = torch.zeros_like(src), torch.zeros_like(src)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zds.zds_newton_schulz(plan, src, out, ws)
    for _ in range(4):
        src.normal_()
        out.zero_()
        graph.replay()
        zds.zds_newton_schulz(plan, src, want.zero_(), ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and out.abs().max() > 0
    plan.close()


def test_streams_and_graph_replays():
    """On a stream of the caller's; captured once and replayed with the grads
    refilled in place, eager work in between, every replay against the eager
    result."""
    mats, total = layout([(48, 80), (300, 200), (1030, 1100)], gap=7)
    plan = zds.zds_matrix_plan_create(mats)
    ws, ws2 = (zds.new_newton_schulz_workspace(plan, torch.bfloat16) for _ in range(2))
    src = to_dev(fill(mats, total, 1, "bf16"), "bf16")
    want = torch.zeros_like(src)
    zds.zds_newton_schulz(plan, src, want, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(src)
    with torch.cuda.stream(side):
        zds.zds_newton_schulz(plan, src, got, ws2)
    zds.zds_newton_schulz(plan, src, want, ws)         # at the same time, its own workspace
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(src)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zds.zds_newton_schulz(plan, src, out, ws)
    for seed in (2, 3, 4, 5):
        src.copy_(to_dev(fill(mats, total, seed, "bf16"), "bf16"))
        out.zero_()
        graph.replay()
        zds.zds_newton_schulz(plan, src, want.zero_(), ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    plan.close()


# ------------------------------------------------------------------ the whole step

def _oracle_step(O, x, master, mom, m, v, st, hp, mats, split, cfg):
    """One MuonStep in plain NumPy: (the new arrays, or None when skipped; the step scalars)."""
    sc = O.overflow_and_norm(x, "fp16", st.scale, cfg["K"], cfg["max_norm"])
    if sc["overflow"]:
        return None, sc
    gs = sc["grad_scale"]
    mom, u = M.muon_momentum(x[:split], "fp16", mom, gs, 0.95, True, "bf16")
    master = master.copy()
    for o, r, c in mats:
        s = slice(o, o + r * c)
        q = narrow(M.newton_schulz(widen(u[s], "bf16").astype(np.float64).reshape(r, c)).reshape(-1).astype(np.float32), "bf16")
        master[s], _ = M.muon_apply(q, "bf16", master[s], r, c, cfg["lr"], cfg["wd"], "rms", "fp16")
    con = O.adamw_constants(hp, st.beta1_pow, st.beta2_pow)
    p, m, v = O.adamw_update(x[split:], "fp16", gs, master[split:], m, v, con)
    master[split:] = p
    return (master, mom, m, v), sc


def test_muon_step_follows_the_definition():
    """Three steps and one with an overflow between them, matrices and other
    tensors together, eager and from a captured graph. The momentum and
    AdamW's arrays are bit-exact; the matrices' weights are off by at most
    lr * scale * (the orthogonalisation's error) in each step."""
    import oracle as O
    from zero_sharded_mixed_tensor_amd.step import MuonStep
    mats, split = layout([(96, 160), (200, 72), (64, 64), (300, 300)], gap=64)
    split = -(-split // 64) * 64
    n = split + 5000
    rng = np.random.default_rng(17)
    master = (rng.standard_normal(n) * 0.02).astype(np.float32)
    pad = np.ones(split, bool)
    for o, r, c in mats:
        pad[o:o + r * c] = False
    master[:split][pad] = 0
    xs = [(rng.standard_normal(n) * 1e-2 * 2.0 ** 10).astype(np.float16).view(np.uint16) for _ in range(4)]
    for x in xs:
        x[:split][pad] = 0
    xs[2][7] = 0x7C00  # an infinity
    cfg = dict(K=2, max_norm=1.0, lr=2e-2, wd=0.1)
    muon = zds.muon_hparams(lr=cfg["lr"], momentum=0.95, weight_decay=cfg["wd"], scale="rms")

    def fresh():
        st = MuonStep(n, split, mats, zds.hparams(), muon, zds.scaler_config(initial_scale_power=10), 1.0, 2)
        dev = [torch.from_numpy(master.copy()).cuda(), torch.zeros(split, device="cuda"),
               torch.zeros(n - split, device="cuda"), torch.zeros(n - split, device="cuda"),
               torch.zeros(n, dtype=torch.float16, device="cuda")]
        return st, dev

    st, dev = fresh()
    want = [master.copy(), np.zeros(split, np.float32), np.zeros(n - split, np.float32), np.zeros(n - split, np.float32)]
    ost = O.scaler_init(initial_scale_power=10)
    hp = O.AdamW()
    norms = {k: 0.2 * np.sqrt(max(r, c)) * np.sqrt(min(r, c)) * 1.3 for k, (_, r, c) in enumerate(mats)}
    eager, steps = [], 0
    for x in xs:
        st.step(to_dev(x, "fp16"), dev[0], dev[1], dev[2], dev[3], dev[4])
        new, sc = _oracle_step(O, x, want[0], want[1], want[2], want[3], ost, hp, mats, split, cfg)
        ost = O.scaler_update(ost, sc["overflow"], hp.beta1, hp.beta2)
        s = st.read_state()
        assert (s.t, s.scale, s.steps_skipped) == (ost.t, ost.scale, int(x is xs[2] or x is xs[3]))
        if new is not None:
            want, steps = list(new), steps + 1
        got = [to_host(t) for t in dev]
        assert np.array_equal(got[1], want[1])
        assert np.array_equal(got[0][split:], want[0][split:])
        assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])
        assert (got[0][:split][pad] == 0).all()
        for k, (o, r, c) in enumerate(mats):
            a, b = got[0][o:o + r * c].astype(np.float64), want[0][o:o + r * c].astype(np.float64)
            assert np.linalg.norm(a - b) <= steps * cfg["lr"] * norms[k] * TOL["bf16"] + 1e-6 * np.linalg.norm(b)
            assert np.array_equal(got[4][o:o + r * c], narrow(got[0][o:o + r * c], "fp16"))
        eager.append([t.clone() for t in dev])
    # the same steps replayed from a graph
    st, dev = fresh()
    g = to_dev(xs[0], "fp16")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        st.step(g, dev[0], dev[1], dev[2], dev[3], dev[4])
    for x, e in zip(xs, eager):
        g.copy_(to_dev(x, "fp16"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(dev, e):
            assert torch.equal(a, b)


def test_muon_step_from_config_and_refusals():
    from zero_sharded_mixed_tensor_amd.config import from_ds_config
    from zero_sharded_mixed_tensor_amd.step import MuonStep
    cfg = from_ds_config({"optimizer": {"type": "Muon", "params": {"lr": 1e-2, "ns_steps": 3}}, "bf16": {"enabled": True}})
    st = MuonStep.from_config(64 * 64, 64 * 64, [(0, 64, 64)], cfg)
    assert st.ns_steps == 3 and st.split == 4096
    g = torch.randn(4096, device="cuda").bfloat16()
    w, m = torch.randn(4096, device="cuda"), torch.zeros(4096, device="cuda")
    e = torch.empty(0, device="cuda")
    before = w.clone()
    st.step(g, w, m, e, e, None)                 # nothing but matrices, no 16-bit copy
    assert not torch.equal(w, before) and torch.isfinite(w).all()
    for split in (4095, -1, 4097):
        with pytest.raises(zds.ZdsError):
            MuonStep(4096, split, [(0, 64, 64)])

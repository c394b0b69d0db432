"""The accuracy of the orthogonalisation against 64 bits, next to that of the
same steps in plain fp32 (FP32 results) or of one rounding (BF16 results)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from zero_sharded_mixed_tensor_amd import zds  # noqa: E402

QUINTIC = (3.4445, -4.7750, 2.0315)


def steps_of(x, coef):
    """The steps in x's type; in 64 bits with the coefficients the call gets."""
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    x = x / (x.norm() + 1e-7)
    for a, b, c in torch.tensor(coef, dtype=torch.float32).double().tolist():
        g = x @ x.T.contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T.contiguous() if tall else x


def orthogonalise(shapes, dtype, coef=None, seed=1):
    """{(rows, cols): (err, ref)}: squared errors summed over a shape's
    matrices, the library's and the reference's (plain fp32, or the exact
    result rounded to bf16)."""
    mats, pos = [], 0
    for r, c in shapes:
        mats.append((pos, r, c))
        pos += r * c
    x = torch.randn(pos, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, dtype)
    ws.fill_(0xFF)
    y = torch.zeros_like(x)
    coef = [QUINTIC] * 5 if coef is None else coef
    zds.zds_newton_schulz(plan, x, y, ws, steps=len(coef), coef=coef)
    again = torch.zeros_like(x)
    zds.zds_newton_schulz(plan, x, again, ws, steps=len(coef), coef=coef)
    assert torch.equal(again, y)
    out = {}
    for o, r, c in mats:
        g = x[o:o + r * c].view(r, c)
        want = steps_of(g.double(), coef)
        ref = steps_of(g, coef) if dtype == torch.float32 else want.bfloat16()
        e, f = out.get((r, c), (0.0, 0.0))
        out[r, c] = (e + (y[o:o + r * c].view(r, c).double() - want).square().sum().item(),
                     f + (ref.double() - want).square().sum().item())
    plan.close()
    return out


@pytest.mark.parametrize("rows,cols", [(2, 2), (2, 64), (4, 5), (8, 8), (8, 9), (16, 16), (16, 17), (17, 16), (16, 300),
                                       (24, 3000), (31, 31), (32, 32), (1000, 32), (48, 48), (64, 64), (64, 2000)])
def test_fp32_results_of_few_rows(rows, cols):
    """A pair of fp16 numbers holds a value to half a step of fp32 (11 bits,
    then 11 bits of a remainder of at most 2^-12), and the product of two low
    halves, which is left out, is at most as large again. So each operation is
    off by at most twice what plain fp32's is. Many matrices together, as few
    roundings decide about one of them."""
    n = max(4, min(400, 20000 // (rows * cols)))
    err, plain = orthogonalise([(rows, cols)] * n, torch.float32)[rows, cols]
    assert err <= 4 * plain, (err / plain) ** 0.5


def test_fp32_results_of_a_mixed_set():
    shapes = [(16, 32)] * 24 + [(64, 64)] * 16 + [(96, 160)] * 12 + [(256, 128)] * 8 + [(200, 333)] * 4
    for shape, (err, plain) in orthogonalise(shapes, torch.float32).items():
        assert err <= 4 * plain, (shape, (err / plain) ** 0.5)


MIXED = [
    [(16, 32)] * 24 + [(64, 64)] * 16 + [(96, 160)] * 12 + [(256, 128)] * 8 + [(200, 333)] * 4,
    [(16, 32)] * 24 + [(256, 256)],
    [(32, 1000)] * 4 + [(1024, 4096)] * 4,
    [(3000, 24)] * 2 + [(600, 700)] + [(5, 64)] * 60,
    [(1000, 4096)] * 2 + [(777, 1333)] * 3 + [(40, 513)] * 2 + [(1025, 1023)],   # tiles of 128 and 256
    [(1100, 1110)] * 12 + [(30, 4000)] * 2,                # tiles of 128, two to a unit
    [(2000, 2040)] * 8 + [(33, 70)] * 20,                  # tiles of 256, the last ones in pieces
    [(4000, 4090), (64, 4096)],                            # tiles of 192
    [(128, 4096), (48, 4090), (250, 2000), (256, 256), (100, 120)],   # pieces of tiles of 128
    # the larger tiles' kernels that carry pairs: 128 alone on a unit, sums in pieces, 256, 192
    [(131, 4946)] + [(4, 2208)] * 4,
    [(1203, 89)] + [(9, 3284)] * 2,
    [(2874, 3390)] * 2 + [(26, 974)] * 4,
    [(3390, 3460)] * 3 + [(37, 1860)] * 3 + [(340, 327)] * 14 + [(89, 72)] * 5,
    [(1190, 1158)] * 13 + [(6, 677)] * 6,
    [(1516, 1196)] * 5 + [(145, 70)] * 13 + [(30, 106)] * 3,
    [(2956, 2953), (273, 339), (2423, 69), (2423, 69), (61, 726)] + [(83, 930)] * 14,
]


@pytest.mark.parametrize("shapes", MIXED, ids=lambda s: "+".join("%dx%d" % x for x in dict.fromkeys(s)))
def test_bf16_results_of_a_mixed_set_are_about_one_rounding(shapes):
    """Each shape's error: that of rounding the exact result and, independent
    of it, at most as much again from the roundings of X, A and B to fp16. Up
    to 64 rows A and B are pairs, which leaves a third of that (its square), in
    whatever company the matrix is. 5 % for the draw."""
    for shape, (err, rounding) in orthogonalise(shapes, torch.bfloat16).items():
        before = 1 / 3 if min(shape) <= 64 else 1
        assert err <= (1 + before) * 1.05 ** 2 * rounding, (shape, (err / rounding) ** 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("coef", [(1.0, 1e-39, 0.0), (1.0, 0.0, -1e-36), (2.0, 1e-30, 1e-30), (1.0, 0.0, 0.0)])
def test_coefficients_next_to_zero(dtype, coef):
    """B next to nothing: the result is a X. The norm is off by an fp32 rounding
    or two, and a BF16 result is rounded once."""
    x = torch.randn(40 * 70, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    plan = zds.zds_matrix_plan_create([(0, 40, 70)])
    y = torch.full_like(x, 9.0)
    zds.zds_newton_schulz(plan, x, y, zds.new_newton_schulz_workspace(plan, dtype), steps=1, coef=[coef])
    want = coef[0] * x.double() / x.double().norm()
    assert ((y.double() - want).abs() <= want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -21) + 2.0 ** -24).all()
    plan.close()


# Steps that start steep and flatten; every value stays below 2.
STEEP = [(8.2052, -22.9018, 16.4607), (4.0664, -2.8612, 0.5184), (3.9096, -2.8234, 0.5250), (3.2856, -2.4153, 0.4853),
         (2.2779, -1.6199, 0.3985), (1.8726, -1.2307, 0.3585), (1.875, -1.25, 0.375)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (40, 70), (96, 160), (600, 512), (2000, 2040)])
@pytest.mark.parametrize("steps", [1, 2, 3, 7])
def test_steep_steps_do_not_diverge(dtype, shape, steps):
    """A matrix of equal elements has the singular value 1, where the first
    step is steepest, and its roundings all point one way. No
    step takes a value of up to 1 + 2^-8 past 1.992; 5 % for the roundings."""
    r, c = shape
    x = torch.full((r * c,), 0.7, device="cuda").to(dtype)
    plan = zds.zds_matrix_plan_create([(0, r, c)])
    y = torch.zeros_like(x)
    zds.zds_newton_schulz(plan, x, y, zds.new_newton_schulz_workspace(plan, dtype), steps=steps, coef=STEEP[:steps])
    assert torch.isfinite(y).all() and y.double().norm().item() < 2.1
    plan.close()


@pytest.mark.parametrize("coef", [STEEP, [(1.875, -1.25, 0.375)] * 16, [(1.5, -0.5, 0.0)] * 12, [QUINTIC] * 3],
                         ids=["steep", "quintic16", "cubic12", "default3"])
def test_bf16_results_of_other_steps_are_about_one_rounding(coef):
    """As for the default steps: one rounding and as much again of everything
    before it, 5 % for the draw. What the product leaves out of X (its
    remainder behind 11 bits) must then follow the coefficients that are given."""
    shapes = [(65, 65)] * 4 + [(96, 160)] * 3 + [(256, 128)] * 3 + [(400, 1500)] * 2 + [(1500, 2000)]
    for shape, (err, rounding) in orthogonalise(shapes, torch.bfloat16, coef).items():
        assert err <= 2 * 1.05 ** 2 * rounding, (shape, (err / rounding) ** 0.5)

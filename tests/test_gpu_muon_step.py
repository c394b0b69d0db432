"""MuonStep on the GPU: what a refused step leaves, and a rank's set of more
than one group of matrices."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from zero_sharded_mixed_tensor_amd import zds  # noqa: E402
from zero_sharded_mixed_tensor_amd.step import MuonStep  # noqa: E402


def test_a_refused_step_changes_nothing():
    n, split = 64 * 64 + 1000, 64 * 64
    st = MuonStep(n, split, [(0, 64, 64)])
    a = dict(grads=torch.randn(n, device="cuda").bfloat16(), master=torch.randn(n, device="cuda"),
             momentum=torch.randn(split, device="cuda"), exp_avg=torch.randn(n - split, device="cuda"),
             exp_avg_sq=torch.rand(n - split, device="cuda"), params_out=torch.zeros(n, device="cuda").bfloat16())
    before = {k: t.clone() for k, t in a.items()}
    for change in (dict(params_out=a["params_out"][:split]), dict(exp_avg_sq=a["exp_avg_sq"][:-1]),
                   dict(exp_avg=a["exp_avg"].cpu()), dict(params_out=a["master"].view(torch.bfloat16)[:n])):
        with pytest.raises(zds.ZdsError):
            st.step(**dict(a, **change))
    torch.cuda.synchronize()
    for k, t in a.items():
        assert torch.equal(t, before[k]), k
    t0 = st.read_state().t
    st.step(**a)
    assert st.read_state().t == t0 + 1
    for k in ("master", "momentum", "exp_avg", "exp_avg_sq", "params_out"):
        assert not torch.equal(a[k], before[k]), k


@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, 2.0 ** -7), (torch.float32, 3e-5)])
def test_a_set_of_two_groups(dtype, tol):
    """Matrices of more than 2^28 elements together go through the launches in
    groups, one after another in one workspace; the second here also with sums
    in pieces. Tolerances as for the other sets of these sizes (2-norm): a BF16
    rounding and as much again; for FP32 22-bit operands and fp32 sums."""
    mats, pos = [], 0
    for r, c in [(4096, 4096)] * 16 + [(2000, 2040)] * 8:
        mats.append((pos, r, c))
        pos += r * c + 8
    x = torch.empty(pos, device="cuda", dtype=dtype).normal_(generator=torch.Generator("cuda").manual_seed(4))
    plan = zds.zds_matrix_plan_create(mats)
    ws = zds.new_newton_schulz_workspace(plan, dtype)
    one = zds.zds_matrix_plan_create(mats[:1])
    assert ws.numel() < 17 * zds.zds_newton_schulz_workspace_bytes(one, dtype)      # one group's, not all's
    one.close()
    ws.fill_(0xFF)
    y = torch.full_like(x, 9.0)
    zds.zds_newton_schulz(plan, x, y, ws)
    for k in (0, 15, 16, 23):
        o, r, c = mats[k]
        g = x[o:o + r * c].view(r, c).double()
        g = g / (g.norm() + 1e-7)
        for _ in range(5):
            a = g @ g.T.contiguous()
            g = 3.4445 * g + (-4.7750 * a + 2.0315 * (a @ a)) @ g
        assert ((y[o:o + r * c].view(r, c).double() - g).norm() / g.norm()).item() <= tol, k
        assert (y[o + r * c:o + r * c + 8] == 9).all()
    again = torch.full_like(x, 9.0)
    zds.zds_newton_schulz(plan, x, again, ws)
    assert torch.equal(again, y)
    plan.close()


def test_a_muon_rank_is_saved_and_resumed(tmp_path):
    """Three steps, a save, a load into fresh buffers and two more end on the
    bits of five straight; the merged file holds every tensor."""
    shapes = [(96, 160), (200, 72), (64, 64), (777,), (5000,)]
    numels = [torch.Size(s).numel() for s in shapes]
    offs, n = zds.zds_flat_layout(numels, 64)
    offs, split = list(offs), offs[3]
    mats = [(o, *s) for o, s in zip(offs, shapes[:3])]
    g = torch.Generator("cuda").manual_seed(6)
    grads = [torch.empty(n, device="cuda").normal_(0, 1e-2, generator=g).bfloat16() for _ in range(5)]
    start = torch.empty(n, device="cuda").normal_(0, 0.02, generator=g)
    for x in grads + [start]:                            # the layout's padding is zero
        for o, k, e in zip(offs, numels, offs[1:] + [n]):
            x[o + k:e] = 0

    def fresh():
        st = MuonStep(n, split, mats, muon=zds.muon_hparams(lr=1e-2, scale="rms"))
        p, m, v = start.clone(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        return st, p, m, v, torch.zeros(n, dtype=torch.bfloat16, device="cuda")

    def run(st, p, m, v, out, some):
        for x in some:
            st.step(x, p, m[:split], m[split:], v[split:], out)

    straight = fresh()
    run(*straight, grads)
    first = fresh()
    run(*first, grads[:3])
    meta, path = zds.checkpoint_meta(numels, 1, 0, 64), str(tmp_path / "rank0.zckpt")
    zds.zds_checkpoint_save(path, meta, numels, first[1], first[2], first[3], first[0].base.state)
    second = fresh()
    zds.zds_checkpoint_load(path, meta, numels, second[1], second[2], second[3], second[0].base.state)
    assert second[0].read_state().t == 3
    run(*second, grads[3:])
    torch.cuda.synchronize()
    for a, b in zip(straight[1:], second[1:]):
        assert torch.equal(a, b)
    assert second[0].read_state().t == straight[0].read_state().t == 5
    for section, whole in ((0, first[1]), (1, first[2])):
        parts = zds.split_consolidated(zds.zds_consolidate_fp32([path], section), numels)
        for o, k, part in zip(offs, numels, parts):
            assert torch.equal(torch.from_numpy(part), whole[o:o + k].cpu())


def test_a_step_on_another_stream_than_the_current_one():
    """Built while the current stream is busy and run on one of the caller's at
    once: nothing that the construction left on the current stream comes later."""
    n, split = 200 * 72 + 3000, 200 * 72
    g = torch.randn(n, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    start = torch.randn(n, generator=torch.Generator().manual_seed(10)).cuda()

    def run(stream, busy):
        a = [g, start.clone(), torch.zeros(split, device="cuda"), torch.zeros(n - split, device="cuda"),
             torch.zeros(n - split, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
        torch.cuda.synchronize()
        if busy:
            x = torch.ones(4096, 4096, device="cuda")
            for _ in range(20):
                x = x @ x * 1e-4
        st = MuonStep(n, split, [(0, 200, 72)], stream=stream)
        for _ in range(2):
            st.step(*a, stream=stream)
        torch.cuda.synchronize()
        return st, a

    want, a = run(None, False)
    got, b = run(torch.cuda.Stream(), True)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert torch.equal(got.update, want.update) and got.update.abs().max() > 0
    assert got.read_state().t == want.read_state().t == 2

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

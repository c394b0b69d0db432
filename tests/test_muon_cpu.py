"""CPU checks of Muon's entry points: everything they refuse is refused before
the device is touched, and the plain definitions agree with each other."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import muon as M

zds = pytest.importorskip("zero_sharded_mixed_tensor_amd.zds", reason="libzds.so not built")


def _raises(text, fn):
    with pytest.raises(zds.ZdsError) as e:
        fn()
    assert text in str(e.value), str(e.value)


@pytest.mark.parametrize("mats,text", [
    ([(0, -1, 4)], "sizes must lie"),
    ([(0, 4, 1 << 17)], "sizes must lie"),
    ([(0, 60000, 60000)], "2^31 elements"),
    ([(-1, 4, 4)], "offset must lie"),
    ([(1 << 40, 4, 4)], "offset must lie"),
    ([(0, 4, 4), (15, 4, 4)], "overlap"),
    ([(100, 3, 3), (0, 10, 11)], "overlap"),
    ([(0, 4, 4), (0, 4, 4)], "overlap"),
    ([(0, 1 << 40, 4)], "out of range"),
])
def test_plan_refusals(mats, text):
    _raises(text, lambda: zds.zds_matrix_plan_create(mats))


def test_plan_null_arguments():
    lib = zds.lib
    h = ctypes.c_void_p()
    assert lib.zds_matrix_plan_create(None, None, None, None, 0) == zds.ZDS_EINVAL
    assert lib.zds_matrix_plan_create(ctypes.byref(h), None, None, None, 1) == zds.ZDS_EINVAL
    assert lib.zds_matrix_plan_create(ctypes.byref(h), None, None, None, -1) == zds.ZDS_EINVAL
    lib.zds_matrix_plan_destroy(None)
    assert lib.zds_matrix_plan_num_matrices(None) == -1 and lib.zds_matrix_plan_span(None) == -1
    assert lib.zds_newton_schulz_workspace_bytes(None, zds.ZDS_BF16) == 0


@pytest.mark.parametrize("change,text", [
    (dict(lr=-1.0), "lr"), (dict(lr=float("nan")), "lr"), (dict(lr=float("inf")), "lr"),
    (dict(weight_decay=-0.1), "weight_decay"), (dict(weight_decay=float("inf")), "weight_decay"),
    (dict(momentum=1.0), "momentum"), (dict(momentum=-0.1), "momentum"), (dict(momentum=float("nan")), "momentum"),
])
def test_hparam_refusals(change, text):
    hp = zds.muon_hparams(**change)
    p = ctypes.c_void_p(64)
    args = (ctypes.byref(hp), p, zds.ZDS_BF16, p, p, zds.ZDS_BF16, 8, p, None)
    assert zds.lib.zds_muon_momentum(*args) == zds.ZDS_EINVAL and text in zds.zds_last_error()
    assert zds.lib.zds_muon_apply(ctypes.byref(hp), None, p, zds.ZDS_BF16, p, p, zds.ZDS_BF16, p, None) == zds.ZDS_EINVAL
    assert text in zds.zds_last_error()


def test_enum_refusals():
    p = ctypes.c_void_p(64)
    for f, v in (("nesterov", 2), ("nesterov", -1), ("scale", 3), ("scale", -1)):
        hp = zds.muon_hparams()
        setattr(hp, f, v)
        assert zds.lib.zds_muon_momentum(ctypes.byref(hp), p, zds.ZDS_BF16, p, p, zds.ZDS_BF16, 8, p, None) == zds.ZDS_EINVAL
    _raises("scale must be", lambda: zds.muon_hparams(scale="fan"))
    assert zds.lib.zds_muon_momentum(None, p, zds.ZDS_BF16, p, p, zds.ZDS_BF16, 8, p, None) == zds.ZDS_EINVAL


def test_momentum_refusals():
    hp = ctypes.byref(zds.muon_hparams())
    f = zds.lib.zds_muon_momentum
    p, odd = ctypes.c_void_p(64), ctypes.c_void_p(65)
    assert f(hp, p, 7, p, p, zds.ZDS_BF16, 8, p, None) == zds.ZDS_EINVAL
    assert f(hp, p, zds.ZDS_BF16, p, p, zds.ZDS_FP16, 8, p, None) == zds.ZDS_EINVAL
    assert f(hp, p, zds.ZDS_BF16, p, p, zds.ZDS_BF16, -1, p, None) == zds.ZDS_EINVAL
    assert f(hp, p, zds.ZDS_BF16, p, p, zds.ZDS_BF16, 1 << 40, p, None) == zds.ZDS_EINVAL
    for k in range(4):
        a = [p, p, p, p]
        a[k] = None
        assert f(hp, a[0], zds.ZDS_BF16, a[1], a[2], zds.ZDS_BF16, 8, a[3], None) == zds.ZDS_EINVAL
        a[k] = odd
        assert f(hp, a[0], zds.ZDS_BF16, a[1], a[2], zds.ZDS_BF16, 8, a[3], None) == zds.ZDS_EALIGN
    assert f(hp, None, zds.ZDS_BF16, None, None, zds.ZDS_BF16, 0, None, None) == zds.ZDS_OK


def test_momentum_overlaps_are_refused():
    hp = ctypes.byref(zds.muon_hparams())
    f = zds.lib.zds_muon_momentum
    at = lambda k: ctypes.c_void_p(1 << 20 | k)
    sc = ctypes.c_void_p(1 << 24)
    for g, m, u, gdt in ((0, 1996, 65536, zds.ZDS_BF16), (0, 65536, 1998, zds.ZDS_BF16), (0, 65536, 0, zds.ZDS_FP32),
                         (0, 65536, 2, zds.ZDS_BF16), (65536, 0, 3998, zds.ZDS_BF16), (3998, 0, 65536, zds.ZDS_BF16)):
        assert f(hp, at(g), gdt, at(m), at(u), zds.ZDS_BF16, 1000, sc, None) == zds.ZDS_EINVAL, (g, m, u)
        assert "overlap" in zds.zds_last_error()


def test_momentum_binding_lengths():
    hp, sc = zds.muon_hparams(), torch.zeros(64, dtype=torch.uint8)
    g, m, u = torch.zeros(100, dtype=torch.bfloat16), torch.zeros(100), torch.zeros(100, dtype=torch.bfloat16)
    _raises("grads holds 99", lambda: zds.zds_muon_momentum(hp, g[:99], m, u, sc))
    _raises("update holds 99", lambda: zds.zds_muon_momentum(hp, g, m, u[:99], sc))
    _raises("momentum holds 100", lambda: zds.zds_muon_momentum(hp, g, m, u, sc, n=101))
    _raises("must be fp32", lambda: zds.zds_muon_momentum(hp, g, m.double(), u, sc))
    _raises("scalars holds", lambda: zds.zds_muon_momentum(hp, g, m, u, sc[:8]))
    _raises("device tensor", lambda: zds.zds_muon_momentum(hp, g, m, u, sc))


def _ns(steps=5, coef=None, dtype=None):
    arr = None if coef is None else (ctypes.c_float * len(coef))(*coef)
    return zds.lib.zds_newton_schulz(None, None, None, zds.ZDS_BF16 if dtype is None else dtype, arr, steps, None, None, 0,
                                     None)


def test_newton_schulz_refusals():
    for kw, text in ((dict(dtype=zds.ZDS_FP16), "bf16 or fp32"), (dict(dtype=9), "bf16 or fp32"),
                     (dict(steps=0), "steps"), (dict(steps=17), "steps"),
                     (dict(steps=1, coef=[9.0, 0.0, 0.0]), "past 8"),
                     (dict(steps=1, coef=[float("nan"), 0.0, 0.0]), "past 8"),
                     (dict(steps=1, coef=[1.0, float("inf"), 0.0]), "past 8"),
                     # 1.9 s in every step: 13 after four
                     (dict(steps=4, coef=[1.9, 0.0, 0.0] * 4), "step 3"),
                     (dict(), "null plan"),
                     (dict(steps=3, coef=[2.0, 0.0, 0.0, 1.8, 0.0, 0.0, 2.0, 0.0, 0.0]), "null plan")):
        assert _ns(**kw) == zds.ZDS_EINVAL
        assert text in zds.zds_last_error(), (kw, zds.zds_last_error())


def test_newton_schulz_moves_singular_values_only():
    """The definition against its effect: the same singular vectors, each
    singular value through the steps' polynomial."""
    rng = np.random.default_rng(3)
    for r, c in ((20, 33), (33, 20), (16, 16)):
        g = rng.standard_normal((r, c))
        u, s, vt = np.linalg.svd(g, full_matrices=False)
        s = s / (np.linalg.norm(g) + 1e-7)
        for _ in range(5):
            a, b, k = np.float32(M.QUINTIC).astype(np.float64)
            s = a * s + b * s ** 3 + k * s ** 5
        assert np.abs(M.newton_schulz(g) - (u * s) @ vt).max() < 1e-12
        assert 0.3 < s.min() and s.max() < 1.3


def test_apply_scales():
    assert M.muon_scale(400, 100, "aspect") == np.float32(2.0) and M.muon_scale(100, 400, "aspect") == np.float32(1.0)
    assert M.muon_scale(100, 400, "rms") == np.float32(0.2 * 20.0) and M.muon_scale(3, 7, "none") == 1.0


def test_config_maps_muon():
    from zero_sharded_mixed_tensor_amd.config import ConfigError, from_ds_config
    c = from_ds_config({"optimizer": {"type": "Muon", "params": {"lr": 2e-2, "weight_decay": 0.1}},
                        "bf16": {"enabled": True}, "gradient_clipping": 1.0})
    assert (c.muon.lr, c.muon.momentum, c.muon.nesterov, c.muon.ns_steps, c.muon.scale) == (2e-2, 0.95, True, 5, "aspect")
    assert c.lr == 2e-2 and c.param_dtype == "bf16"
    hp = c.muon_hparams()
    assert abs(hp.lr - 2e-2) < 1e-8 and hp.scale == zds.ZDS_MUON_SCALE_ASPECT and abs(hp.weight_decay - 0.1) < 1e-8
    c = from_ds_config({"optimizer": {"type": "muon", "params": {
        "lr": 1e-3, "muon_lr": 5e-3, "adam_lr": 3e-4, "momentum": 0.9, "nesterov": False, "ns_steps": 6, "scale": "rms",
        "betas": [0.8, 0.95]}}})
    assert (c.muon.lr, c.lr, c.beta1, c.beta2) == (5e-3, 3e-4, 0.8, 0.95)
    assert (c.muon.momentum, c.muon.nesterov, c.muon.ns_steps, c.muon.scale) == (0.9, False, 6, "rms")
    assert from_ds_config({}).muon is None
    with pytest.raises(ConfigError):
        from_ds_config({}).muon_hparams()
    for bad in ({"momentum": 1.0}, {"ns_steps": 0}, {"ns_steps": 17}, {"scale": "fan"}, {"nesterov": 1}, {"momentum": "x"}):
        with pytest.raises(ConfigError):
            from_ds_config({"optimizer": {"type": "Muon", "params": bad}})
    with pytest.raises(ConfigError):
        from_ds_config({"optimizer": {"type": "Muon"}, "zero_optimization": {"offload_optimizer": {"device": "cpu"}}})

"""MuonStep and the Muon configuration: what is refused, and before what.
Nothing here reaches a device."""

import pytest
import torch

from zero_sharded_mixed_tensor_amd.config import ConfigError, from_ds_config

zds = pytest.importorskip("zero_sharded_mixed_tensor_amd.zds", reason="libzds.so not built")
from zero_sharded_mixed_tensor_amd.step import MuonStep, ShardStep  # noqa: E402


def muon_config(**params):
    return from_ds_config({"optimizer": {"type": "Muon", "params": params}})


def test_a_muon_configuration_is_no_adamw_step():
    """Its hparams() are those of the tensors that AdamW updates next to the
    matrices: a step of them alone would update the matrices by AdamW, too."""
    with pytest.raises(zds.ZdsError) as e:
        ShardStep.from_config(64, muon_config(lr=1e-2))
    assert "MuonStep" in str(e.value)
    with pytest.raises(ConfigError):
        MuonStep.from_config(64, 64, [(0, 8, 8)], from_ds_config({}))


def test_auto_takes_the_default():
    auto = muon_config(lr="auto", muon_lr="auto", adam_lr="auto", momentum="auto", nesterov="auto", ns_steps="auto",
                       scale="auto", weight_decay="auto")
    assert auto == muon_config()
    assert muon_config(nesterov=None, scale=None) == muon_config()
    for bad in ({"nesterov": "yes"}, {"nesterov": 0}, {"scale": "automatic"}, {"scale": 1}):
        with pytest.raises(ConfigError):
            muon_config(**bad)


def test_one_set_of_defaults():
    """A recipe that names no value is the same step from the configuration and
    from the library."""
    for want, got in ((zds.muon_hparams(), muon_config().muon_hparams()), (zds.hparams(), muon_config().hparams())):
        assert bytes(want) == bytes(got)
    from inspect import signature
    assert muon_config().muon.ns_steps == signature(MuonStep).parameters["ns_steps"].default
    assert muon_config().muon.ns_steps == signature(zds.zds_newton_schulz).parameters["steps"].default


class Recorder:
    """Stands in for the four calls of a step, in order."""

    def __init__(self, monkeypatch):
        self.calls, self.args = [], []
        for name in ("zds_muon_momentum", "zds_newton_schulz", "zds_muon_apply", "zds_adam_step"):
            monkeypatch.setattr(zds, name, lambda *a, _n=name, **k: (self.calls.append(_n), self.args.append(a)))
        monkeypatch.setattr(zds, "_here", lambda t, what: t.data_ptr())   # (the tensors here lie on the host)


def host_step(n=200, split=128, steps=5):
    st = MuonStep.__new__(MuonStep)
    st.n, st.split, st.ns_steps, st.muon = n, split, steps, zds.muon_hparams()
    st.base = ShardStep.__new__(ShardStep)
    st.base.hp, st.base.scalars, st.base.state = zds.hparams(), torch.zeros(64, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8)
    st.plan, st.ws = None, None
    st.update = torch.zeros(split, dtype=torch.bfloat16)
    return st


def arrays(n=200, split=128):
    return dict(grads=torch.zeros(n, dtype=torch.bfloat16), master=torch.zeros(n), momentum=torch.zeros(split),
                exp_avg=torch.zeros(n - split), exp_avg_sq=torch.zeros(n - split),
                params_out=torch.zeros(n, dtype=torch.bfloat16))


def test_a_step_makes_its_calls_in_order(monkeypatch):
    rec = Recorder(monkeypatch)
    host_step().apply(**arrays())
    host_step().apply(**dict(arrays(), params_out=None))
    assert rec.calls == ["zds_muon_momentum", "zds_newton_schulz", "zds_muon_apply", "zds_adam_step"] * 2


def test_adamw_gets_what_lies_behind_the_split(monkeypatch):
    """Of arrays of any shape, and the grads' own place may take the params."""
    rec = Recorder(monkeypatch)
    a = arrays()
    a["grads"], a["master"] = torch.zeros(50, 4), torch.zeros(4, 50)
    host_step().apply(**a)
    for t, whole in ((rec.args[3][1], a["grads"]), (rec.args[3][2], a["master"]), (rec.args[3][5], a["params_out"])):
        assert t.numel() == 72 and t.data_ptr() == whole.data_ptr() + 128 * whole.element_size()
    a = arrays()
    host_step().apply(**dict(a, params_out=a["grads"]))
    assert len(rec.calls) == 8


@pytest.mark.parametrize("change", [
    dict(grads=torch.zeros(199, dtype=torch.bfloat16)), dict(grads=torch.zeros(200, dtype=torch.int16)),
    dict(grads=None), dict(grads=torch.zeros(400)[::2]),
    dict(master=torch.zeros(199)), dict(master=torch.zeros(200, dtype=torch.float64)),
    dict(momentum=torch.zeros(127)), dict(momentum=torch.zeros(128, dtype=torch.bfloat16)),
    dict(exp_avg=torch.zeros(71)), dict(exp_avg=torch.zeros(72, dtype=torch.bfloat16)), dict(exp_avg=None),
    dict(exp_avg_sq=torch.zeros(71)), dict(exp_avg_sq=torch.zeros(72, dtype=torch.float16)),
    dict(params_out=torch.zeros(199, dtype=torch.bfloat16)), dict(params_out=torch.zeros(200)),
    dict(params_out=torch.zeros(128, dtype=torch.bfloat16)),
    dict(params_out=torch.zeros(400, dtype=torch.bfloat16)[::2]), dict(master=torch.zeros(400)[::2]),
], ids=lambda c: "-".join("%s%s" % (k, "" if v is None else "%s%s" % (tuple(v.shape), str(v.dtype)[6:])) for k, v in c.items()))
def test_what_any_call_of_a_step_would_refuse_is_refused_before_the_first(monkeypatch, change):
    """Half a step cannot be repeated: the momentum has moved."""
    rec = Recorder(monkeypatch)
    with pytest.raises(zds.ZdsError):
        host_step().apply(**dict(arrays(), **change))
    assert rec.calls == []


def test_overlaps_and_settings_are_refused_before_the_first_call(monkeypatch):
    rec = Recorder(monkeypatch)
    a = arrays()
    with pytest.raises(zds.ZdsError):
        host_step().apply(**dict(a, params_out=a["master"].view(torch.bfloat16)[:200]))
    both = torch.zeros(300)
    for x, y in (("master", "exp_avg"), ("momentum", "exp_avg_sq"), ("master", "momentum"), ("exp_avg", "exp_avg_sq")):
        with pytest.raises(zds.ZdsError):
            host_step().apply(**dict(a, **{x: both[:a[x].numel()], y: both[1:1 + a[y].numel()]}))
    for steps in (0, 17):
        with pytest.raises(zds.ZdsError):
            host_step(steps=steps).apply(**a)
    st = host_step()
    st.base.hp = zds.hparams(beta1=1.0)
    with pytest.raises(zds.ZdsError):
        st.apply(**a)
    assert rec.calls == []
    side = torch.zeros(200 + 128 + 72 + 72)            # one after another in one buffer is fine
    host_step().apply(a["grads"], side[:200], side[200:328], side[328:400], side[400:], a["params_out"])
    assert len(rec.calls) == 4

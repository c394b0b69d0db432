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

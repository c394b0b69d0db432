"""Moments in fewer bits and gradient dropout without a GPU: the generator
against its published vectors, the oracle's own pins, and what the entry
points, the binding, the step classes and the configuration refuse. No call
here reaches a device: each is refused before anything is enqueued, or handles
no element."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import quantised as Q
from zero_sharded_mixed_tensor_amd.config import ConfigError, from_ds_config

zds = pytest.importorskip("zero_sharded_mixed_tensor_amd.zds", reason="libzds.so not built")
from zero_sharded_mixed_tensor_amd.step import DropoutExchange, QuantisedStep, ShardStep  # noqa: E402

FORMATS = (Q.E4M3, Q.UE5M3)


# ------------------------------------------------------------------ the generator

@pytest.mark.parametrize("key,counter,want", [
    # the test vectors published with the generator
    (0, (0, 0, 0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    (2 ** 64 - 1, (0xFFFFFFFF,) * 4, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    (0x299F31D0A4093822, (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_generator_published_vectors(key, counter, want):
    call = counter[0] | counter[1] << 32
    assert tuple(zds.zds_random_words_host(key, call, counter[2], counter[3])) == want
    assert tuple(int(w) for w in Q.random_words(key, [call], counter[2], counter[3])[0]) == want


def test_generator_host_equals_oracle():
    rng = np.random.default_rng(3)
    for _ in range(50):
        seed, call = int(rng.integers(0, 2 ** 63)) * 2 + 1, int(rng.integers(0, 2 ** 62))
        step, stream = int(rng.integers(0, 2 ** 32)), int(rng.integers(0, 3))
        assert zds.zds_random_words_host(seed, call, step, stream) == [int(w) for w in
                                                                      Q.random_words(seed, [call], step, stream)[0]]


# ------------------------------------------------------------------ the oracle's pins

def _draw(fmt, n, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal(n) * 2.0 ** rng.integers(-30, 10, n)).astype(np.float32)
    return np.abs(x) if fmt == Q.UE5M3 else x


@pytest.mark.parametrize("fmt", FORMATS)
def test_nearest_code_by_exact_arithmetic(fmt):
    """Every element's code is the one of least distance, halves to the even one."""
    x = _draw(fmt, 32 * 7 + 5, 11)
    codes, exps = Q.quantise(x, fmt)
    table = [Fraction(v) for v in Q.code_values(fmt)]
    for i, v in enumerate(x):
        unit = Fraction(2) ** (int(exps[i // 32]) - 127)
        dist = [abs(abs(Fraction(float(v))) - t * unit) for t in table]
        best = min(dist)
        wanted = [c for c, d in enumerate(dist) if d == best]
        c = int(codes[i]) & Q.BAD[fmt]
        assert c in wanted or (fmt == Q.UE5M3 and c == 1 and wanted == [0])
        if len(wanted) == 2 and c != 1:
            assert c % 2 == 0
    # the largest magnitude of a block lies in its top binade, and below the top code
    for b in range(exps.size):
        top = np.abs(x[32 * b:32 * b + 32]).max()
        assert 0.875 * 2.0 ** (int(exps[b]) - 127) <= top <= 1.75 * 2.0 ** (int(exps[b]) - 127)


@pytest.mark.parametrize("fmt", FORMATS + (Q.BF16,))
def test_random_rounding_is_right_on_average(fmt):
    """Over all 65536 values of the random bits the mean of what is read back
    is the value itself: to half a step of 2^-16 (BF16: exactly, as its 16
    dropped bits are the 16 random ones)."""
    r = np.arange(65536)
    x = np.concatenate([_draw(fmt if fmt != Q.BF16 else Q.UE5M3, 31, 5)[:31], [np.float32(900.0)]]).astype(np.float32)
    for i in range(0, 31, 3):
        reads = []
        tiled = np.tile(x, 512)
        for k in range(0, 65536, 512):
            rr = np.repeat(r[k:k + 512], 32)
            codes, exps = Q.quantise(tiled, fmt, rr)
            reads.append(Q.read_back(codes, exps, fmt).reshape(-1, 32)[:, i])
        got = np.concatenate(reads)
        lo, hi = got.min(), got.max()
        if fmt == Q.UE5M3 and lo == 0 or hi == lo:
            continue
        assert abs(got.mean() - float(x[i])) <= (hi - lo) * 2.0 ** -17 * (0 if fmt == Q.BF16 else 1) + 1e-12 * abs(x[i])
        break
    else:
        pytest.fail("no element was rounded")


@pytest.mark.parametrize("fmt", FORMATS + (Q.BF16,))
@pytest.mark.parametrize("random", [False, True])
def test_values_survive_a_round_trip(fmt, random):
    """A block whose largest value lay just over 1.75 * 2^k may read back as
    1.75 * 2^k and then gets an exponent byte that is one less: other codes,
    but every value of the wider grid up to 1.75 * 2^k is one of the finer."""
    x = _draw(Q.UE5M3, 32 * 40 + 9, 2)
    codes, exps = Q.quantise(x, fmt)
    back = Q.read_back(codes, exps, fmt).astype(np.float32)
    r = np.full(x.size, 0xFFFF) if random else None
    again, exps2 = Q.quantise(back, fmt, r)
    assert np.array_equal(Q.read_back(again, exps2, fmt), Q.read_back(codes, exps, fmt))
    if exps is not None:
        assert (exps.astype(int) - exps2).min() >= 0 and (exps.astype(int) - exps2).max() <= 1


def test_special_values_of_the_oracle():
    x = np.zeros(96, np.float32)
    x[0], x[40], x[41], x[64], x[65] = np.inf, -1.0, 2.0 ** -149, 3.0, 2.0 ** -149
    codes, exps = Q.quantise(x, Q.UE5M3)
    assert codes[0] == 0xFF and exps[0] == 255 and codes[40] == 0xFF and codes[41] == 1
    assert codes[65] == 1 and codes[66] == 0 and np.isnan(Q.read_back(codes, exps, Q.UE5M3)[[0, 40]]).all()
    codes, exps = Q.quantise(np.float32([-np.inf, np.nan, -0.0, 1.75]), Q.E4M3)
    assert list(codes[:3]) == [0xFF, 0x7F, 0x80]


def test_kept_places_are_even():
    """Each of a group's places is kept equally often: the byte's top bits are
    the place, so all places have 256 / ratio of the byte's values; and the
    generator's bytes are even (a chi-square of 255 degrees of freedom lies
    below 255 + 5 sqrt(510) but for 1 in 10^5 seeds)."""
    n = 256 * 40000
    at = Q.kept_places(n, 256, 99, 512, 7)
    count = np.bincount(at % 256, minlength=256)
    chi = ((count - 40000 / 256) ** 2 / (40000 / 256)).sum()
    assert chi < 255 + 5 * 510 ** 0.5
    # the same numbers wherever a call begins
    part = Q.kept_places(256 * 17, 256, 99, 512 + 256 * 1000, 7)
    assert np.array_equal(part, at[1000:1017] - 256 * 1000)


# ------------------------------------------------------------------ refusals of the entry points

FAKE = 1 << 20        # an address that nothing reads: every call below is refused first


def _status(fn, *args):
    st = getattr(zds.lib, fn)(*args)
    return st, zds.lib.zds_last_error().decode()


def _refused(fn, args, text, status=None):
    st, msg = _status(fn, *args)
    assert st == (zds.ZDS_EINVAL if status is None else status) and text in msg, (st, msg)


def quantise_args(**kw):
    a = dict(src=FAKE, n=100, fmt=0, rounding=1, seed=1, first=0, state=FAKE * 2, codes=FAKE * 3, exps=FAKE * 4, stream=None)
    a.update(kw)
    return list(a.values())


def test_quantise_refusals():
    fn = "zds_state_quantise"
    for kw, text in ((dict(fmt=3), "format"), (dict(fmt=-1), "format"), (dict(rounding=2), "rounding"),
                     (dict(n=-1), "n must"), (dict(n=1 << 40), "n must"), (dict(first=-32), "first"),
                     (dict(first=16), "first"), (dict(first=(1 << 63) - 64), "first"), (dict(state=None), "state"), (dict(src=None), "null"),
                     (dict(codes=None), "null"), (dict(exps=None), "exps"), (dict(fmt=2), "no exps"),
                     (dict(codes=FAKE), "overlap"), (dict(exps=FAKE * 3), "overlap"), (dict(exps=FAKE + 396), "overlap")):
        _refused(fn, quantise_args(**kw), text)
    for kw in (dict(src=FAKE + 2), dict(state=FAKE * 2 + 4), dict(fmt=2, exps=None, codes=FAKE * 3 + 1)):
        _refused(fn, quantise_args(**kw), "aligned", zds.ZDS_EALIGN)
    assert _status(fn, *quantise_args(n=0))[0] == zds.ZDS_OK
    assert _status(fn, *quantise_args(n=0, rounding=0, first=5, state=None))[0] == zds.ZDS_OK


def test_dequantise_refusals():
    fn = "zds_state_dequantise"

    def args(**kw):
        a = dict(codes=FAKE, exps=FAKE * 2, n=100, fmt=1, dst=FAKE * 3, dtype=2, stream=None)
        a.update(kw)
        return list(a.values())
    for kw, text in ((dict(fmt=7), "format"), (dict(dtype=0), "dst dtype"), (dict(dtype=9), "dst dtype"),
                     (dict(n=-5), "n must"), (dict(codes=None), "null"), (dict(dst=None), "null"),
                     (dict(exps=None), "exps"), (dict(fmt=2), "no exps"), (dict(dst=FAKE - 396), "overlap"),
                     (dict(dst=FAKE * 2), "overlap")):
        _refused(fn, args(**kw), text)
    _refused(fn, args(dst=FAKE * 3 + 2), "aligned", zds.ZDS_EALIGN)
    assert _status(fn, *args(n=0))[0] == zds.ZDS_OK


def step_args(**kw):
    a = dict(hp=zds.hparams(), grads=FAKE, gdt=1, master=2 * FAKE, m=3 * FAKE, me=4 * FAKE, v=5 * FAKE, fmt=1, ve=6 * FAKE,
             out=7 * FAKE, pdt=1, n=100, seed=0, first=0, scalars=8 * FAKE, state=9 * FAKE, stream=None)
    a.update(kw)
    if a["hp"] is not None:
        a["hp"] = ctypes.byref(a["hp"])
    return list(a.values())


def test_step_refusals():
    fn = "zds_adam_step_q8"
    for kw, text in ((dict(hp=None), "hparams"), (dict(hp=zds.hparams(beta1=0.3)), "betas"),
                     (dict(hp=zds.hparams(eps=0.0)), "eps"), (dict(hp=zds.hparams(eps=1e-31)), "eps"), (dict(hp=zds.hparams(lr=float("nan"))), "lr"),
                     (dict(gdt=5), "grad dtype"), (dict(pdt=2), "param dtype"), (dict(fmt=0), "second moment"),
                     (dict(fmt=3), "second moment"), (dict(n=-1), "n must"), (dict(n=1 << 40), "n must"),
                     (dict(first=33), "first"), (dict(first=-32), "first"), (dict(first=(1 << 63) - 64), "first"),
                     (dict(fmt=2), "no exps"), (dict(fmt=2, ve=None, v=2 * FAKE + 398), "overlap"),
                     (dict(out=2 * FAKE), "overlap"), (dict(m=4 * FAKE + 3), "overlap"), (dict(ve=4 * FAKE), "overlap"),
                     (dict(gdt=2, out=FAKE), "overlap"), (dict(out=FAKE + 2), "overlap")):
        _refused(fn, step_args(**kw), text)
    for name in ("grads", "master", "m", "me", "v", "ve", "scalars", "state"):
        _refused(fn, step_args(**{name: None}), "null pointer")
    for kw in (dict(grads=FAKE + 1), dict(master=2 * FAKE + 2), dict(out=7 * FAKE + 1), dict(scalars=8 * FAKE + 4),
               dict(state=9 * FAKE + 4), dict(fmt=2, ve=None, v=5 * FAKE + 1)):
        _refused(fn, step_args(**kw), "aligned", zds.ZDS_EALIGN)
    assert _status(fn, *step_args(n=0))[0] == zds.ZDS_OK


def test_dropout_refusals():
    def comp(**kw):
        a = dict(x=FAKE, xdt=1, error=2 * FAKE, n=1000, ratio=4, seed=0, first=0, sc=None, state=3 * FAKE,
                 values=4 * FAKE, vdt=1, stream=None)
        a.update(kw)
        return list(a.values())
    fn = "zds_dropout_compress"
    for kw, text in ((dict(ratio=1), "ratio"), (dict(ratio=3), "ratio"), (dict(ratio=512), "ratio"),
                     (dict(ratio=-4), "ratio"), (dict(ratio=0), "ratio"), (dict(vdt=3), "value dtype"),
                     (dict(xdt=3), "x dtype"), (dict(n=-1), "n must"), (dict(n=1 << 40), "n must"),
                     (dict(first=2), "first"), (dict(first=-4), "first"), (dict(first=(1 << 63) - 64), "first"), (dict(x=None), "null"),
                     (dict(values=None), "null"), (dict(state=None), "null"), (dict(values=FAKE), "overlap"),
                     (dict(error=FAKE + 1996), "overlap"), (dict(values=2 * FAKE), "overlap")):
        _refused(fn, comp(**kw), text)
    for kw in (dict(x=FAKE + 1), dict(error=2 * FAKE + 2), dict(values=4 * FAKE + 1), dict(state=3 * FAKE + 4),
               dict(sc=5 * FAKE + 4)):
        _refused(fn, comp(**kw), "aligned", zds.ZDS_EALIGN)
    assert _status(fn, *comp(n=0))[0] == zds.ZDS_OK

    def dec(peers=(FAKE, 2 * FAKE), **kw):
        a = dict(peers=(ctypes.c_void_p * max(1, len(peers)))(*peers) if peers is not None else None,
                 num=2 if peers is None else len(peers), vdt=1, n=1000, ratio=4, seed=0, first=0, state=3 * FAKE,
                 dst=4 * FAKE, odt=2, mode=1, stream=None)
        a.update(kw)
        return list(a.values())
    fn = "zds_dropout_decompress"
    for kw, text in ((dict(num=0), "num_peers"), (dict(num=17), "num_peers"), (dict(mode=0), "mode"),
                     (dict(mode=3), "mode"), (dict(ratio=6), "ratio"), (dict(odt=0), "dst"), (dict(vdt=2, odt=1), "dst"),
                     (dict(first=6), "first"), (dict(first=(1 << 63) - 64), "first"), (dict(peers=None), "null"), (dict(dst=None), "null"),
                     (dict(state=None), "null"), (dict(peers=(FAKE, None)), "peer 1"), (dict(dst=2 * FAKE - 8), "overlaps peer 1")):
        _refused(fn, dec(**kw), text)
    for kw, text in ((dict(dst=4 * FAKE + 2), "aligned"), (dict(peers=(FAKE + 1, 2 * FAKE)), "peer 0")):
        _refused(fn, dec(**kw), text, zds.ZDS_EALIGN)
    assert _status(fn, *dec(n=0))[0] == zds.ZDS_OK


def test_random_words_refuses_null():
    assert _status("zds_random_words_host", 0, 0, 0, 0, None)[0] == zds.ZDS_EINVAL


# ------------------------------------------------------------------ the binding

def _raises(fn, text):
    with pytest.raises(zds.ZdsError) as e:
        fn()
    assert text in str(e.value), str(e.value)


def _f32(n):
    return torch.zeros(n)


def test_binding_lengths():
    st, sc = torch.zeros(64, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8)
    m = zds.new_quantised_state(100, zds.ZDS_STATE_E4M3, "cpu")
    v = zds.new_quantised_state(100, zds.ZDS_STATE_UE5M3, "cpu")
    w = zds.new_quantised_state(100, zds.ZDS_STATE_BF16, "cpu")
    assert m.exps.numel() == 4 and w.exps is None and w.codes.dtype == torch.bfloat16
    _raises(lambda: zds.new_quantised_state(4, 9, "cpu"), "format")
    _raises(lambda: zds.zds_state_quantise(_f32(99), m, n=100), "src holds 99")
    _raises(lambda: zds.zds_state_quantise(_f32(101), m), "codes holds 100")
    _raises(lambda: zds.zds_state_quantise(_f32(100).double(), m), "fp32")
    _raises(lambda: zds.zds_state_quantise(_f32(100), m, state=st[:63]), "state holds 63")
    _raises(lambda: zds.zds_state_quantise(_f32(100), zds.QuantisedState(0, m.codes, m.exps[:3])), "exps holds 3")
    _raises(lambda: zds.zds_state_quantise(_f32(100), zds.QuantisedState(0, m.codes)), "exps is missing")
    _raises(lambda: zds.zds_state_quantise(_f32(100), zds.QuantisedState(2, w.codes, m.exps)), "no exps")
    _raises(lambda: zds.zds_state_quantise(_f32(100), zds.QuantisedState(2, m.codes)), "must be bf16")
    _raises(lambda: zds.zds_state_quantise(_f32(100), m.codes), "QuantisedState")
    _raises(lambda: zds.zds_state_quantise(_f32(100), m, seed=-1), "device tensor")   # (buffers come first)
    _raises(lambda: zds.zds_state_dequantise(m, _f32(101)), "codes holds 100")
    _raises(lambda: zds.zds_state_dequantise(m, _f32(99), n=100), "dst holds 99")
    ok = dict(grads=_f32(100), master=_f32(100), params=torch.zeros(100, dtype=torch.bfloat16))
    call = lambda m=m, v=v, st=st, sc=sc, **k: zds.zds_adam_step_q8(  # noqa: E731
        zds.hparams(), *(k.get(x, ok[x]) for x in ("grads", "master")), m, v, k.get("params", ok["params"]), 0, 0, sc, st,
        n=100)
    _raises(lambda: call(grads=_f32(99)), "grads holds 99")
    _raises(lambda: call(master=_f32(99)), "master holds 99")
    _raises(lambda: call(params=torch.zeros(99, dtype=torch.bfloat16)), "params_out holds 99")
    _raises(lambda: call(sc=sc[:60]), "scalars holds 60")
    _raises(lambda: call(st=st[:60]), "state holds 60")
    _raises(lambda: call(), "device tensor")
    _raises(lambda: zds.zds_dropout_compress(_f32(100), _f32(99), 4, _f32(25), 0, 0, st), "error holds 99")
    _raises(lambda: zds.zds_dropout_compress(_f32(100), None, 4, _f32(24), 0, 0, st), "values holds 24")
    _raises(lambda: zds.zds_dropout_compress(_f32(101), None, 4, _f32(25), 0, 0, st), "values holds 25")
    _raises(lambda: zds.zds_dropout_compress(_f32(100), None, 0, _f32(25), 0, 0, st), "ratio")
    _raises(lambda: zds.zds_dropout_decompress([_f32(25), _f32(24)], 4, _f32(100), 0, 0, st), "peer 1 holds 24")
    _raises(lambda: zds.zds_dropout_decompress([_f32(25), _f32(25).half()], 4, _f32(100), 0, 0, st), "one dtype")
    _raises(lambda: zds.zds_dropout_decompress([_f32(25)], 4, _f32(99), 0, 0, st, n=100), "dst holds 99")
    _raises(lambda: zds.zds_random_words_host(1 << 64, 0, 0, 1), "64-bit")
    assert zds.dropout_groups(100, 8) == 13 and zds.dropout_groups(0, 8) == 0


@pytest.mark.parametrize("ratio", [2 ** 32 + 2, 2 ** 32 + 4, -2 ** 32 + 8, 2 ** 64 + 256, 512, 1])
def test_binding_refuses_a_ratio_that_ctypes_would_cut(ratio):
    """The messages' lengths are checked with the whole number: cut to 32 bits,
    a ratio of 2^32 + 4 would be one of 4, whose message is not of one value."""
    st = torch.zeros(64, dtype=torch.uint8)
    _raises(lambda: zds.zds_dropout_compress(_f32(1000), None, ratio, _f32(1000), 0, 0, st), "ratio")
    _raises(lambda: zds.zds_dropout_decompress([_f32(1000)], ratio, _f32(1000), 0, 0, st), "ratio")


def test_binding_refuses_a_length_that_ctypes_would_cut():
    """n = 1000 - 2^64 is no longer than any buffer, and is 1000 in 64 bits."""
    n, st, sc = 1000 - 2 ** 64, torch.zeros(64, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8)
    m, v = (zds.new_quantised_state(32, f, "cpu") for f in (zds.ZDS_STATE_E4M3, zds.ZDS_STATE_UE5M3))
    x = _f32(32)
    for call in (lambda: zds.zds_state_quantise(x, m, n=n), lambda: zds.zds_state_dequantise(m, x, n=n),
                 lambda: zds.zds_adam_step_q8(zds.hparams(), x, x, m, v, None, 0, 0, sc, st, n=n),
                 lambda: zds.zds_dropout_compress(x, None, 4, x, 0, 0, st, n=n),
                 lambda: zds.zds_dropout_decompress([x], 4, x, 0, 0, st, n=n),
                 lambda: zds.zds_adam_step(zds.hparams(), x, x, x, x, None, sc, st, n=n),
                 lambda: zds.zds_overflow_and_norm(x, 1, 0.0, st, sc, x, n=n),
                 lambda: zds.zds_muon_momentum(zds.muon_hparams(), x, x, x, sc, n=n),
                 lambda: zds.zds_reduce_peer_slices([x.half()], x, zds.ZDS_OVERWRITE, n=n),
                 lambda: zds.zds_onebit_compress(x, None, 64, x, x, n=n)):
        _raises(call, "out of range")
    for n in (2 ** 64 + 4, 2 ** 63):
        _raises(lambda: zds.zds_state_quantise(x, m, n=n), "src holds 32")


# ------------------------------------------------------------------ configuration and step classes

def config(kind="AdamW8bit", **params):
    return from_ds_config({"optimizer": {"type": kind, "params": params}})


def test_configuration_of_the_moments():
    assert config().second_moment == "bf16"                       # beta2 0.999
    assert config(betas=[0.9, 0.95]).second_moment == "8bit"
    assert config(betas=[0.9, 0.98], second_moment="auto").second_moment == "8bit"
    assert config("Adam8bit", second_moment="8bit").second_moment == "8bit"
    assert config("AdamW").second_moment is None and config("AdamW") == from_ds_config({})
    a, b = config(lr=2e-4), config("AdamW", lr=2e-4)
    assert bytes(a.hparams()) == bytes(b.hparams())
    for bad in (dict(second_moment="fp8"), dict(second_moment=8)):
        with pytest.raises(ConfigError):
            config(**bad)
    with pytest.raises(ConfigError):
        config("Adam8bit", adam_w_mode=False, weight_decay=0.1)
    with pytest.raises(ConfigError):
        from_ds_config({"optimizer": {"type": "AdamW8bit"},
                        "zero_optimization": {"stage": 1, "offload_optimizer": {"device": "cpu"}}})


def test_the_wrong_step_for_a_configuration():
    with pytest.raises(zds.ZdsError) as e:
        ShardStep.from_config(64, config())
    assert "QuantisedStep" in str(e.value)
    with pytest.raises(zds.ZdsError) as e:
        QuantisedStep.from_config(64, config("AdamW"))
    assert "ShardStep" in str(e.value)


def test_step_classes_refuse():
    for kw in (dict(second=zds.ZDS_STATE_E4M3), dict(first=8), dict(first=-32)):
        with pytest.raises(zds.ZdsError):
            QuantisedStep(64, **kw)
    for args, kw in (((64, 3), {}), ((64, 512), {}), ((64, 8), dict(first=4)), ((64, 8), dict(seed=-1))):
        with pytest.raises(zds.ZdsError):
            DropoutExchange(*args, device="cpu", **kw)
    ex = DropoutExchange(100, 8, device="cpu", feedback=False)
    assert ex.groups == 13 and ex.values.numel() == 13 and ex.error is None
    with pytest.raises(zds.ZdsError):
        ex.compress(_f32(100), type("S", (), dict(state=torch.zeros(64, dtype=torch.uint8), scalars=None)))


def test_buffers_are_cleared_before_they_are_handed_out(monkeypatch):
    """Each construction that clears memory waits for the stream that does it,
    after the last of its buffers is made: the calls may come on another one."""
    log = []
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: log.append("clear") or zeros(*a, **dict(k, device="cpu")))
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: type("S", (), dict(synchronize=lambda self: log.append("wait")))())
    monkeypatch.setattr(zds, "new_workspace", lambda n, device: None)      # (nothing in it is read first)
    DropoutExchange(64, 8, device="cuda")
    assert log == ["clear", "clear", "wait"]
    log.clear()
    DropoutExchange(64, 8, feedback=False, device=torch.device("cuda", 0))
    assert log == ["clear", "wait"]
    log.clear()
    step = object.__new__(QuantisedStep)
    step.n, step.second, step.state = 64, zds.ZDS_STATE_UE5M3, type("T", (), dict(device=torch.device("cuda", 0)))
    step.new_moments()
    assert log == ["clear"] * 4 + ["wait"]
    log.clear()
    DropoutExchange(64, 8, device="cpu")
    assert log == ["clear", "clear"]


def test_a_span_of_an_exchange():
    """A shard begins and ends with whole groups (or at the end), and its values
    are those of its groups in a whole message."""
    ex = DropoutExchange(1000, 16, torch.float32, first=32, device="cpu")
    values, dst = torch.arange(63, dtype=torch.float32), _f32(1000)
    step = type("S", (), dict(state=torch.zeros(64, dtype=torch.uint8)))
    for span in ((-16, 16), (8, 32), (0, 1001), (0, 24), (32, 16), (1008, 1008), (0, 1008)):
        _raises(lambda: ex.decompress([values], dst, step, span=span), "span")
    _raises(lambda: ex.decompress([values[:62]], dst, step, span=(0, 16)), "peer 0 holds 62")
    _raises(lambda: ex.decompress([torch.zeros(63, 2)[:, 0]], dst, step, span=(0, 16)), "contiguous")
    _raises(lambda: ex.decompress([values], dst[:15], step, span=(16, 32)), "dst holds 15")


def test_what_a_span_passes_on(monkeypatch):
    ex = DropoutExchange(1000, 16, torch.float32, seed=5, first=32, device="cpu")
    values, step, got = torch.arange(63, dtype=torch.float32), type("S", (), dict(state=None)), []
    monkeypatch.setattr(zds, "zds_dropout_decompress",
                        lambda peers, ratio, dst, seed, first, state, mode, stream, n: got.append(
                            (peers[0].tolist(), ratio, seed, first, n)))
    for span in ((0, 1000), (16, 48), (992, 1000), (64, 64), None):
        ex.decompress([values], None, step, span=span)
    assert got == [(list(range(63)), 16, 5, 32, 1000), ([1, 2], 16, 5, 48, 32), ([62], 16, 5, 32 + 992, 8),
                   ([], 16, 5, 96, 0), (list(range(63)), 16, 5, 32, 1000)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [0, 1, 100, 1000, 1024, 733953])
def test_a_message_with_its_padding(dtype, n):
    """Rows of this length follow each other at multiples of 16 bytes."""
    ex = DropoutExchange(n, 8, dtype, device="cpu", feedback=False)
    assert ex.values.numel() == ex.groups and ex.values.dtype == dtype and ex.values.data_ptr() == ex.padded.data_ptr()
    size = ex.padded.numel() * ex.padded.element_size()
    assert size % 16 == 0 and 0 <= size - ex.groups * ex.padded.element_size() < 16 and not ex.padded.any()

"""Gradient dropout on the GPU against the plain definitions, bit for bit: a
message and an error are one or two fp32 operations from the inputs."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import quantised as Q  # noqa: E402
from oracle.zero_step import narrow, widen  # noqa: E402
from tests.test_gpu_quantised import scalars, state  # noqa: E402
from tests.util import to_dev, to_host  # noqa: E402
from zero_sharded_mixed_tensor_amd import zds  # noqa: E402
from zero_sharded_mixed_tensor_amd.step import DropoutExchange, MuonStep, OffloadStep, QuantisedStep, ShardStep  # noqa: E402

TDT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SEED = 0xC0FFEE1234567


def host(x32, dtype):
    return x32.astype(np.float32) if dtype == "fp32" else narrow(x32.astype(np.float32), dtype)


def same(got, want, dtype):
    """Bit for bit; NaN is NaN."""
    nan = np.isnan(widen(want, dtype))
    assert np.array_equal(np.isnan(widen(got, dtype)), nan)
    view = (lambda a: a.view(np.uint32)) if dtype == "fp32" else (lambda a: a)
    assert np.array_equal(view(got)[~nan], view(want)[~nan])


def shifted(a, dtype, pad, room=0):
    return to_dev(np.concatenate([a[:1].repeat(pad), a, a[:1].repeat(room)]), dtype)[pad:]


@pytest.mark.parametrize("ratio", [2, 4, 8, 64, 256])
@pytest.mark.parametrize("xdt,vdt", [("fp16", "fp16"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"),
                                     ("fp32", "fp16")])
@pytest.mark.parametrize("n,pad", [(1, 0), (5, 0), (257, 0), (4096, 0), (4097, 1), (50003, 0), (50003, 3)])
def test_compress_bit_exact(ratio, xdt, vdt, n, pad):
    rng = np.random.default_rng(n + ratio)
    x = host(rng.standard_normal(n) * 64, xdt)
    e = (rng.standard_normal(n) * 0.3).astype(np.float32)
    if n > 1000:
        e[rng.integers(0, n, 40)] *= np.float32(1e5)         # past fp16's range
    first, steps, scale = ratio * (16 * 999 + n % 16), 5, 128.0
    for feedback in (True, False):
        err = e if feedback else None
        want, werr = Q.dropout_compress(x, xdt, err, ratio, SEED, first, steps, scale, vdt)
        dx = shifted(x, xdt, pad)
        de = shifted(e, "fp32", pad, 8) if feedback else None
        dv = torch.full((want.size + 8,), 7.0, dtype=TDT[vdt], device="cuda")
        zds.zds_dropout_compress(dx, de, ratio, dv, SEED, first, state(steps, scale), scalars(), n=n)
        same(to_host(dv)[:want.size], want, vdt)
        assert (dv[want.size:] == 7.0).all()
        if feedback:
            same(to_host(de)[:n], werr, "fp32")
            assert (to_host(de)[n:] == e[0]).all()


@pytest.mark.parametrize("ratio", [2, 4, 16, 256])
@pytest.mark.parametrize("vdt,odt", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("n,pad,peers", [(1, 0, 1), (5, 0, 3), (4096, 0, 2), (4099, 1, 16), (50003, 0, 8), (50003, 2, 1)])
def test_decompress_bit_exact(ratio, vdt, odt, n, pad, peers):
    rng = np.random.default_rng(n + ratio)
    groups = -(-n // ratio)
    msgs = [host(rng.standard_normal(groups), vdt) for _ in range(peers)]
    dst = host(rng.standard_normal(n), odt)
    first, steps = ratio * (77 + n % 16), 9
    dev = [to_dev(m, vdt) for m in msgs]
    for mode in (zds.ZDS_OVERWRITE, zds.ZDS_ACCUMULATE):
        want = Q.dropout_decompress(msgs, vdt, n, ratio, SEED, first, steps, dst, odt, mode == zds.ZDS_ACCUMULATE)
        dd = shifted(dst, odt, pad, 8)
        zds.zds_dropout_decompress(dev, ratio, dd, SEED, first, state(steps), mode, n=n)
        got = to_host(dd)
        same(got[:n], want, odt)
        same(got[n:], dst[:1].repeat(8), odt)


@pytest.mark.parametrize("ratio", [2, 4, 16, 256])
@pytest.mark.parametrize("vdt,odt", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("n,peers", [(257, 2), (50003, 8), (16 * 4096 + 40, 16)])
def test_messages_at_any_address(ratio, vdt, odt, n, peers):
    """Rows of one gathered buffer, of a length that is no multiple of 16 bytes,
    and one odd message among aligned ones, under an aligned dst: what separate
    allocations give."""
    rng = np.random.default_rng(n + ratio)
    groups = -(-n // ratio)
    msgs = [host(rng.standard_normal(groups), vdt) for _ in range(peers)]
    dst = host(rng.standard_normal(n), odt)
    rows = torch.zeros(peers, groups, dtype=TDT[vdt], device="cuda")
    for row, m in zip(rows, msgs):
        row.copy_(to_dev(m, vdt))
    one = [to_dev(m, vdt) for m in msgs]
    one[peers // 2] = shifted(msgs[peers // 2], vdt, 1)
    for mode in (zds.ZDS_OVERWRITE, zds.ZDS_ACCUMULATE):
        want = Q.dropout_decompress(msgs, vdt, n, ratio, SEED, 0, 9, dst, odt, mode == zds.ZDS_ACCUMULATE)
        for messages in (list(rows), one):
            dd = shifted(dst, odt, 0, 8)
            zds.zds_dropout_decompress(messages, ratio, dd, SEED, 0, state(9), mode, n=n)
            same(to_host(dd)[:n], want, odt)
            same(to_host(dd)[n:], dst[:1].repeat(8), odt)


@pytest.mark.parametrize("vdt,odt", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("ratio", [64, 128, 256])
@pytest.mark.parametrize("n", [128 * 4096, 259 * 4096 + 5])
def test_decompress_tiles_in_runs(ratio, vdt, odt, n):
    """Long enough for the order of tiles that shares lines between them."""
    rng = np.random.default_rng(ratio)
    msgs = [host(rng.standard_normal(-(-n // ratio)), vdt) for _ in range(3)]
    dst = host(rng.standard_normal(n), odt)
    want = Q.dropout_decompress(msgs, vdt, n, ratio, SEED, ratio, 5, dst, odt, False)
    dd = shifted(dst, odt, 0, 8)
    zds.zds_dropout_decompress([to_dev(m, vdt) for m in msgs], ratio, dd, SEED, ratio, state(5), n=n)
    got = to_host(dd)
    same(got[:n], want, odt)
    same(got[n:], dst[:1].repeat(8), odt)


@pytest.mark.parametrize("odt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("ratio", [2, 4, 8, 32, 64, 128])
def test_adding_keeps_the_other_bits(ratio, odt):
    """Any bits: NaN payloads, subnormal numbers, signed zeros."""
    n, first, steps = 3 * 4096 + 17, ratio * 3, 4
    rng = np.random.default_rng(ratio)
    dst = rng.integers(0, 2 ** 32, n, np.uint32).view(np.float32) if odt == "fp32" else \
        rng.integers(0, 2 ** 16, n, np.uint16)
    msg = host(rng.standard_normal(-(-n // ratio)), odt)
    kept = np.isin(np.arange(n), Q.kept_places(n, ratio, SEED, first, steps))
    want = Q.dropout_decompress([msg], odt, n, ratio, SEED, first, steps, dst, odt, True)
    dd = to_dev(dst, odt)
    zds.zds_dropout_decompress([to_dev(msg, odt)], ratio, dd, SEED, first, state(steps), zds.ZDS_ACCUMULATE, n=n)
    got = to_host(dd)
    bits = (lambda a: a.view(np.uint32)) if odt == "fp32" else (lambda a: a)
    assert np.array_equal(bits(got)[~kept], bits(dst)[~kept])
    same(got, want, odt)


def test_infinities_and_nan():
    """Where the caller does not look first, they stay where they are: a kept
    one is sent, another one is kept in the error."""
    n, ratio = 64, 8
    x = np.ones(n, np.float32)
    x[::3], x[1] = np.inf, np.nan
    e = np.zeros(n, np.float32)
    want, werr = Q.dropout_compress(x, "fp32", e, ratio, 1, 0, 0, 1.0, "fp32")
    de, dv = to_dev(e, "fp32"), torch.zeros(8, device="cuda")
    zds.zds_dropout_compress(to_dev(x, "fp32"), de, ratio, dv, 1, 0, state())
    same(to_host(dv), want, "fp32")
    same(to_host(de), werr, "fp32")


@pytest.mark.parametrize("vdt", ["fp16", "bf16", "fp32"])
def test_overflow_poisons_the_message(vdt):
    n, ratio = 10007, 4
    e = np.random.default_rng(0).standard_normal(n).astype(np.float32)
    x = torch.ones(n, dtype=torch.float16, device="cuda")
    for feedback in (True, False):
        de = to_dev(e, "fp32") if feedback else None
        dv = torch.zeros(2502 + 3, dtype=TDT[vdt], device="cuda")
        zds.zds_dropout_compress(x, de, ratio, dv, 1, 0, state(), scalars(overflow=1))
        assert torch.isnan(dv[:2502]).all() and (dv[2502:] == 0).all()
        assert not feedback or np.array_equal(to_host(de), e)


def test_nothing_is_lost():
    """Every element is either sent or still in the error, exactly: over the
    steps the decoded messages and the last error add up to the inputs. Whole
    numbers below 2^24 in all, so fp32 sums are exact."""
    n, ratio = 3000, 8
    rng = np.random.default_rng(4)
    err, total, sent = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    values = torch.empty(375, device="cuda")
    seen = torch.zeros(n, device="cuda")
    for k in range(64):
        x = to_dev(rng.integers(-100, 101, n).astype(np.float32), "fp32")
        total += x
        zds.zds_dropout_compress(x, err, ratio, values, 3, 0, state(k))
        zds.zds_dropout_decompress([values], ratio, sent, 3, 0, state(k), zds.ZDS_ACCUMULATE)
        one = torch.empty(n, device="cuda")
        zds.zds_dropout_decompress([torch.ones_like(values)], ratio, one, 3, 0, state(k))
        seen += one
        assert (one.view(-1, ratio).sum(1) == 1).all()
    assert torch.equal(total, sent + err)
    # an element is kept in 64 of 8 * 64 draws: 8 on average, a deviation of 2.6
    assert seen.sum() == 375 * 64 and seen.max() <= 8 + 6 * 2.7


def test_offsets_past_32_bits():
    n, ratio = (1 << 32) + 4133, 16
    a = n - n % 4096 - 8192
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_()
    err = torch.zeros(n, device="cuda")
    v, v2 = torch.empty(-(-n // ratio), device="cuda"), torch.empty(-(-(n - a) // ratio), device="cuda")
    zds.zds_dropout_compress(x, err, ratio, v, 3, 0, state(2))
    e2 = torch.zeros(n - a, device="cuda")
    zds.zds_dropout_compress(x[a:].clone(), e2, ratio, v2, 3, a, state(2))
    assert torch.equal(v[a // ratio:], v2) and torch.equal(err[a:], e2)
    zds.zds_dropout_decompress([v], ratio, err, 3, 0, state(2))
    zds.zds_dropout_decompress([v2], ratio, e2, 3, a, state(2))
    assert torch.equal(err[a:], e2) and int((e2 != 0).sum()) <= v2.numel()
    zds.zds_dropout_decompress([v], ratio, err, 3, 0, state(2), zds.ZDS_ACCUMULATE)
    zds.zds_dropout_decompress([v2], ratio, e2, 3, a, state(2), zds.ZDS_ACCUMULATE)
    assert torch.equal(err[a:], e2)
    # without feedback
    zds.zds_dropout_compress(x, None, ratio, v, 3, 0, state(2))
    zds.zds_dropout_compress(x[a:].clone(), None, ratio, v2, 3, a, state(2))
    assert torch.equal(v[a // ratio:], v2)


def test_exchange_of_two_ranks_with_quantised_moments():
    """Two ranks' whole steps as they would run: each compresses its own grads,
    the messages are summed, both decode, step and update their loss scale;
    one rank's overflow at step 3 is skipped by both and costs no rank its
    error; eager, and one rank's step replayed from a graph."""
    n, ratio, world = 70003, 4, 2

    def rank():
        st = QuantisedStep(n, zds.hparams(lr=1e-3, beta2=0.95), zds.scaler_config(initial_scale_power=8), max_norm=1.0,
                           accum_steps=world, seed=9, first=0)
        return dict(st=st, ex=DropoutExchange(n, ratio, torch.bfloat16, seed=21, first=0),
                    master=torch.full((n,), 0.01, device="cuda"), mv=st.new_moments(),
                    params=torch.zeros(n, dtype=torch.float16, device="cuda"), g=torch.empty(n, device="cuda"),
                    x=torch.zeros(n, dtype=torch.float16, device="cuda"))

    def grads(k, r):
        g = torch.Generator(device="cuda").manual_seed(1000 * k + r)
        x = torch.randn(n, device="cuda", generator=g).mul_(0.3).half()
        if k == 3 and r == 1:
            x[123] = float("inf")
        return x

    def send(q):
        q["st"].norm(q["x"])
        q["ex"].compress(q["x"], q["st"])

    def take(q, total):
        q["ex"].norm(total, q["st"])
        q["ex"].decompress([total], q["g"], q["st"])
        q["st"].adam(q["g"], q["master"], *q["mv"], q["params"])
        q["st"].scaler()

    total = torch.empty(-(-n // ratio), device="cuda")
    ranks = [rank(), rank()]
    scales, log = [], []
    for k in range(8):
        scales.append(ranks[0]["st"].read_state().scale)
        for r, q in enumerate(ranks):
            q["x"].copy_(grads(k, r))
            send(q)
        total.copy_(ranks[0]["ex"].values.float() + ranks[1]["ex"].values.float())
        errors = [q["ex"].error.clone() for q in ranks]
        for q in ranks:
            take(q, total)
        log.append((ranks[0]["master"].clone(), ranks[0]["ex"].values.clone(), ranks[1]["ex"].values.clone()))
        # the norm of the message is the gradient's
        sc = zds.new_scalars()
        zds.zds_overflow_and_norm(ranks[0]["g"], world, 1.0, ranks[0]["st"].state, sc, ranks[0]["st"].ws)
        a, b = zds.read_scalars(sc), ranks[0]["st"].read_scalars()
        assert a.overflow == b.overflow == (1 if k == 3 else 0)
        if k != 3:
            assert abs(a.sumsq - b.sumsq) <= 1e-12 * a.sumsq
        for q, before in zip(ranks, errors):
            assert torch.equal(q["ex"].error, before) and torch.isfinite(q["ex"].error).all()
    for name in ("master", "params"):
        assert torch.equal(ranks[0][name], ranks[1][name])
    assert bytes(ranks[0]["st"].read_state()) == bytes(ranks[1]["st"].read_state())
    assert ranks[0]["st"].read_state().steps_skipped == 1 and scales[4] == scales[3] / 2
    assert torch.equal(log[3][0], log[2][0]) and not torch.equal(log[4][0], log[3][0])

    # rank 0 from a graph: its two halves around the exchange
    q = rank()
    peer = torch.empty_like(ranks[1]["ex"].values)
    other = torch.empty(-(-n // ratio), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        send(q)
        other.copy_(q["ex"].values.float() + peer.float())
        take(q, other)
    for k in range(8):
        q["x"].copy_(grads(k, 0))
        peer.copy_(log[k][2])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q["master"], log[k][0]), k


def test_dense_step_after_an_exchange():
    """The decoded gradient feeds the fp32 step, too; without feedback the
    message is right on average: over 2048 steps of one gradient the mean of
    the decoded ones is the gradient, to five deviations of the mean (an
    element is x * ratio in one of ratio steps: x^2 (ratio - 1) a step)."""
    n, ratio, steps = 1000, 4, 2048
    x = torch.linspace(-1, 1, n, device="cuda")
    ex = DropoutExchange(n, ratio, torch.float32, seed=4, feedback=False)
    mean = torch.zeros(n, dtype=torch.float64, device="cuda")
    g = torch.empty(n, device="cuda")
    st = ShardStep(n, zds.hparams(lr=0.0), zds.scaler_config(dynamic=False), max_norm=0.0)
    p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    for _ in range(steps):
        ex.compress(x, st)
        ex.norm(ex.values, st)
        ex.decompress([ex.values], g, st)
        st.adam(g, p, m, v, None)
        st.scaler()
        mean += g
    off = (mean / steps - x).abs()
    assert (off <= 5 * x.abs() * ((ratio - 1) / steps) ** 0.5 + 1e-6).all()


def test_first_calls_on_another_stream_than_the_current_one():
    """Built while the current stream is busy and used on one of the caller's at
    once: nothing that the constructions left on the current stream comes later."""
    n, ratio = 300007, 8
    x = torch.randn(n, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    start = torch.randn(n, generator=torch.Generator().manual_seed(4)).cuda()

    def run(stream, busy):
        p, g, out = start.clone(), torch.empty(n, device="cuda"), torch.empty(n, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        if busy:
            y = torch.ones(4096, 4096, device="cuda")
            for _ in range(20):
                y = y @ y * 1e-4
        st = QuantisedStep(n, zds.hparams(lr=1e-3, beta2=0.95), zds.scaler_config(dynamic=False), seed=2, stream=stream)
        ex = DropoutExchange(n, ratio, torch.float32, seed=6)
        m, v = st.new_moments()
        for _ in range(2):
            ex.compress(x, st, stream)
            ex.norm(ex.values, st, stream)
            ex.decompress([ex.values], g, st, stream=stream)
            st.adam(g, p, m, v, out, stream)
            st.scaler(stream)
        torch.cuda.synchronize()
        return p, g, out, m.codes, m.exps, v.codes, v.exps, ex.values, ex.error

    want = run(None, False)
    for a, b in zip(run(torch.cuda.Stream(), True), want):
        assert torch.equal(a, b)
    assert want[8].abs().max() > 0


@pytest.mark.parametrize("ratio,world", [(16, 2), (4, 3), (64, 4)])
def test_ranks_that_each_update_their_shard(ratio, world):
    """Every rank sends its gradient of all elements and decodes its own shard:
    what the ranks' shards become, put together, is what one rank that updates
    everything makes of the same messages, bit for bit, the 8-bit moments'
    roundings included, as they follow the flat element."""
    numels = [50003, 777, 20000]
    align = max(64, ratio)
    total = zds.zds_shard_range(zds.zds_flat_layout(numels, align)[1], world, world - 1, align)[1]
    hp, cfg = zds.hparams(lr=1e-3, beta2=0.95), zds.scaler_config(initial_scale_power=8)
    start = torch.randn(total, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.02

    def rank(lo, hi):
        st = QuantisedStep(hi - lo, hp, cfg, max_norm=1.0, accum_steps=world, seed=9, first=lo)
        return dict(st=st, ex=DropoutExchange(total, ratio, torch.bfloat16, seed=21), lo=lo, hi=hi, mv=st.new_moments(),
                    p=start[lo:hi].clone(), g=torch.empty(hi - lo, device="cuda"),
                    o=torch.empty(hi - lo, dtype=torch.bfloat16, device="cuda"))

    def take(q, message, span):
        q["ex"].norm(message, q["st"])
        q["ex"].decompress([message], q["g"], q["st"], span=span)
        q["st"].adam(q["g"], q["p"], *q["mv"], q["o"])
        q["st"].scaler()

    ranks = [rank(*zds.zds_shard_range(total, world, r, align)) for r in range(world)]
    assert len({q["lo"] for q in ranks}) == world
    whole = rank(0, total)
    for k in range(5):
        for r, q in enumerate(ranks):
            x = torch.randn(total, device="cuda", generator=torch.Generator(device="cuda").manual_seed(10 * k + r)).half()
            if k == 2 and r == 1:
                x[-5] = float("inf")                       # outside the shards of most ranks
            q["ex"].flag(x, q["st"])
            assert q["st"].read_scalars().overflow == (1 if k == 2 and r == 1 else 0)
            q["ex"].compress(x, q["st"])
        message = sum(q["ex"].values.float() for q in ranks).bfloat16()
        for q in ranks:
            take(q, message, (q["lo"], q["hi"]))
        take(whole, message, None)
        scalars = whole["st"].read_scalars()
        assert scalars.overflow == (1 if k == 2 else 0) and (k == 2 or scalars.norm > 0)
        for q in ranks:
            assert bytes(q["st"].read_state()) == bytes(whole["st"].read_state())
            assert bytes(q["st"].read_scalars())[:32] == bytes(scalars)[:32]
        for name in ("g", "p", "o"):
            got = torch.cat([q[name] for q in ranks])
            assert torch.equal(got.view(torch.uint8), whole[name].view(torch.uint8)), (k, name)
        assert torch.equal(torch.cat([q["mv"][0].codes for q in ranks]), whole["mv"][0].codes)
        assert torch.equal(torch.cat([q["mv"][1].codes for q in ranks]), whole["mv"][1].codes)
    assert not torch.equal(whole["p"], start)


@pytest.mark.parametrize("combined", [False, True])
def test_what_an_overflow_leaves_in_the_errors(combined):
    """Two ranks, one of which overflows at step 3. Its message is NaN and both
    skip the step; its error stays as it was. The other rank's error is what
    its compress made of it, so that what it sent is lost, unless the flags were
    combined first: then its error stays, too, and over the other steps decoded
    messages and errors add up to the gradients, exactly (whole numbers)."""
    n, ratio, world = 20005, 8, 2

    def rank():
        st = ShardStep(n, zds.hparams(lr=0.0), zds.scaler_config(initial_scale_power=4), max_norm=0.0, accum_steps=world)
        return dict(st=st, ex=DropoutExchange(n, ratio, torch.float32, seed=21))

    ranks = [rank() for _ in range(world)]
    given, taken = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for k in range(6):
        scale = ranks[0]["st"].read_state().scale
        flags, xs, before = [], [], [q["ex"].error.clone() for q in ranks]
        for r, q in enumerate(ranks):
            x = np.random.default_rng(10 * k + r).integers(-100, 101, n).astype(np.float32) * np.float32(scale)
            if k == 3 and r == 1:
                x[123] = np.inf
            xs.append(x)
            flags.append(q["ex"].flag(to_dev(x, "fp32"), q["st"]))
        assert [int(f) for f in flags] == ([0, 1] if k == 3 else [0, 0])
        if combined:
            top = torch.maximum(*flags)
            for f in flags:
                f.copy_(top)
        for x, q in zip(xs, ranks):
            q["ex"].compress(to_dev(x, "fp32"), q["st"])
        total = ranks[0]["ex"].values + ranks[1]["ex"].values
        for r, (x, q, e) in enumerate(zip(xs, ranks, before)):
            skipped = k == 3 and (combined or r == 1)
            assert torch.isnan(q["ex"].values).all() == skipped
            want = to_host(e) if skipped else Q.dropout_compress(x, "fp32", to_host(e), ratio, 21, 0, k, scale, "fp32")[1]
            same(to_host(q["ex"].error), want, "fp32")
        if k == 3:
            assert torch.equal(ranks[0]["ex"].error, before[0]) == combined
        g = torch.empty(n, device="cuda")
        for q in ranks:
            q["ex"].norm(total, q["st"])
            q["ex"].decompress([total], g, q["st"])
            assert q["st"].read_scalars().overflow == (1 if k == 3 else 0)
            q["st"].scaler()
        if k != 3:
            given += sum(to_dev(x, "fp32") for x in xs) / scale
            taken += g / scale
    left = ranks[0]["ex"].error + ranks[1]["ex"].error
    assert torch.equal(given, taken + left) == combined


def _gradient(ex, k):
    """What the exchange's message makes in step k, by the plain call, in the message's type."""
    g = torch.empty(ex.n, dtype=ex.values.dtype, device="cuda")
    zds.zds_dropout_decompress([ex.values], ex.ratio, g, ex.seed, ex.first, state(k))
    return g


def test_exchange_in_front_of_a_muon_step():
    """The state and scalars of its base: two steps end where steps on the
    gradient that the messages make end (no clipping, so that the norm's order
    of sums does not come in)."""
    n, split, ratio = 200 * 72 + 3000, 200 * 72, 4

    def fresh():
        g = torch.Generator(device="cuda").manual_seed(5)
        return MuonStep(n, split, [(0, 200, 72)], max_norm=0.0, scaler=zds.scaler_config(dynamic=False)), [
            torch.randn(n, device="cuda", generator=g), torch.zeros(split, device="cuda"),
            torch.zeros(n - split, device="cuda"), torch.zeros(n - split, device="cuda"),
            torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
    (a, sa), (b, sb) = fresh(), fresh()
    ex, got = DropoutExchange(n, ratio, torch.bfloat16, seed=3), torch.empty(n, dtype=torch.bfloat16, device="cuda")
    for k in range(2):
        x = torch.randn(n, generator=torch.Generator().manual_seed(k)).bfloat16().cuda()
        assert int(ex.flag(x, a)) == 0
        ex.compress(x, a)
        ex.norm(ex.values, a)
        ex.decompress([ex.values], got, a)
        want = _gradient(ex, k)
        assert torch.equal(got, want) and (want != 0).any()
        a.apply(got, *sa)
        a.base.scaler()
        b.step(want, *sb)
    for x, y in zip(sa, sb):
        assert torch.equal(x, y)
    assert a.read_state().t == 2 and bytes(a.read_state()) == bytes(b.read_state())


def test_exchange_in_front_of_an_offloaded_step():
    """The state and scalars on the device: two steps, one of them skipped, end
    where steps on the gradient that the messages make end."""
    n, ratio = 70001, 8

    def fresh():
        host = [torch.zeros(n).pin_memory() for _ in range(3)]
        host[0].copy_(torch.randn(n, generator=torch.Generator().manual_seed(5)))
        return OffloadStep(n, *host, torch.float16, torch.float16, chunk=1 << 15), host
    (a, ha), (b, hb) = fresh(), fresh()
    ex = DropoutExchange(n, ratio, torch.float16, seed=3)
    pa, pb = (torch.zeros(n, dtype=torch.float16, device="cuda") for _ in range(2))
    got = torch.empty(n, dtype=torch.float16, device="cuda")
    for k in range(3):
        x = torch.randn(n, generator=torch.Generator().manual_seed(k)).half().cuda()
        if k == 1:
            x[7] = float("inf")
        assert int(ex.flag(x, a)) == (1 if k == 1 else 0)
        ex.compress(x, a)
        ex.decompress([ex.values], got, a)
        want = _gradient(ex, k)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        for q, g, p in ((a, got, pa), (b, want, pb)):
            assert q.step(g, p).overflow == (1 if k == 1 else 0)
    torch.cuda.synchronize()
    for x, y in zip(ha + [pa], hb + [pb]):
        assert torch.equal(x, y)
    assert bytes(a.dev.read_state()) == bytes(b.dev.read_state()) and a.dev.read_state().steps_skipped == 1


def test_an_exchange_is_resumed():
    """Steps with a save and a resume between them: the checkpoint's arrays and
    the exchange's error are all that goes on, bit for bit."""
    n, ratio = 30011, 16

    def fresh():
        st = QuantisedStep(n, zds.hparams(lr=1e-3, beta2=0.95), zds.scaler_config(initial_scale_power=6), seed=8)
        return st, DropoutExchange(n, ratio, torch.bfloat16, seed=9), torch.ones(n, device="cuda"), *st.new_moments()

    def go(st, ex, p, m, v, some):
        g = torch.empty(n, device="cuda")
        for k in some:
            x = torch.randn(n, generator=torch.Generator().manual_seed(k)).half().cuda()
            ex.flag(x, st)
            ex.compress(x, st)
            ex.norm(ex.values, st)
            ex.decompress([ex.values], g, st)
            st.adam(g, p, m, v, None)
            st.scaler()

    straight, first, second = fresh(), fresh(), fresh()
    go(*straight, range(6))
    go(*first, range(3))
    m32, v32 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    first[0].read_back(first[3], first[4], m32, v32)
    second[0].state.copy_(first[0].state)
    second[0].quantise(m32, v32, second[3], second[4])
    second[2].copy_(first[2])
    assert first[1].error.abs().max() > 0
    second[1].error.copy_(first[1].error)
    go(*second, range(3, 6))
    assert torch.equal(second[2], straight[2]) and torch.equal(second[1].error, straight[1].error)
    assert torch.equal(second[1].values, straight[1].values)


@pytest.mark.parametrize("span", [None, (128, 9000)])
def test_gathered_messages(span):
    """Four ranks' padded messages as rows of one buffer: decoded from the rows
    as from the messages themselves, the padding untouched."""
    n, ratio = 10007, 8
    st = ShardStep(n, scaler=zds.scaler_config(dynamic=False))
    exs = [DropoutExchange(n, ratio, torch.bfloat16, seed=4) for _ in range(4)]
    for r, ex in enumerate(exs):
        ex.compress(torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(r)).bfloat16(), st)
        assert not ex.padded[ex.groups:].any()
    rows = torch.cat([ex.padded for ex in exs]).view(4, -1)
    assert all(row.data_ptr() % 16 == 0 for row in rows) and rows.shape[1] > exs[0].groups
    lo, hi = span or (0, n)
    a, b = torch.empty(hi - lo, device="cuda"), torch.empty(n, device="cuda")
    exs[0].decompress(list(rows), a, st, span=span)
    exs[0].decompress([ex.values for ex in exs], b, st)
    assert torch.equal(a, b[lo:hi]) and (a != 0).any()

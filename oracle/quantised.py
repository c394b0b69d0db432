"""AdamW's moments in fewer bits and gradient dropout, plain NumPy.

The codes are looked up in the table of the values they stand for, in float64;
the generator is written out on Python's and NumPy's whole numbers. Nothing
here follows the kernels' way through the bits of an fp32 number, but for the
16-bit format, whose definition they are."""

import numpy as np

from .zero_step import adamw_update, narrow, widen

BLOCK = 32
E4M3, UE5M3, BF16 = 0, 1, 2
TOP = {E4M3: 15, UE5M3: 31}
LEAST = {E4M3: 0, UE5M3: 11}
BAD = {E4M3: 0x7F, UE5M3: 0xFF}
ROUNDING, DROPOUT = 1, 2


# ------------------------------------------------------------------ the generator

def random_words(seed, calls, steps_seen, stream):
    """(len(calls), 4) uint32: Philox4x32-10 of key `seed` and counters (call
    low, call high, steps_seen, stream)."""
    low = np.uint64(0xFFFFFFFF)
    c = np.asarray(calls, np.uint64)
    x = [c & low, c >> np.uint64(32), np.full(c.shape, steps_seen, np.uint64), np.full(c.shape, stream, np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)   # both below 2^64
        x = [(q >> np.uint64(32)) ^ x[1] ^ np.uint64(k0), q & low, (p >> np.uint64(32)) ^ x[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(x, -1).astype(np.uint32)


def rounding_bits(seed, first, n, steps_seen, fmt):
    """The 16 random bits of n elements from flat index `first`."""
    f = first + np.arange(n, dtype=np.uint64)
    calls, at = np.unique(f // np.uint64(8), return_inverse=True)
    words = random_words(seed, calls, steps_seen, ROUNDING)[at, (f // np.uint64(2) % np.uint64(4)).astype(int)]
    r = (words >> (f % np.uint64(2) * np.uint64(16)).astype(np.uint32)) & np.uint32(0xFFFF)
    if fmt != E4M3:
        r = (r >> np.uint32(8)) | ((r & np.uint32(0xFF)) << np.uint32(8))
    return r.astype(np.int64)


# ------------------------------------------------------------------ the formats

def code_values(fmt):
    """Values of the magnitude codes below the top one, for an exponent byte
    of 127 (largest binade [1, 2))."""
    codes = np.arange(BAD[fmt], dtype=np.float64)
    field, frac = codes // 8, codes % 8
    return np.where(field > 0, (1 + frac / 8) * 2.0 ** field, frac / 4) * 2.0 ** -TOP[fmt]


def exponent_bytes(x, fmt):
    """Exponent byte of each block of 32."""
    pad = np.zeros(-x.size % BLOCK, np.float32)
    mag = np.abs(np.concatenate([x, pad])).reshape(-1, BLOCK)
    out = []
    for row in mag:
        if not np.isfinite(row).all():
            out.append(255)
            continue
        a = float(row.max())
        e = 0 if a < 2.0 ** -126 else int(np.floor(np.log2(np.float64(a)))) + 127
        while e > 0 and 2.0 ** (e - 127) > a:      # (log2 next to a power of two)
            e -= 1
        while a >= 2.0 ** (e - 126):
            e += 1
        if e == 0:                                 # subnormal: the mantissa is a / 2^-126
            e += a > 0.75 * 2.0 ** -126
        elif a > 1.75 * 2.0 ** (e - 127):
            e += 1
        out.append(min(max(e, LEAST[fmt]), 255))
    return np.array(out, np.uint8)


def quantise(x, fmt, r=None):
    """(codes, exponent bytes) of fp32 x; r: 16 random bits an element, None
    for the nearest code (halves to the even one)."""
    x = np.asarray(x, np.float32)
    if fmt == BF16:
        bits = x.view(np.uint32).astype(np.int64)
        mag = bits & 0x7FFFFFFF
        code = (mag + (r if r is not None else 0x7FFF + (mag >> 16 & 1))) >> 16
        code = np.where(np.isnan(x), (mag >> 16) | 0x40, np.where(np.isinf(x), 0x7F80, code))
        code = np.where((code == 0) & (mag > 0), 1, code)
        return (code | (bits >> 16 & 0x8000)).astype(np.uint16), None
    exps = exponent_bytes(x, fmt)
    s = np.repeat(exps.astype(np.float64), BLOCK)[:x.size]
    with np.errstate(over="ignore", invalid="ignore"):
        mag = np.abs(x.astype(np.float64)) * 2.0 ** (127 - s)
        # what fp32 leaves of it next to its least numbers (2^-20 of the codes' least step)
        grain = 2.0 ** (-149 + 127 - TOP[fmt])
        mag = np.where(mag < grain * 2.0 ** 24, np.round(mag / grain) * grain, mag)
    table = code_values(fmt)
    fine = np.isfinite(x) & ((x >= 0) | (fmt == E4M3))
    mag = np.where(fine, mag, 0.0)
    lo = np.searchsorted(table, mag, "right") - 1
    step = np.where(lo < 8, table[1], table[np.minimum(lo, table.size - 2) + 1] - table[np.minimum(lo, table.size - 2)])
    frac = (mag - table[lo]) / step                 # in [0, 1), exact
    if r is None:
        up = (frac > 0.5) | ((frac == 0.5) & (lo % 2 == 1))
    else:
        up = np.floor(frac * 2.0 ** 20) + 16 * r + 8 >= 2 ** 20
    code = lo + up
    if fmt == UE5M3:
        code = np.where((code == 0) & (x > 0), 1, code)
    code = np.where(fine, code, BAD[fmt])
    if fmt == E4M3:
        code = code | np.where(np.signbit(x), 0x80, 0)
    return code.astype(np.uint8), exps


def read_back(codes, exps, fmt):
    """float64 values of the codes (fp32 numbers, but for an overflow)."""
    if fmt == BF16:
        return widen(codes, "bf16").astype(np.float64)
    c = codes.astype(np.int64)
    mag = c & BAD[fmt]
    s = np.repeat(exps.astype(np.float64), BLOCK)[:c.size]
    value = np.append(code_values(fmt), np.nan)[mag] * 2.0 ** (s - 127)
    return np.where((c > 0x7F) & (fmt == E4M3), -value, value)


def adam_step_q8(x, gdtype, grad_scale, master, m, v, sq_fmt, consts, seed, first, steps_seen, pdtype):
    """(master, (codes, exps) of the first moment, of the second, params16).
    m, v: (codes, exps); consts: adamw_constants' of the step."""
    with np.errstate(over="ignore"):
        m32 = read_back(*m, E4M3).astype(np.float32)
        v32 = read_back(*v, sq_fmt).astype(np.float32)
    p, m32, v32 = adamw_update(x, gdtype, grad_scale, master, m32, v32, consts)[:3]
    r = [rounding_bits(seed, first, m32.size, steps_seen, f) for f in (E4M3, sq_fmt)]
    return p, quantise(m32, E4M3, r[0]), quantise(v32, sq_fmt, r[1]), narrow(p, pdtype)


# ------------------------------------------------------------------ gradient dropout

def kept_places(n, ratio, seed, first, steps_seen):
    """Flat place of each group's kept element (past the end: nothing kept)."""
    groups = -(-n // ratio)
    j = first // ratio + np.arange(groups, dtype=np.int64)
    words = random_words(seed, j // 16, steps_seen, DROPOUT)
    byte = words[np.arange(groups), j % 16 // 4] >> (8 * (j % 4)).astype(np.uint32) & np.uint32(255)
    return np.arange(groups) * ratio + byte.astype(np.int64) * ratio // 256


def _store(x, dtype):
    return x.astype(np.float32) if dtype == "fp32" else narrow(x.astype(np.float32), dtype)


def dropout_compress(x, xdtype, error, ratio, seed, first, steps_seen, scale, vdtype, overflow=False):
    """(values, new error) of one rank's gradient."""
    f = np.float32
    x = widen(x, xdtype)
    at = kept_places(x.size, ratio, seed, first, steps_seen)
    inside = at < x.size
    if overflow:
        return _store(np.full(at.size, np.nan, f), vdtype), error
    values = np.zeros(at.size, f)
    with np.errstate(over="ignore", invalid="ignore"):
        if error is None:
            values[inside] = x[at[inside]] * f(ratio)
            return _store(values, vdtype), None
        c = x + f(scale) * error
        values[inside] = c[at[inside]]
        stored = _store(values, vdtype)
        sent = widen(stored, vdtype)
        ok = inside & np.isfinite(sent)
        c[at[ok]] = c[at[ok]] - sent[ok]
        return stored, c * (f(1) / f(scale))


def dropout_decompress(peers, vdtype, n, ratio, seed, first, steps_seen, dst, odtype, accumulate):
    """The gradient: dst's elements with the messages' sum written or added."""
    at = kept_places(n, ratio, seed, first, steps_seen)
    inside = at < n
    t = widen(peers[0], vdtype).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        for p in peers[1:]:
            t = t + widen(p, vdtype)
        out = widen(dst, odtype).astype(np.float32) if accumulate else np.zeros(n, np.float32)
        out[at[inside]] = out[at[inside]] + t[inside] if accumulate else t[inside]
    if not accumulate:
        return _store(out, odtype)
    stored = np.array(dst, copy=True)
    stored[at[inside]] = _store(out[at[inside]], odtype)
    return stored

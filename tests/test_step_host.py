"""The serving-step entry points on the host: refused arguments (checked before
anything is launched) and the rotary table against its definition in extended
precision.  No kernel is launched here."""
import ctypes
import math

import numpy as np
import pytest

P = ctypes.c_void_p


def _tables(kvq, **kw):
    a = dict(ring=P(0x1000), capacity=8, state=P(0x1100), state_out=P(0x1200), lens=P(0x1300), target=P(0x1400),
             lens_out=P(0x1500), batch=1, table=P(0x1600), width=4, cu=P(0x1700), n=4, pos=P(0x1800), seq=P(0x1900),
             slots=P(0x1A00))
    a.update(kw)
    return kvq.lib().kvq_update_tables(*a.values(), None)


def test_update_tables_refusals(kvq):
    for kw in (dict(capacity=0), dict(batch=-1), dict(width=-1), dict(n=-1), dict(ring=None), dict(state=None),
               dict(state_out=None), dict(cu=None), dict(lens=None), dict(target=None), dict(lens_out=None),
               dict(table=None), dict(pos=None), dict(seq=None), dict(slots=None)):
        assert _tables(kvq, **kw) == kvq.KVQ_ERR_INVALID, kw
    assert _tables(kvq, batch=16385) == kvq.KVQ_ERR_UNSUPPORTED


def _rope(kvq, desc, **kw):
    a = dict(turns=P(0x1000), mag=1.0, pos=P(0x2000), n=3, q=P(0x3000), qs=512, qo=P(0x4000), qos=512, hq=4,
             k=P(0x5000), ks=256, ko=P(0x6000), kos=256, hk=2, dtype=kvq.KVQ_BF16)
    a.update(kw)
    return kvq.lib().kvq_rope(ctypes.byref(desc), *a.values(), None)


def test_rope_refusals(kvq):
    d = kvq.make_rope()
    assert _rope(kvq, d, n=0) == kvq.KVQ_OK                       # nothing to rotate
    assert _rope(kvq, d, hq=0, hk=0) == kvq.KVQ_OK
    for kw in (dict(n=-1), dict(hq=-1), dict(mag=math.inf), dict(mag=math.nan), dict(dtype=7), dict(turns=None),
               dict(turns=P(0x1004)), dict(pos=None), dict(q=None), dict(q=P(0x3008)), dict(qs=504), dict(qs=516),
               dict(qo=P(0x4002)), dict(k=None), dict(ks=248), dict(kos=252), dict(ko=None),
               dict(qo=P(0x3000), qos=1024)):                     # in place with another stride
        assert _rope(kvq, d, **kw) == kvq.KVQ_ERR_INVALID, kw
    assert _rope(kvq, d, dtype=kvq.KVQ_F32) == kvq.KVQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=8), "UNSUPPORTED"), (dict(rotary_dim=136), "UNSUPPORTED"), (dict(rotary_dim=120), "UNSUPPORTED"),
    (dict(rotary_dim=-16), "UNSUPPORTED"), (dict(base=1.0), "INVALID"), (dict(base=math.nan), "INVALID"),
    (dict(scaling="linear", factor=0.5), "INVALID"), (dict(scaling="ntk", factor=math.inf), "INVALID"),
    (dict(scaling="bands", factor=2.0, original_len=0, low=1, high=4), "INVALID"),
    (dict(scaling="bands", factor=2.0, original_len=64, low=4, high=4), "INVALID"),
    (dict(scaling="yarn", factor=2.0, original_len=64, low=0, high=4), "INVALID"),
    (dict(scaling="yarn", factor=2.0, original_len=64, low=math.nan, high=4), "INVALID")])
def test_rope_descriptors_refused(kvq, kw, status):
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_rope_table(kvq.make_rope(**kw))
    assert e.value.status == getattr(kvq, "KVQ_ERR_" + status)


def test_unknown_rope_scaling(kvq):
    with pytest.raises(kvq.KvqError):
        kvq.make_rope(scaling="other")
    d = kvq.make_rope()
    d.scaling = 5
    assert _rope(kvq, d) == kvq.KVQ_ERR_INVALID
    d = kvq.make_rope()
    d.interleaved = 2
    assert _rope(kvq, d) == kvq.KVQ_ERR_INVALID


def _definition(dim, base, scaling, factor, length, low, high):
    """Turns per position of each pair and the magnitude, in extended precision."""
    f = np.longdouble
    i = np.arange(dim // 2, dtype=f)
    b = f(base)
    if scaling == "ntk":
        b = b * f(factor) ** (f(dim) / f(dim - 2))
    g = b ** (-2 * i / f(dim))
    mag = 1.0
    if scaling == "linear":
        g = g / f(factor)
    elif scaling == "bands":
        k = (f(length) * g / (2 * f(np.pi)) - f(low)) / (f(high) - f(low))
        k = np.clip(k, 0, 1)
        g = k * g + (1 - k) * g / f(factor)
    elif scaling == "yarn":
        def index(n):
            return dim * math.log(length / (2 * math.pi * n)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(high)), 0), min(math.ceil(index(low)), dim - 1)
        d = np.clip((i - lo) / f(max(hi - lo, 0.001)), 0, 1)
        g = d * g / f(factor) + (1 - d) * g
        mag = 0.1 * math.log(factor) + 1
    return g / (2 * f("3.14159265358979323846264338327950288")), mag


@pytest.mark.parametrize("dim", [16, 48, 64, 128])
@pytest.mark.parametrize("scaling,base,factor,length,low,high", [
    ("none", 10000.0, 1.0, 0, 0, 0), ("linear", 10000.0, 4.0, 0, 0, 0), ("ntk", 10000.0, 8.0, 0, 0, 0),
    ("bands", 500000.0, 8.0, 8192, 1.0, 4.0), ("yarn", 10000.0, 16.0, 4096, 1.0, 32.0),
    ("yarn", 1000000.0, 1.0, 32768, 1.0, 32.0)])
def test_rope_table_follows_its_definition(kvq, dim, scaling, base, factor, length, low, high):
    """Within 2^-56 of a turn per position: 2^-25 of a turn at position 2^31."""
    turns, mag = kvq.kvq_rope_table(kvq.make_rope(dim, base, False, scaling, factor, length, low, high))
    want, wmag = _definition(dim, base, scaling, factor, length, low, high)
    assert turns.shape == (dim // 2,)
    got = turns.astype(np.longdouble) / np.longdouble(2) ** 64
    # numpy's pi is a double: its error (2^-53 relative) moves the ramps of "bands" by as much
    assert np.max(np.abs(got - want)) < 2.0 ** (-50 if scaling == "bands" else -56)
    assert abs(mag - wmag) <= 2.0 ** -23 * wmag


def test_scored_decode_refusals(kvq):
    L = kvq.lib()
    d = kvq.make_desc(4, 2)
    d.pool = 0x1000
    one = P(0x4000)

    def call(o, ws=one, nbytes=1 << 20, hq=4, batch=1):
        return L.kvq_decode_attention_scored(ctypes.byref(d), ctypes.byref(o) if o is not None else None, one,
                                             kvq.KVQ_BF16, batch, hq, one, 1, one, 16, one, kvq.KVQ_F32, ws, nbytes,
                                             None)

    for window in (-1, 2 ** 31, 2 ** 32):
        with pytest.raises(kvq.KvqError):
            kvq.make_score_opts(window=window)
    o = kvq.make_score_opts()
    o.window = -1
    assert call(o) == kvq.KVQ_ERR_INVALID
    for bad in (dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=math.inf), dict(softmax_scale=math.nan)):
        assert call(kvq.make_score_opts(**bad)) == kvq.KVQ_ERR_INVALID, bad
    o = kvq.make_score_opts()
    o.alibi_slopes = 0x1002
    assert call(o) == kvq.KVQ_ERR_INVALID
    ok = kvq.make_score_opts(softcap=30.0)
    assert call(ok, hq=6) == kvq.KVQ_ERR_UNSUPPORTED
    assert call(ok, ws=None) == kvq.KVQ_ERR_WORKSPACE
    assert call(ok, nbytes=16) == kvq.KVQ_ERR_WORKSPACE
    assert call(None, ws=None) == kvq.KVQ_ERR_WORKSPACE          # no options: all off
    assert call(ok, batch=0) == kvq.KVQ_OK


def test_scored_workspace_follows_the_window(kvq):
    """A window shortens the span that the splits cover: never more records
    than without it, and those of the window's span (window + 15 tokens)."""
    full = kvq.kvq_decode_scored_workspace_bytes(1024, 8, 2, 64, 131072)
    assert full == kvq.kvq_decode_workspace_bytes(1024, 8, 2, 64, 131072)
    w = kvq.kvq_decode_scored_workspace_bytes(1024, 8, 2, 64, 131072, window=1024)
    assert w == kvq.kvq_decode_workspace_bytes(1024, 8, 2, 64, 1024 + 15) <= full
    assert kvq.kvq_decode_scored_workspace_bytes(1024, 8, 2, 64, 131072, window=2 ** 31 - 1) == full
    assert kvq.kvq_decode_scored_workspace_bytes(1024, 8, 2, 64, 131072, window=-1) == 0


def test_prefill_refusals(kvq):
    L = kvq.lib()

    def call(o=None, **kw):
        a = dict(q=P(0x10000), qs=512, k=P(0x20000), ks=256, v=P(0x30000), vs=256, out=P(0x40000), os=512, n=3, hq=4,
                 hk=2, cu=P(0x5000), batch=1, prefix=None, dtype=kvq.KVQ_BF16)
        a.update(kw)
        return L.kvq_prefill_attention(ctypes.byref(o) if o is not None else None, *a.values(), None)

    assert call(n=0) == kvq.KVQ_OK and call(batch=0) == kvq.KVQ_OK
    for kw in (dict(n=-1), dict(batch=-1), dict(hq=0), dict(hk=0), dict(q=None), dict(k=P(0x20008)), dict(v=None),
               dict(out=None), dict(cu=None), dict(qs=504), dict(ks=260), dict(vs=128), dict(os=0), dict(dtype=9),
               dict(out=P(0x10000)), dict(out=P(0x20000)), dict(out=P(0x30000)), dict(ks=1 << 40)):
        assert call(**kw) == kvq.KVQ_ERR_INVALID, kw
    for kw in (dict(hq=6), dict(hq=5), dict(hq=32, qs=4096, os=4096), dict(dtype=kvq.KVQ_F32)):
        assert call(**kw) == kvq.KVQ_ERR_UNSUPPORTED, kw
    for bad in (dict(softcap=-1.0), dict(softcap=math.inf), dict(softmax_scale=math.nan)):
        assert call(kvq.make_score_opts(**bad)) == kvq.KVQ_ERR_INVALID, bad
    o = kvq.make_score_opts()
    o.alibi_slopes = 0x1001
    assert call(o) == kvq.KVQ_ERR_INVALID


def _exact_turns(dim, base, scaling, factor, length, low, high):
    """Turns per position of each pair in 60 decimal digits."""
    from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal as D, getcontext
    getcontext().prec = 60
    two_pi = 2 * D("3.14159265358979323846264338327950288419716939937510582097494459")
    base, factor, low, high = D(base), D(factor), D(low), D(high)
    if scaling == "ntk":
        base *= (factor.ln() * dim / (dim - 2)).exp()
    ramp = [D(0)] * (dim // 2)  # how much of each pair is divided by the factor
    g = [(base.ln() * (-2 * i) / dim).exp() for i in range(dim // 2)]
    if scaling == "linear":
        ramp = [D(1)] * (dim // 2)
    elif scaling == "bands":
        ramp = [1 - min(max((length * x / two_pi - low) / (high - low), D(0)), D(1)) for x in g]
    elif scaling == "yarn":
        def index(n):
            return dim * (length / (n * two_pi)).ln() / (2 * base.ln())
        lo = max(index(high).to_integral_value(ROUND_FLOOR), D(0))
        hi = min(index(low).to_integral_value(ROUND_CEILING), D(dim - 1))
        ramp = [min(max((i - lo) / max(hi - lo, D("0.001")), D(0)), D(1)) for i in range(dim // 2)]
    return [(x * r / factor + x * (1 - r)) / two_pi for x, r in zip(g, ramp)]


@pytest.mark.parametrize("dim", [16, 48, 128])
@pytest.mark.parametrize("scaling,base,factor,length,low,high", [
    ("none", 10000.0, 1.0, 0, 0, 0), ("none", 1e6, 1.0, 0, 0, 0), ("linear", 10000.0, 4.0, 0, 0, 0),
    ("ntk", 10000.0, 8.0, 0, 0, 0), ("bands", 500000.0, 8.0, 8192, 1.0, 4.0), ("yarn", 10000.0, 16.0, 4096, 1.0, 32.0)])
def test_rope_table_in_units_of_its_last_place(kvq, dim, scaling, base, factor, length, low, high):
    """Extended precision (2^-64 of a value) throughout, then cut to 2^-64: exponent and logarithm of a frequency
    f < 1 are off by a few 2^-64 of f ln f (at most 0.37), the ramps by as many of (length f / 2 pi) / (high - low), some
    hundreds for the longest wavelengths that "bands" still blends, times a slope 1 / (high - low) and f below
    2 pi high / length: within 2^-61 of a turn in all.  A table formed in doubles is off by up to 2^-54."""
    turns, _ = kvq.kvq_rope_table(kvq.make_rope(dim, base, False, scaling, factor, length, low, high))
    want = _exact_turns(dim, base, scaling, factor, length, low, high)
    assert max(abs(int(t) - w * 2 ** 64) for t, w in zip(turns, want)) <= 8

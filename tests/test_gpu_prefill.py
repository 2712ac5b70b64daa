"""kvq_prefill_attention against its definition in 64 bits.

Tolerance of an output o = sum p v / sum p, with A = sum p |v| / sum p:
  - eps/2 of |o|: the output's rounding; eps/2 of A: that of each p;
  - 2 e A for a score error e on both sums: the fp32 accumulation of 128
    products over up to 128 additions of at most a step each, 2^-23 * 2^4 (the
    sums inside a product are wider than their sequence) of sum |q k| tau, the
    softcap's 2^-21 cap, the distance bias's 2^-23 of it, exponentials 2^-21;
  - fp16: a p below 2^-14 is rounded to 2^-25, l is at least 1: n 2^-25 max |v|.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _t(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _reference(q, k, v, lens, starts, prefixes, scale=0.0, softcap=0.0, window=0, slopes=None):
    """-> outputs in 64 bits (rows of no prompt NaN), tolerance."""
    import torch
    G = q.shape[1] // k.shape[1]
    tau = scale if scale > 0 else 1 / math.sqrt(128)
    eps = torch.finfo(q.dtype).eps
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for n, s0, pre in zip(lens, starts, prefixes):
        if n == 0:
            continue
        for h in range(q.shape[1]):
            qq, kk, vv = (x.double() for x in (q[s0:s0 + n, h], k[s0:s0 + n, h // G], v[s0:s0 + n, h // G]))
            t, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
            ok = (j <= t) | (j < pre)
            if window:
                ok &= t - j < window
            s = qq @ kk.nan_to_num(0, 0, 0).T * tau
            size = (qq.abs() @ kk.nan_to_num(0, 0, 0).abs().T * tau).masked_fill(~ok, 0).amax(1, keepdim=True)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            bias = 0.0
            if slopes is not None:
                bias = float(slopes[h]) * (t - j).abs().double()
                s = s - bias
                bias = bias.masked_fill(~ok, 0).amax(1, keepdim=True)
            p = torch.softmax(s.masked_fill(~ok, -math.inf), 1)
            vz = vv.nan_to_num(0, 0, 0)
            out[s0:s0 + n, h] = p @ vz
            A = p @ vz.abs()
            e = 2.0 ** -19 * size + 2.0 ** -21 * (1 + softcap) + 2.0 ** -23 * bias
            x = (eps / 2) * (out[s0:s0 + n, h].abs() + A) + 2 * e * A + 1e-30
            if q.dtype == torch.float16:
                x = x + 2.0 ** -24 + n * 2.0 ** -25 * vz.abs().amax()
            tol[s0:s0 + n, h] = x
    return out, tol


def _rows(n, heads, dtype, g, mul=1.0):
    import torch
    x = torch.randn(n, heads, 128, device="cuda", generator=g)
    x[..., ::41] *= mul
    return x.to(_t(dtype))


def _run(kvq, lens, hq, hkv, dtype="bf16", prefixes=None, pad=0, seed=0, mutate=None, **opts):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    n = sum(lens) + pad
    q, k, v = _rows(n, hq, dtype, g), _rows(n, hkv, dtype, g, 15.0), _rows(n, hkv, dtype, g)
    if mutate:
        mutate(q, k, v)
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    slopes = opts.get("alibi_slopes")
    dev = dict(opts, alibi_slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    out = torch.full_like(q, 7.0)
    kvq.kvq_prefill_attention(q, k, v, torch.from_numpy(starts).cuda(), out, opts=kvq.make_score_opts(**dev),
                              prefix_lens=None if prefixes is None else
                              torch.tensor(prefixes, dtype=torch.int32, device="cuda"))
    assert kvq.kvq_last_device_status() == 0
    want, tol = _reference(q, k, v, lens, starts, prefixes or [0] * len(lens), opts.get("softmax_scale", 0.0),
                           opts.get("softcap", 0.0), opts.get("window", 0),
                           None if slopes is None else np.float32(slopes))
    _close(out[:sum(lens)], want[:sum(lens)], tol[:sum(lens)])
    assert (out[sum(lens):] == 7.0).all()  # rows behind the last prompt
    return out


def _close(out, want, tol):
    import torch
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all(), (~torch.isfinite(out)).nonzero()[:4]
    worst = (err - tol).argmax()
    assert (err <= tol).all(), (float(err.flatten()[worst]), float(tol.flatten()[worst]), np.unravel_index(
        int(worst), tuple(out.shape)))


def _slopes(n):
    return [2.0 ** (-8.0 * (h + 1) / n) for h in range(n)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("lens", [[1], [20], [128], [129], [257], [700]], ids=str)
def test_one_prompt(kvq, cuda, group, lens, dtype):
    _run(kvq, lens, 2 * group, 2, dtype, seed=group)


@pytest.mark.parametrize("opts", [
    {}, dict(softcap=50.0), dict(softcap=5.0), dict(window=1), dict(window=2), dict(window=128), dict(window=129),
    dict(window=300), dict(alibi_slopes=_slopes(8)), dict(softcap=30.0, window=77, alibi_slopes=_slopes(8)),
    dict(softmax_scale=0.03, softcap=20.0)], ids=lambda o: "-".join(f"{k}{v if k == 'window' else ''}" for k, v in
                                                                   o.items()) or "none")
@pytest.mark.parametrize("hkv", [1, 8])
@pytest.mark.parametrize("prefix", [False, True])
def test_options_ragged(kvq, cuda, opts, hkv, prefix):
    lens = [17, 0, 500, 1, 128, 333, 0, 64, 1025]
    _run(kvq, lens, 8, hkv, "fp16" if prefix else "bf16", prefixes=[n // 3 if i % 3 else n for i, n in enumerate(lens)]
         if prefix else None, pad=13, seed=hkv, **opts)


@pytest.mark.parametrize("prefixes", [[0, 5000], [-3, 1], [300, 299], [2 ** 31 - 1, 150]])
def test_prefix_bounds(kvq, cuda, prefixes):
    """Cut to the prompt; negative ones are none."""
    import torch
    lens = [300, 300]
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (_rows(600, 2, "bf16", g) for _ in range(3))
    out = torch.empty_like(q)
    kvq.kvq_prefill_attention(q, k, v, torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda"), out,
                              prefix_lens=torch.tensor(prefixes, dtype=torch.int32, device="cuda"))
    want, tol = _reference(q, k, v, lens, [0, 300], prefixes)
    _close(out, want, tol)


def test_many_short_prompts(kvq, cuda):
    """More prompts than threads; the order of the items over them."""
    rng = np.random.default_rng(3)
    _run(kvq, [int(x) for x in rng.integers(0, 9, 900)], 4, 2, "bf16")


def test_thousands_of_single_tokens(kvq, cuda):
    """Each attends to itself alone: its output is its value, bit for bit; every fourth prompt is empty."""
    import torch
    n = 20011
    g = torch.Generator(device="cuda").manual_seed(21)
    q, k, v = _rows(n, 8, "fp16", g), _rows(n, 2, "fp16", g), _rows(n, 2, "fp16", g)
    lens = np.ones(n * 4 // 3 + 2, np.int32)
    lens[3::4] = 0
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cu = cu[:int(np.searchsorted(cu, n)) + 1]
    out = torch.empty_like(q)
    kvq.kvq_prefill_attention(q, k, v, torch.from_numpy(cu).cuda(), out, opts=kvq.make_score_opts(window=7))
    assert torch.equal(out, v.repeat_interleave(4, dim=1))
    assert kvq.kvq_last_device_status() == 0


@pytest.mark.parametrize("group", [1, 8])
def test_long_prompt(kvq, cuda, group):
    _run(kvq, [5000], group, 1, "bf16", seed=9)


def test_large_scores_and_saturated_caps(kvq, cuda):
    """Scores of hundreds: the running max moves in most tiles; then the same under a small and a huge cap."""
    def louder(q, k, v):
        q.mul_(30)
    _run(kvq, [600, 40], 4, 2, "bf16", mutate=louder)
    _run(kvq, [600, 40], 4, 2, "bf16", mutate=louder, softcap=2.0)
    _run(kvq, [600, 40], 4, 2, "bf16", softcap=3e5)
    _run(kvq, [300], 4, 2, "fp16", softcap=1e-3, softmax_scale=20.0)
    _run(kvq, [300], 4, 2, "fp16", softcap=9.0)  # most rows below half of it, below it, some beyond


@pytest.mark.parametrize("at", [0.55, 0.75, 0.95])
@pytest.mark.parametrize("scale,cap", [(1 / 128, 30.0), (1 / 128, 50.0), (0.0, 200.0), (0.0, 1000.0), (0.0, 10000.0)])
def test_scores_near_their_cap(kvq, cuda, scale, cap, at):
    """Scores around `at` of the cap, a few units apart, whatever scale / cap is; those of the second key tile are
    next to one beyond the cap, so equal scores stand in tiles of both forms of the cap."""
    import torch

    def near(q, k, v):
        g = torch.Generator(device="cuda").manual_seed(17)
        tau = scale or 1 / math.sqrt(128)
        noise = torch.randn(k.shape, device="cuda", generator=g) / (tau * math.sqrt(128))
        k.copy_(at * cap / (tau * 128) + noise * (torch.arange(len(k), device="cuda") % 3 == 0)[:, None, None])
        k[130] = -2 * cap / (tau * 128)
        q.fill_(1.0)
    _run(kvq, [300, 40], 2, 1, "fp16", mutate=near, softmax_scale=scale, softcap=cap)


def test_rising_scores_move_the_maximum(kvq, cuda):
    """Keys of one direction whose length falls with the position: the oldest tile has the largest scores."""
    import torch

    def rising(q, k, v):
        n = k.shape[0]
        q.copy_(torch.ones_like(q))
        k.copy_((torch.linspace(12, 0.1, n, device="cuda")[:, None, None] * torch.ones_like(k.float())).to(k.dtype))
    _run(kvq, [900], 2, 1, "bf16", mutate=rising)
    _run(kvq, [900], 2, 1, "fp16", mutate=rising)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("group", [1, 4])
def test_masked_places_do_not_reach_a_row(kvq, cuda, bad, group):
    """NaN and infinities in later tokens' keys and values, in rows behind the last prompt and before the window:
    every row that does not read them is as without them."""
    import torch
    lens, pad = [300, 70], 40

    def spoil(q, k, v):
        v[250, :, 3] = bad
        k[250, :, 100] = bad
        v[370:] = bad
        k[370:] = bad
        q[370:] = bad
    starts = [0, 300]
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = _rows(410, 2 * group, "bf16", g), _rows(410, 2, "bf16", g), _rows(410, 2, "bf16", g)
    spoil(q, k, v)
    cu = torch.tensor([0, 300, 370], dtype=torch.int32, device="cuda")
    for window in (0, 20):
        out = torch.full_like(q, 7.0)
        kvq.kvq_prefill_attention(q, k, v, cu, out, opts=kvq.make_score_opts(window=window))
        want, tol = _reference(q, k, v, lens, starts, [0, 0], window=window)
        for rows in (slice(0, 250), slice(300, 370)) + ((slice(270, 300),) if window else ()):
            _close(out[rows], want[rows], tol[rows])
        assert (out[370:] == 7.0).all()
        assert not torch.isfinite(out[250:250 + (window or 50)]).all(-1).any()  # those that read them
    # a value row only: the rows that read it are spoilt in that dim alone
    v[250, :, 4], k[250] = bad, 0
    out = torch.empty_like(q)
    kvq.kvq_prefill_attention(q, k, v, cu, out)
    keep = [d for d in range(128) if d not in (3, 4)]
    assert torch.isfinite(out[250:300][..., keep]).all() and not torch.isfinite(out[250:300, :, 3:5]).any()


@pytest.mark.parametrize("junk", [float("inf"), float("nan"), 3e4])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("softcap", [20.0, 1e5])
def test_masked_places_do_not_choose_the_form_of_the_cap(kvq, cuda, softcap, window, junk):
    """Infinities and loud numbers in the keys of later tokens, of tokens before the window, of the next prompt and of
    padding, and in the padding's queries: every bit of the rows that read none of them is as without them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(23)
    q, k, v = _rows(460, 8, "bf16", g), _rows(460, 2, "bf16", g), _rows(460, 2, "bf16", g)
    cu = torch.tensor([0, 300, 417], dtype=torch.int32, device="cuda")
    opts = kvq.make_score_opts(softcap=softcap, window=window)
    want, out = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    kvq.kvq_prefill_attention(q, k, v, cu, want, opts=opts)
    k[250] = k[400] = junk  # a key in either prompt: rows behind it read it, up to the window
    k[417:] = q[417:] = junk
    kvq.kvq_prefill_attention(q, k, v, cu, out, opts=opts)
    for rows in (slice(0, 250), slice(300, 400)) + ((slice(290, 300),) if window else ()):
        assert torch.equal(out[rows], want[rows])
    assert (out[417:] == 7.0).all() and kvq.kvq_last_device_status() == 0


def test_a_loud_head_leaves_the_others_their_precision(kvq, cuda):
    """A cap of 1e5 that one head's scores pass; the others' are a few units: their cap is as good as none, whatever
    form the loud head's scores in the same tile need."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(29)
    q, k, v = _rows(300, 4, "fp16", g), _rows(300, 1, "fp16", g), _rows(300, 1, "fp16", g)
    q[:, 1] *= 400
    k *= 50
    q[:, [0, 2, 3]] /= 50
    out = torch.empty_like(q)
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    kvq.kvq_prefill_attention(q, k, v, cu, out, opts=kvq.make_score_opts(softcap=2e4))
    assert (q[:, 1].double() @ k[:, 0].double().T / math.sqrt(128)).abs().max() > 3e4
    want, tol = _reference(q, k, v, [300], [0], [0])  # tanh(x) is x up to 2e-7 of it for scores below 15
    for h in (0, 2, 3):
        _close(out[:, h], want[:, h], tol[:, h])


def test_a_long_prompt_before_rows_that_are_not_numbers(kvq, cuda):
    """65536 tokens and then padding full of NaN; and a later token's value that is not finite: the rows before it
    are formed again within the wait limit."""
    import torch
    n = 65536
    g = torch.Generator(device="cuda").manual_seed(31)
    q, k, v = _rows(n + 50, 8, "bf16", g), _rows(n + 50, 1, "bf16", g), _rows(n + 50, 1, "bf16", g)
    cu = torch.tensor([0, n - 70], dtype=torch.int32, device="cuda")
    want, out = torch.empty_like(q), torch.full_like(q, 7.0)
    kvq.kvq_prefill_attention(q, k, v, cu, want)
    for x in (q, k, v):
        x[n - 70:] = float("nan")
    kvq.kvq_prefill_attention(q, k, v, cu, out)
    assert torch.equal(out[:n - 70], want[:n - 70]) and (out[n - 70:] == 7.0).all()
    v[n - 80] = float("inf")
    kvq.kvq_prefill_attention(q, k, v, cu, out)
    assert kvq.kvq_last_device_status() == 0
    # formed again without the rounding of p: half a step of each output and of p on one side, the latter at most
    # 2^-8 sum p |v| / sum p <= 2^-8 max |v|
    a, b = out[:n - 80].double(), want[:n - 80].double()
    assert ((a - b).abs() <= 2.0 ** -8 * (a.abs() + b.abs() + v[:n - 80].double().abs().max()) + 1e-4).all()
    assert not torch.isfinite(out[n - 80:n - 70]).any()


@pytest.mark.parametrize("dtype,group,opts", [("bf16", 4, {}), ("fp16", 1, dict(window=150)), ("bf16", 8, dict(softcap=9.0)),
                                              ("fp16", 2, dict(prefix=200)), ("bf16", 1, dict(window=33, prefix=40))])
def test_values_that_are_not_finite_reach_their_readers_alone(kvq, cuda, dtype, group, opts):
    """Infinities and NaN in a few dims of values: an output dim that reads one is as its formula says (infinite, or
    not a number if it reads a NaN or both infinities), every other one as without them, bit for bit."""
    import torch
    lens, inf, nan = [300, 1, 420, 128], float("inf"), float("nan")
    cu = np.concatenate([[0], np.cumsum(lens)])
    g = torch.Generator(device="cuda").manual_seed(37)
    q, k, v = _rows(849, 2 * group, dtype, g), _rows(849, 2, dtype, g), _rows(849, 2, dtype, g)
    prefixes, o = [opts.get("prefix", 0)] * 4, kvq.make_score_opts(softcap=opts.get("softcap", 0.0),
                                                                   window=opts.get("window", 0))
    pre = torch.tensor(prefixes, dtype=torch.int32, device="cuda") if "prefix" in opts else None
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    want, out = torch.empty_like(q), torch.empty_like(q)
    kvq.kvq_prefill_attention(q, k, v, dcu, want, opts=o, prefix_lens=pre)
    for key, head, dim, x in ((0, 0, 5, inf), (100, 0, 5, -inf), (120, 0, 7, inf), (127, 1, 7, nan), (128, 0, 64, -inf),
                              (299, 0, 127, nan), (300, 0, 1, inf), (301, 1, 0, nan), (450, 0, 70, inf),
                              (451, 0, 70, nan), (560, 1, 33, -inf), (720, 1, 33, inf), (721, 0, 2, inf), (848, 1, 90, nan)):
        v[key, head, dim] = x
    v[60, 0], v[400:404, 1, 100:] = nan, inf
    kvq.kvq_prefill_attention(q, k, v, dcu, out, opts=o, prefix_lens=pre)
    assert kvq.kvq_last_device_status() == 0
    for s, n, p in zip(cu, lens, prefixes):
        t, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
        reads = (j <= t) | (j < p)
        if o.window:
            reads &= t - j < o.window
        vv = v[s:s + n]
        has = lambda m: torch.einsum("tj,jhd->thd", reads.double(), m.double()) > 0  # noqa: E731
        up, down, no = has(vv == inf), has(vv == -inf), has(vv.isnan())
        no |= up & down
        up, down, no = (x.repeat_interleave(group, 1) for x in (up & ~no, down & ~no, no))
        got, clean = out[s:s + n], want[s:s + n]
        assert got[no].isnan().all() and (got[up] == inf).all() and (got[down] == -inf).all()
        rest = ~(no | up | down)
        assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("bad", ["everywhere", "one dim", "infinite", "last"])
def test_values_that_are_not_finite_cost_little_time(kvq, cuda, bad):
    """Values that are NaN throughout, in one dim, infinite throughout, or one of them near a prompt's end: the call
    takes at most a few times as long (looking at the keys of two or three tiles an item takes each warp some tens of
    microseconds; forming rows again would take a hundred times as long)."""
    import torch
    n = 8192
    g = torch.Generator(device="cuda").manual_seed(41)
    q, k, v = _rows(n, 32, "bf16", g), _rows(n, 8, "bf16", g), _rows(n, 8, "bf16", g)
    cu, out = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.empty_like(q)

    def ms():
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        kvq.kvq_prefill_attention(q, k, v, cu, out)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b)
    ms()
    clean = min(ms() for _ in range(3))
    if bad == "everywhere":
        v.fill_(float("nan"))
    elif bad == "one dim":
        v[:, :, 17] = float("nan")
    elif bad == "infinite":
        v.fill_(float("inf"))
    else:
        v[n - 2] = float("inf")
    took = min(ms() for _ in range(2))
    assert kvq.kvq_last_device_status() == 0
    assert took <= 12 * clean, (took, clean)


def test_a_key_that_is_not_a_number_spoils_its_readers(kvq, cuda):
    """Every query that reads it gets NaN, in the masked tile of the diagonal and in plain ones; the others nothing."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(13)
    q, k, v = _rows(500, 2, "bf16", g), _rows(500, 2, "bf16", g), _rows(500, 2, "bf16", g)
    k[130, 0, 7] = float("nan")
    out = torch.empty_like(q)
    for opts in (kvq.make_score_opts(), kvq.make_score_opts(softcap=20.0), kvq.make_score_opts(window=200)):
        kvq.kvq_prefill_attention(q, k, v, torch.tensor([0, 500], dtype=torch.int32, device="cuda"), out, opts=opts)
        end = 330 if opts.window else 500
        assert torch.isnan(out[130:end, 0]).all() and torch.isfinite(out[:130]).all() and torch.isfinite(out[:, 1]).all()
        assert torch.isfinite(out[end:]).all()


def test_rows_with_equal_scores(kvq, cuda):
    """Zero queries: the mean of the values."""
    def zero(q, k, v):
        q.zero_()
    _run(kvq, [400], 2, 2, "bf16", mutate=zero)


def test_strided_rows_and_offsets_beyond_32_bits(kvq, cuda):
    """q, k, v slices of one fused projection whose last rows lie beyond 2^31 elements."""
    import torch
    hq, hkv, lens = 8, 1, [150, 170]
    n = 320
    stride = 1 << 23  # 320 rows: 2.7e9 elements, 5.4 GB
    buf = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
    qkv = buf.as_strided((n, hq + 2 * hkv, 128), (stride, 128, 1))
    g = torch.Generator(device="cuda").manual_seed(8)
    qkv.copy_(_rows(n, hq + 2 * hkv, "bf16", g))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    out = torch.empty(n, 2 * hq, 128, dtype=torch.bfloat16, device="cuda")[:, 3:3 + hq]
    kvq.kvq_prefill_attention(q, k, v, torch.tensor([0, 150, 320], dtype=torch.int32, device="cuda"), out)
    want, tol = _reference(q, k, v, lens, [0, 150], [0, 0])
    _close(out, want, tol)


def test_bad_bounds_are_left_out(kvq, cuda):
    """Descending bounds and bounds behind the rows: recorded, the other prompts computed, nothing else written."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = (_rows(200, 2, "bf16", g) for _ in range(3))
    for cu, good in (([0, 60, 50, 120], [(0, 60), (50, 70)]), ([0, 90, 300], [(0, 90)]), ([-5, 20, 40], [(20, 20)])):
        out = torch.full_like(q, 7.0)
        kvq.kvq_prefill_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), out)
        assert kvq.kvq_last_device_status() == kvq.KVQ_ERR_OUT_OF_RANGE
        left = torch.ones(200, dtype=torch.bool, device="cuda")
        for s, n in good[::-1]:
            left[s:s + n] = False
        assert (out[left] == 7.0).all()
        s, n = good[-1]
        want, tol = _reference(q, k, v, [n], [s], [0])
        _close(out[s + 10:s + n], want[s + 10:s + n], tol[s + 10:s + n])


def test_empty_calls(kvq, cuda):
    import torch
    e = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    kvq.kvq_prefill_attention(e, e, e, torch.zeros(3, dtype=torch.int32, device="cuda"), e)
    x = torch.full((4, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = x.clone()
    kvq.kvq_prefill_attention(x, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"), out)
    kvq.kvq_prefill_attention(x, x, x, torch.zeros(3, dtype=torch.int32, device="cuda"), out)
    assert kvq.kvq_last_device_status() == 0 and (out == 7.0).all()


def test_same_answer_again_and_in_graphs_on_two_streams(kvq, cuda):
    """Calls repeat bit for bit, eager, captured and replayed next to each other."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(12)
    q, k, v = _rows(700, 8, "bf16", g), _rows(700, 1, "bf16", g), _rows(700, 1, "bf16", g)
    cu = torch.tensor([0, 100, 700], dtype=torch.int32, device="cuda")
    opts = kvq.make_score_opts(softcap=30.0)
    want = torch.empty_like(q)
    kvq.kvq_prefill_attention(q, k, v, cu, want, opts=opts)
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, o in zip(streams, outs):
        s.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            kvq.kvq_prefill_attention(q, k, v, cu, o, opts=opts)
    for _ in range(5):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    cu.copy_(torch.tensor([0, 333, 650], dtype=torch.int32))  # other prompts through the same graph
    kvq.kvq_prefill_attention(q, k, v, cu, want, opts=opts)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][:650], want[:650])
    assert kvq.kvq_last_device_status() == 0


def test_wrapper_refusals(kvq, cuda):
    import torch
    q, k = torch.zeros(6, 4, 128, device="cuda").half(), torch.zeros(6, 2, 128, device="cuda").half()
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    good = dict(q=q, k=k, v=k.clone(), cu_seqlens=cu, out=torch.empty_like(q))
    kvq.kvq_prefill_attention(**good)
    for bad in (dict(q=q.bfloat16()), dict(q=q[:5]), dict(k=k[:, :1]), dict(k=k.cpu()), dict(cu_seqlens=cu.long()),
                dict(out=q), dict(out=torch.empty(6, 4, 128, device="cuda")), dict(q=q[:, :3]), dict(cu_seqlens=cu[:0]),
                dict(v=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(prefix_lens=torch.zeros_like(cu)),
                dict(opts=kvq.make_score_opts(alibi_slopes=torch.ones(3, device="cuda"))),
                dict(opts=kvq.make_score_opts(softcap=-1.0))):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_prefill_attention(**{**good, **bad})

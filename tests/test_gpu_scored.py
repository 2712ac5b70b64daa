"""kvq_decode_attention_scored against its definition in 64 bits, over pools
written by the oracle.

Tolerance: that of the plain decode (2e-3 for fp32 outputs of values of a few
units; the score options add to a score of up to softcap 50 an error of 2^-22
of it, 1.2e-5 of a probability) and half a step of a narrower output type.
"""
import math

import numpy as np
import pytest

import helpers
import oracle
import synth

pytestmark = pytest.mark.gpu


def _pool(wl, preset=(4, 2)):
    g = oracle.geom(num_blocks=wl.num_blocks, num_kv_heads=wl.hkv, k_bits=preset[0], v_bits=preset[1])
    pool = oracle.new_pool(g)
    k = wl.kv_rows(synth.TID_K, 0, wl.total_tokens)
    v = wl.kv_rows(synth.TID_V, 0, wl.total_tokens)
    assert oracle.quantize_append(g, pool, k, v, wl.dtype, wl.slots()) == 0
    return pool


def _rows(wl, pool, slots, preset):
    """K and V of the cache in 64 bits, [tokens, Hkv, 128] in the original domain."""
    kb, vb = preset
    raw = helpers._token_bytes(pool, wl.num_blocks, wl.hkv, slots, preset)  # [n, hkv, bytes]
    f = np.ascontiguousarray(raw[..., -8:]).view(np.float16).astype(np.float64)  # S_K, Z_K, S_V, Z_V
    h = np.array([[1.0]])
    while h.shape[0] < 128:
        h = np.block([[h, h], [h, -h]])
    h /= math.sqrt(128)

    def unpack(x, bits):
        e = np.arange(128) * bits
        return ((x[..., e // 8] >> (e % 8).astype(np.uint8)) & (2 ** bits - 1)).astype(np.float64)

    k = unpack(raw[..., :16 * kb], kb) * f[..., 0:1] + f[..., 1:2]
    v = unpack(raw[..., 16 * kb:16 * (kb + vb)], vb) * f[..., 2:3] + f[..., 3:4]
    return k @ h, v @ h


def _want(wl, pool, q, preset=(4, 2), scale=0.0, softcap=0.0, window=0, slopes=None):
    G = wl.hq // wl.hkv
    out = np.zeros((wl.batch, wl.hq, 128))
    for b in range(wl.batch):
        L = int(wl.seq_lens[b])
        lo = max(0, L - window) if window else 0
        if L == 0:
            continue
        t = np.arange(lo, L)
        k, v = _rows(wl, pool, wl.block_table[b, t // 16].astype(np.int64) * 16 + t % 16, preset)
        for h in range(wl.hq):
            s = k[:, h // G] @ q[b, h] * (scale if scale > 0 else 1 / math.sqrt(128))
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes[h] * (L - 1 - t)
            p = np.exp(s - s.max())
            out[b, h] = p @ v[:, h // G] / p.sum()
    return out


def _got(kvq, wl, pool, q, opts, preset=(4, 2), window=0, out_dtype=None, table=None):
    import torch
    msl = max(int(wl.seq_lens.max()), 1)
    out = torch.empty((wl.batch, wl.hq, 128), dtype=out_dtype or torch.float32, device="cuda")
    ws = kvq.new_scored_workspace(wl.num_blocks, wl.hkv, wl.batch, wl.hq, msl, window=window, preset=preset)
    kvq.kvq_decode_attention_scored(torch.from_numpy(pool).cuda(), wl.num_blocks, wl.hkv, q,
                                    torch.from_numpy(wl.block_table if table is None else table).cuda(),
                                    torch.from_numpy(wl.seq_lens).cuda(), msl, out, ws, opts, preset=preset)
    torch.cuda.synchronize()
    assert kvq.kvq_last_device_status() == 0
    return out


def _run(kvq, wl, preset=(4, 2), q_mul=1.0, out_dtype=None, **opts):
    import torch
    pool = _pool(wl, preset)
    q = (q_mul * torch.from_numpy(np.ascontiguousarray(wl.query()).view(np.int16)).view(torch.bfloat16).float())
    q = q.bfloat16().cuda()
    slopes = opts.get("alibi_slopes")
    dev = dict(opts, alibi_slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda())
    got = _got(kvq, wl, pool, q, kvq.make_score_opts(**dev), preset, opts.get("window", 0), out_dtype)
    want = _want(wl, pool, q.double().cpu().numpy(), preset, opts.get("softmax_scale", 0.0), opts.get("softcap", 0.0),
                 opts.get("window", 0), None if slopes is None else np.float32(slopes).astype(np.float64))
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - want) - half * np.abs(want)
    assert err.max() <= helpers.ATTN_TOL, err.max()
    return want


# lengths across blocks and chunks, an empty sequence and single tokens
_RAGGED = [1, 15, 16, 17, 300, 0, 2100, 129]


def _wl(lens, hq, hkv, seed, **kw):
    return synth.Workload("s", len(lens), hq, hkv, 128, lens, 16, synth.BF16, 3, 10.0, 30.0, seed=seed, **kw)


def _slopes(n):
    return [2.0 ** (-8.0 * (h + 1) / n) for h in range(n)]


@pytest.mark.parametrize("opts", [
    {}, dict(softcap=50.0), dict(softcap=5.0), dict(window=1), dict(window=16), dict(window=100), dict(window=129),
    dict(window=5000), dict(alibi_slopes=_slopes(16)), dict(softcap=30.0, window=77, alibi_slopes=_slopes(16)),
    dict(softmax_scale=0.05, softcap=20.0)], ids=lambda o: "-".join(o) or "none")
def test_options_ragged(kvq, cuda, opts):
    _run(kvq, _wl(_RAGGED, 16, 2, 61, extra_blocks=3), **opts)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("preset", [(4, 2), (4, 4), (2, 2), (8, 4)])
def test_groups_and_presets(kvq, cuda, G, preset):
    """Small grids (one CTA per multiprocessor) with every group and preset, splits included."""
    _run(kvq, _wl([777, 4130], 2 * G, 2, 70 + G), preset=preset, softcap=40.0, window=2000, alibi_slopes=_slopes(2 * G))


@pytest.mark.parametrize("G", [1, 8])
def test_full_grids(kvq, cuda, G):
    """More CTAs than multiprocessors (the other layout of the warps)."""
    _run(kvq, _wl([700 + 31 * i for i in range(40)], 4 * G, 4, 80 + G), softcap=25.0, alibi_slopes=_slopes(4 * G))


def test_large_scores_saturate_the_cap(kvq, cuda):
    """Scores far beyond the cap in both directions: e^2x is 0 and infinity."""
    _run(kvq, _wl([500, 33], 16, 2, 91), q_mul=200.0, softcap=2.0)


@pytest.mark.parametrize("softcap", [1e-3, 6.0, 1e5])
def test_caps_of_any_size(kvq, cuda, softcap):
    """Tiny, around the scores (both forms of the cap in one row), huge (no cap in effect)."""
    _run(kvq, _wl([500, 33], 16, 2, 96), softcap=softcap)


@pytest.mark.parametrize("q_mul", [1e4, 3e6, 1e9])
def test_two_scores_around_half_of_a_large_cap(kvq, cuda, q_mul):
    """Nearly equal keys, the best just beyond half of the cap and the second just below: both forms of the cap keep
    their order, so the best takes everything."""
    import torch
    wl = _wl([300], 1, 1, 97)
    g = oracle.geom(num_blocks=wl.num_blocks, num_kv_heads=1, k_bits=8, v_bits=4)
    pool = oracle.new_pool(g)
    k, v = wl.kv_rows(synth.TID_K, 0, 300).copy(), wl.kv_rows(synth.TID_V, 0, 300)
    k[:] = k[:1] ^ np.random.default_rng(2).integers(0, 2, k.shape).astype(k.dtype)  # the last bit of some elements
    assert oracle.quantize_append(g, pool, k, v, wl.dtype, wl.slots()) == 0
    kk = _rows(wl, pool, wl.slots(), (8, 4))[0][:, 0]
    q = torch.from_numpy(q_mul * kk[0] / np.abs(kk[0]).max()).float().view(1, 1, 128)
    s = np.sort(kk @ q.double().numpy()[0, 0] / math.sqrt(128))
    cap = float(np.float32(s[-1] + s[-2]))
    assert 1e-5 < s[-1] / s[-2] - 1 < 1e-3
    want = _want(wl, pool, q.double().numpy(), (8, 4), softcap=cap)
    got = _got(kvq, wl, pool, q.cuda(), kvq.make_score_opts(softcap=cap), (8, 4))
    assert np.abs(got.double().cpu().numpy() - want).max() <= helpers.ATTN_TOL


def test_steep_and_zero_and_growing_biases(kvq, cuda):
    """A slope that leaves the newest token alone, a slope of zero, one that favours distant tokens."""
    _run(kvq, _wl([900, 33], 8, 1, 92), alibi_slopes=[100.0, 0.0, -0.01, 1e-6, 3.0, 1e30, 0.5, 0.01])


@pytest.mark.parametrize("name", ["bfloat16", "float16"])
def test_output_types(kvq, cuda, name):
    import torch
    _run(kvq, _wl([900, 64, 129], 32, 4, 77), out_dtype=getattr(torch, name), softcap=50.0, window=512)


def test_blocks_before_the_window_are_not_read(kvq, cuda):
    """Their entries may name blocks given back: ids outside the pool change nothing and record nothing."""
    import torch
    wl = _wl([1000, 300], 16, 2, 93)
    pool = _pool(wl)
    q = torch.from_numpy(np.ascontiguousarray(wl.query()).view(np.int16)).view(torch.bfloat16).cuda()
    opts = kvq.make_score_opts(window=200)
    want = _got(kvq, wl, pool, q, opts, window=200)
    table = wl.block_table.copy()
    table[0, :(1000 - 200) // 16] = 10 ** 6
    table[1, :(300 - 200) // 16] = -3
    got = _got(kvq, wl, pool, q, opts, window=200, table=table)
    assert torch.equal(got, want)


def test_without_options_it_is_the_plain_decode(kvq, cuda):
    """Same pool, same query: both within their tolerance of one answer, so of each other."""
    import torch
    wl = _wl([2000, 77], 16, 2, 94)
    pool = _pool(wl)
    q = torch.from_numpy(np.ascontiguousarray(wl.query()).view(np.int16)).view(torch.bfloat16).cuda()
    got = _got(kvq, wl, pool, q, kvq.make_score_opts())
    out = torch.empty_like(got)
    ws = kvq.new_workspace(wl.num_blocks, wl.hkv, wl.batch, wl.hq, 2000)
    kvq.kvq_decode_attention(torch.from_numpy(pool).cuda(), wl.num_blocks, wl.hkv, q,
                             torch.from_numpy(wl.block_table).cuda(), torch.from_numpy(wl.seq_lens).cuda(), 2000, out, ws)
    assert (got - out).abs().max().item() <= 2 * helpers.ATTN_TOL


def test_graph_replays_with_growing_lengths(kvq, cuda):
    """One captured call; the lengths in device memory move on between replays, across the window's block edges."""
    import torch
    wl = _wl([400, 90], 16, 2, 95)
    pool_np = _pool(wl)
    pool = torch.from_numpy(pool_np).cuda()
    q = torch.from_numpy(np.ascontiguousarray(wl.query()).view(np.int16)).view(torch.bfloat16).cuda()
    opts = kvq.make_score_opts(softcap=30.0, window=64)
    bt = torch.from_numpy(wl.block_table).cuda()
    lens = torch.tensor([300, 60], dtype=torch.int32, device="cuda")
    ws = kvq.new_scored_workspace(wl.num_blocks, wl.hkv, 2, 16, 400, window=64)
    out = torch.empty(2, 16, 128, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kvq.kvq_decode_attention_scored(pool, wl.num_blocks, wl.hkv, q, bt, lens, 400, out, ws, opts)
    for step in (0, 1, 20, 30):
        wl.seq_lens = np.array([300 + step, 60 + step], dtype=np.int32)
        lens.copy_(torch.from_numpy(wl.seq_lens))
        g.replay()
        torch.cuda.synchronize()
        want = _want(wl, pool_np, q.double().cpu().numpy(), softcap=30.0, window=64)
        assert np.abs(out.cpu().numpy() - want).max() <= helpers.ATTN_TOL
    assert kvq.kvq_last_device_status() == 0


def test_wrapper_refusals(kvq, cuda):
    import torch
    pool = kvq.new_pool(8, 2)
    q = torch.zeros(2, 4, 128, device="cuda").half()
    bt, lens = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    ws = kvq.new_scored_workspace(8, 2, 2, 4, 64)
    good = dict(pool=pool, num_blocks=8, num_kv_heads=2, q=q, block_table=bt, seq_lens=lens, max_seq_len=64,
                out=torch.empty_like(q), workspace=ws, opts=kvq.make_score_opts())
    kvq.kvq_decode_attention_scored(**good)
    short = torch.ones(3, device="cuda")
    for bad in (dict(num_blocks=9), dict(q=q[:, :, :64]), dict(q=q.transpose(0, 1)), dict(block_table=bt.long()),
                dict(block_table=bt[:1]), dict(seq_lens=lens.cpu()), dict(out=torch.empty(2, 4, 64, device="cuda")),
                dict(opts=kvq.make_score_opts(alibi_slopes=short)), dict(workspace=ws[:16])):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_decode_attention_scored(**{**good, **bad})
    for bad in (short.double(), short.cpu(), torch.ones(8, device="cuda")[::2]):
        with pytest.raises(kvq.KvqError):
            kvq.make_score_opts(alibi_slopes=bad)
    assert kvq.kvq_last_device_status() == 0

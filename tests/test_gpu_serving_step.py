"""A serving loop from the library's parts, as an engine would run it: step
tables, rotary positions, the write into the packed cache, prompt attention
for the new prompts, then decode steps over the cache from one captured graph,
with one sliding-window, softcapped model.  Against the definitions in 64 bits
on the same cache; the plain bookkeeping is done again on the host."""
import math

import numpy as np
import pytest

import helpers
import oracle

pytestmark = pytest.mark.gpu

HQ, HKV, B, WIDTH, CAP, WINDOW, SOFTCAP = 16, 2, 16, 24, 96, 100, 30.0


def _rotated(x, pos, turns, mag):
    """Half layout, 64 bits, rounded to bf16 as the kernel's output is."""
    import torch
    phase = np.array([[(int(p) * int(t) % 2 ** 64) / 2 ** 64 for t in turns] for p in pos])
    t = torch.from_numpy(2 * np.pi * phase)[:, None, :]
    h = len(turns)
    x = x.double().cpu()
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([mag * (a * t.cos() - b * t.sin()), mag * (b * t.cos() + a * t.sin()), x[..., 2 * h:]], -1)


def _attend(q, k, v, t):
    """One query [Hq, 128] at position t over keys 0 .. t (numpy, 64 bits)."""
    lo = max(0, t - WINDOW + 1)
    out = np.zeros((HQ, 128))
    for h in range(HQ):
        s = k[lo:t + 1, h * HKV // HQ] @ q[h] / math.sqrt(128)
        s = SOFTCAP * np.tanh(s / SOFTCAP)
        p = np.exp(s - s.max())
        out[h] = p @ v[lo:t + 1, h * HKV // HQ] / p.sum()
    return out


def _cache_rows(pool, row, n):
    """K and V of a sequence's n tokens from the pool's bytes, original domain."""
    g = oracle.geom(num_blocks=CAP, num_kv_heads=HKV)
    had = np.array([[1.0]])
    while had.shape[0] < 128:
        had = np.block([[had, had], [had, -had]])
    had /= math.sqrt(128)
    k, v = np.zeros((n, HKV, 128)), np.zeros((n, HKV, 128))
    for t in range(n):
        for h in range(HKV):
            kc, sk, zk, vc, sv, zv = oracle.unpack_token(g, pool, int(row[t // B]), t % B, h)
            k[t, h] = (kc * oracle.f16_to_f64(sk) + oracle.f16_to_f64(zk)) @ had
            v[t, h] = (vc * oracle.f16_to_f64(sv) + oracle.f16_to_f64(zv)) @ had
    return k, v


def test_prompts_then_captured_decode_steps(kvq, cuda):
    import torch
    batch, rows = 3, 256
    gen = torch.Generator(device="cuda").manual_seed(4)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = kvq.new_pool(CAP, HKV)
    ring = torch.randperm(CAP, generator=torch.Generator().manual_seed(1)).to(**i32)
    state = torch.tensor([0, CAP, 0, 0], **i32)
    lens, target = torch.zeros(batch, **i32), torch.tensor([120, 33, 1], **i32)
    table, cu, maps = torch.full((batch, WIDTH), -1, **i32), torch.zeros(batch + 1, **i32), torch.zeros(3, rows, **i32)
    desc = kvq.make_rope(64, 10000.0, False, "yarn", 4.0, 64, 1.0, 32.0)
    turns, mag = kvq.kvq_rope_table(desc)
    rope, _ = kvq.new_rope_table(desc)
    opts = kvq.make_score_opts(softcap=SOFTCAP, window=WINDOW)
    out = torch.zeros(rows, HQ, 128, dtype=torch.bfloat16, device="cuda")

    # one fused projection's rows: q, k and v heads of each token
    def project(n):
        return torch.randn(n, HQ + 2 * HKV, 128, device="cuda", generator=gen).bfloat16()

    def step(qkv, n):
        """Tables, rotation (in place) and the write of a step of at most n tokens."""
        kvq.kvq_update_tables(ring, state, state, lens, target, lens, table, cu, maps[0][:n], maps[1][:n], maps[2][:n])
        kvq.kvq_rope(desc, rope, mag, maps[0][:n], qkv[:, :HQ], qkv[:, HQ:HQ + HKV])
        kvq.kvq_quantize_append(pool, CAP, HKV, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], maps[2][:n],
                                token_stride=(HQ + 2 * HKV) * 128)

    qkv = project(rows)
    raw = qkv.clone()
    step(qkv, rows)
    kvq.kvq_prefill_attention(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], cu, out, opts=opts)
    assert kvq.kvq_last_device_status() == 0
    assert cu.tolist() == [0, 120, 153, 154] and lens.tolist() == [120, 33, 1]
    pos = maps[0].cpu().numpy()
    assert pos.tolist() == [*range(120), *range(33), 0] + [-1] * (rows - 154)
    assert torch.equal(qkv[154:], raw[154:])
    want = _rotated(raw[:154, :HQ + HKV], pos[:154], turns, mag)
    got = qkv[:154, :HQ + HKV].double().cpu()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 6e-6).all()  # rounding; 6e-7 of |a| + |b| < 10
    # the prompts' attention on the rotated rows: half a bf16 step (2^-8) of each p and of the output
    x = qkv[:154].double().cpu().numpy()
    k, v = x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
    o = out.double().cpu().numpy()
    for s, n in ((0, 120), (120, 33), (153, 1)):
        for t in range(n):
            w = _attend(x[s + t, :HQ], k[s:s + n], v[s:s + n], t)
            assert np.abs(o[s + t] - w).max() <= 2 * 2.0 ** -8 * np.abs(v[s:s + t + 1]).max() + 1e-4

    # decode: one graph, three requests of which the second ends and starts again from nothing
    qkv1, out1 = project(batch), torch.zeros(batch, HQ, 128, dtype=torch.bfloat16, device="cuda")
    ws = kvq.new_scored_workspace(CAP, HKV, batch, HQ, WIDTH * B, window=WINDOW)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(qkv1, batch)
        kvq.kvq_decode_attention_scored(pool, CAP, HKV, qkv1[:, :HQ].contiguous(), table, lens, WIDTH * B, out1, ws,
                                        opts)
    for i in range(20):
        target.copy_(lens + 1)
        if i == 7:
            target[1] = 0  # finished: its blocks go back, its output is zero
        qkv1.copy_(project(batch))
        graph.replay()
        assert kvq.kvq_last_device_status() == 0
        now = lens.tolist()
        assert now == [121 + i, 0 if i == 7 else (34 + i if i < 7 else i - 7), 2 + i]
        if i in (0, 6, 7, 8, 19):
            bytes_, rows_ = pool.cpu().numpy(), table.cpu().numpy()
            order = [b for b in range(batch) if now[b] > 0]  # packed rows of the step, by sequence
            q = qkv1.double().cpu().numpy()
            for b in range(batch):
                if now[b] == 0:
                    assert not out1[b].any()
            if len(order) == batch:
                for b in order:
                    ck, cv = _cache_rows(bytes_, rows_[b], now[b])
                    w = _attend(q[b, :HQ], ck, cv, now[b] - 1)
                    err = np.abs(out1[b].double().cpu().numpy() - w) - 2.0 ** -8 * np.abs(w)
                    assert err.max() <= helpers.ATTN_TOL
        # no block is owned twice, none is lost
        s = state.tolist()
        free = [ring[(s[0] + j) % CAP].item() for j in range(s[1])]
        owned = [p for b in range(batch) for p in table[b, :-(-now[b] // B)].tolist()]
        assert sorted(free + owned) == list(range(CAP))


def test_decode_queries_gathered_from_the_packed_rows(kvq, cuda):
    """Steps in which requests end, wait and start: the packed rows behind one without a token move up, so the decode's
    queries are row cu_seqlens[b] for sequence b, in one graph with the rest.  Every sequence with a new token gets
    its own attention, an ended one zeros."""
    import torch
    batch = 5
    gen = torch.Generator(device="cuda").manual_seed(14)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool, ws = kvq.new_pool(CAP, HKV), kvq.new_scored_workspace(CAP, HKV, batch, HQ, WIDTH * B, window=WINDOW)
    ring, state = torch.arange(CAP, **i32), torch.tensor([0, CAP, 0, 0], **i32)
    lens, target = torch.zeros(batch, **i32), torch.zeros(batch, **i32)
    table, cu, maps = torch.full((batch, WIDTH), -1, **i32), torch.zeros(batch + 1, **i32), torch.zeros(3, batch, **i32)
    desc = kvq.make_rope(128)
    rope, mag = kvq.new_rope_table(desc)
    opts = kvq.make_score_opts(softcap=SOFTCAP, window=WINDOW)
    qkv = torch.zeros(batch, HQ + 2 * HKV, 128, dtype=torch.bfloat16, device="cuda")
    out, q = torch.zeros(batch, HQ, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(qkv[:, :HQ])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvq.kvq_update_tables(ring, state, state, lens, target, lens, table, cu, maps[0], maps[1], maps[2])
        kvq.kvq_rope(desc, rope, mag, maps[0], qkv[:, :HQ], qkv[:, HQ:HQ + HKV])
        kvq.kvq_quantize_append(pool, CAP, HKV, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], maps[2],
                                token_stride=(HQ + 2 * HKV) * 128)
        torch.index_select(qkv[:, :HQ], 0, cu[:-1].clamp(max=batch - 1), out=q)
        kvq.kvq_decode_attention_scored(pool, CAP, HKV, q, table, lens, WIDTH * B, out, ws, opts)
    at = [0] * batch
    # one target per sequence and step: "+" a token more, "." waits, "0" ends
    for i, step in enumerate(("+++++", "+++++", "+.+0+", "++.++", "0+++.", "+++++")):
        at = [n + 1 if x == "+" else n if x == "." else 0 for n, x in zip(at, step)]
        target.copy_(torch.tensor(at, dtype=torch.int32))
        qkv.copy_(torch.randn(qkv.shape, device="cuda", generator=gen).bfloat16())
        graph.replay()
        assert kvq.kvq_last_device_status() == 0 and lens.tolist() == at
        live = [b for b in range(batch) if step[b] == "+"]
        assert maps[1].tolist() == live + [-1] * (batch - len(live))
        bytes_, rows, rotated = pool.cpu().numpy(), table.cpu().numpy(), qkv.double().cpu().numpy()
        for b in range(batch):
            if step[b] == "0":
                assert not out[b].any()
        for n, b in enumerate(live):
            ck, cv = _cache_rows(bytes_, rows[b], at[b])
            w = _attend(rotated[n, :HQ], ck, cv, at[b] - 1)
            err = np.abs(out[b].double().cpu().numpy() - w) - 2.0 ** -8 * np.abs(w)
            assert err.max() <= helpers.ATTN_TOL


def test_calls_on_several_streams_at_once(kvq, cuda):
    """Prompts, decodes over two pools, writes and tables of different steps side by side: each as it is alone."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(9)
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = lambda n, h: torch.randn(n, h, 128, device="cuda", generator=gen).bfloat16()  # noqa: E731
    q, k, v = rows(1500, 16), rows(1500, 2), rows(1500, 2)
    cu = torch.tensor([0, 700, 1500], **i32)
    nblk, batch = 640, 5
    slots = torch.arange(nblk * B, **i32)
    table = torch.arange(nblk, **i32).view(batch, -1)
    lens = torch.tensor([2048, 1, 777, 0, 1900], **i32)
    kk, vv, q1 = rows(nblk * B, 2), rows(nblk * B, 2), rows(batch, 16)
    opts = kvq.make_score_opts(softcap=20.0)
    pools = [kvq.new_pool(nblk, 2) for _ in range(2)]
    ws = [kvq.new_scored_workspace(nblk, 2, batch, 16, 2048) for _ in range(2)]
    target = torch.tensor([2049, 1, 800, 16, 0], **i32)

    def fresh():
        return dict(prompt=torch.zeros_like(q), pools=[torch.zeros_like(p) for p in pools],
                    decode=[torch.zeros_like(q1) for _ in range(2)], ring=torch.arange(64, **i32),
                    state=torch.tensor([60, 30, 0, 0], **i32), lens=torch.empty_like(lens), table=table.clone(),
                    cu=torch.empty(batch + 1, **i32), maps=torch.empty(3, 64, **i32))

    def prompt(o):
        kvq.kvq_prefill_attention(q, k, v, cu, o["prompt"], opts=opts)

    def cache(o, i):
        kvq.kvq_quantize_append(o["pools"][i], nblk, 2, kk, vv, slots)
        kvq.kvq_decode_attention_scored(o["pools"][i], nblk, 2, q1, table, lens, 2048, o["decode"][i], ws[i], opts)

    def tables(o):
        kvq.kvq_update_tables(o["ring"], o["state"], o["state"], lens, target, o["lens"], o["table"], o["cu"],
                              o["maps"][0], o["maps"][1], o["maps"][2])

    alone = fresh()
    for call in (prompt, lambda o: cache(o, 0), lambda o: cache(o, 1), tables):
        call(alone)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(10):
        o = fresh()
        torch.cuda.synchronize()
        for s, call in zip(streams, (prompt, lambda o: cache(o, 0), lambda o: cache(o, 1), tables)):
            with torch.cuda.stream(s):
                call(o)
        torch.cuda.synchronize()
        for name, want in alone.items():
            for a, b in zip(o[name] if isinstance(want, list) else [o[name]], want if isinstance(want, list) else [want]):
                assert torch.equal(a, b), name
    # (request 0 asks for a token more than its table row holds: left as it was, and recorded)
    assert alone["lens"].tolist() == [2048, 1, 800, 16, 0]
    assert kvq.kvq_last_device_status() == kvq.KVQ_ERR_OUT_OF_RANGE

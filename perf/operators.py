"""The serving step's operators, as measured cases.

Four operators that stand next to the packed cache's write and read paths in
a serving program: the block tables and slot maps of a step, rotary positions
of its queries and keys, the attention of whole prompts over their own rows,
and the single-token attention over the packed cache with the same score
options (softcap, distance bias, sliding window).

`run` computes a case in elementary torch operations, or, when `own` is true,
through the package's entry points; `exact` computes it from the definition
in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

D = 128          # head dimension
BLOCK = 16       # token slots per cache block
DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 running requests: each grows by a token
        {"name": "tables-64-decode", "op": "tables", "batch": 64, "mean_new": 1, "churn": False, "pool_blocks": 40960},
        # a busy scheduler step: new prompts, growing and finished requests together
        {"name": "tables-2048-churn", "op": "tables", "batch": 2048, "mean_new": 64, "churn": True,
         "pool_blocks": 262144},
        # a decode step's 64 tokens, 64 query and 8 kv heads (the mixed workload's step)
        {"name": "rope-64-decode", "op": "rope", "tokens": 64, "hq": 64, "hkv": 8, "rotary_dim": 128,
         "interleaved": False, "scaling": "none", "dtype": "bf16", "far": False},
        # a chunk of ragged prompts with part of the head rotated, pairs interleaved
        {"name": "rope-2047-interleaved-part", "op": "rope", "tokens": 2047, "hq": 32, "hkv": 8, "rotary_dim": 64,
         "interleaved": True, "scaling": "linear", "dtype": "fp16", "far": False},
        # four prompts of 16384 tokens, frequencies scaled for long contexts
        {"name": "rope-65536-yarn", "op": "rope", "tokens": 65536, "hq": 64, "hkv": 8, "rotary_dim": 128,
         "interleaved": False, "scaling": "yarn", "dtype": "bf16", "far": True},
        # one short question: the latency of a prompt's attention
        {"name": "prefill-1x20-softcap", "op": "prefill", "lens": "20", "hq": 64, "hkv": 8, "dtype": "bf16",
         "softcap": 50.0, "window": 0, "alibi": False, "prefix": False},
        # a packed batch of ordinary prompts with distance-biased heads
        {"name": "prefill-12-ragged-alibi", "op": "prefill",
         "lens": "17,1500,333,64,901,1,128,1203,777,49,256,1027", "hq": 32, "hkv": 8, "dtype": "bf16", "softcap": 0.0,
         "window": 0, "alibi": True, "prefix": False},
        # two documents with a bidirectional prefix, windowed and capped scores, one kv head per query head
        {"name": "prefill-2-prefix-window-softcap", "op": "prefill", "lens": "4096,2047", "hq": 16, "hkv": 16,
         "dtype": "fp16", "softcap": 30.0, "window": 1024, "alibi": False, "prefix": True},
        # one long prompt at the long-context model's head counts
        {"name": "prefill-1x16384", "op": "prefill", "lens": "16384", "hq": 64, "hkv": 8, "dtype": "bf16",
         "softcap": 0.0, "window": 0, "alibi": False, "prefix": False},
        # one user's chat: the latency of a single-token step
        {"name": "decode-1x2047-softcap", "op": "decode", "batch": 1, "min_len": 2047, "max_len": 2047, "hq": 32,
         "hkv": 8, "kb": 4, "vb": 2, "dtype": "bf16", "softcap": 50.0, "window": 0, "alibi": False},
        # the mixed workload's 64 sequences of 8192 with a sliding window layer
        {"name": "decode-64x8192-window-softcap", "op": "decode", "batch": 64, "min_len": 8192, "max_len": 8192,
         "hq": 64, "hkv": 8, "kb": 8, "vb": 4, "dtype": "fp16", "softcap": 50.0, "window": 4096, "alibi": False},
        # the batched workload's ragged lengths, distance-biased heads
        {"name": "decode-32-ragged-alibi", "op": "decode", "batch": 32, "min_len": 4096, "max_len": 16384, "hq": 64,
         "hkv": 8, "kb": 4, "vb": 2, "dtype": "bf16", "softcap": 0.0, "window": 0, "alibi": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "prefill", "decode"])
    if op == "tables":
        batch = _log_int(rng, 1, 4096)
        return {"op": op, "batch": batch, "mean_new": _log_int(rng, 1, max(1, min(4096, 131072 // batch))),
                "churn": rng.random() < 0.7, "pool_blocks": _log_int(rng, 4096, 262144)}
    if op == "rope":
        hq, hkv = rng.choice([(64, 8), (32, 8), (16, 16), (8, 1), (14, 2), (40, 8)])
        return {"op": op, "tokens": _log_int(rng, 1, 65536), "hq": hq, "hkv": hkv,
                "rotary_dim": rng.choice([16, 32, 48, 64, 96, 128]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                "dtype": rng.choice(["bf16", "fp16"]), "far": rng.random() < 0.5}
    hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    softcap = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
    alibi = rng.random() < 0.3
    dtype = rng.choice(["bf16", "fp16"])
    if op == "prefill":
        n = _log_int(rng, 1, 48)
        lens = [_log_int(rng, 1, 8192 if n <= 4 else 2048) for _ in range(n)]
        return {"op": op, "lens": ",".join(str(x) for x in lens), "hq": hkv * group, "hkv": hkv, "dtype": dtype,
                "softcap": softcap, "window": rng.choice([0, 0, 1, _log_int(rng, 2, 4096)]), "alibi": alibi,
                "prefix": rng.random() < 0.3}
    batch = _log_int(rng, 1, 64)
    top = _log_int(rng, 1, min(65536, 524288 // batch))
    kb, vb = rng.choice([(4, 2), (4, 4), (2, 2), (8, 4)])
    return {"op": op, "batch": batch, "min_len": rng.choice([0, 1, top // 2, top]), "max_len": top, "hq": hkv * group,
            "hkv": hkv, "kb": kb, "vb": vb, "dtype": dtype, "softcap": softcap,
            "window": rng.choice([0, 0, _log_int(rng, 1, 8192)]), "alibi": alibi}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _prefixes(case):
    """Bidirectional prefix of each prompt: a third of it (a whole prompt for every fourth)."""
    return [(n if i % 4 == 3 else n // 3) if case["prefix"] else 0 for i, n in enumerate(_lens(case))]


def _decode_lens(case, seed):
    r = np.random.default_rng(1000003 * seed + 17)
    return [int(x) for x in r.integers(case["min_len"], case["max_len"] + 1, case["batch"])]


def _pairs(n, window, prefix):
    """(query, key) pairs that a prompt of n tokens reads."""
    t = np.arange(n, dtype=np.int64)
    lo = np.maximum(t - window + 1, 0) if window else np.zeros(n, dtype=np.int64)
    return int((np.maximum(t + 1, min(prefix, n)) - lo).sum())


def work(case):
    op = case["op"]
    if op == "tables":
        tokens = case["batch"] * case["mean_new"]
        # three lengths and a running sum per request, an entry read and written per block, three maps per token
        return {"bytes": 16 * case["batch"] + 8 * (tokens // BLOCK + case["batch"]) + 12 * tokens, "flops": 0}
    if op == "rope":
        rows = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": rows * D * 2 * 2 + 4 * case["tokens"], "flops": 3 * rows * case["rotary_dim"]}
    if op == "prefill":
        lens = _lens(case)
        pairs = sum(_pairs(n, case["window"], p) for n, p in zip(lens, _prefixes(case)))
        return {"bytes": sum(lens) * D * 2 * 2 * (case["hq"] + case["hkv"]), "flops": 4 * D * case["hq"] * pairs}
    mean = (case["min_len"] + case["max_len"]) / 2
    if case["window"]:
        mean = min(mean, case["window"])
    tokens = int(case["batch"] * mean)
    token_bytes = D * (case["kb"] + case["vb"]) // 8 + 8
    return {"bytes": tokens * case["hkv"] * token_bytes + case["batch"] * case["hq"] * D * 4 + 4 * (tokens // BLOCK),
            "flops": 4 * D * case["hq"] * tokens}


# ---- what a user's program has in hand -----------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _rows(g, n, heads, dtype, outliers):
    """n token rows of head vectors: N(0, 1), a few channels per head much larger when outliers."""
    scale = torch.ones(heads, D, device=DEVICE)
    if outliers:
        idx = torch.argsort(torch.rand(heads, D, device=DEVICE, generator=g), dim=1)[:, :3]
        scale.scatter_(1, idx, 10 + 20 * torch.rand(heads, 3, device=DEVICE, generator=g))
    x = torch.empty(n, heads, D, device=DEVICE, dtype=dtype)
    for a in range(0, n, 65536):
        m = min(65536, n - a)
        x[a:a + m] = (torch.randn(m, heads, D, device=DEVICE, generator=g) * scale).to(dtype)
    return x


def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device=DEVICE)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(D)


def _quantized_pool(g, tables, lens, case):
    """A pool whose blocks hold the quantized rows of the sequences (packed as the cache's layout says)."""
    hkv, kb, vb = case["hkv"], case["kb"], case["vb"]
    seg = BLOCK * D * (kb + vb) // 8 + 8 * BLOCK
    pool = torch.zeros(case["num_blocks"], hkv, seg, dtype=torch.uint8, device=DEVICE)
    rot = _hadamard(torch.float32)
    used = torch.cat([tables[b, :-(-n // BLOCK)] for b, n in enumerate(lens)]).long()
    scale = torch.ones(hkv, D, device=DEVICE)
    idx = torch.argsort(torch.rand(hkv, D, device=DEVICE, generator=g), dim=1)[:, :3]
    scale.scatter_(1, idx, 10 + 20 * torch.rand(hkv, 3, device=DEVICE, generator=g))

    def quantize(x, bits):  # [n, heads, BLOCK, D] -> packed codes and fp16 scale and zero as bytes
        r = x @ rot
        lo, hi = r.amin(-1, keepdim=True), r.amax(-1, keepdim=True)
        s, z = ((hi - lo) / (2 ** bits - 1)).half(), lo.half()
        c = torch.clamp(torch.round((r - z.float()) / s.float()), 0, 2 ** bits - 1).to(torch.uint8)
        per = 8 // bits
        c = c.view(*c.shape[:-1], D // per, per)
        packed = c[..., 0].clone()
        for j in range(1, per):
            packed |= c[..., j] << (bits * j)
        return (packed.flatten(-2), s.squeeze(-1).contiguous().view(torch.uint8),
                z.squeeze(-1).contiguous().view(torch.uint8))

    for a in range(0, len(used), 4096):
        ids = used[a:a + 4096]
        shape = (len(ids), hkv, BLOCK, D)
        kc, ks, kz = quantize(torch.randn(shape, device=DEVICE, generator=g) * scale[:, None, :], kb)
        vc, vs, vz = quantize(torch.randn(shape, device=DEVICE, generator=g), vb)
        pool[ids] = torch.cat([kc, vc, ks, kz, vs, vz], -1)
    return pool


def _inv_freq(case):
    """Radians per position of each pair, in 64 bits, and the factor on cosine and sine."""
    dim, base, factor, original = case["rotary_dim"], 10000.0, 8.0, 8192
    i = torch.arange(dim // 2, dtype=torch.float64)
    scaling, mag = case["scaling"], 1.0
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    f = base ** (-2 * i / dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":  # long wavelengths divided, short ones kept, a ramp between
        turns = original * f / (2 * math.pi)
        keep = torch.clamp((turns - 1.0) / (4.0 - 1.0), 0, 1)
        f = keep * f + (1 - keep) * f / factor
    elif scaling == "yarn":  # the ramp runs over the pair index between two numbers of turns
        def index(turns):
            return dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), dim - 1)
        divided = torch.clamp((i - lo) / max(hi - lo, 0.001), 0, 1)
        f = divided * f / factor + (1 - divided) * f
        mag = 0.1 * math.log(factor) + 1.0
    return f, mag


def _rope_desc(kvq, case):
    low, high = {"bands": (1.0, 4.0), "yarn": (1.0, 32.0)}.get(case["scaling"], (0.0, 0.0))
    return kvq.make_rope(rotary_dim=case["rotary_dim"], base=10000.0, interleaved=case["interleaved"],
                         scaling=case["scaling"], factor=8.0, original_len=8192, low=low, high=high)


def _slopes(hq):
    h = torch.arange(1, hq + 1, dtype=torch.float32, device=DEVICE)
    return torch.exp2(-8.0 * h / hq)


def _prepare_tables(case, seed, st):
    r = np.random.default_rng(seed)
    batch, mean, cap = case["batch"], case["mean_new"], case["pool_blocks"]
    max_blocks = min(4096, max(64, -(-4 * mean // BLOCK) + 64))
    old = r.integers(0, 16 * BLOCK, batch)
    new = old + (r.integers(0, 2 * mean + 1, batch) if case["churn"] else mean)
    if case["churn"]:
        kind = r.random(batch)
        new = np.where(kind < 0.1, 0, new)                     # finished
        new = np.where((kind >= 0.1) & (kind < 0.15), old // 2, new)  # rolled back
        old = np.where(kind > 0.8, 0, old)                     # new prompts
    new = np.minimum(new, max_blocks * BLOCK)
    have = -(-old // BLOCK)
    table = np.full((batch, max_blocks), -1, dtype=np.int32)
    order = r.permutation(cap).astype(np.int32)
    pos = 0
    for b in range(batch):
        n = min(int(have[b]), cap - pos)
        old[b] = min(old[b], n * BLOCK)
        if new[b] < old[b] or not case["churn"]:
            new[b] = min(new[b], old[b] + mean)
        table[b, :n] = order[pos:pos + n]
        pos += n
    free = order[pos:]
    head = int(r.integers(0, cap))
    ring = np.full(cap, -1, dtype=np.int32)
    ring[(head + np.arange(len(free))) % cap] = free
    # a step's fixed buffers are a little longer than the tokens that it usually has
    st["max_tokens"] = 37 + batch * (mean + mean // 4 + 48 if case["churn"] else mean)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEVICE)  # noqa: E731
    st.update(ring=dev(ring), state=dev(np.array([head, len(free), 0, 0])), lens=dev(old), target=dev(new),
              table=dev(table))
    n = st["max_tokens"]
    st.update(state_out=torch.zeros(4, dtype=torch.int32, device=DEVICE), lens_out=torch.empty_like(st["lens"]),
              cu=torch.empty(batch + 1, dtype=torch.int32, device=DEVICE),
              maps=torch.empty(3, n, dtype=torch.int32, device=DEVICE))


def _prepare_rope(case, seed, st):
    g = _gen(seed)
    n, dtype = case["tokens"], DTYPES[case["dtype"]]
    start = (1 << 20) if case["far"] else 0
    # ragged prompts packed one after the other
    pos = torch.arange(n, device=DEVICE)
    cut = int(torch.randint(1, n + 1, (1,), device=DEVICE, generator=g).item())
    st["positions"] = (torch.where(pos < cut, pos, pos - cut) + start).to(torch.int32)
    st["q"] = _rows(g, n, case["hq"], dtype, False)
    st["k"] = _rows(g, n, case["hkv"], dtype, True)
    f, mag = _inv_freq(case)
    st["inv_freq"], st["mag"] = f.to(DEVICE), mag
    if own:
        import bit_kv_cache_18_b200 as kvq
        st["desc"] = _rope_desc(kvq, case)
        st["table"], st["magnitude"] = kvq.new_rope_table(st["desc"])
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])


def _prepare_prefill(case, seed, st):
    g = _gen(seed)
    lens, dtype = _lens(case), DTYPES[case["dtype"]]
    n = sum(lens)
    st["lens"], st["prefixes"] = lens, _prefixes(case)
    st["q"] = _rows(g, n, case["hq"], dtype, False)
    st["k"] = _rows(g, n, case["hkv"], dtype, True)
    st["v"] = _rows(g, n, case["hkv"], dtype, False)
    st["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEVICE)
    st["prefix"] = torch.tensor(st["prefixes"], dtype=torch.int32, device=DEVICE) if case["prefix"] else None
    st["slopes"] = _slopes(case["hq"]) if case["alibi"] else None
    if own:
        import bit_kv_cache_18_b200 as kvq
        st["opts"] = kvq.make_score_opts(softcap=case["softcap"], window=case["window"], alibi_slopes=st["slopes"])
        st["out"] = torch.empty_like(st["q"])


def _prepare_decode(case, seed, st):
    g = _gen(seed)
    lens = _decode_lens(case, seed)
    blocks = [-(-n // BLOCK) for n in lens]
    width = max(1, -(-case["max_len"] // BLOCK))
    num_blocks = sum(blocks) + 8
    order = torch.randperm(num_blocks, device=DEVICE, generator=g).to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEVICE)
    pos = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[pos:pos + n]
        pos += n
    st["host_lens"], st["table"] = lens, table
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    st["pool"] = _quantized_pool(g, table, lens, dict(case, num_blocks=num_blocks))
    st["q"] = torch.randn(case["batch"], case["hq"], D, device=DEVICE, generator=g).to(DTYPES[case["dtype"]])
    st["slopes"] = _slopes(case["hq"]) if case["alibi"] else None
    if own:
        import bit_kv_cache_18_b200 as kvq
        preset = (case["kb"], case["vb"])
        st["opts"] = kvq.make_score_opts(softcap=case["softcap"], window=case["window"], alibi_slopes=st["slopes"])
        st["ws"] = kvq.new_scored_workspace(num_blocks, case["hkv"], case["batch"], case["hq"], case["max_len"],
                                            window=case["window"], preset=preset)
        st["out"] = torch.empty_like(st["q"])


def prepare(case, seed):
    st = {"case": case}
    {"tables": _prepare_tables, "rope": _prepare_rope, "prefill": _prepare_prefill,
     "decode": _prepare_decode}[case["op"]](case, seed, st)
    return st


# ---- plain forms ----------------------------------------------------------------------

def _plain_tables(st):
    ring, state, lens, target, table = st["ring"], st["state"], st["lens"].long(), st["target"].long(), st["table"]
    cap, width, batch, n = ring.numel(), table.shape[1], lens.numel(), st["max_tokens"]
    head, count = state[0].long(), state[1].long()
    have, want = (lens + BLOCK - 1) // BLOCK, (target + BLOCK - 1) // BLOCK
    grow = target > lens
    zero = torch.zeros_like(lens)
    need = torch.where(grow, want - have, zero)
    tok = torch.where(grow, target - lens, zero)
    fits = grow & (torch.cumsum(need, 0) <= count) & (torch.cumsum(tok, 0) <= n)
    need, tok = torch.where(fits, need, zero), torch.where(fits, tok, zero)
    back = torch.where(target < lens, have - want, zero)
    need_end, back_end = torch.cumsum(need, 0), torch.cumsum(back, 0)
    cu = torch.cat([zero[:1], torch.cumsum(tok, 0)])
    col = torch.arange(width, device=DEVICE)[None, :]
    taken = (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (head + (need_end - need)[:, None] + col - have[:, None]) % cap
    new_table = torch.where(taken, ring[at], table)
    freed = (col >= want[:, None]) & (col < (want + back)[:, None])
    to = (head + count + (back_end - back)[:, None] + col - want[:, None]) % cap
    new_ring = ring.clone()
    new_ring[to[freed]] = table[freed]
    i = torch.arange(n, device=DEVICE)
    live = i < cu[-1]
    seq = torch.clamp(torch.searchsorted(cu, i, right=True) - 1, max=batch - 1)
    pos = torch.where(live, lens[seq] + i - cu[seq], zero[:1])
    blk = new_table[seq, torch.clamp(pos // BLOCK, max=width - 1)].long()
    minus = torch.full_like(i, -1)
    new_state = torch.stack([(head + need_end[-1]) % cap, count - need_end[-1] + back_end[-1]])
    new_lens = torch.where(fits | (target < lens), target, lens)
    return [x.to(torch.int32) for x in (new_table, new_ring, new_state, new_lens, cu, torch.where(live, pos, minus),
                                        torch.where(live, seq, minus),
                                        torch.where(live, blk * BLOCK + pos % BLOCK, minus))]


def _plain_rope(st):
    case = st["case"]
    half = case["rotary_dim"] // 2
    angle = st["positions"].double()[:, None] * st["inv_freq"][None, :]
    cos = (torch.cos(angle) * st["mag"]).float()[:, None, :]
    sin = (torch.sin(angle) * st["mag"]).float()[:, None, :]
    outs = []
    for x in (st["q"], st["k"]):
        y = x.float()
        if case["interleaved"]:
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:2 * half]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        outs.append(torch.cat([r, y[..., 2 * half:]], -1).to(x.dtype))
    return outs


def _plain_prefill(st):
    case = st["case"]
    q, k, v, hkv = st["q"], st["k"], st["v"], case["hkv"]
    group = case["hq"] // hkv
    out = torch.empty_like(q)
    start = 0
    for n, prefix in zip(st["lens"], st["prefixes"]):
        kk = k[start:start + n].float().permute(1, 2, 0)                 # [Hkv, D, n]
        vv = v[start:start + n].float().permute(1, 0, 2)                 # [Hkv, n, D]
        qq = q[start:start + n].float().view(n, hkv, group, D).permute(1, 2, 0, 3)
        step = max(16, min(n, (1 << 28) // (case["hq"] * n)))
        for a in range(0, n, step):
            b = min(n, a + step)
            lo = max(0, a - case["window"] + 1) if case["window"] else 0
            hi = min(n, max(b, prefix))
            s = qq[:, :, a:b].reshape(hkv, group * (b - a), D) @ kk[:, :, lo:hi]
            s = s.view(hkv, group, b - a, hi - lo).mul_(1.0 / math.sqrt(D))
            if case["softcap"]:
                s = s.div_(case["softcap"]).tanh_().mul_(case["softcap"])
            t = torch.arange(a, b, device=DEVICE)[:, None]
            j = torch.arange(lo, hi, device=DEVICE)[None, :]
            if case["alibi"]:
                s = s - st["slopes"].view(hkv, group, 1, 1) * (t - j).abs().float()
            allowed = (j <= t) | (j < prefix)
            if case["window"]:
                allowed &= t - j < case["window"]
            s = s.masked_fill_(~allowed, float("-inf"))
            p = s.sub_(s.amax(-1, keepdim=True)).exp_()
            l = p.sum(-1, keepdim=True)
            o = p.view(hkv, group * (b - a), hi - lo) @ vv[:, lo:hi]
            o = o.view(hkv, group, b - a, D) / l
            out[start + a:start + b] = o.permute(2, 0, 1, 3).reshape(b - a, case["hq"], D).to(out.dtype)
        start += n
    return out


def _unpack(seg, bits, offset):
    """[blocks, Hkv, bytes] -> codes [Hkv, blocks*BLOCK, D] as uint8 of the rows at byte offset."""
    n, hkv, _ = seg.shape
    row = D * bits // 8
    x = seg[..., offset:offset + BLOCK * row].view(n, hkv, BLOCK, row)
    c = torch.stack([(x >> (bits * j)) & (2 ** bits - 1) for j in range(8 // bits)], -1)
    return c.view(n, hkv, BLOCK, D).permute(1, 0, 2, 3).reshape(hkv, n * BLOCK, D)


def _factors(seg, offset):
    n, hkv, _ = seg.shape
    x = seg[..., offset:offset + 2 * BLOCK].contiguous().view(torch.float16)
    return x.permute(1, 0, 2).reshape(hkv, n * BLOCK, 1)


def _plain_decode(st):
    case = st["case"]
    hkv, kb, vb = case["hkv"], case["kb"], case["vb"]
    group = case["hq"] // hkv
    meta = BLOCK * D * (kb + vb) // 8
    rot = _hadamard(torch.float32)
    out = torch.zeros_like(st["q"])
    for b, n in enumerate(st["host_lens"]):
        if n == 0:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        blk0 = first // BLOCK
        seg = st["pool"][st["table"][b, blk0:-(-n // BLOCK)].long()]
        cut = slice(first - blk0 * BLOCK, n - blk0 * BLOCK)
        k = (_unpack(seg, kb, 0).float() * _factors(seg, meta).float() + _factors(seg, meta + 32).float())[:, cut]
        v = (_unpack(seg, vb, BLOCK * D * kb // 8).float() * _factors(seg, meta + 64).float()
             + _factors(seg, meta + 96).float())[:, cut]
        q = st["q"][b].float().view(hkv, group, D) @ rot
        s = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
        if case["softcap"]:
            s = torch.tanh(s / case["softcap"]) * case["softcap"]
        if case["alibi"]:
            dist = (n - 1 - torch.arange(first, n, device=DEVICE)).float()
            s = s - st["slopes"].view(hkv, group, 1) * dist
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        out[b] = (o @ rot).view(case["hq"], D).to(out.dtype)
    return out


# ---- the package's entry points -----------------------------------------------------------

def _own_tables(kvq, st):
    kvq.kvq_update_tables(st["ring"], st["state"], st["state_out"], st["lens"], st["target"], st["lens_out"],
                          st["table"], st["cu"], st["maps"][0], st["maps"][1], st["maps"][2])
    return [st["table"], st["ring"], st["state_out"][:2], st["lens_out"], st["cu"], st["maps"][0], st["maps"][1],
            st["maps"][2]]


def _own_rope(kvq, st):
    kvq.kvq_rope(st["desc"], st["table"], st["magnitude"], st["positions"], st["q"], st["k"], q_out=st["q_out"],
                 k_out=st["k_out"])
    return [st["q_out"], st["k_out"]]


def _own_prefill(kvq, st):
    kvq.kvq_prefill_attention(st["q"], st["k"], st["v"], st["cu"], st["out"], opts=st["opts"],
                              prefix_lens=st["prefix"])
    return st["out"]


def _own_decode(kvq, st):
    case = st["case"]
    kvq.kvq_decode_attention_scored(st["pool"], st["pool"].shape[0], case["hkv"], st["q"], st["table"],
                                    st["seq_lens"], case["max_len"], st["out"], st["ws"], st["opts"],
                                    preset=(case["kb"], case["vb"]))
    return st["out"]


def run(st):
    op = st["case"]["op"]
    if own:
        import bit_kv_cache_18_b200 as kvq
        return {"tables": _own_tables, "rope": _own_rope, "prefill": _own_prefill, "decode": _own_decode}[op](kvq, st)
    return {"tables": _plain_tables, "rope": _plain_rope, "prefill": _plain_prefill, "decode": _plain_decode}[op](st)


# ---- the definitions in 64 bits -----------------------------------------------------------

def _exact_rope(case, seed):
    st = {"case": case}
    _prepare_rope(case, seed, st)
    half = case["rotary_dim"] // 2
    z = torch.polar(torch.full_like(st["inv_freq"], st["mag"]).expand(case["tokens"], half).contiguous(),
                    torch.outer(st["positions"].double(), st["inv_freq"]))[:, None, :]
    outs = []
    for x in (st["q"], st["k"]):
        y = x.double()
        i = torch.arange(half, device=DEVICE)
        ia, ib = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        w = torch.complex(y[..., ia], y[..., ib]) * z
        y[..., ia], y[..., ib] = w.real, w.imag
        outs.append(y)
    return outs


def _exact_prefill(case, seed):
    st = {"case": case}
    _prepare_prefill(case, seed, st)
    group = case["hq"] // case["hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
    base = 0
    for n, prefix in zip(st["lens"], st["prefixes"]):
        for h in range(case["hq"]):
            k = st["k"][base:base + n, h // group].double()
            v = st["v"][base:base + n, h // group].double()
            for a in range(0, n, 4096):
                t = torch.arange(a, min(n, a + 4096), device=DEVICE)
                s = st["q"][base + t, h].double() @ k.T / math.sqrt(D)
                if case["softcap"]:
                    s = case["softcap"] * torch.tanh(s / case["softcap"])
                dist = t[:, None] - torch.arange(n, device=DEVICE)[None, :]
                if case["alibi"]:
                    s = s - float(st["slopes"][h]) * dist.abs()
                hidden = (dist < 0) & (torch.arange(n, device=DEVICE) >= prefix)
                if case["window"]:
                    hidden |= dist >= case["window"]
                s[hidden] = -math.inf
                out[base + t, h] = torch.exp(s - torch.logsumexp(s, 1, keepdim=True)) @ v
        base += n
    return out


def _exact_decode(case, seed):
    st = {"case": case}
    _prepare_decode(case, seed, st)
    hkv, kb, vb = case["hkv"], case["kb"], case["vb"]
    group, krow, vrow = case["hq"] // hkv, D * kb // 8, D * vb // 8
    rot = _hadamard(torch.float64)

    def rows(seg, bits, start, width, s_at):  # [blocks, bytes] -> rows in the original domain
        raw = seg[:, start:start + BLOCK * width].reshape(-1, width).to(torch.int32)
        e = torch.arange(D, device=DEVICE) * bits
        c = (raw[:, e // 8] >> (e % 8)) & (2 ** bits - 1)
        f = seg[:, s_at:s_at + 4 * BLOCK].contiguous().view(torch.float16).double().view(-1, 2, BLOCK)
        return (c.double() * f[:, 0].reshape(-1, 1) + f[:, 1].reshape(-1, 1)) @ rot

    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
    meta = BLOCK * (krow + vrow)
    for b, n in enumerate(st["host_lens"]):
        if n == 0:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        for h in range(hkv):
            seg = st["pool"][st["table"][b, :-(-n // BLOCK)].long(), h]
            k = rows(seg, kb, 0, krow, meta)[first:n]
            v = rows(seg, vb, BLOCK * krow, vrow, meta + 4 * BLOCK)[first:n]
            s = st["q"][b, h * group:(h + 1) * group].double() @ k.T / math.sqrt(D)
            if case["softcap"]:
                s = case["softcap"] * torch.tanh(s / case["softcap"])
            if case["alibi"]:
                dist = torch.arange(n - 1 - first, -1, -1, device=DEVICE, dtype=torch.float64)
                s = s - st["slopes"][h * group:(h + 1) * group].double()[:, None] * dist
            out[b, h * group:(h + 1) * group] = torch.softmax(s, 1) @ v
    return out


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    return {"rope": _exact_rope, "prefill": _exact_prefill, "decode": _exact_decode}[op](case, seed)

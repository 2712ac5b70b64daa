"""kvq_update_tables against the rules of include/kvq.h, one sequence after the
other in plain Python.  Whole numbers: every output is equal."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

B = 16


def _reference(ring, state, lens, target, table, max_tokens):
    ring, table = ring.copy(), table.copy()
    cap, (head, count) = len(ring), state
    longest = table.shape[1] * B
    out = list(lens)
    cu, maps, status, stopped, taken, freed = [0], [], 0, False, 0, []
    for b, (n, t) in enumerate(zip(lens, target)):
        new = 0
        if not (0 <= n <= longest and 0 <= t <= longest):
            status = status or -5
        elif t > n:
            have, want = -(-n // B), -(-t // B)
            if stopped or taken + want - have > count or cu[-1] + t - n > max_tokens:
                if not stopped:
                    status = status or (-4 if taken + want - have > count else -5)
                stopped = True
            else:
                for e in range(have, want):
                    table[b, e] = ring[(head + taken) % cap]
                    taken += 1
                for p in range(n, t):
                    maps.append((p, b, table[b, p // B] * B + p % B))
                new, out[b] = t - n, t
        else:
            freed += list(table[b, -(-t // B):-(-n // B)])
            out[b] = t
        cu.append(cu[-1] + new)
    for i, p in enumerate(freed):
        ring[(head + count + i) % cap] = p
    maps += [(-1, -1, -1)] * (max_tokens - len(maps))
    return (ring, [(head + taken) % cap, count - taken + len(freed)], out, table, cu,
            np.array(maps, dtype=np.int32).reshape(-1, 3).T, status)


def _case(rng, batch, mean, cap, width, churn=True, head=None, spare=None):
    """Sequences that own distinct blocks, the rest free in a ring from `head` on."""
    lens = rng.integers(0, 6 * B, batch)
    kind = rng.random(batch)
    target = np.where(kind < 0.2, 0, np.where(kind < 0.35, lens // 2, lens + rng.integers(0, 2 * mean + 1, batch)))
    if not churn:
        target = lens + mean
    lens = np.minimum(np.where(kind > 0.8, 0, lens), width * B) if churn else np.minimum(lens, width * B)
    target = np.minimum(target, width * B)
    ids = rng.permutation(cap).astype(np.int32)
    table = np.full((batch, width), -1, dtype=np.int32)
    used = 0
    for b in range(batch):
        n = -(-int(lens[b]) // B)
        table[b, :n] = ids[used:used + n]
        used += n
    assert used <= cap
    free = ids[used:] if spare is None else ids[used:used + spare]
    head = int(rng.integers(0, cap)) if head is None else head
    ring = np.full(cap, -7, dtype=np.int32)
    ring[(head + np.arange(len(free))) % cap] = free
    return ring, [head, len(free)], lens.astype(np.int32), target.astype(np.int32), table


def _run(kvq, case, max_tokens, in_place=False, stream=None):
    import torch
    ring, state, lens, target, table = case
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    r, s, n, t, tb = dev(ring), dev([*state, 0, 0]), dev(lens), dev(target), dev(table)
    s2 = s if in_place else torch.zeros(4, dtype=torch.int32, device="cuda")
    n2 = n if in_place else torch.full_like(n, -9)
    cu = torch.full((len(lens) + 1,), -9, dtype=torch.int32, device="cuda")
    maps = torch.full((3, max_tokens), -9, dtype=torch.int32, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    kvq.kvq_update_tables(r, s, s2, n, t, n2, tb, cu, maps[0], maps[1], maps[2], stream=stream)
    status = kvq.kvq_last_device_status(stream)
    assert s2[2].item() == 0
    return [x.cpu().numpy() for x in (r, s2[:2], n2, tb, cu, maps)] + [status]


def _check(kvq, case, max_tokens, **kw):
    got, want = _run(kvq, case, max_tokens, **kw), _reference(*case, max_tokens)
    for name, g, w in zip(("ring", "state", "lens", "table", "cu", "maps", "status"), got, want):
        assert np.array_equal(g, np.asarray(w)), name
    return got


@pytest.mark.parametrize("batch,mean,max_tokens", [(1, 1, 200), (1, 700, 1500), (3, 5, 400), (64, 1, 3001), (33, 40, 4000),
                                                   (257, 9, 9000), (1025, 30, 70001), (4096, 2, 90000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_churn(kvq, cuda, batch, mean, max_tokens, in_place):
    rng = np.random.default_rng(batch + mean)
    case = _case(rng, batch, mean, 8 * batch + 200 + batch * mean // 4, 90)
    got = _check(kvq, case, max_tokens, in_place=in_place)
    assert got[-1] == 0


def test_decode_step(kvq, cuda):
    rng = np.random.default_rng(3)
    _check(kvq, _case(rng, 64, 1, 1024, 8, churn=False), 64)


@pytest.mark.parametrize("spare", [0, 1, 7, 40])
def test_blocks_run_out(kvq, cuda, spare):
    """The first growing sequence that the free blocks do not cover stops every later one that grows."""
    rng = np.random.default_rng(spare)
    got = _check(kvq, _case(rng, 50, 60, 500, 20, spare=spare), 6000)
    assert got[-1] == kvq.KVQ_ERR_POOL_EXHAUSTED


@pytest.mark.parametrize("max_tokens", [0, 1, 100, 4000])
def test_batch_buffer_runs_out(kvq, cuda, max_tokens):
    rng = np.random.default_rng(11)
    got = _check(kvq, _case(rng, 300, 60, 4000, 20), max_tokens)
    assert got[-1] == kvq.KVQ_ERR_OUT_OF_RANGE


def test_lengths_out_of_range(kvq, cuda):
    rng = np.random.default_rng(5)
    ring, state, lens, target, table = _case(rng, 40, 20, 400, 10)
    target[3], target[9], lens[17], lens[20] = -1, 10 * B + 1, -5, 2 ** 31 - 1
    got = _check(kvq, (ring, state, lens, target, table), 3000)
    assert got[-1] == kvq.KVQ_ERR_OUT_OF_RANGE


@pytest.mark.parametrize("state", [[-1, 3], [400, 0], [0, 401], [0, -1]])
def test_state_outside_the_ring(kvq, cuda, state):
    """Nothing is taken or returned, nothing outside the buffers is touched, and it is recorded."""
    rng = np.random.default_rng(6)
    ring, _, lens, target, table = _case(rng, 40, 20, 400, 10)
    lens, target = np.where(target > lens, 0, lens).astype(np.int32), np.where(target > lens, 30, 0).astype(np.int32)
    got = _run(kvq, (ring, state, lens, target, table), 3000)
    assert got[-1] == kvq.KVQ_ERR_OUT_OF_RANGE
    assert np.array_equal(got[0], ring) and np.array_equal(got[3], table) and list(got[1]) == state
    assert np.array_equal(got[2], lens) and not got[4].any() and (got[5] == -1).all()


@pytest.mark.parametrize("ticket", [1 << 20, 1, 5, -1, 147, -2 ** 31])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_ticket_that_is_not_zero_is_recorded(kvq, cuda, ticket, in_place):
    """State words that were never zeroed, in a call of several CTAs: every sequence is left as it was, no block moves,
    and it is recorded."""
    import torch
    ring, state, lens, target, table = _case(np.random.default_rng(13), 300, 20, 4000, 20)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    r, s, n, t, tb = dev(ring), dev([*state, ticket, 0]), dev(lens), dev(target), dev(table)
    s2 = s if in_place else dev([-9, -9, ticket, 0])
    n2 = n if in_place else torch.full_like(n, -9)
    cu, maps = torch.full((301,), -9, dtype=torch.int32, device="cuda"), torch.full((3, 9000), -9, dtype=torch.int32,
                                                                                   device="cuda")
    kvq.kvq_update_tables(r, s, s2, n, t, n2, tb, cu, maps[0], maps[1], maps[2])
    assert kvq.kvq_last_device_status() == kvq.KVQ_ERR_OUT_OF_RANGE
    assert np.array_equal(r.cpu().numpy(), ring) and np.array_equal(tb.cpu().numpy(), table)
    assert s2[:2].tolist() == state and np.array_equal(n2.cpu().numpy(), lens)
    assert not cu.any() and (maps == -1).all()
    s2[2] = 0  # and then it works
    kvq.kvq_update_tables(r, s, s2, n, t, n2, tb, cu, maps[0], maps[1], maps[2])
    want = _reference(ring, state, lens, target, table, 9000)
    assert kvq.kvq_last_device_status() == 0 and s2[:2].tolist() == want[1] and s2[2].item() == 0
    assert np.array_equal(n2.cpu().numpy(), np.asarray(want[2])) and np.array_equal(r.cpu().numpy(), want[0])


def test_bad_block_ids_give_no_slot(kvq, cuda):
    table = np.array([[3, -1], [134217727, 5]], dtype=np.int32)  # 2^27 - 1: its slots would pass 2^31
    ring = np.array([-2, 4, 9, 9], dtype=np.int32)
    got = _run(kvq, (ring, [0, 2], np.array([15, 3], np.int32), np.array([18, 5], np.int32), table), 5)
    assert got[-1] == kvq.KVQ_ERR_OUT_OF_RANGE
    assert got[5][2].tolist() == [3 * B + 15, -1, -1, -1, -1] and got[3].tolist() == [[3, -2], [134217727, 5]]


def test_empty_batch(kvq, cuda):
    z = np.zeros(0, np.int32)
    got = _run(kvq, (np.arange(4, dtype=np.int32), [1, 3], z, z, np.zeros((0, 4), np.int32)), 7)
    assert got[-1] == 0 and list(got[1]) == [1, 3] and got[4].tolist() == [0] and (got[5] == -1).all()


def test_largest_batch(kvq, cuda):
    rng = np.random.default_rng(8)
    _check(kvq, _case(rng, 16384, 1, 16384 * 7, 8, churn=False), 16384)


def test_replayed_steps_and_a_side_stream(kvq, cuda):
    """A captured step, replayed on its own state: forty decode steps from one graph."""
    import torch
    rng = np.random.default_rng(9)
    ring, state, lens, _, table = _case(rng, 20, 1, 400, 10, churn=False)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    r, s, n, tb = dev(ring), dev([*state, 0, 0]), dev(lens), dev(table)
    t, cu, maps = torch.empty_like(n), torch.zeros(21, dtype=torch.int32, device="cuda"), \
        torch.zeros(3, 24, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        torch.add(n, 1, out=t)
        kvq.kvq_update_tables(r, s, s, n, t, n, tb, cu, maps[0], maps[1], maps[2])
    want = (ring, state, list(lens), table)
    for _ in range(40):
        g.replay()
        want = _reference(want[0], want[1], want[2], [x + 1 for x in want[2]], want[3], 24)
        got = [x.cpu().numpy() for x in (r, s[:2], n, tb, cu, maps)]
        for a, b in zip(got, want[:6]):
            assert np.array_equal(a, np.asarray(b))
    assert kvq.kvq_last_device_status() == 0
    _check(kvq, _case(rng, 64, 1, 1024, 8, churn=False), 64, stream=side)


def test_wrapper_refusals(kvq, cuda):
    import torch
    z = lambda *s, **k: torch.zeros(*s, dtype=k.get("dtype", torch.int32), device=k.get("device", "cuda"))  # noqa: E731
    good = dict(ring=z(8), state_in=z(4), state_out=z(4), seq_lens=z(2), target_lens=z(2), lens_out=z(2),
                block_table=z(2, 3), cu_seqlens=z(3), positions=z(4), seq_ids=z(4), slots=z(4))
    kvq.kvq_update_tables(**good)
    for bad in (dict(ring=z(8, dtype=torch.int64)), dict(state_in=z(3)), dict(target_lens=z(3)), dict(lens_out=z(1)),
                dict(block_table=z(3, 2)), dict(block_table=z(2, 6)[:, ::2]), dict(cu_seqlens=z(2)), dict(slots=z(5)),
                dict(seq_ids=z(4, device="cpu"))):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_update_tables(**{**good, **bad})

"""kvq_rope against the definition in 64 bits.

Tolerance of an output y = m (a cos t - b sin t): half a step of its type
(eps/2 of |y|, or half the smallest subnormal) plus the fp32 arithmetic on
values of size |a| + |b|: the angle's rounding to fp32 half turns, 2^-25 pi =
9.4e-8, and its cut at 2^-32 turns, 1.5e-9; two units of sincospif, 2.4e-7;
the factor m and its rounding, 1.2e-7; product and sum, 1.2e-7: 6e-7 in all.
The cosine and sine of the definition come from the exact phase modulo a turn.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


def _t(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _want(x, positions, turns, mag, interleaved):
    """x [n, H, 128] in 64 bits -> rotated, and |a| + |b| of each element (0 behind the rotated part)."""
    half = len(turns)
    phase = [[(int(p) * int(t) % 2 ** 64) / 2 ** 64 for t in turns] for p in positions]
    t = 2 * np.pi * np.array(phase)[:, None, :]
    y, size = x.copy(), np.zeros_like(x)
    ia = 2 * np.arange(half) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = mag * (a * np.cos(t) - b * np.sin(t)), mag * (b * np.cos(t) + a * np.sin(t))
    size[..., ia] = size[..., ib] = mag * (np.abs(a) + np.abs(b))
    return y, size


def _check(got, x, positions, turns, mag, interleaved, dtype):
    import torch
    want, size = _want(x.double().cpu().numpy(), positions, turns, mag, interleaved)
    err = np.abs(got.double().cpu().numpy() - want)
    tol = np.abs(want) * torch.finfo(_t(dtype)).eps / 2 + TINY[dtype] + 6e-7 * size
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,hq,hkv,n", [(128, 64, 8, 5), (16, 8, 1, 1), (48, 14, 2, 3), (64, 3, 3, 33), (96, 40, 8, 2),
                                          (112, 1, 0, 7), (128, 130, 70, 2)])
def test_layouts_and_parts(kvq, cuda, dtype, interleaved, dim, hq, hkv, n):
    import torch
    d = kvq.make_rope(dim, 10000.0, interleaved, "yarn", 8.0, 4096, 1.0, 32.0)
    table, mag = kvq.new_rope_table(d)
    turns, _ = kvq.kvq_rope_table(d)
    g = torch.Generator(device="cuda").manual_seed(dim + hq)
    pos = np.random.default_rng(dim).integers(0, 200000, n).astype(np.int32)
    q = torch.randn(n, hq, 128, device="cuda", generator=g).to(_t(dtype))
    k = (30 * torch.randn(n, hkv, 128, device="cuda", generator=g)).to(_t(dtype)) if hkv else None
    qo, ko = torch.empty_like(q), torch.empty_like(k) if hkv else None
    p = torch.from_numpy(pos).cuda()
    kvq.kvq_rope(d, table, mag, p, q, k, qo, ko)
    _check(qo, q, pos, turns, mag, interleaved, dtype)
    if hkv:
        _check(ko, k, pos, turns, mag, interleaved, dtype)
    # in place: the same values
    kvq.kvq_rope(d, table, mag, p, q, k)
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "bands", "yarn"])
def test_far_positions(kvq, cuda, scaling):
    """Exact angles up to the last position an int32 holds."""
    import torch
    d = kvq.make_rope(128, 10000.0, False, scaling, 8.0, 8192, 1.0, 4.0)
    table, mag = kvq.new_rope_table(d)
    pos = np.array([0, 1, 8191, 2 ** 20 + 3, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1], dtype=np.int32)
    q = torch.randn(len(pos), 4, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).half()
    out = torch.empty_like(q)
    kvq.kvq_rope(d, table, mag, torch.from_numpy(pos).cuda(), q, q_out=out)
    _check(out, q, pos, kvq.kvq_rope_table(d)[0], mag, False, "fp16")


def test_strided_rows_of_a_fused_projection(kvq, cuda):
    """q and k are slices of one [n, (Hq + 2 Hkv), 128] buffer, rotated in place: the v part and the padding rows
    (negative positions) keep their bytes."""
    import torch
    n, hq, hkv = 21, 8, 2
    qkv = torch.randn(n, hq + 2 * hkv, 128, device="cuda").bfloat16()
    before = qkv.clone()
    d = kvq.make_rope(64, 10000.0, True)
    table, mag = kvq.new_rope_table(d)
    pos = np.arange(n, dtype=np.int32)
    pos[-4:] = -1
    kvq.kvq_rope(d, table, mag, torch.from_numpy(pos).cuda(), qkv[:, :hq], qkv[:, hq:hq + hkv])
    assert torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:]) and torch.equal(qkv[-4:], before[-4:])
    _check(qkv[:-4, :hq + hkv], before[:-4, :hq + hkv], pos[:-4], kvq.kvq_rope_table(d)[0], mag, True, "bf16")


def test_offsets_beyond_32_bits(kvq, cuda):
    """Rows whose element offset passes 2^31."""
    import torch
    n, h = 16400, 1024
    q = torch.zeros(n, h, 128, dtype=torch.bfloat16, device="cuda")  # 4.3 GB, 2.15e9 elements
    rows = torch.randn(2, h, 128, device="cuda").bfloat16()
    q[-2:] = rows
    d = kvq.make_rope()
    table, mag = kvq.new_rope_table(d)
    pos = np.zeros(n, dtype=np.int32)
    pos[-2:] = (77, 123456)
    kvq.kvq_rope(d, table, mag, torch.from_numpy(pos).cuda(), q)
    _check(q[-2:], rows, pos[-2:], kvq.kvq_rope_table(d)[0], mag, False, "bf16")


def test_infinities_stay_in_their_pair(kvq, cuda):
    import torch
    q = torch.randn(1, 1, 128, device="cuda").half()
    q[0, 0, 5] = float("inf")
    d = kvq.make_rope(rotary_dim=64)
    table, mag = kvq.new_rope_table(d)
    out = torch.empty_like(q)
    kvq.kvq_rope(d, table, mag, torch.tensor([3], dtype=torch.int32, device="cuda"), q, q_out=out)
    bad = (~torch.isfinite(out[0, 0])).nonzero().flatten().tolist()
    assert bad == [5, 37]


def test_graph_and_side_stream(kvq, cuda):
    import torch
    d = kvq.make_rope()
    table, mag = kvq.new_rope_table(d)
    q = torch.randn(9, 4, 128, device="cuda").half()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    want, out = torch.empty_like(q), torch.empty_like(q)
    kvq.kvq_rope(d, table, mag, pos, q, q_out=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kvq.kvq_rope(d, table, mag, pos, q, q_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    q.mul_(0.5)
    g.replay()
    kvq.kvq_rope(d, table, mag, pos, q, q_out=want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_wrapper_refusals(kvq, cuda):
    import torch
    d = kvq.make_rope()
    table, mag = kvq.new_rope_table(d)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    q, k = torch.zeros(3, 4, 128, device="cuda").half(), torch.zeros(3, 2, 128, device="cuda").half()
    kvq.kvq_rope(d, table, mag, pos, q, k)
    kvq.kvq_rope(d, table, mag, pos[:0], q[:0], k[:0])
    for bad in (dict(positions=pos.long()), dict(positions=pos[:2]), dict(q=q.float()), dict(q=q[:, :, ::2]),
                dict(q=q.transpose(0, 1)), dict(k=k.bfloat16()), dict(k=k.cpu()), dict(table=table[:32]),
                dict(q_out=torch.zeros(3, 5, 128, device="cuda").half()), dict(k=None, k_out=k)):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_rope(**{**dict(desc=d, table=table, magnitude=mag, positions=pos, q=q, k=k), **bad})

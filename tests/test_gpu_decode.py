"""gdn_decode against the 64-bit token recurrence, through the public binding."""
import pytest
import torch

import operator_reference as R
from linear_attention_ssm_gdn_b200 import GdnError, gdn_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _setup(lens, Hk, Hv, d, seed, pad=(), spare=3):
    gen = torch.Generator().manual_seed(seed)
    n = len(lens)
    pool = torch.randn(n + spare, Hv, d, d, generator=gen) * 0.1
    slots = torch.randperm(n + spare, generator=gen)[:n].tolist()
    rows = R.rows(gen, sum(lens), Hk, Hv, d)
    pool_gpu = pool.to(DEV)
    table = torch.tensor([0 if b in pad else pool_gpu[s].data_ptr() for b, s in enumerate(slots)],
                         dtype=torch.int64, device=DEV)
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    return pool, pool_gpu, slots, table, cu, rows


def _check(lens, pool, pool_gpu, slots, rows, o, scale, pad=()):
    o_ref, h_ref = R.forward(*rows, lens, pool[slots], scale)
    cu = R.offsets(lens)
    for b in pad:
        o_ref[cu[b]:cu[b + 1]] = 0
        h_ref[b] = pool[slots[b]].double()
        assert not o[cu[b]:cu[b + 1]].any()
    assert R.rel(o, o_ref) <= R.BF16_REL + R.F32_REL
    got = pool_gpu.cpu()
    # per row two products of d terms: d 2^-24 each of the state's size, at the most
    most, d = max(max(lens), 1), pool.shape[-1]
    assert R.rel(got[slots], h_ref) <= most * 2 * (d + 8) * 2.0 ** -24
    others = [s for s in range(pool.shape[0]) if s not in slots]
    for s in others + [slots[b] for b in range(len(lens)) if lens[b] == 0 or b in pad]:
        assert torch.equal(got[s], pool[s])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (2, 6), (3, 3)])
@pytest.mark.parametrize("n", [1, 5])
def test_one_row_each(d, heads, n):
    lens = [1] * n
    pool, pg, slots, table, cu, rows = _setup(lens, *heads, d, seed=n + d)
    dev = [x.to(DEV) for x in rows]
    o = gdn_decode(table, *dev, scale=0.5)
    _check(lens, pool, pg, slots, rows, o, 0.5)
    # the same through row offsets, bit for bit
    pg2 = pool.to(DEV)
    table2 = torch.tensor([pg2[s].data_ptr() for s in slots], dtype=torch.int64, device=DEV)
    o2 = gdn_decode(table2, *dev, cu_seqlens=cu, scale=0.5)
    assert torch.equal(o, o2) and torch.equal(pg, pg2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[3], [0, 1, 7, 0, 2], [0, 0, 1], [40, 1]])
def test_ragged_rows(d, lens):
    pool, pg, slots, table, cu, rows = _setup(lens, 2, 4, d, seed=d + sum(lens))
    o = gdn_decode(table, *[x.to(DEV) for x in rows], cu_seqlens=cu)
    _check(lens, pool, pg, slots, rows, o, 1.0)


def test_padding_entries_and_rows_behind_the_last_sequence():
    lens = [2, 3, 1, 2]
    pool, pg, slots, table, cu, rows = _setup(lens, 2, 4, 128, seed=3, pad=(1, 3))
    spare = 5
    dev = [torch.cat([x, torch.full((spare, *x.shape[1:]), float("nan"), dtype=x.dtype)]).to(DEV)
           for x in rows]
    o = torch.full((sum(lens) + spare, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    gdn_decode(table, *dev, cu_seqlens=cu, o=o)
    assert (o[sum(lens):] == 7.0).all()
    _check(lens, pool, pg, slots, rows, o[:sum(lens)], 1.0, pad=(1, 3))


def test_offsets_outside_the_rows_are_clamped():
    lens = [2, 2]
    pool, pg, slots, table, _, rows = _setup(lens, 1, 2, 64, seed=4)
    cu = torch.tensor([-3, 2, 1000], dtype=torch.int32, device=DEV)
    o = gdn_decode(table, *[x.to(DEV) for x in rows], cu_seqlens=cu)
    _check(lens, pool, pg, slots, rows, o, 1.0)


def test_strided_views():
    lens = [1] * 6
    Hk, Hv, d = 2, 4, 64
    pool, pg, slots, table, _, (q, k, v, g, beta) = _setup(lens, Hk, Hv, d, seed=5)
    qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).to(DEV)
    ba = torch.cat([g, beta], 1).to(DEV)
    s = qkv.split([Hk * d, Hk * d, Hv * d], 1)
    o = gdn_decode(table, s[0].unflatten(1, (Hk, d)), s[1].unflatten(1, (Hk, d)),
                   s[2].unflatten(1, (Hv, d)), ba[:, :Hv], ba[:, Hv:])
    _check(lens, pool, pg, slots, (q, k, v, g, beta), o, 1.0)


def test_gates_at_their_ends():
    """g = -inf forgets the state, g = 0 keeps it, beta = 0 writes nothing."""
    lens = [1] * 4
    pool, pg, slots, table, _, (q, k, v, g, beta) = _setup(lens, 1, 2, 128, seed=6)
    g[0], g[1], beta[2], g[3] = -float("inf"), 0.0, 0.0, -200.0
    o = gdn_decode(table, *[x.to(DEV) for x in (q, k, v, g, beta)])
    _check(lens, pool, pg, slots, (q, k, v, g, beta), o, 1.0)


def test_many_sequences_many_heads():
    lens = [1] * 64
    pool, pg, slots, table, _, rows = _setup(lens, 4, 12, 64, seed=7)
    o = gdn_decode(table, *[x.to(DEV) for x in rows])
    _check(lens, pool, pg, slots, rows, o, 1.0)


def test_captured_steps_on_another_stream():
    """Two steps of new rows in one graph, replayed twice: four steps in a row."""
    lens, Hk, Hv, d = [1, 1, 1], 2, 4, 128
    pool, pg, slots, table, _, _ = _setup(lens, Hk, Hv, d, seed=8)
    gen = torch.Generator().manual_seed(9)
    steps = [R.rows(gen, 3, Hk, Hv, d) for _ in range(4)]
    bufs = [[x.to(DEV) for x in s] for s in steps[:2]]
    outs = [torch.zeros(3, Hv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for x, o in zip(bufs, outs):
            gdn_decode(table, *x, o=o)
    h = pool[slots]
    for rep in range(2):
        for x, s in zip(bufs, steps[2 * rep:]):
            for dst, src in zip(x, s):
                dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for o, s in zip(outs, steps[2 * rep:]):
            o_ref, h = R.forward(*s, lens, h)
            assert R.rel(o, o_ref) <= R.BF16_REL + R.F32_REL
    assert R.rel(pg.cpu()[slots], h) <= 4 * 2 * (d + 8) * 2.0 ** -24


def test_explicit_stream_and_empty_calls():
    lens = [1, 1]
    pool, pg, slots, table, _, rows = _setup(lens, 1, 2, 64, seed=10)
    dev = [x.to(DEV) for x in rows]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = gdn_decode(table, *dev, stream=side)
    side.synchronize()
    _check(lens, pool, pg, slots, rows, o, 1.0)
    none = [x[:0] for x in dev]
    assert gdn_decode(table[:0], *none).shape == (0, 2, 64)
    assert gdn_decode(table, *none, cu_seqlens=torch.zeros(3, dtype=torch.int32, device=DEV)).shape[0] == 0


def test_refusals():
    lens = [1, 1]
    _, _, _, table, cu, rows = _setup(lens, 1, 2, 64, seed=11)
    q, k, v, g, beta = [x.to(DEV) for x in rows]
    with pytest.raises(ValueError, match="one row per sequence"):
        gdn_decode(table[:1], q, k, v, g, beta)
    with pytest.raises(ValueError, match="cu_seqlens"):
        gdn_decode(table, q, k, v, g, beta, cu_seqlens=cu[:2])
    with pytest.raises(TypeError, match="v"):
        gdn_decode(table, q, k, v.float(), g, beta)
    with pytest.raises(GdnError, match="16-byte"):
        wide = torch.zeros(2, 72, dtype=torch.bfloat16, device=DEV)[:, 2:66].unflatten(1, (1, 64))
        gdn_decode(table, wide, wide, v, g, beta)

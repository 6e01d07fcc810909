"""gdn_state_tables against the definition, and the tables in the calls that read them."""
import numpy as np
import pytest
import torch

import operator_reference as R
from linear_attention_ssm_gdn_b200 import (_lib, gdn_chunk_backward, gdn_chunk_prefill,
                                           gdn_decode, gdn_state_tables)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _expect(lens, slots, pool):
    chunks = [-(-x // 64) for x in lens]
    row_seq = np.repeat(np.arange(len(lens)), lens)
    return {"cu_seqlens": R.offsets(lens), "cu_chunks": R.offsets(chunks), "row_seq": row_seq,
            "row_slot": np.maximum(np.array(slots, dtype=np.int64), -1)[row_seq],
            "chunk_seq": np.repeat(np.arange(len(lens)), chunks),
            "h_table": [pool[s].data_ptr() if s >= 0 else 0 for s in slots]}


def _lens(n, seed):
    rng = np.random.default_rng(seed)
    return [int(x) for x in rng.choice([0, 1, 1, 63, 64, 65, 300], n)]


@pytest.mark.parametrize("n", [1, 2, 31, 256, 1023, 1024, 1025, 5000])
def test_tables(n):
    lens = [1] if n == 1 else _lens(n, n)
    slots = list(np.random.default_rng(n).permutation(n + 3)[:n])
    if n > 2:
        slots[1] = -1
    pool = torch.empty(n + 3, 1, 8, 8, device=DEV)
    flag = _int([0])
    t = gdn_state_tables(_int(lens), _int(slots), pool, total_rows=sum(lens), flag=flag)
    want = _expect(lens, slots, pool)
    assert set(t) == set(want)
    for name, x in want.items():
        got = t[name].cpu().numpy()
        assert np.array_equal(got[:len(x)], np.asarray(x)), name
        assert name == "chunk_seq" or len(got) == len(x)
    assert int(flag) == 0


def test_only_what_is_asked_for_and_longer_buffers():
    lens, spare = [0, 70, 0, 0, 5, 1, 0], 50
    full = _expect(lens, [0] * 7, torch.empty(1, 1, 8, 8, device=DEV))
    for keys in (("cu_seqlens",), ("cu_chunks", "chunk_seq"), ("row_seq",),
                 ("cu_seqlens", "row_seq", "chunk_seq")):
        out = {x: torch.full((len(full[x]) + (spare if "seq" in x and "cu" not in x else 0),), -9,
                             dtype=torch.int32, device=DEV) for x in keys}
        assert gdn_state_tables(_int(lens), out=out) is out
        for x in keys:
            got = out[x].cpu().numpy()
            assert np.array_equal(got[:len(full[x])], np.asarray(full[x])), x
            assert (got[len(full[x]):] == -9).all(), x


def test_no_sequences_and_no_rows():
    t = gdn_state_tables(_int([]), total_rows=0)
    assert t["cu_seqlens"].tolist() == [0] and t["cu_chunks"].tolist() == [0]
    t = gdn_state_tables(_int([0, 0, 0]), total_rows=0)
    assert t["cu_seqlens"].tolist() == [0] * 4 and t["cu_chunks"].tolist() == [0] * 4


def test_one_long_sequence_among_short_ones():
    lens = [1, 3_000_000, 0, 2]
    t = gdn_state_tables(_int(lens), total_rows=sum(lens))
    assert torch.equal(t["row_seq"].cpu(), torch.repeat_interleave(
        torch.arange(4, dtype=torch.int32), torch.tensor(lens)))


@pytest.mark.parametrize("what", ["length", "slot", "rows", "chunks"])
def test_bad_values_set_the_flag_and_stay_in_bounds(what):
    lens, slots = [3, 200, 5], [0, 1, 2]
    pool = torch.empty(3, 1, 8, 8, device=DEV)
    if what == "length":
        lens[1] = -7
    if what == "slot":
        slots[1] = 3
    rows = 100 if what == "rows" else 208
    chunks = 2 if what == "chunks" else 10
    guard = 64
    buf = {"row_seq": torch.full((rows + guard,), -9, dtype=torch.int32, device=DEV),
           "row_slot": torch.full((rows + guard,), -9, dtype=torch.int32, device=DEV),
           "chunk_seq": torch.full((chunks + guard,), -9, dtype=torch.int32, device=DEV)}
    out = {"row_seq": buf["row_seq"][:rows], "row_slot": buf["row_slot"][:rows],
           "chunk_seq": buf["chunk_seq"][:chunks], "cu_seqlens": _int([0] * 4),
           "cu_chunks": _int([0] * 4), "h_table": torch.zeros(3, dtype=torch.int64, device=DEV)}
    flag = _int([1])  # another bit: kept
    gdn_state_tables(_int(lens), _int(slots), pool, out=out, flag=flag)
    assert int(flag) == 1 | _lib.GDN_FLAG_ERROR
    for x in buf:
        assert (buf[x][-guard:] == -9).all()
    cu, cc = out["cu_seqlens"].tolist(), out["cu_chunks"].tolist()
    assert cu == {"length": [0, 3, 3, 8], "rows": [0, 3, 100, 100]}.get(what, [0, 3, 203, 208])
    assert cc == {"length": [0, 1, 1, 2], "chunks": [0, 1, 2, 2]}.get(what, [0, 1, 5, 6])
    if what == "slot":
        assert out["h_table"][1] == 0 and (out["row_slot"][3:203] == -1).all()


def test_largest_lengths_do_not_overflow():
    flag = _int([0])
    out = {"cu_seqlens": _int([0] * 4), "cu_chunks": _int([0] * 4)}
    gdn_state_tables(_int([2**31 - 1] * 3), out=out, flag=flag)
    assert out["cu_seqlens"].tolist() == [0, 2**31 - 2, 2**31 - 2, 2**31 - 2]
    assert int(flag) == _lib.GDN_FLAG_ERROR


def test_refusals():
    lens, pool = _int([1, 2]), torch.empty(4, 1, 8, 8, device=DEV)
    for kw in (dict(), dict(slots=lens, total_rows=3), dict(pool=pool, total_rows=3),
               dict(slots=lens, pool=pool, out={}), dict(slots=_int([1]), pool=pool, total_rows=3),
               dict(out={"cu_seqlens": _int([0])}), dict(out={"row_slot": lens}),
               dict(slots=lens, pool=pool, out={"h_table": torch.zeros(2, dtype=torch.int64, device=DEV),
                                                "row_seq": lens, "row_slot": _int([1])}),
               dict(slots=lens, pool=pool.transpose(2, 3), total_rows=3)):
        with pytest.raises(ValueError):
            gdn_state_tables(lens, **kw)
    with pytest.raises(TypeError):
        gdn_state_tables(lens.long(), total_rows=3)


def test_a_captured_step_follows_its_lengths():
    lens, pool = _int([1, 1, 1, 1]), torch.empty(6, 1, 8, 8, device=DEV)
    slots = _int([5, 0, 3, 1])
    out = gdn_state_tables(lens, slots, pool, total_rows=400)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn_state_tables(lens, slots, pool, out=out)
    for new in ([3, 0, 70, 1], [0, 0, 0, 400]):
        lens.copy_(_int(new))
        graph.replay()
        want = _expect(new, [5, 0, 3, 1], pool)
        for x in ("cu_seqlens", "cu_chunks", "row_seq", "row_slot", "chunk_seq", "h_table"):
            assert np.array_equal(out[x].cpu().numpy()[:len(want[x])], np.asarray(want[x])), x


def test_an_engine_step_and_a_training_step_together():
    """Tables, prompts through the prefill, their states into the pool, then decode
    steps through the tables' pointers; and the backward pass over the same rows."""
    gen = torch.Generator().manual_seed(1)
    Hk, Hv, d, lens = 2, 4, 128, [70, 1, 0, 130]
    n, pool = len(lens), torch.zeros(7, Hv, d, d, device=DEV)
    slots = [6, 2, 0, 3]
    rows = R.rows(gen, sum(lens), Hk, Hv, d)
    dev = [x.to(DEV) for x in rows]
    t = gdn_state_tables(_int(lens), _int(slots), pool, total_rows=sum(lens))
    o, hT = gdn_chunk_prefill(*dev, t["cu_seqlens"])
    pool[torch.tensor(slots, device=DEV)] = hT
    o_ref, h = R.forward(*rows, lens)
    assert R.rel(o, o_ref) <= 5e-3  # the prefill's own bound
    new = [1, 2, 1, 0]
    more = R.rows(gen, sum(new), Hk, Hv, d)
    t2 = gdn_state_tables(_int(new), _int(slots), pool, total_rows=sum(new))
    got = gdn_decode(t2["h_table"], *[x.to(DEV) for x in more], cu_seqlens=t2["cu_seqlens"])
    want, h2 = R.forward(*more, new, hT.cpu())
    assert R.rel(got, want) <= R.BF16_REL + R.F32_REL
    assert R.rel(pool.cpu()[slots], h2) <= 4 * (d + 8) * 2.0 ** -24
    do = torch.randn(sum(lens), Hv, d, generator=gen).to(torch.bfloat16)
    grads = gdn_chunk_backward(*dev, t["cu_seqlens"], do.to(DEV))
    for x, y in zip(grads[:5], R.backward(*rows, lens, do)):
        assert R.rel(x, y) <= (R.BF16_REL if x.dtype == torch.bfloat16 else 0) + R.F32_REL

"""gdn_chunk_backward where rows, decays or values leave the ordinary range."""
import pytest
import torch

import operator_reference as R
from linear_attention_ssm_gdn_b200 import (debug_device_errors, gdn_chunk_backward,
                                           gdn_chunk_backward_workspace_bytes)
from test_gpu_chunk_backward import DEV, NAMES, _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("empty", [2, 40])
@pytest.mark.parametrize("given", [True, False])
def test_rows_but_only_empty_sequences(empty, d, given):
    """No sequence owns a row: dh0 is dhT (or zeros) as soon as the call has ended in its
    stream, and no row's gradient is touched.  (Above 32 sequences another kernel makes the map.)"""
    rows, do, h0, dhT = _case([200], 2, 4, d, seed=1)
    dhT = torch.randn(empty, 4, d, d, device=DEV)
    cu = torch.zeros(empty + 1, dtype=torch.int32, device=DEV)
    dev = [x.to(DEV) for x in rows]
    do = do.to(DEV)
    for _ in range(3):
        dh0 = torch.full_like(dhT, float("nan"))
        gdn_chunk_backward(*dev, cu, do, dhT=dhT if given else None, dh0=dh0)
        assert torch.equal(dh0, dhT if given else torch.zeros_like(dhT))
    assert debug_device_errors() == [0, 0, 0, 0]


def test_a_captured_call_replayed_without_rows():
    """A step of fixed size whose sequences are all empty at one replay and full at the next."""
    lens, d = [70, 130], 64
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=2)
    dev = [x.to(DEV) for x in rows]
    do, h0, dhT = do.to(DEV), h0.to(DEV), dhT.to(DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    ws = torch.empty(gdn_chunk_backward_workspace_bytes(200, 2, 1, 2, d, d), dtype=torch.uint8,
                     device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn_chunk_backward(*dev, cu, do, h0=h0, dhT=dhT, workspace=ws)
        copy = got[5].clone()
    want = gdn_chunk_backward(*dev, torch.tensor([0, 70, 200], dtype=torch.int32, device=DEV),
                              do, h0=h0, dhT=dhT)
    for lens_now in ([0, 0], [70, 130], [0, 0], [70, 130]):
        cu.copy_(torch.tensor(R.offsets(lens_now), dtype=torch.int32))
        graph.replay()
        if sum(lens_now):
            for x, y in zip(got, want):
                assert torch.equal(x, y)
        else:
            assert torch.equal(copy, dhT)


@pytest.mark.parametrize("rise", [20.0, 70.0])
@pytest.mark.parametrize("fall", [5.0, 120.0, 1e4])
def test_gates_that_rise_and_then_fall(rise, fall):
    """A rise within the documented bound, and within the same 16 rows a fall far below where it
    began: no decay of a pair of rows overflows, though those to the block's end differ by more
    than f32 holds."""
    lens, d = [100], 64
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=3)
    rows[3].fill_(-0.01)
    rows[3][20], rows[3][26] = rise, -fall
    rows[2][:20] *= 2.0 ** -60  # what the rise enlarges
    h0 = h0 * 2.0 ** -60
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))
    want = R.backward(*dev, lens, do.to(DEV), h0.to(DEV), dhT.to(DEV))
    for name, x, y in zip(NAMES, got, want):
        assert torch.isfinite(x).all(), name
        if name != "dg":
            assert R.rel(x, y) <= (R.BF16_REL if name in NAMES[:3] else 0) + R.F32_REL, name


def _row_errors(x, y):
    """Of each row (all heads): 2-norm of the difference over that of y."""
    x, y = x.double().flatten(1), y.flatten(1)
    return ((x - y).norm(dim=1) / y.norm(dim=1)).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gate, rows_", [(-0.3, 64), (-0.5, 64), (-1.0, 64), (-0.3, 200), (-2.0, 40)])
@pytest.mark.parametrize("what", ["last row", "final state", "first row of v"])
def test_masked_gradients_behind_strong_decays(what, gate, rows_, d):
    """All that reaches the chunk's first rows comes through its decays (of e^-19 to e^-80, f32's
    range is e^-87): every row is as near to its own size as where nothing decays."""
    lens = [rows_]
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=4)
    rows[3].fill_(gate)
    rows[3][::5] *= 0.7  # (not the same for all)
    if what == "final state":
        do = torch.zeros_like(do)
    else:
        do[:-1] = 0
        dhT = torch.zeros_like(dhT)
    if what == "first row of v":  # the forward scan's counterpart
        rows[2][1:] = 0
        h0 = torch.zeros_like(h0)
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor([0, rows_], dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))
    want = R.backward(*dev, lens, do.to(DEV), h0.to(DEV), dhT.to(DEV))
    errs = {"dv": _row_errors(got[2], want[2]), "dh0": R.rel(got[5], want[5]),
            "dbeta": R.rel(got[4], want[4])}
    print(errs)
    assert errs["dv"] <= R.BF16_REL + R.F32_REL
    assert errs["dh0"] <= R.F32_REL and errs["dbeta"] <= R.F32_REL


@pytest.mark.parametrize("rise, fall, where", [(70.0, 90.0, 26), (70.0, 75.0, 26), (70.0, 110.0, 40)])
def test_a_rise_and_a_fall_beyond_f32_between_them(rise, fall, where):
    """From the top of the rise to the end of the fall it is e^-75 to e^-110: what f32 no longer
    holds (below e^-87) is lost on the way back to the first rows, in any form in 32 bits, but
    nothing overflows, and the rows from the fall on are right."""
    lens, d = [100], 64
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=5)
    rows[3].fill_(-0.01)
    rows[3][20], rows[3][where] = rise, -fall
    rows[2][:20] *= 2.0 ** -60
    h0 = h0 * 2.0 ** -60
    do[:where] = 0
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))
    want = R.backward(*dev, lens, do.to(DEV), h0.to(DEV), dhT.to(DEV))
    for name, x, y in zip(NAMES, got, want):
        assert torch.isfinite(x).all(), name
        if name in ("dv", "dbeta"):
            assert R.rel(x[where:], y[where:]) <= (R.BF16_REL if name == "dv" else 0) + R.F32_REL
    if fall < 87:
        assert R.rel(got[5], want[5]) <= R.F32_REL


@pytest.mark.parametrize("heads", [(2, 2), (1, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_rounded_once(d, heads):
    """dq, dk and dv are the exact gradients rounded to bf16, but for elements that the f32
    arithmetic moves over the middle of two neighbours.  An error of e times the tensor's
    root mean square r moves an element x, whose neighbours are at least 2^-8 |x| apart, with
    probability 2 e r / (2^-8 |x|) at most; over normally distributed x (1 / |x| cut off where that
    is 1) this is about 2^9 e (0.8 ln(1 / (2^9 e)) + 1), 4.6 % for e = F32_REL.  One operand of 11
    bits (e = 1.4e-4, the root mean square of its rounding) gives 22 %."""
    lens = [300, 70]
    case = _case(lens, *heads, d, seed=6)
    rows, do, h0, dhT = case
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    dev = [x.to(DEV) for x in rows]
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))
    want = R.backward(*dev, lens, do.to(DEV), h0.to(DEV), dhT.to(DEV))
    other = [float((x != y.to(torch.bfloat16)).double().mean()) for x, y in zip(got[:3], want)]
    assert max(other) <= 0.046, other


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what, power", [("do", -40), ("do", -90), ("q", -40), ("k", -40),
                                         ("do", 30), ("q", 30)])
def test_single_rows_far_from_the_others(what, power, d):
    """A few rows are 2^-90 to 2^30 times the others: every row of dq, dk and dv keeps its own
    accuracy.  (The factor 8: a row is a sum of up to four products that partly cancel.)"""
    lens = [100, 30]
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=7)
    x = {"q": rows[0], "k": rows[1], "do": do}[what]
    for r in (7, 50, 70, 120):
        x[r] = x[r] * 2.0 ** power
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))
    want = R.backward(*dev, lens, do.to(DEV), h0.to(DEV), dhT.to(DEV))
    for name, x, y in list(zip(NAMES, got, want))[:3]:
        assert _row_errors(x, y) <= R.BF16_REL + 8 * R.F32_REL, name


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("d", [64, 128])
def test_a_bad_output_gradient_stays_in_its_row_of_dq(value, d):
    """Row r of dq depends on row r of do alone (and on the forward pass)."""
    lens = [100, 30]
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=8)
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    want = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))[0]
    do[40, 1, 3] = value
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))[0]
    assert torch.equal(got[:40], want[:40]) and torch.equal(got[41:], want[41:])
    assert not torch.isfinite(got[40]).all() or value == 3e38


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift", [0.0, -1.0, -3.0, -5.0, -8.0, -30.0])
def test_gate_gradients_under_decays(shift, d):
    """dg_r has the decay e^g_r itself: its accuracy is relative to that, however strong it is."""
    lens = [150, 7]
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=9)
    rows[3] += shift
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))[3]
    want = R.backward(*dev, lens, do.to(DEV), h0.to(DEV), dhT.to(DEV))[3]
    print(R.rel(got, want))
    assert R.rel(got, want) <= R.F32_REL
    # against e^g as well: with gates of many sizes the norm alone shows the weakest
    size = rows[3].double().exp().to(DEV)
    assert R.rel(got.double() / size, want / size) <= R.F32_REL


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cut", [1, 15, 16, 31, 32, 33, 47, 63, 64, 100])
def test_one_strong_gate(cut, d):
    """One row forgets nearly everything: its dg is e^-25 of its neighbours'."""
    lens = [130]
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=10)
    rows[3][cut] = -25.0
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*dev, cu, do.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))[3]
    want = R.backward(*dev, lens, do.to(DEV), h0.to(DEV), dhT.to(DEV))[3]
    assert R.rel(got, want) <= R.F32_REL
    # a single sum of some 10^4 products, which may cancel to a tenth of their size
    assert R.rel(got[cut], want[cut]) <= 10 * R.F32_REL


@pytest.mark.parametrize("given", [("dq", "dk", "dv", "dg", "dbeta"), ("dk", "dg")])
def test_gradients_into_given_buffers(given):
    """Rows before, between and behind the sequences keep what the buffers hold."""
    lens, spare, d = [70, 0, 33], 5, 64
    rows, do, h0, dhT = _case(lens, 2, 4, d, seed=11)
    T = sum(lens) + 2 * spare
    dev = [torch.cat([x[:spare], x, x[:spare]]).to(DEV) for x in (*rows, do)]
    cu = torch.tensor([spare + x for x in R.offsets(lens)], dtype=torch.int32, device=DEV)
    shapes = {"dq": (T, 2, d), "dk": (T, 2, d), "dv": (T, 4, d), "dg": (T, 4), "dbeta": (T, 4)}
    bufs = {n: torch.full(shapes[n], 7.0, device=DEV,
                          dtype=torch.bfloat16 if n in NAMES[:3] else torch.float32) for n in given}
    got = gdn_chunk_backward(*dev[:5], cu, dev[5], h0=h0.to(DEV), dhT=dhT.to(DEV), **bufs)
    want = gdn_chunk_backward(*[x[spare:-spare].contiguous() for x in dev[:5]],
                              (cu - spare).contiguous(), dev[5][spare:-spare].contiguous(),
                              h0=h0.to(DEV), dhT=dhT.to(DEV))
    for name, x, y in zip(NAMES, got, want):
        if name != "dh0":
            assert torch.equal(x[spare:-spare], y), name
        if name in bufs:
            assert x is bufs[name]
            assert (x[:spare] == 7).all() and (x[-spare:] == 7).all()


def test_refused_buffers():
    rows, do, _, _ = _case([4], 1, 2, 64, seed=12)
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    good = gdn_chunk_backward(*dev, cu, do.to(DEV))
    for name, x in zip(NAMES[:5], good):
        with pytest.raises(ValueError, match=name):
            gdn_chunk_backward(*dev, cu, do.to(DEV), **{name: x[:3]})
        with pytest.raises(TypeError, match=name):
            gdn_chunk_backward(*dev, cu, do.to(DEV), **{name: x.double()})
        with pytest.raises(ValueError, match=name):
            gdn_chunk_backward(*dev, cu, do.to(DEV), **{name: x.cpu()})


@pytest.mark.parametrize("cut", [64, 100])
def test_a_sequence_in_two_parts(cut):
    """Last part first, its dh0 as the first part's dhT, the state between them as its h0."""
    lens, d = [230], 128
    rows, do, h0, dhT = _case(lens, 1, 2, d, seed=13)
    dev, do, h0, dhT = [x.to(DEV) for x in rows], do.to(DEV), h0.to(DEV), dhT.to(DEV)
    want = R.backward(*dev, lens, do, h0, dhT)
    between = R.forward(*[x[:cut] for x in dev], [cut], h0)[1].float()

    def part(rows, do, h0, dhT):
        cu = torch.tensor([0, do.shape[0]], dtype=torch.int32, device=DEV)
        return gdn_chunk_backward(*rows, cu, do, h0=h0, dhT=dhT)

    last = part([x[cut:] for x in dev], do[cut:], between, dhT)
    first = part([x[:cut] for x in dev], do[:cut], h0, last[5])
    for name, a, b, y in zip(NAMES, first, last, want):
        x = a if name == "dh0" else torch.cat([a, b])
        # (a part's h0 and dhT are rounded to f32 once more: 2^-24 each)
        assert R.rel(x, y) <= (R.BF16_REL if name in NAMES[:3] else 0) + R.F32_REL, name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gates, keys, what", [(0.0, 0, "values"), (-0.1, 0, "values"),
                                               (-3.0, -10, "values"), (0.0, 2, "queries")])
def test_rows_that_data_sets_apart(what, gates, keys, d):
    """Ordinary gates, but most rows have no value (the rows behind the last one that has live on
    what decays left of it) or hardly any query: a 16-row block holds rows 2^-35 and less of its
    largest, and each keeps its own accuracy.  (dbeta: the product of two vectors that may cancel
    to a hundredth.)"""
    lens = [128, 65]
    rows, do, _, _ = _case(lens, 2, 2, d, seed=14)
    rows[3] += gates
    rows[1] = rows[1] * 2.0 ** keys
    rows[4] = rows[4] * 2.0 ** (-2 * max(0, keys))
    if what == "values":
        rows[2][6:54] = rows[2][58:99] = rows[2][130:] = 0
        if keys == 0:
            rows[2][6:99] = 0
    else:
        rows[0][[62, 126, 127, 189, 190, 191, 192]] *= 2.0 ** -35
    dev = [x.to(DEV) for x in rows]
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*dev, cu, do.to(DEV))
    want = R.backward(*dev, lens, do.to(DEV))
    for name, x, y in zip(NAMES[:5], got, want):
        keep = y.double().flatten(1).norm(dim=1) > 1e-28  # (what f32 has digits for on the way there)
        tol = R.BF16_REL + 8 * R.F32_REL if name in NAMES[:3] else 100 * R.F32_REL
        if name != "dg":
            assert _row_errors(x[keep], y[keep]) <= tol, name

"""gdn_chunk_backward against the 64-bit token recurrence's gradients."""
import numpy as np
import pytest
import torch

import operator_reference as R
import oracle
from helpers import f64
from linear_attention_ssm_gdn_b200 import (GdnError, gdn_chunk_backward,
                                           gdn_chunk_backward_workspace_bytes)

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def _case(lens, Hk, Hv, d, seed, states=True):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rows = list(R.rows(gen, T, Hk, Hv, d))
    do = torch.randn(T, Hv, d, generator=gen).to(torch.bfloat16)
    h0 = torch.randn(N, Hv, d, d, generator=gen) * 0.1 if states else None
    dhT = torch.randn(N, Hv, d, d, generator=gen) * 0.1 if states else None
    return rows, do, h0, dhT


def _gpu(x):
    return None if x is None else x.to(DEV)


def _run(lens, rows, do, h0, dhT, scale=1.0, **kw):
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    return gdn_chunk_backward(*[x.to(DEV) for x in rows], cu, do.to(DEV), h0=_gpu(h0),
                              dhT=_gpu(dhT), scale=scale, **kw)


def _check(lens, got, rows, do, h0, dhT, scale=1.0, dg_size=0.0):
    """dg_size: the size of the terms whose sum dg is, where they cancel to far less."""
    want = R.backward(*[x.to(DEV) for x in rows], lens, do.to(DEV), _gpu(h0), _gpu(dhT), scale)
    for name, x, y in zip(NAMES, got, want):
        if x is None:
            assert name == "dh0" and h0 is None
            continue
        tol = (R.BF16_REL if x.dtype == torch.bfloat16 else 0) + R.F32_REL
        err = R.rel(x, y)
        print(f"{name} {err:.2e}", end=" ")
        if name == "dg":
            tol *= 1.0 + dg_size / float(y.norm())
        assert err <= tol, f"{name}: {err:.3e}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [63], [64], [65], [200], [1, 0, 63, 64, 65, 0, 130]])
def test_lengths(d, lens):
    case = _case(lens, 1, 2, d, seed=d + len(lens) + sum(lens))
    _check(lens, _run(lens, *case), *case)


@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (2, 6), (1, 4), (2, 10)])
def test_shared_key_heads(heads):
    lens = [100, 40]
    case = _case(lens, *heads, 64, seed=sum(heads))
    _check(lens, _run(lens, *case, scale=0.125), *case, scale=0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(2, 4), (1, 3), (1, 8), (1, 9)])
@pytest.mark.parametrize("lens", [[1], [33, 0, 2], [64, 65], [700, 1500]])
def test_value_heads_apart_and_in_turn(lens, heads, d):
    """Few chunks take a CTA per value head, summed in clusters of up to 8; many, or more
    value heads a key head, take them in turn."""
    case = _case(lens, *heads, d, seed=sum(lens) + sum(heads))
    got = _run(lens, *case, scale=0.5)
    _check(lens, got, *case, scale=0.5)
    again = _run(lens, *case, scale=0.5)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("d", [64, 128])
def test_without_states(d):
    lens = [130, 5]
    rows, do, _, _ = _case(lens, 2, 4, d, seed=5)
    got = _run(lens, rows, do, None, None)
    assert got[5] is None
    _check(lens, got, rows, do, None, None)


@pytest.mark.parametrize("h0", [None, "zeros"])
@pytest.mark.parametrize("lens", [[1], [1, 0, 1], [3, 70]])
def test_gate_of_a_zero_state_has_no_gradient(lens, h0):
    """The first row decays a state that is zero: its gate's gradient is 0 exactly."""
    rows, do, _, dhT = _case(lens, 1, 2, 64, seed=24)
    h0 = None if h0 is None else torch.zeros(len(lens), 2, 64, 64)
    dg = _run(lens, rows, do, h0, dhT)[3]
    first = [x for x, n in zip(R.offsets(lens), lens) if n]
    assert not dg[first].any()
    want = R.backward(*rows, lens, do, h0, dhT)[3]
    assert R.rel(dg, want) <= R.F32_REL


def test_only_one_of_the_state_arguments():
    lens = [70]
    rows, do, h0, dhT = _case(lens, 1, 2, 64, seed=6)
    _check(lens, _run(lens, rows, do, h0, None), rows, do, h0, None)
    dh0 = torch.empty(1, 2, 64, 64, device=DEV)
    got = _run(lens, rows, do, None, dhT, dh0=dh0)
    assert got[5] is dh0
    _check(lens, got[:5], rows, do, None, dhT)
    want = R.backward(*rows, lens, do, None, dhT)[5]
    assert R.rel(dh0, want) <= R.F32_REL


def test_state_gradient_in_place_and_alone():
    """dh0 over dhT, and no output gradient at all."""
    lens = [70, 0, 3]
    rows, do, h0, dhT = _case(lens, 1, 2, 128, seed=7)
    do = torch.zeros_like(do)
    buf = dhT.to(DEV)
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*[x.to(DEV) for x in rows], cu, do.to(DEV), h0=h0.to(DEV), dhT=buf,
                             dh0=buf)
    assert got[5] is buf and torch.equal(buf[1].cpu(), dhT[1])
    _check(lens, got, rows, do, h0, dhT)


@pytest.mark.parametrize("kind", ["weak", "strong", "cut", "forget", "mixed"])
def test_decays(kind):
    lens = [150]
    rows, do, h0, dhT = _case(lens, 1, 2, 64, seed=8)
    g = rows[3]
    if kind == "weak":
        g *= 1e-3
    elif kind == "strong":
        g -= 30.0
    elif kind == "cut":  # a very strong decay that later rows must not lose precision to
        g[10], g[100] = -3000.0, -1e5
    elif kind == "forget":
        g[20], g[64], g[127] = -float("inf"), -float("inf"), -float("inf")
    else:  # gates that rise within the documented bound
        g[::7] = 0.5
    size = 0.0
    if kind == "strong":
        # dg_r = <H', dH'> + sum over s >= r of the chunk of (q_s . dq_s - v_s . dv_s), every
        # term rounded to f32 relative to its own size.  Here the states forget all but the
        # last row, the terms are of size 1 and their sum, e^-30 and less, is below that
        # rounding: the error is F32_REL of the terms' absolute sum.
        q, k, v, g, b = rows
        dq, _, dv, _, _, _ = R.backward(q.repeat_interleave(2, 1), k.repeat_interleave(2, 1), v, g,
                                        b, lens, do, h0, dhT)
        terms = (q.double() * dq).abs().sum(-1) + (v.double() * dv).abs().sum(-1)
        terms[-1] += (R.forward(*rows, lens, h0)[1] * dhT).abs().sum((0, 2, 3))
        ends = [min(len(terms), 64 * (c + 1)) for c in range(-(-len(terms) // 64))]
        size = float(torch.cat([terms[64 * c:e].flip(0).cumsum(0) for c, e in enumerate(ends)]).norm())
    _check(lens, _run(lens, rows, do, h0, dhT), rows, do, h0, dhT, dg_size=size)


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_beta_at_its_ends(beta):
    lens = [90]
    rows, do, h0, dhT = _case(lens, 2, 2, 64, seed=9)
    rows[4].fill_(beta)
    _check(lens, _run(lens, rows, do, h0, dhT), rows, do, h0, dhT)
    rows[4][::3] = 1.0 - beta
    _check(lens, _run(lens, rows, do, h0, dhT), rows, do, h0, dhT)


def test_repeated_keys():
    """The same key in every other row: the chunk's triangular system at its fullest."""
    lens = [128]
    rows, do, h0, dhT = _case(lens, 1, 1, 64, seed=10)
    rows[1][::2] = rows[1][0].clone()
    _check(lens, _run(lens, rows, do, h0, dhT), rows, do, h0, dhT)


@pytest.mark.parametrize("size", [(1e-3, 1e4, 1e-4), (1.0, 1e-5, 1e6), (0.25, 1e3, 1.0)])
def test_sizes_of_values(size):
    """Small keys and queries, large and small values and output gradients."""
    lens = [100, 30]
    rows, do, h0, dhT = _case(lens, 1, 2, 128, seed=11)
    rows[0], rows[1], rows[2] = rows[0] * size[0], rows[1] * size[0], rows[2] * size[1]
    do = do * size[2]
    h0, dhT = h0 * size[1], dhT * size[2]
    _check(lens, _run(lens, rows, do, h0, dhT), rows, do, h0, dhT)


def test_rows_of_very_different_sizes():
    lens = [64, 64]
    rows, do, h0, dhT = _case(lens, 1, 1, 64, seed=12)
    for x in (rows[0], rows[1], rows[2], do):
        x[::5] = x[::5] * 2.0 ** -30
        x[3::7] = 0
    _check(lens, _run(lens, rows, do, h0, dhT), rows, do, h0, dhT)


def test_strided_views_and_rows_behind_the_last_sequence():
    lens, Hk, Hv, d, spare = [70, 9], 2, 4, 64, 6
    rows, do, h0, dhT = _case(lens, Hk, Hv, d, seed=13)
    T = sum(lens)
    q, k, v, g, beta = [torch.cat([x, torch.full((spare, *x.shape[1:]), float("nan"),
                                                 dtype=x.dtype)]) for x in rows]
    do_ = torch.cat([do, torch.full((spare, Hv, d), float("nan"), dtype=do.dtype)])
    qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).to(DEV)
    ba = torch.cat([g, beta], 1).to(DEV)
    s = qkv.split([Hk * d, Hk * d, Hv * d], 1)
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(s[0].unflatten(1, (Hk, d)), s[1].unflatten(1, (Hk, d)),
                             s[2].unflatten(1, (Hv, d)), ba[:, :Hv], ba[:, Hv:], cu,
                             do_.to(DEV), h0=h0.to(DEV), dhT=dhT.to(DEV))
    _check(lens, [x[:T] for x in got[:5]] + [got[5]], rows, do, h0, dhT)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [-0.7, 0.0, 1e-20, 3e4])
def test_scales(scale, d):
    lens = [70, 3, 130]
    case = _case(lens, 1, 2, d, seed=24)
    _check(lens, _run(lens, *case, scale=scale), *case, scale=scale)


def test_first_offset_above_zero():
    """Rows before the first sequence belong to none, as those behind the last."""
    lens, spare = [70, 0, 33], 9
    rows, do, h0, dhT = _case(lens, 2, 4, 128, seed=25)

    def padded(x):
        nan = torch.full((spare, *x.shape[1:]), float("nan"), dtype=x.dtype)
        return torch.cat([nan, x, nan]).to(DEV)

    cu = torch.tensor([spare + x for x in R.offsets(lens)], dtype=torch.int32, device=DEV)
    got = gdn_chunk_backward(*[padded(x) for x in rows], cu, padded(do), h0=h0.to(DEV),
                             dhT=dhT.to(DEV))
    _check(lens, [x[spare:-spare] for x in got[:5]] + [got[5]], rows, do, h0, dhT)


def test_nan_stays_in_its_sequence():
    lens = [70, 130, 64]
    rows, do, h0, dhT = _case(lens, 2, 4, 128, seed=26)
    want = _run(lens, rows, do, h0, dhT)
    rows[2][100, 1, 5] = float("nan")
    got = _run(lens, rows, do, h0, dhT)
    for x, y in zip(got[:5], want):
        assert torch.equal(x[:70], y[:70]) and torch.equal(x[200:], y[200:])
    assert torch.isnan(got[1][70:200]).any()


def test_negative_beta():
    lens = [300]
    case = _case(lens, 2, 2, 128, seed=27)
    case[0][4] = case[0][4] * 2 - 1
    _check(lens, _run(lens, *case), *case)


def test_many_chunks_and_the_same_bits_twice():
    lens = [2000, 333]
    case = _case(lens, 2, 4, 128, seed=14)
    a, b = _run(lens, *case), _run(lens, *case)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    _check(lens, a, *case)


@pytest.mark.parametrize("n", [32, 33, 64, 65])
def test_numbers_of_sequences(n):
    lens = [(7 * i * i) % 150 for i in range(n)]
    case = _case(lens, 1, 3, 64, seed=n)
    _check(lens, _run(lens, *case), *case)


def test_many_sequences():
    lens = [int(x) for x in np.random.default_rng(15).integers(0, 90, 60)]
    case = _case(lens, 1, 2, 64, seed=15)
    _check(lens, _run(lens, *case), *case)


def test_against_differences_of_the_oracle():
    """The gradient along a random direction against central differences in 64 bits."""
    lens = [75]
    rows, do, h0, dhT = _case(lens, 1, 2, 64, seed=16)
    got = _run(lens, rows, do, h0, dhT)
    base = [f64(x) for x in rows] + [f64(h0)]
    cu = np.array(R.offsets(lens))

    def loss(x):
        o, hT = oracle.gdn_token(*x[:5], cu, x[5])
        return float((o * f64(do)).sum() + (hT * f64(dhT)).sum())

    rng = np.random.default_rng(17)
    for i, gr in enumerate(got):
        gr = f64(gr.float())
        step = rng.standard_normal(base[i].shape)
        eps = 1e-5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + eps * step, base[i] - eps * step
        diff = (loss(up) - loss(down)) / (2 * eps)
        # the gradient's own error (bf16 or f32), times the direction's size
        tol = (R.BF16_REL if i < 3 else R.F32_REL) + 1e-7
        assert abs(diff - float((gr * step).sum())) <= \
            tol * np.linalg.norm(gr) * np.linalg.norm(step), NAMES[i]


def test_captured_and_replayed_on_new_inputs():
    lens, Hk, Hv, d = [70, 64], 1, 2, 64
    cases = [_case(lens, Hk, Hv, d, seed=s) for s in (18, 19)]
    rows, do, h0, dhT = cases[0]
    buf = [x.to(DEV) for x in rows] + [do.to(DEV), h0.to(DEV), dhT.to(DEV)]
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32, device=DEV)
    ws = torch.empty(gdn_chunk_backward_workspace_bytes(sum(lens), 2, Hk, Hv, d, d),
                     dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn_chunk_backward(*buf[:5], cu, buf[5], h0=buf[6], dhT=buf[7], workspace=ws)
    for rows, do, h0, dhT in cases[::-1]:
        for x, y in zip(buf, [*rows, do, h0, dhT]):
            x.copy_(y)
        ws.fill_(255)  # whatever the workspace holds on entry
        graph.replay()
        torch.cuda.synchronize()
        _check(lens, got, rows, do, h0, dhT)


def test_two_calls_at_once_on_two_streams():
    lens = [500]
    cases = [_case(lens, 1, 2, 128, seed=s) for s in (20, 21)]
    cu = torch.tensor([0, 500], dtype=torch.int32, device=DEV)
    dev = [[[x.to(DEV) for x in c[0]], c[1].to(DEV), c[2].to(DEV), c[3].to(DEV)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [gdn_chunk_backward(*x[0], cu, x[1], h0=x[2], dhT=x[3], stream=s)
           for x, s in zip(dev, streams)]
    torch.cuda.synchronize()
    for x, c in zip(got, cases):
        _check(lens, x, *c)


def test_no_rows():
    rows, do, h0, dhT = _case([0, 0], 1, 2, 64, seed=22)
    got = _run([0, 0], rows, do, h0, dhT)
    assert [tuple(x.shape) for x in got[:5]] == [(0, 1, 64)] * 2 + [(0, 2, 64)] + [(0, 2)] * 2
    assert torch.equal(got[5].cpu(), dhT)
    got = _run([0, 0], rows, do, h0, None)
    assert not got[5].any()


def test_refusals():
    lens = [4]
    rows, do, h0, dhT = _case(lens, 1, 2, 64, seed=23)
    with pytest.raises(ValueError, match="do"):
        _run(lens, rows, do[:3], h0, dhT)
    with pytest.raises(ValueError, match="dhT"):
        _run(lens, rows, do, h0, dhT[:, :1])
    with pytest.raises(TypeError, match="h0"):
        _run(lens, rows, do, h0.double(), dhT)
    with pytest.raises(GdnError, match="workspace"):
        _run(lens, rows, do, h0, dhT, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        _run(lens, rows, do, h0.transpose(2, 3), dhT)

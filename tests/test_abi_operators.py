"""Host-only checks of gdn_decode, gdn_state_tables and gdn_chunk_backward: their
guards refuse bad arguments with the named error before anything is launched,
empty calls succeed, and the binding refuses tensors it cannot pass on."""
import types

import pytest
import torch

import linear_attention_ssm_gdn_b200 as gdn
from linear_attention_ssm_gdn_b200 import _lib
from linear_attention_ssm_gdn_b200.build import build
from linear_attention_ssm_gdn_b200.gdn import _switched

P = 0x10000  # fake, aligned device address: never reached behind a refusing guard
NULL = None


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def _err(lib):
    return lib.gdn_last_error().decode()


def _decode(lib, **kw):
    a = {**dict(table=P, q=P, k=P, qks=2048, v=P, vs=6144, g=P, beta=P, gbs=48, cu=P, o=P,
                batch=64, rows=64, Hk=16, Hv=48, dk=128, dv=128), **kw}
    return lib.gdn_decode(a["table"], a["q"], a["k"], a["qks"], a["v"], a["vs"], a["g"],
                          a["beta"], a["gbs"], a["cu"], a["o"], a["batch"], a["rows"], a["Hk"],
                          a["Hv"], a["dk"], a["dv"], 1.0, None)


def test_decode_guards(lib):
    for x in ("table", "q", "k", "v", "g", "beta", "o"):
        assert _decode(lib, **{x: NULL}) == _lib.GDN_ERR_NULL, x
    for kw in (dict(Hk=0), dict(Hk=5), dict(dk=64), dict(dk=96, dv=96), dict(batch=-1),
               dict(rows=-1), dict(cu=NULL, rows=65), dict(batch=1 << 24, rows=1 << 24)):
        assert _decode(lib, **kw) == _lib.GDN_ERR_SHAPE, kw
    for kw in (dict(qks=2040), dict(vs=6136), dict(gbs=47)):
        assert _decode(lib, **kw) == _lib.GDN_ERR_STRIDE, kw
    for kw in (dict(q=P + 8), dict(k=P + 2), dict(v=P + 8), dict(o=P + 8), dict(qks=2052),
               dict(vs=6148)):
        assert _decode(lib, **kw) == _lib.GDN_ERR_ALIGN, kw
    assert "gdn_decode" in _err(lib)
    assert _decode(lib, rows=0, q=NULL, k=NULL, v=NULL, g=NULL, beta=NULL, o=NULL) == _lib.GDN_OK
    assert _decode(lib, batch=0, table=NULL) == _lib.GDN_OK and _err(lib) == ""


def _tables(lib, **kw):
    a = {**dict(lens=P, slots=P, n=4, pool=P, sf=4096, ns=8, cu=P, table=P, rs=P, rl=P, rcap=100,
                cc=P, cs=P, ccap=10, flag=P), **kw}
    return lib.gdn_state_tables(a["lens"], a["slots"], a["n"], a["pool"], a["sf"], a["ns"],
                                a["cu"], a["table"], a["rs"], a["rl"], a["rcap"], a["cc"],
                                a["cs"], a["ccap"], a["flag"], None)


def test_state_tables_guards(lib):
    for kw in (dict(lens=NULL), dict(pool=NULL), dict(table=NULL), dict(slots=NULL)):
        assert _tables(lib, **kw) == _lib.GDN_ERR_NULL, kw
    for kw in (dict(n=-1), dict(ns=-1), dict(sf=-4), dict(rcap=-1), dict(ccap=-1),
               dict(rcap=0x7FFFFFFF), dict(ccap=0x7FFFFFFF)):
        assert _tables(lib, **kw) == _lib.GDN_ERR_SHAPE, kw
    for kw in (dict(pool=P + 4), dict(sf=4098)):
        assert _tables(lib, **kw) == _lib.GDN_ERR_ALIGN, kw
    assert "gdn_state_tables" in _err(lib)


def _backward(lib, **kw):
    a = {**dict(q=P, k=P, qks=2048, v=P, vs=6144, g=P, beta=P, gbs=48, cu=P, N=1, T=4576,
                h0=NULL, do=P, dhT=NULL, dq=P, dk=P, dv=P, dg=P, db=P, dh0=NULL, Hk=16, Hv=48,
                d_k=128, d_v=128, ws=P, wsb=1 << 40), **kw}
    return lib.gdn_chunk_backward(a["q"], a["k"], a["qks"], a["v"], a["vs"], a["g"], a["beta"],
                                  a["gbs"], a["cu"], a["N"], a["T"], a["h0"], a["do"], a["dhT"],
                                  a["dq"], a["dk"], a["dv"], a["dg"], a["db"], a["dh0"], a["Hk"],
                                  a["Hv"], a["d_k"], a["d_v"], 1.0, a["ws"], a["wsb"], None)


def test_chunk_backward_guards(lib):
    for x in ("q", "k", "v", "g", "beta", "cu", "do", "dq", "dk", "dv", "dg", "db"):
        assert _backward(lib, **{x: NULL}) == _lib.GDN_ERR_NULL, x
    for kw in (dict(Hk=0), dict(Hk=5), dict(d_k=64), dict(d_k=32, d_v=32), dict(N=0),
               dict(T=-1), dict(Hk=1, Hv=65536, vs=65536 * 128, gbs=65536), dict(N=1 << 28)):
        assert _backward(lib, **kw) == _lib.GDN_ERR_SHAPE, kw
    for kw in (dict(qks=2040), dict(vs=6136), dict(gbs=47)):
        assert _backward(lib, **kw) == _lib.GDN_ERR_STRIDE, kw
    for kw in (dict(q=P + 8), dict(v=P + 8), dict(do=P + 8), dict(h0=P + 4), dict(dhT=P + 4),
               dict(dq=P + 2), dict(dk=P + 2), dict(dv=P + 2), dict(dh0=P + 4), dict(qks=2052),
               dict(vs=6148)):
        assert _backward(lib, **kw) == _lib.GDN_ERR_ALIGN, kw
    need = lib.gdn_chunk_backward_workspace_bytes(4576, 1, 16, 48, 128, 128)
    for kw in (dict(ws=NULL), dict(wsb=need - 1), dict(ws=P + 128)):
        assert _backward(lib, **kw) == _lib.GDN_ERR_WORKSPACE, kw
    assert "gdn_chunk_backward" in _err(lib)
    # nothing to do: no rows, and no dh0 wanted
    assert _backward(lib, T=0, ws=NULL, wsb=0, q=NULL, dq=NULL) == _lib.GDN_OK
    assert _err(lib) == ""


def test_chunk_backward_workspace_grows_past_32_bits(lib):
    f = lib.gdn_chunk_backward_workspace_bytes
    assert f(0, 1, 16, 48, 128, 128) == 0 and f(64, 0, 16, 48, 128, 128) == 0
    assert f(1, 1, 1, 1, 64, 64) > 0
    # at least the chunks' entry states and their gradients
    assert f(1 << 20, 1, 16, 48, 128, 128) >= (1 << 14) * 48 * 128 * 128 * 8


def test_binding_refuses_cpu_tensors_and_wrong_types():
    z = torch.zeros
    q, v = z(3, 2, 64, dtype=torch.bfloat16), z(3, 2, 64, dtype=torch.bfloat16)
    g = z(3, 2)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_decode(z(3, dtype=torch.int64), q, q, v, g, g)
    with pytest.raises(TypeError, match="h_table"):
        gdn.gdn_decode(z(3, dtype=torch.int32), q, q, v, g, g)
    with pytest.raises(TypeError, match="lens"):
        gdn.gdn_state_tables(z(3), total_rows=1)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_chunk_backward(q, q, v, g, g, z(2, dtype=torch.int32), v)
    with pytest.raises(TypeError, match="q"):
        gdn.gdn_chunk_backward(q.float(), q, v, g, g, z(2, dtype=torch.int32), v)


def test_a_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        with _switched(torch.device("cuda", 0), stream):
            pass

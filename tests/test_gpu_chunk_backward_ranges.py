"""gdn_chunk_backward where rows, decays or values leave the ordinary range."""
import pytest
import torch

import operator_reference as R
from linear_attention_ssm_gdn_b200 import (debug_device_errors, gdn_chunk_backward,
                                           gdn_chunk_backward_workspace_bytes)
from test_gpu_chunk_backward import DEV, _case

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

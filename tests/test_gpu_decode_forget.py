"""gdn_decode on state slots that hold anything: g = -inf forgets it."""
import pytest
import torch

import operator_reference as R
from linear_attention_ssm_gdn_b200 import gdn_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("held", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("gate", [-float("inf"), -1000.0])
def test_a_forgotten_state_may_hold_anything(held, gate, d):
    """A recycled slot: the first row forgets it, the others (and the other sequence) go on."""
    gen = torch.Generator().manual_seed(d)
    lens = [3, 2]
    rows = [x.to(DEV) for x in R.rows(gen, 5, 1, 2, d)]
    pool = torch.randn(2, 2, d, d, generator=gen).to(DEV)
    rows[3][0] = gate
    zero = pool.clone()
    zero[0] = 0
    want, states = R.forward(*rows, lens, zero)
    pool[0] = held
    table = torch.tensor([x.data_ptr() for x in pool], dtype=torch.int64, device=DEV)
    cu = torch.tensor([0, 3, 5], dtype=torch.int32, device=DEV)
    o = gdn_decode(table, *rows, cu_seqlens=cu)
    assert R.rel(o, want) <= R.BF16_REL + R.F32_REL
    assert R.rel(pool, states) <= R.F32_REL

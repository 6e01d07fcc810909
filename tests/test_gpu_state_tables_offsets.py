"""gdn_state_tables where not every table is made."""
import json
import tempfile

import numpy as np
import pytest
import torch
from torch.profiler import ProfilerActivity, profile

from linear_attention_ssm_gdn_b200 import gdn_state_tables

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _lens(n, seed):
    return [int(x) for x in np.random.default_rng(seed).choice([0, 1, 1, 63, 64, 65, 300], n)]


@pytest.mark.parametrize("n", [1, 64, 1024, 1025, 2048, 5000, 200_000])
def test_offsets_alone(n):
    """No map, so no position that asks for a CTA: the tiles of lengths do."""
    lens = _lens(n, n + 1)
    out = {"cu_seqlens": torch.full((n + 1,), -9, dtype=torch.int32, device=DEV),
           "cu_chunks": torch.full((n + 1,), -9, dtype=torch.int32, device=DEV)}
    gdn_state_tables(_int(lens), out=out)
    x = torch.tensor(lens)
    for name, y in (("cu_seqlens", x), ("cu_chunks", (x + 63) // 64)):
        assert out[name][0] == 0 and torch.equal(out[name][1:].cpu().long(), y.cumsum(0)), name


@pytest.mark.parametrize("n", [3, 1025, 5000])
def test_launch_is_as_large_as_what_is_made(n):
    """Offsets alone take a CTA for every 1024 lengths, not one for every 2048 rows that there
    might be."""

    lens = _int(_lens(n, n))
    out = {"cu_seqlens": torch.empty(n + 1, dtype=torch.int32, device=DEV)}
    gdn_state_tables(lens, out=out)
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        gdn_state_tables(lens, out=out)
        torch.cuda.synchronize()
    with tempfile.NamedTemporaryFile(suffix=".json") as f:
        p.export_chrome_trace(f.name)
        with open(f.name) as trace:
            events = json.load(trace)["traceEvents"]
    grids = [e["args"]["grid"] for e in events if "tables_kernel" in e.get("name", "")]
    if not grids:
        pytest.skip("the profiler records no kernels here")
    assert grids == [[-(-n // 1024), 1, 1]]

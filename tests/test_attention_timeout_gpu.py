"""The attention kernels' bounded waits, in the starved test build (GPU): no copy is
issued, every wait on one runs out, and each kernel must stop, write NaN for every row
it could not finish (and what no wait stands before as always), and free its tensor
memory: the same call on the normal library right after must be right."""
import pytest
import torch

from attention_cases import Problem
from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    normal = B.load(build_mod.build())
    starved = B.load(build_mod.build_starved())
    saved = B._lib
    yield normal, starved
    B._lib = saved


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("kind", ["decode", "runs", "prefix"])
def test_stops_and_writes_nan(libs, kind, dtype):
    normal, starved = libs
    flags = B.MSA_LAUNCH_QUERY_RUNS if kind == "runs" else 0
    if kind == "prefix":
        p = Problem(31, lens=(40, 300, 7, 0), prefixes=(700,), groups=(0, 3), ids=None, dtype=dtype)
        seen = [0, 1, 2]
    else:
        p = Problem(32, lens=(0, 5, 700, 129), seq_of=(0, 1, 1, 1), dtype=dtype)
        seen = [1, 2, 3]
    B._lib = starved
    d = p.device()
    d.run(flags)
    torch.cuda.synchronize()
    rest = [t for t in range(p.T) if t not in seen]
    assert torch.isnan(d.out[seen]).all() and torch.isnan(d.lse[seen]).all()
    assert (d.out[rest] == 0).all() and torch.isneginf(d.lse[rest]).all()
    B._lib = normal
    p.device().run(flags).check()

"""The adapters' bounded waits, in the starved test build (GPU): no copy is issued, every wait on
one runs out, and the kernel must stop, leave NaN in the rows of every request with an adapter (the
others' as they were) and free its tensor memory: the same call on the normal library right after
must be right."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod
from test_adapter_gpu import Case, mixed, runs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    normal = B.load(build_mod.build())
    starved = B.load(build_mod.build_starved())
    saved = B._lib
    yield normal, starved
    B._lib = saved


@pytest.mark.parametrize("order", [mixed, runs], ids=["mixed", "runs"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_stops_and_writes_nan(libs, order, fp8):
    normal, starved = libs
    c = Case(order(1300, 3), k=1000, adapters=3, rank=64, fp8=fp8)      # tiles of 128 tokens
    B._lib = starved
    c.run()
    torch.cuda.synchronize()
    on = (c.ids >= 0) & (c.ids < 3)
    assert c.out[on].isnan().all()
    assert torch.equal(c.out[~on].view(torch.int16), c.rows[~on].view(torch.int16))
    B._lib = normal
    c.run().check()


@pytest.mark.parametrize("rank,k", [(64, 1000), (24, 2100), (96, 640)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_gives_up_while_copies_land(libs, rank, k, fp8):
    """Rows that are given up with copies in flight are NaN, not what the copies bring: every row,
    over many calls.  (Nothing else uses the memory that the copies land in.)"""
    normal, _ = libs
    given_up = B.load(build_mod.build_given_up())
    c = Case(runs(2048, 3), k=k, adapters=3, rank=rank, fp8=fp8)
    on = (c.ids >= 0) & (c.ids < 3)
    B._lib = given_up
    try:
        for _ in range(3):
            c.out.zero_()
            c.run()
            torch.cuda.synchronize()
            assert c.out[on].isnan().all()
            assert torch.equal(c.out[~on].view(torch.int16), c.rows[~on].view(torch.int16))
    finally:
        B._lib = normal
    c.run().check()

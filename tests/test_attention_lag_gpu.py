"""The attention kernels with one softmax warp behind the others (GPU): in the lagging test
build a warp sleeps for 20 us after each exchange through shared memory, far longer than
the others take to their next one.  Results must be those of the definition, and the same
bits from call to call."""
import pytest
import torch

from attention_cases import Problem
from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lagging():
    saved = B._lib
    B._lib = B.load(build_mod.build_lagging())
    yield
    B._lib = saved


# queries large enough that the maximum of a list moves from chunk to chunk
@pytest.mark.parametrize("kw", [
    dict(lens=(4000, 3000, 700, 90), topk=16, heads=(64, 8)),
    dict(lens=(4000, 3000, 700, 90), topk=16, heads=(32, 2), dtype="bf16"),
    dict(lens=(4000, 3000, 700, 90), topk=32, heads=(16, 8), dtype="bf16", head_dim=64),
    dict(lens=[300 * i for i in range(40)], ids=None, heads=(16, 1)),
], ids=["e4m3-8", "bf16-16", "bf16-8", "dense-e4m3-16"])
def test_single_queries(kw):
    p = Problem(71, q_gain=6.0, **kw)
    ref = p.reference()
    first = p.device().run().check(ref)
    for _ in range(3):
        d = p.device().run().check(ref)
        assert torch.equal(d.out, first.out) and torch.equal(d.lse, first.lse)


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("kind", ["runs", "prefix"])
def test_tiles_of_queries(kind, dtype):
    if kind == "runs":
        p = Problem(72, lens=list(range(1500, 1570)), seq_of=[0] * 70, topk=8, heads=(16, 2), q_gain=6.0, dtype=dtype)
    else:
        p = Problem(73, lens=(40, 300, 7, 0) * 5, prefixes=(3000, 500), groups=(0, 11, 20), ids=None, heads=(16, 2),
                    q_gain=6.0, dtype=dtype)
    flags = B.MSA_LAUNCH_QUERY_RUNS if kind == "runs" else 0
    ref = p.reference()
    first = p.device().run(flags).check(ref)
    d = p.device().run(flags).check(ref)
    assert torch.equal(d.out, first.out) and torch.equal(d.lse, first.lse)

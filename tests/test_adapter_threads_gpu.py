"""Adapter calls of several host threads at once (GPU), each on a stream of its own with tensors and a
workspace of its own: calls of other ranks and other numbers of adapters, whose kernels take other
amounts of shared memory, none of which may be refused."""
import threading

import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod
from test_adapter_gpu import Case, mixed, runs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def at_once(cases, calls):
    errors = []
    start = threading.Barrier(len(cases))

    def work(case, stream):
        try:
            start.wait()
            for _ in range(calls):
                case.run(stream=stream)
        except Exception as e:       # shown below
            errors.append(e)

    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    for c in cases:
        c.check()


@pytest.mark.parametrize("ranks", [(16, 96), (24, 40, 64, 96)], ids=str)
def test_wide_tiles_of_other_ranks(ranks):
    """Rings of 111 to 217 KB, up-projections of one kernel with other widths and of several."""
    at_once([Case(runs(2600, 3), k=1000, adapters=3, rank=r, fp8=r % 32 == 0, seed=r) for r in ranks], 400)


def test_sorts_of_other_tables():
    at_once([Case(mixed(200, n), k=64, ends=(64,), rank=8, adapters=n, seed=n) for n in (12400, 13000, 16384)], 600)

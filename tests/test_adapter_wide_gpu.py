"""The adapters' tiles of 128 tokens (GPU), at sizes that take them, and the up-projection's stream of
columns: a CTA's share of up to 1,024 columns in stages of 128, two ahead, of every rank's layout in
shared memory.  Tolerances as for the other tests of the adapters (Case.check)."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import build as build_mod
from paged_kv_cache_msa_gb300 import binding as B
from test_adapter_gpu import PACKED, SMALL, Case, mixed, runs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def takes_wide_tiles(t, k, slices, rank, adapters):
    """The rule of msa_adapter_forward: T^2 * rows of down * K from 5e11 on, and 56 tokens for each
    of up to 16 adapters."""
    return t * t * slices * rank * k >= 5e11 and t >= 56 * min(adapters, 16) and t > 17


def columns_of_a_cta(t, k, ends, rank):
    """The up-projection's chunk of columns, as msa_adapter_forward chooses it."""
    units, groups = -(-k // 64), -(-t // 128)
    splits = max(1, min(152 // groups, min(units // 4, 8)))
    chunk = 128
    while chunk < 1024:
        items = groups * -(-ends[-1] // chunk)
        if items <= 2 * 152 or (items <= 8 * 152 and chunk >= 4 * splits * rank):
            break
        chunk *= 2
    return chunk


def wide(ids, k, ends, rank, adapters, chunk=None, **kw):
    t = len(ids)
    assert takes_wide_tiles(t, k, len(ends), rank, adapters)
    assert chunk is None or columns_of_a_cta(t, k, ends, rank) == chunk
    return Case(ids, k=k, ends=ends, rank=rank, adapters=adapters, **kw)


INSIDE = (640, 1984, 2112, 5000)         # chunks begin inside a slice, the last ends inside a stage
ONE = (8192,)


@pytest.mark.parametrize("ends,t,k,chunks", [
    (PACKED, 2048, 1024, {16: 256, 24: 512, 32: 512, 40: 1024, 64: 1024, 96: 1024}),
    (INSIDE, 3001, 1024, {16: 256, 24: 512, 32: 512, 40: 512, 48: 512, 64: 512, 80: 512, 96: 512, 128: 512}),
    (ONE, 5003, 2500, {8: 512, 16: 512, 24: 512, 56: 1024, 64: 1024, 104: 1024, 128: 1024}),
], ids=["packed", "inside", "one"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_columns_in_many_stages(ends, t, k, chunks, fp8):
    """A stage is filled again while the one after it is used: 2 to 8 stages a CTA."""
    for rank, chunk in chunks.items():
        if not takes_wide_tiles(t, k, len(ends), rank, 5):
            continue
        wide(runs(t, 5), k, ends, rank, 5, chunk, fp8=fp8, pad=rank % 3, seed=rank).run().check()


def test_chunks_are_covered():
    """Of the ranks above, every chunk from 256 columns on, in both layouts of a piece of up."""
    seen = {(columns_of_a_cta(2048, 1024, PACKED, r), -(-r // 16)) for r in (16, 24, 32, 40, 64, 96)}
    seen |= {(columns_of_a_cta(3001, 1024, INSIDE, r), -(-r // 16)) for r in (16, 24, 32, 40, 48, 64, 80, 96, 128)}
    assert {c for c, _ in seen} >= {512, 1024}


@pytest.mark.parametrize("seed", range(8))
def test_tiles_of_several_adapters_over_the_packed_row(seed):
    """Batches of wide rows in runs of any length: tiles that are full, short, or of tokens without an adapter."""
    gen = torch.Generator().manual_seed(seed)
    rank, t = (24, 32, 64, 96)[seed % 4], 2048 + 37 * seed
    edges = torch.cat([torch.tensor([0, t]), torch.randint(1, t, (4 + 5 * seed,), generator=gen)]).sort().values
    ids = []
    for i, n in enumerate(edges.diff().tolist()):
        ids += [i % 7 - 1] * n
    wide(ids, 1536, PACKED, rank, 6, seed=seed, fp8=seed % 2 == 1).run().check()


@pytest.mark.parametrize("t,k", [(2100, 2049), (2500, 1001), (6000, 200), (10200, 65), (10300, 64), (13000, 40), (900, 9600),
                                 (720, 15500)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_hidden_sizes(t, k, fp8):
    """K blocks that are whole, short, and one alone."""
    wide(runs(t, 4) if t % 2 else mixed(t, 4), k, SMALL, 40, 4, fp8=fp8, pad=1, seed=k).run().check()


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 48, 56, 64, 72, 80, 96, 100 // 8 * 8])
@pytest.mark.parametrize("order", [mixed, runs], ids=["mixed", "runs"])
def test_ranks(rank, order):
    t = int((5e11 / (5 * rank * 1000)) ** 0.5) + 2
    wide(order(t, 3), 1000, SMALL, rank, 3, fp8=rank % 16 == 8, seed=rank).run().check()


@pytest.mark.parametrize("ends", [(8,), (56,), (72,), (64, 128, 192, 256, 320, 384, 448, 456), (1000,), (4096, 4104)], ids=str)
@pytest.mark.parametrize("t", [2900, 3333])
def test_widths(ends, t):
    rank = 64 if len(ends) > 4 else 128
    wide(mixed(t, 4), 1000, ends, rank, 4, fp8=True, pad=2, seed=t).run().check()


@pytest.mark.parametrize("rank", [24, 64, 96])
def test_in_place_and_again_over_the_packed_row(rank):
    c = wide(runs(2200, 4), 1024, PACKED, rank, 4).run().check()
    rows, want = c.rows.clone(), c.out.clone()
    c.ws.fill_(0x7F)
    c.out.zero_()
    c.run()
    assert torch.equal(c.out.view(torch.int16), want.view(torch.int16))
    c.run(out=c.rows)
    assert torch.equal(c.rows.view(torch.int16), want.view(torch.int16))
    c.check(out=c.rows, rows=rows)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_their_own(bad):
    """Over many stages of columns."""
    for what in ("down", "up", "alpha", "hidden", "hidden_scales", "rows"):
        c = wide(runs(2200, 4), 1024, PACKED, 40, 4).run()
        clean = c.out.clone()
        if what in ("down", "up", "alpha"):
            getattr(c, what)[2] = bad
            mine = c.ids == 2
        else:
            getattr(c, what)[1000] = bad
            mine = torch.arange(c.n, device="cuda") == 1000
        c.run()
        assert torch.equal(c.out[~mine].view(torch.int16), clean[~mine].view(torch.int16)), what
        touched = mine & (c.ids >= 0) & (c.ids < 4) if what != "rows" else mine
        assert not c.out[touched].isfinite().any(), what

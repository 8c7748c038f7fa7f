"""The attention operators against their definition in 64 bits (GPU)."""
import pytest
import torch

from attention_cases import Problem
from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

RUNS = B.MSA_LAUNCH_QUERY_RUNS
PDL = B.MSA_LAUNCH_PDL


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


LENS = (1, 2, 63, 64, 65, 127, 128, 129, 0, 255, 256, 257, 511, 640, 1000, 2049, -3)

SPARSE = [
    dict(),                                                       # fp8, 8/2 heads of 128
    dict(dtype="bf16"),
    dict(head_dim=64, heads=(8, 2)),
    dict(head_dim=64, heads=(8, 2), dtype="bf16"),
    dict(heads=(64, 8), topk=16),
    dict(heads=(32, 2), topk=16),                                 # 16 heads on each
    dict(heads=(32, 2), dtype="bf16"),
    dict(heads=(3, 3)),                                           # one on each
    dict(heads=(10, 2)),                                          # five
    dict(heads=(9, 1), dtype="bf16"),
    dict(heads=(40, 2)),                                          # twenty
    dict(heads=(17, 1), head_dim=64),
    dict(page=8), dict(page=16), dict(page=32, dtype="bf16"), dict(page=128), dict(page=256),
    dict(page=48), dict(page=1), dict(page=7), dict(page=96, dtype="bf16"), dict(page=4, head_dim=64),
    dict(block=64, topk=8), dict(block=32, topk=64, dtype="bf16"), dict(block=96), dict(block=256),
    dict(block=160), dict(block=1024, topk=2),
    dict(topk=1), dict(topk=64), dict(topk=5, ids="messy"), dict(topk=33, ids="messy", dtype="bf16"),
    dict(layout="padded"), dict(layout="padded", dtype="bf16"), dict(layout="nhd"), dict(layout="nhd", dtype="bf16"),
    dict(layout="heads_outer"), dict(layout="odd"), dict(layout="odd", dtype="bf16"),
    dict(layout="interleaved"), dict(layout="interleaved", dtype="bf16", head_dim=64),
    dict(per_head=True), dict(per_head=True, heads=(64, 8)),
    dict(dtype="e4m3", v_dtype="bf16"), dict(dtype="bf16", v_dtype="e4m3"),
    dict(bad_pages=12), dict(bad_pages=12, dtype="bf16", head_dim=64),
    dict(scale=1.0), dict(scale=1e-3), dict(q_gain=40.0), dict(q_gain=1e-4),
]


def _name(d):
    return "-".join(f"{k}={v}" for k, v in d.items()).replace(" ", "") or "default"


@pytest.mark.parametrize("kw", SPARSE, ids=_name)
def test_sparse_decode(kw):
    p = Problem(11, **{**dict(lens=LENS), **kw})
    p.device().run().check()


@pytest.mark.parametrize("lens", [(1,), (0,), (128,), (9000,), (0, 0, 0), (5,) * 130, (700, 0, 3)], ids=str)
@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_sparse_decode_batches(lens, dtype):
    Problem(12, lens=lens, dtype=dtype, topk=16).device().run().check()


@pytest.mark.parametrize("kw", [
    dict(heads=(64, 8), topk=16), dict(heads=(32, 2), topk=16, dtype="bf16"), dict(heads=(8, 2), head_dim=64, topk=9),
    dict(heads=(16, 8), ids=None),                 # dense, no prefix
    dict(heads=(32, 2), ids=None, dtype="bf16"),
], ids=_name)
def test_long_and_short_histories_side_by_side(kw):
    """Histories of one tile between histories of many, on every SM: the pipeline's groups
    get ahead of and behind one another."""
    lens = [(1, 5000, 100, 130, 7000, 3, 3000 + 7 * i, 250)[i % 8] for i in range(60)]
    Problem(16, lens=lens, **kw).device().run().check()


def _runs(*spans):
    """Consecutive queries of sequences: (first visible length, count) each."""
    lens, seq = [], []
    for s, (a, n) in enumerate(spans):
        lens += list(range(a, a + n))
        seq += [s] * n
    return dict(lens=lens, seq_of=seq)


PREFILL = [
    dict(**_runs((1, 150))),
    dict(**_runs((1, 150)), dtype="bf16"),
    dict(**_runs((900, 70)), heads=(64, 8), topk=16),
    dict(**_runs((900, 70)), heads=(32, 2), dtype="bf16"),
    dict(**_runs((500, 40)), head_dim=64),
    dict(**_runs((500, 40)), head_dim=64, dtype="bf16"),
    dict(**_runs((1, 20), (300, 3), (1000, 1), (257, 45))),             # tiles of several sequences
    dict(**_runs((1, 5), (200, 5), (1, 5), (400, 9)), heads=(4, 4)),
    dict(**_runs((800, 33)), heads=(2, 1)),
    dict(**_runs((800, 33)), heads=(10, 2)),
    dict(**_runs((800, 33)), heads=(40, 2)),
    dict(**_runs((800, 9)), heads=(128, 1), head_dim=64),
    dict(**_runs((1500, 60)), block=256),
    dict(**_runs((1500, 30)), block=1024, topk=2),
    dict(**_runs((700, 30)), block=64, topk=8),
    dict(**_runs((700, 30)), page=16), dict(**_runs((700, 30)), page=128, dtype="bf16"),
    dict(**_runs((700, 30)), page=48), dict(**_runs((700, 30)), page=7),
    dict(**_runs((700, 40)), ids="messy", topk=6),
    dict(**_runs((2000, 30)), topk=64, heads=(4, 4)),
    dict(**_runs((700, 40)), bad_pages=6),
    dict(**_runs((700, 40)), layout="nhd"), dict(**_runs((700, 40)), layout="odd"),
    dict(**_runs((700, 40)), layout="padded", per_head=True),
    dict(**_runs((700, 40)), dtype="e4m3", v_dtype="bf16"),
    dict(**_runs((700, 40)), scale=1.0), dict(**_runs((700, 40)), q_gain=40.0),
]


@pytest.mark.parametrize("ids", ["random", "near"])
@pytest.mark.parametrize("kw", PREFILL, ids=lambda d: _name({k: v for k, v in d.items() if k not in ("lens", "seq_of")})
                         + f"-{len(d['lens'])}")
def test_sparse_query_runs(kw, ids):
    p = Problem(13, **{**dict(ids=ids), **kw})
    p.device().run(RUNS).check()


def test_query_runs_on_unrelated_queries():
    """The flag is a hint: a decode batch is answered the same way."""
    p = Problem(14, lens=LENS, topk=8, heads=(64, 8))
    p.device().run(RUNS).check()


PREFIX = [
    dict(lens=(5, 0, 130, 64, 1), prefixes=(300,), groups=(0, 5)),
    dict(lens=(5, 0, 130, 64, 1), prefixes=(300,), groups=(0, 5), dtype="bf16"),
    dict(lens=(0,) * 9, prefixes=(129,), groups=(0, 9)),
    dict(lens=(7,) * 40, prefixes=(1000, 0, 1, 127), groups=(0, 20, 25, 26, 40), heads=(64, 8)),
    dict(lens=(200,) * 40, prefixes=(1000, 333), groups=(3, 20, 31), heads=(32, 2), dtype="bf16"),  # some in no group
    dict(lens=(50,) * 20, prefixes=(500, 400, 300), groups=(0, 12, 5, 20)),                         # not monotone
    dict(lens=(50,) * 20, prefixes=(500, 400), groups=(-4, 12, 99)),                                # past the batch
    dict(lens=(9, 300) * 10, prefixes=(640,), groups=(0, 20), head_dim=64),
    dict(lens=(9, 300) * 10, prefixes=(640,), groups=(0, 20), head_dim=64, dtype="bf16"),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), page=16),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), page=128),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), page=24),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), page=3),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), layout="nhd"),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), layout="odd", dtype="bf16"),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), layout="interleaved", per_head=True),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), heads=(10, 2)),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), heads=(40, 2)),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), heads=(128, 1), head_dim=64),
    dict(lens=(40,) * 140, prefixes=(700,), groups=(0, 140), heads=(2, 2)),
    dict(lens=(300, 40) * 6, prefixes=(700,), groups=(0, 12), bad_pages=8),
    dict(lens=(300, 40) * 6, prefixes=(700,), groups=(0, 12), bad_pages=8, dtype="bf16"),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), dtype="bf16", v_dtype="e4m3"),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), scale=1.0),
    dict(lens=(40,) * 6, prefixes=(700,), groups=(0, 6), q_gain=40.0),
    dict(lens=LENS),                                                     # no prefix: dense paged attention
    dict(lens=LENS, dtype="bf16", heads=(32, 2)),
    dict(lens=(9000,)), dict(lens=(1,)), dict(lens=(0, 0)),
    dict(lens=(0, 0), prefixes=(0,), groups=(0, 2)),
]


@pytest.mark.parametrize("kw", PREFIX, ids=lambda d: _name(
    {k: (v if k != "lens" or len(v) < 7 else len(v)) for k, v in d.items()}))
def test_prefix(kw):
    p = Problem(15, ids=None, **kw)
    p.device().run().check()


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("splits", [False, True], ids=["whole", "split"])
def test_values_of_unseen_tokens_never_reach_a_row(dtype, splits):
    """NaN and infinity written as the value of a token: only the queries that see the
    token get them, although their tile multiplies it for all."""
    n = 1200 if not splits else 40          # enough tiles for a CTA each, or blocks shared by several
    p = Problem(17, lens=list(range(2000, 2000 + n)), seq_of=[0] * n, heads=(16, 8), dtype=dtype, ids="near", topk=4)
    clean = p.device()
    tok = 2000 + n // 2                     # from the middle query on it is visible
    pg, row = int(p.table[0, tok // p.page]), tok % p.page
    dirty = p.device()
    raw = p.v.clone().view(torch.uint8) if dtype == "e4m3" else p.v.clone()
    raw[pg, 3, row, 5] = 0x7F if dtype == "e4m3" else float("inf")
    dirty.vpool = (raw.view(torch.float8_e4m3fn) if dtype == "e4m3" else raw).contiguous().cuda()
    dirty.v = B.cache_from_tensor(dirty.vpool)
    clean.run(RUNS)
    dirty.run(RUNS)
    a, b = clean.out.float(), dirty.out.float()
    sees = torch.zeros(n, 16, p.d, dtype=torch.bool)
    for t in range(n):
        if int(p.lens[t]) > tok and (p.ids[t] == tok // p.block).any():
            sees[t, 6:8, 5] = True          # the two query heads on K/V head 3
    assert sees.any() and not sees.all()
    assert not torch.isfinite(b[sees.cuda()]).any()
    rest = ~sees.cuda()
    # a row computed again sums in another order: as far off as two roundings
    assert torch.isfinite(b[rest]).all()
    _, _, tol, _ = p.reference() if n < 100 else (None, None, None, None)
    if tol is not None:
        assert ((a - b).abs()[rest] <= 2 * tol.cuda()[rest]).all()
    else:
        assert ((a - b).abs()[rest] <= 2.0 ** -6 * a.abs()[rest] + 2.0 ** -6).all()
    assert torch.equal(clean.lse, dirty.lse)


@pytest.mark.parametrize("kw", [dict(), dict(dtype="bf16"), dict(ids=None, prefixes=(900,), groups=(0, 9)),
                                dict(ids=None, prefixes=(900,), groups=(0, 9), dtype="bf16")], ids=_name)
def test_a_call_repeats_bit_for_bit(kw):
    p = Problem(18, **{**dict(lens=(1, 700, 300, 64, 2000, 129, 0, 90, 1500), heads=(16, 2)), **kw})
    d = p.device().run()
    for flags in ([0, PDL] if kw.get("ids", 1) is None else [0, PDL, RUNS, RUNS]):
        e = p.device().run(flags)
        if flags == RUNS:
            e2 = p.device().run(flags)
            assert torch.equal(e.out, e2.out) and torch.equal(e.lse, e2.lse)
        else:
            assert torch.equal(d.out, e.out) and torch.equal(d.lse, e.lse)

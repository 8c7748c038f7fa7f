"""The attention operators on values out of the ordinary (GPU): queries whose heads differ
in size, infinite and NaN queries, key scales of zero, keys of infinity."""
import pytest
import torch

from attention_cases import Problem
from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

RUNS = B.MSA_LAUNCH_QUERY_RUNS


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def _problem(kind, seed=91, **kw):
    """Single queries, a run or queries behind prefixes, and the call's flags."""
    if kind == "prefix":
        base = dict(lens=(5, 0, 300, 64, 1, 777), prefixes=(700,), groups=(0, 6), ids=None)
    elif kind == "dense":
        base = dict(lens=(5, 0, 300, 64, 1, 777), ids=None)
    elif kind == "runs":
        base = dict(lens=list(range(700, 740)), seq_of=[0] * 40, ids="near")
    else:
        base = dict(lens=(5, 0, 300, 64, 1, 2000, 777))
    return Problem(seed, **{**base, **kw}), RUNS if kind == "runs" else 0


KINDS = ["single", "dense", "runs", "prefix"]


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("heads", [(16, 2), (32, 2)], ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_heads_of_unlike_size(kind, heads, dtype):
    """A head's result does not depend on the size of the other heads: the same bits when
    they are 2^17 times larger."""
    p, flags = _problem(kind, heads=heads, dtype=dtype)
    small = p.device().run(flags).check()
    q = p.q.clone()
    p.q[:, 1] *= 2.0 ** 17
    p.q[:, 5] *= 2.0 ** 12
    large = p.device().run(flags)
    rest = [h for h in range(heads[0]) if h not in (1, 5)]
    assert torch.equal(large.out[:, rest], small.out[:, rest]) and torch.equal(large.lse[:, rest], small.lse[:, rest])
    p.q = q


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_queries_that_are_not_finite(kind, dtype, bad):
    """A head of a query that is not finite has no result (NaN; every score it has is
    infinite or NaN); every other row has the same bits as without it."""
    p, flags = _problem(kind, heads=(16, 2), dtype=dtype)
    clean = p.device().run(flags)
    t, h = 2, 9
    p.q[t, h, 7] = bad
    d = p.device().run(flags)
    assert torch.isnan(d.out[t, h]).all() and torch.isnan(d.lse[t, h])
    d.out[t, h], d.lse[t, h] = clean.out[t, h], clean.lse[t, h]
    assert torch.equal(d.out, clean.out) and torch.equal(d.lse, clean.lse)


@pytest.mark.parametrize("which", ["all", "one head"])
@pytest.mark.parametrize("bad_pages", [0, 4])
@pytest.mark.parametrize("kind", KINDS)
def test_key_scale_of_zero(kind, bad_pages, which):
    """Every score is 0: the mean of the visible values, and lse = ln of their number."""
    p, flags = _problem(kind, heads=(16, 4), per_head=True, bad_pages=bad_pages)
    p.scales[2 if which == "one head" else slice(0, 4)] = 0.0
    p.device().run(flags).check()


def test_nan_queries_take_no_longer():
    """Rows without a result are not computed a second time, a token after another."""
    p, flags = _problem("runs", heads=(16, 2), lens=list(range(2000, 2600)), seq_of=[0] * 600, topk=16)

    def time():
        d = p.device()
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            d.run(flags)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return d, best

    _, plain = time()
    p.q[:] = float("nan")
    d, nan = time()
    assert torch.isnan(d.out).all() and torch.isnan(d.lse).all()
    assert nan < 4 * plain, (nan, plain)


@pytest.mark.parametrize("kind", KINDS)
def test_scores_of_minus_infinity(kind):
    """Tokens whose score is -infinity have no weight: the same bits as when their pages are
    not there, whole chunks of them among the first; a query that sees no others has out = 0
    and lse = -inf."""
    p, flags = _problem(kind, heads=(16, 2), dtype="bf16", topk=8,
                        **(dict(lens=(2000, 300, 64, 777)) if kind in ("single", "dense") else {}))
    p.q[:, :, 0] = -p.q[:, :, 0].abs().clamp_min(0.01)
    row = int(p.toff[0]) if kind != "prefix" else int(p.poff[0])
    flat = p.table.view(-1)
    gone = [row + i for i in range(10)]          # ten pages of the first history: 640 tokens
    if kind in ("single", "dense"):              # and all of the last one
        gone += [int(p.toff[-1]) + i for i in range(13)]
    infinite = p.device()
    k = p.k.clone()
    k[flat[gone].long(), :, :, 0] = float("inf")
    infinite.kpool = k.cuda()
    infinite.k = B.cache_from_tensor(infinite.kpool)
    infinite.run(flags)
    flat[gone] = -1
    absent = p.device().run(flags).check()
    assert torch.equal(infinite.out, absent.out) and torch.equal(infinite.lse, absent.lse)


@pytest.mark.parametrize("dtype,bad", [("e4m3", "nan"), ("bf16", "nan"), ("bf16", "inf")])
@pytest.mark.parametrize("n", [40, 900], ids=["split", "whole"])
def test_keys_of_unseen_tokens(n, dtype, bad):
    """A key of NaN or infinity: the queries of a run that do not see its token are as
    without it, although their tile multiplies it; those that do have no finite result or
    (a score of -infinity) give the token no weight."""
    p = Problem(92, lens=list(range(2000, 2000 + n)), seq_of=[0] * n, heads=(16, 8), dtype=dtype, ids="near", topk=4)
    clean = p.device().run(RUNS)
    tok = 2000 + n // 2                     # from the middle query on it is visible
    pg, row = int(p.table[0, tok // p.page]), tok % p.page
    dirty = p.device()
    raw = p.k.clone().view(torch.uint8) if dtype == "e4m3" else p.k.clone()
    raw[pg, 3, row, 5] = 0x7F if dtype == "e4m3" else float(bad)
    dirty.kpool = (raw.view(torch.float8_e4m3fn) if dtype == "e4m3" else raw).contiguous().cuda()
    dirty.k = B.cache_from_tensor(dirty.kpool)
    dirty.run(RUNS)
    sees = torch.zeros(n, 16, dtype=torch.bool)
    for t in range(n):
        if int(p.lens[t]) > tok and (p.ids[t] == tok // p.block).any():
            sees[t, 6:8] = True             # the two query heads on K/V head 3
    assert sees.any() and not sees.all()
    if bad == "inf":                        # the sign of the score is that of the query's element
        none = sees & (p.q[:, :, 5] < 0)
        sees &= p.q[:, :, 5] >= 0
        assert torch.isfinite(dirty.out.cpu()[none]).all() and torch.isfinite(dirty.lse.cpu()[none]).all()
        assert torch.isnan(dirty.out.cpu()[sees]).all()
        sees |= none
    else:
        assert torch.isnan(dirty.out.cpu()[sees]).all() and torch.isnan(dirty.lse.cpu()[sees]).all()
    # rows computed again round their weights otherwise: each call is within the tolerance
    # of the definition, so they are within twice of one another
    rest = ~sees
    assert torch.equal(dirty.lse.cpu()[rest], clean.lse.cpu()[rest])
    a, b = clean.out.cpu().double(), dirty.out.cpu().double()
    assert torch.isfinite(b[rest]).all()
    some = rest & (torch.arange(n) % 37 == 0)[:, None] if n > 100 else rest
    at = torch.nonzero(some.any(1)).flatten().tolist()
    q = Problem(92, lens=list(range(2000, 2000 + n)), seq_of=[0] * n, heads=(16, 8), dtype=dtype, ids="near", topk=4)
    q.q, q.lens, q.toff, q.ids, q.T = q.q[at], q.lens[at], q.toff[at], q.ids[at], len(at)
    out, _, tol, _ = q.reference()
    for x in (a, b):
        assert ((x[at] - out).abs()[rest[at]] <= tol[rest[at]]).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("layout", ["hnd", "odd"])
@pytest.mark.parametrize("v_dtype", ["e4m3", "bf16"])
def test_infinite_queries_of_one_token(v_dtype, layout, bad):
    """Over an E4M3 cache an infinite query has no result even where its only score is
    -infinity, in the kernel for every layout as on the tensor cores."""
    p = Problem(93, lens=(1, 1, 0), heads=(16, 2), v_dtype=v_dtype, layout=layout)
    p.q[:, 9, 7] = bad
    d = p.device().run()
    assert torch.isnan(d.out[:2, 9]).all() and torch.isnan(d.lse[:2, 9]).all()
    assert (d.out[2] == 0).all() and torch.isneginf(d.lse[2]).all()
    rest = [h for h in range(16) if h != 9]
    assert torch.isfinite(d.out[:, rest]).all()

"""The attention operators against their definition in 64 bits (GPU)."""
import numpy as np
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


def _both():
    return [(Problem(19, lens=(1, 700, 300, 64, 2000, 129, 0, 90, 1500), heads=(16, 2), topk=6), 0),
            (Problem(20, **_runs((1000, 90)), heads=(16, 2), topk=6, ids="near"), RUNS),
            (Problem(21, lens=(3, 500, 0, 77) * 6, prefixes=(1500, 200), groups=(0, 20, 24), heads=(16, 2), ids=None), 0)]


def test_captured_and_replayed():
    """A capture of the three kinds of call, replayed on changed queries."""
    items = [(p, p.device(), flags) for p, flags in _both()]
    for _, d, flags in items:
        d.run(flags)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _, d, flags in items:
            d.run(flags)
    for p, d, _ in items:
        p.q = (0.5 * p.q.flip(0)).to(torch.bfloat16).contiguous()
        d.q.copy_(p.q)
        d.out.fill_(float("nan"))
        d.ws.fill_(0xFF)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for _, d, _ in items:
        d.check()


def test_two_calls_at_once_on_other_streams():
    """Calls in flight together on streams that are not the current one, each with its own
    workspace, many times over."""
    items = [(p, p.device(), flags, torch.cuda.Stream()) for p, flags in _both()]
    torch.cuda.synchronize()
    for _ in range(20):
        for _, d, flags, s in items:
            d.run(flags, stream=s)
    torch.cuda.synchronize()
    for _, d, _, _ in items:
        d.check()


@pytest.mark.parametrize("which", [0, 1, 2], ids=["decode", "runs", "prefix"])
def test_nothing_past_the_buffers_is_written(which):
    """Outputs and workspace between guard bands; the caches and inputs as they were."""
    p, flags = _both()[which]
    d = p.device()
    pad = 4096
    bufs = {}
    for name in ("out", "lse", "ws"):
        t = getattr(d, name)
        n = t.numel() * t.element_size()
        raw = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
        raw[pad:pad + n] = 0xFF
        setattr(d, name, raw[pad:pad + n].view(t.dtype).view(t.shape))
        bufs[name] = (raw, n)
    d.ws = bufs["ws"][0][pad:pad + B.msa_attention_workspace_bytes(d.cfg, p.T, 0 if p.groups is None else len(p.prefixes))]
    before = [x.clone() for x in (d.kpool.view(torch.uint8), d.vpool.view(torch.uint8), d.q, d.lens, d.toff, d.table)]
    d.run(flags)
    torch.cuda.synchronize()
    for raw, n in bufs.values():
        assert (raw[:pad] == 0xA5).all() and (raw[pad + n:] == 0xA5).all()
    for a, b in zip(before, (d.kpool.view(torch.uint8), d.vpool.view(torch.uint8), d.q, d.lens, d.toff, d.table)):
        assert torch.equal(a, b)
    d.check()


def test_without_lse_and_without_a_workspace():
    for p, flags in _both():
        d = p.device().run(flags)
        e = p.device()
        e.ws = None
        e.run(flags, lse=False)
        torch.cuda.synchronize()
        assert torch.equal(d.out, e.out) and torch.isnan(e.lse).all()


def test_more_queries_than_a_window():
    """Several launches of the decode kernel, and windows that cut groups."""
    n = 900
    lens = [(i * 37) % 200 for i in range(n)]
    Problem(22, lens=lens, heads=(4, 2), topk=2).device().run().check()
    Problem(23, lens=lens, heads=(4, 2), ids=None, prefixes=(300, 150, 70), groups=(10, 350, 500, 880)).device().run().check()


def test_offsets_past_32_bits():
    """Cache elements past 2^32, page strides that leave holes between the pages."""
    P, D, pages = 64, 128, 40
    stride = 2**32 // 32 + 1024                       # elements: page 33 lies past 2^32
    for dtype, tdt in ((B.MSA_DTYPE_FP8_E4M3, torch.float8_e4m3fn),):
        raw = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
        view = torch.as_strided(raw, (pages, 2, P, D), (stride, P * D, D, 1))
        g = torch.Generator(device="cuda").manual_seed(5)
        vals = (torch.randn(pages, 2, P, D, generator=g, device="cuda") / 0.05).to(tdt).view(torch.uint8)
        view.copy_(vals)
        table = torch.randperm(pages, generator=torch.Generator().manual_seed(6)).to(torch.int32).cuda()
        T, n = 3, pages * P
        q = torch.randn(T, 8, D, generator=g, device="cuda").to(torch.bfloat16)
        cfg = B.make_attention_cfg(8, 2, D, P, 128, 8)
        lens = torch.full((T,), n, dtype=torch.int32, device="cuda")
        off = torch.zeros(T, dtype=torch.int64, device="cuda")
        ids = torch.arange(20, dtype=torch.int32, device="cuda").flip(0)[:8].repeat(T, 1).contiguous()
        scales = torch.tensor([0.05, 0.05], device="cuda")
        c = B.cache_from_tensor(view)
        outs = []
        for flags in (0, RUNS):
            out = torch.empty_like(q)
            B.sparse_attention_tensors(cfg, q, ids, lens, off, table, c, c, scales, out, launch_flags=flags)
            outs.append(out)
        kv = vals[table.long()].view(tdt).double() * float(scales[0])         # [pages, 2, P, D] in token order
        kv = kv.permute(1, 0, 2, 3).reshape(2, n, D)[:, 12 * 128:]
        s = torch.einsum("thgd,hnd->thgn", q.double().view(T, 2, 4, D), kv) * D ** -0.5
        ref = torch.einsum("thgn,hnd->thgd", s.softmax(-1), kv).reshape(T, 8, D)
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -7 * kv.abs().mean() * 1.5
        for out in outs:
            assert ((out.double() - ref).abs() <= tol).all()


def test_a_decode_layer_end_to_end():
    """Producer, indexer and sparse attention of one decode step, the attention against its
    definition on what the producer and the indexer wrote; then, on the same caches, dense
    attention behind a shared prefix."""
    from paged_kv_cache_msa_gb300 import workloads as wl
    from paged_kv_cache_msa_gb300.device import DecodeLayer, DeviceWorkload
    w = wl.config2_decode64()
    pools = {k: torch.randint(0, 120, (n,), dtype=torch.uint8, device="cuda") for k, n in w.pools.items()}
    dw = DeviceWorkload(w, pools_on_device=pools)
    layer = DecodeLayer(dw, 144, attention=True)
    s = torch.cuda.current_stream()
    for flags in (0, PDL):
        layer.run(s, flags)
    torch.cuda.synchronize()
    K, V = (pools[k][4096:] for k in ("k", "v"))
    kc = w.caches["k"]
    table, toff, kv_len = dw.page_table.cpu(), layer.table_offset.cpu(), layer.kv_len.cpu()
    ids = layer.topk_ids.cpu()
    q = dw.q_out.view(torch.bfloat16).double()
    out = layer.attn_out.view(torch.bfloat16).double()
    ks, vs = float(w.scales[0]), float(w.scales[1])

    def rows(pool, t, js):
        pg = table[int(toff[t]) + js // 64].long()
        base = pg * kc.stride_page + (js % 64) * kc.stride_token
        idx = base[:, None, None] + (torch.arange(8) * kc.stride_head)[None, :, None] + torch.arange(128)
        return pool[idx.cuda()].view(torch.float8_e4m3fn).double()

    for t in (0, 7, 20, 41, 63):
        n = int(kv_len[t])
        js = torch.cat([torch.arange(b * 128, min(n, b * 128 + 128)) for b in sorted(ids[t][ids[t] >= 0].tolist())])
        k, v = rows(K, t, js) * ks, rows(V, t, js) * vs
        z = torch.einsum("hgd,nhd->hgn", q[t].view(8, 8, 128), k) * 128 ** -0.5
        ref = torch.einsum("hgn,nhd->hgd", z.softmax(-1), v).reshape(64, 128)
        p = z.softmax(-1)
        mean = torch.einsum("hgn,nhd->hgd", p, v.abs()).reshape(64, 128)
        mag = torch.einsum("hgd,nhd->hgn", q[t].view(8, 8, 128).abs(), k.abs()).amax(-1).reshape(64, 1) * 128 ** -0.5
        # The tolerance of attention_cases, in E4M3.  Weights w_j = l p_j, the largest 1 and so
        # 1 / l = max p: an error of 2^-14 in each moves the result by at most
        # sum_j 2^-14 |v_j| / l = 2^-14 max(p) sum_j |v_j|.  (2^-14 times the tokens times
        # mean = sum_j p_j |v_j| is no bound of that: with p_1 near 1 and v_1 = 0 the mean
        # vanishes and the sum does not.)
        qmax = q[t].view(8, 8, 128).abs().amax((1, 2))
        ds = mag * 2.0 ** -16 + 2.0 ** -17 * 128 ** -0.5 * (qmax * k.abs().sum(2).amax(0)).repeat_interleave(8)[:, None]
        floor = 2.0 ** -14 * p.amax(-1).reshape(64, 1) * v.abs().sum(0).repeat_interleave(8, 0)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * ds) * mean + floor
        assert ((out[t] - ref).abs() <= tol).all(), t
    # dense attention of the same queries, the first 8 behind sequence 0's first 512 tokens
    cfg = layer.attn_cfg
    T = w.num_tokens
    plen = min(512, int(kv_len.max()))
    row = int(toff[int(kv_len.argmax())])
    args = dict(kv_len=layer.kv_len, table_offset=layer.table_offset, page_table=dw.page_table,
                k_cache=dw.caches["k"], v_cache=dw.caches["v"], scales=dw.scales)
    a, b = torch.empty_like(dw.q_out), torch.empty_like(dw.q_out)
    B.prefix_attention_tensors(cfg, dw.q_out, torch.tensor([0, 8], dtype=torch.int32, device="cuda"),
                               torch.tensor([plen], dtype=torch.int32, device="cuda"),
                               torch.tensor([row], dtype=torch.int64, device="cuda"), out=a, **args)
    B.prefix_attention_tensors(cfg, dw.q_out, None, None, None, out=b, **args)
    torch.cuda.synchronize()
    assert torch.equal(a[8:], b[8:]) or (a[8:].view(torch.bfloat16).double() - b[8:].view(torch.bfloat16).double()).abs().max() <= 2.0 ** -7 * b.view(torch.bfloat16).abs().max()
    assert not torch.equal(a[:8], b[:8])
    assert torch.isfinite(a.view(torch.bfloat16)).all()


@pytest.mark.parametrize("layout", ["hnd", "odd"])
@pytest.mark.parametrize("kind", ["decode", "runs", "dense", "prefix"])
def test_lengths_past_the_table(kind, layout):
    """Tokens whose table index lies past the table are not visible, however long the
    history is said to be; neither are those before it."""
    kw = dict(prefixes=(700,), groups=(0, 3), ids=None) if kind == "prefix" else dict(ids=None) if kind == "dense" else {}
    lens = (300, 640, 90, 500)
    p = Problem(51, lens=lens, layout=layout, **kw)
    n = p.table.numel() * p.page
    # what the table holds after the start of a row, and the length that says more
    p.lens = torch.tensor([n - int(o) * p.page for o in p.toff], dtype=torch.int32)
    p.toff[2] = -3                                    # three pages before the table
    p.lens[2] = 200 + 3 * p.page
    if p.groups is not None:
        p.prefixes = torch.tensor([n - int(p.poff[0]) * p.page], dtype=torch.int32)
    # every cell that may be seen now is written
    raw_k, raw_v = p._raw(p.k), p._raw(p.v)
    for raw in (raw_k, raw_v):
        raw[(raw & 0x7F) == 0x7F] = 0x11
    if p.ids is not None:
        p.ids = p._ids(np.random.default_rng(52), "random")
    ref = p.reference()
    p.lens = torch.where(torch.arange(4) == 2, p.lens, torch.tensor(2**31 - 1, dtype=torch.int32))
    if p.groups is not None:
        p.prefixes = torch.tensor([2**31 - 1], dtype=torch.int32)
    flags = B.MSA_LAUNCH_QUERY_RUNS if kind == "runs" else 0
    p.device().run(flags).check(ref)


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("kind", ["decode", "runs", "prefix"])
def test_zero_queries_and_negative_scales(kind, dtype):
    """A query of zeros weighs its tokens alike; a negative key scale turns the scores."""
    kw = dict(prefixes=(300,), groups=(0, 5), ids=None) if kind == "prefix" else {}
    p = Problem(61, lens=(500, 130, 700, 0, 129), seq_of=(0, 1, 1, 1, 0), dtype=dtype, **kw)
    p.q[1] = 0.0
    p.q[2, 3:6] = 0.0                                 # some heads of a group
    p.scales = -p.scales
    p.device().run(RUNS if kind == "runs" else 0).check()


@pytest.mark.parametrize("n", [400, 512])
def test_a_group_for_every_query(n):
    """As many groups as the call takes, more than a window of queries."""
    p = Problem(62, lens=[i % 5 for i in range(n)], prefixes=[(70 * i) % 300 for i in range(n)],
                groups=list(range(n + 1)), heads=(4, 2), head_dim=64, ids=None)
    p.device().run().check()


def test_a_decode_layer_behind_a_prefix():
    """Dense attention of a decode layer's queries over its caches, the first eight behind a
    prefix: the prefix's tokens, then each query's own, against the definition."""
    from paged_kv_cache_msa_gb300 import workloads as wl
    from paged_kv_cache_msa_gb300.device import DecodeLayer, DeviceWorkload
    w = wl.config2_decode64()
    pools = {k: torch.randint(0, 120, (n,), dtype=torch.uint8, device="cuda") for k, n in w.pools.items()}
    for raw in pools.values():                         # values of both signs
        raw[::3] += 128
    dw = DeviceWorkload(w, pools_on_device=pools)
    layer = DecodeLayer(dw, 144, attention=True)
    layer.run(torch.cuda.current_stream())
    K, V = (pools[k][4096:] for k in ("k", "v"))
    kc = w.caches["k"]
    table = dw.page_table.flatten()
    own, toff = layer.kv_len.tolist(), layer.table_offset.tolist()
    longest = max(range(64), key=lambda i: own[i])
    plen, prow = min(500, own[longest]), toff[longest]
    out, lse = torch.empty_like(dw.q_out), torch.empty(64, 64, device="cuda")
    B.prefix_attention_tensors(layer.attn_cfg, dw.q_out, torch.tensor([0, 8], dtype=torch.int32, device="cuda"),
                               torch.tensor([plen], dtype=torch.int32, device="cuda"),
                               torch.tensor([prow], dtype=torch.int64, device="cuda"), layer.kv_len, layer.table_offset,
                               dw.page_table, dw.caches["k"], dw.caches["v"], dw.scales, out, lse)
    q, got = dw.q_out.view(torch.bfloat16).double(), out.view(torch.bfloat16).double()

    def rows(pool, spans, scale):
        pg = torch.cat([table[off + torch.arange(n, device="cuda") // 64] for off, n in spans]).long()
        at = torch.cat([torch.arange(n, device="cuda") % 64 for _, n in spans])
        base = pg * kc.stride_page + at * kc.stride_token
        heads = torch.arange(8, device="cuda") * kc.stride_head
        idx = base[:, None, None] + heads[None, :, None] + torch.arange(128, device="cuda")
        return pool[idx].view(torch.float8_e4m3fn).double() * scale

    for t in (0, 3, 7, 8, 40, 63):
        spans = [(prow, plen)] * (t < 8) + [(toff[t], own[t])]
        k, v = (rows(pool, spans, float(w.scales[i])) for i, pool in enumerate((K, V)))
        qt = q[t].view(8, 8, 128)
        z = torch.einsum("hgd,nhd->hgn", qt, k) * 128 ** -0.5
        ref_lse = torch.logsumexp(z, -1)
        p = z.softmax(-1)
        ref = torch.einsum("hgn,nhd->hgd", p, v)
        mean = torch.einsum("hgn,nhd->hgd", p, v.abs())
        # scores: fp32 accumulation, and the query halves' floor of each row; weights: 2^-8
        mag = torch.einsum("hgd,nhd->hgn", qt.abs(), k.abs()).amax(-1) * 128 ** -0.5
        ds = mag * 2.0 ** -16 + 2.0 ** -17 * 128 ** -0.5 * qt.abs().amax(-1) * k.abs().sum(2).amax(0)[:, None]
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * ds[..., None]) * mean
        assert ((got[t].view(8, 8, 128) - ref).abs() <= tol).all(), t
        assert ((lse[t].view(8, 8).double() - ref_lse).abs() <= ds + 2.0 ** -20 * (1 + ref_lse.abs())).all(), t

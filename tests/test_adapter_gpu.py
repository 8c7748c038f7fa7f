"""Low-rank adapters beside a packed projection against their formula in 64 bits (GPU).

Tolerance.  With A = sum_i |up| sum_k |hidden| |down| (times the scales), fp32 sums of K and of rank
products are off by at most (K + rank + 8) 2^-24 A, and u's two bf16 parts by 2^-16 A; then the
output's rounding, 2^-8 of it."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

PACKED = (8192, 9216, 10240, 11264, 11392)      # the big shapes' sections
SMALL = (512, 640, 768, 896, 960)               # the small shapes'


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def wide(x, pad, fill):
    """The same rows, 16 * pad elements further apart than whole vectors need, `fill` between."""
    t, k = x.shape
    w = torch.full((t, -(-k // 16) * 16 + 16 * pad), 0, dtype=torch.uint8, device="cuda").to(x.dtype)
    w.view(torch.uint8).fill_(fill)
    w[:, :k] = x
    return w[:, :k]


class Case:
    def __init__(self, ids, k=256, ends=SMALL, rank=16, adapters=4, fp8=False, scaled=True, pad=0, seed=0, alpha=True):
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        t, w, s = len(ids), ends[-1], len(ends)
        self.n, self.k, self.ends, self.rank, self.adapters = t, k, ends, rank, adapters
        gen = torch.Generator(device="cuda").manual_seed(91 + seed)
        x = torch.randn(t, k, generator=gen, device="cuda") * 2
        x = x.to(torch.float8_e4m3fn) if fp8 else x.bfloat16()
        self.hidden = wide(x, pad, 0x7F)                    # NaN behind the rows
        self.hidden_scales = 0.1 + torch.rand(t, generator=gen, device="cuda") if scaled else None
        d = torch.randn(adapters * s * rank, k, generator=gen, device="cuda") / k ** 0.5
        self.down = wide(d.bfloat16(), pad, 0xFF).unflatten(0, (adapters, s * rank))
        self.up = torch.randn(adapters, w, rank, generator=gen, device="cuda").bfloat16()
        self.alpha = torch.randn(adapters, generator=gen, device="cuda") if alpha else None
        self.rows = wide((3 * torch.randn(t, w, generator=gen, device="cuda")).bfloat16(), pad, 0x21)
        self.raw = torch.full((t + 2, -(-w // 16) * 16 + 16 * pad), 0, dtype=torch.int16, device="cuda").fill_(0x4242)
        self.out = self.raw.view(torch.bfloat16)[1:-1, :w]
        self.cfg = B.make_adapter_cfg(k, ends, rank, adapters, B.MSA_DTYPE_FP8_E4M3 if fp8 else B.MSA_DTYPE_BF16)
        n = B.msa_adapter_workspace_bytes(self.cfg, t)
        self.ws_raw = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")    # NaN
        self.ws = self.ws_raw[256:256 + n]

    def run(self, flags=0, stream=None, out=None, workspace="own"):
        B.adapter_tensors(self.cfg, self.hidden, self.down, self.up, self.ids, self.rows, self.out if out is None else out,
                          hidden_scales=self.hidden_scales, adapter_scales=self.alpha,
                          workspace=self.ws if workspace == "own" else workspace, launch_flags=flags, stream=stream)
        return self

    def formula(self, rows=None):
        """out, and what its tolerance goes by, in 64 bits."""
        rows = self.rows if rows is None else rows
        x = self.hidden.to(torch.float64)
        if self.hidden_scales is not None:
            x = x * self.hidden_scales.double()[:, None]
        out, size = rows.double().clone(), torch.zeros(self.n, self.ends[-1], dtype=torch.float64, device="cuda")
        start = [0, *self.ends]
        for a in range(self.adapters):
            on = self.ids == a
            c = 1.0 if self.alpha is None else float(self.alpha[a])
            for s in range(len(self.ends)):
                d = self.down[a, s * self.rank:(s + 1) * self.rank].double()
                up, cols = self.up[a, start[s]:start[s + 1]].double(), slice(start[s], start[s + 1])
                out[on, cols] += c * (x[on] @ d.T @ up.T)
                size[on, cols] = abs(c) * (x[on].abs() @ d.abs().T @ up.abs().T)
        return out, size

    def check(self, out=None, rows=None):
        got = self.out if out is None else out
        want, size = self.formula(rows)
        tol = 2.0 ** -8 * want.abs() + size * ((self.k + self.rank + 8) * 2.0 ** -24 + 2.0 ** -16)
        off = ((got.double() - want).abs() - tol)
        assert (off <= 0).all(), float(off.max())
        none = (self.ids < 0) | (self.ids >= self.adapters)
        base = self.rows if rows is None else rows
        assert torch.equal(got[none].view(torch.int16), base[none].view(torch.int16))
        assert (self.raw[0] == 0x4242).all() and (self.raw[-1] == 0x4242).all()
        assert (self.raw[1:-1, self.ends[-1]:] == 0x4242).all()
        assert (self.ws_raw[:256] == 0xFF).all() and (self.ws_raw[-256:] == 0xFF).all()
        return self


def mixed(t, n, seed=5):
    """Adapters in no order, ids outside on both sides among them."""
    gen = torch.Generator().manual_seed(seed + t)
    ids = torch.randint(-1, n + 1, (t,), generator=gen).tolist()
    if t > 3:
        ids[2], ids[3] = 2**31 - 1, -2**31
    return ids


def runs(t, n):
    return [(i * (n + 1)) // t - 1 for i in range(t)]


@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 64, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("order", [mixed, runs], ids=["mixed", "runs"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_batches(t, order, fp8):
    Case(order(t, 4), fp8=fp8, seed=t).run().check()


@pytest.mark.parametrize("k", [1, 5, 8, 16, 40, 63, 64, 65, 127, 200, 1000, 1001, 2049, 6144])
@pytest.mark.parametrize("t", [5, 400])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_hidden_sizes(k, t, fp8):
    Case(runs(t, 3), k=k, adapters=3, fp8=fp8, pad=1, seed=k).run().check()


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 56, 64, 96, 128])
@pytest.mark.parametrize("t", [3, 150, 700])
@pytest.mark.parametrize("ends", [(960,), (64, 72), (64, 640, 704, 1024)], ids=str)
def test_ranks_and_slices(rank, t, ends):
    Case(runs(t, 4), k=320, ends=ends, rank=rank, seed=rank).run().check()


@pytest.mark.parametrize("ends", [(8,), (64,), (56,), (64, 128, 192, 256, 320, 384, 448, 456), (200,), (1000,), (4096, 4104)], ids=str)
@pytest.mark.parametrize("t", [1, 33, 260])
def test_widths(ends, t):
    Case(mixed(t, 4), k=96, ends=ends, rank=8, pad=2, seed=t).run().check()


@pytest.mark.parametrize("t", [1, 64, 2048])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_packed_projection(t, fp8):
    """The big shapes' hidden size and packed row."""
    Case(mixed(t, 24) if t <= 64 else runs(t, 5), k=6144, ends=PACKED, adapters=24, fp8=fp8).run().check()


def test_many_adapters_in_one_batch():
    Case([i % 130 for i in range(260)], k=128, rank=8, adapters=130).run().check()
    Case([i % 130 for i in range(520)], k=128, rank=8, adapters=130).run().check()


@pytest.mark.parametrize("t", [1, 40, 600])
def test_one_adapter_and_none(t):
    Case([0] * t, adapters=1).run().check()
    Case([-1] * t, adapters=1).run().check()
    Case([7] * t, adapters=1).run().check()


@pytest.mark.parametrize("kw", [dict(scaled=False), dict(alpha=False), dict(scaled=False, alpha=False, fp8=True)], ids=str)
def test_without_scales(kw):
    Case(mixed(50, 4), **kw).run().check()
    Case(runs(500, 4), **kw).run().check()


@pytest.mark.parametrize("t", [6, 64, 300, 1200])
def test_in_place(t):
    c = Case(mixed(t, 4), pad=1).run().check()
    rows = c.rows.clone()
    want = c.out.clone()
    c.run(out=c.rows)
    assert torch.equal(c.rows, want)
    c.check(out=c.rows, rows=rows)


@pytest.mark.parametrize("t", [20, 64, 300, 1000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_one_requests_values_stay_its_own(t, bad):
    """What is not finite in an adapter, in a request's hidden states, scales or rows reaches only the
    rows of that adapter or request."""
    for what in ("down", "up", "alpha", "hidden", "hidden_scales", "rows"):
        c = Case(mixed(t, 4), pad=1)
        c.run()
        clean = c.out.clone()
        if what in ("down", "up", "alpha"):
            getattr(c, what)[2] = bad
            mine = c.ids == 2
        else:
            getattr(c, what)[1] = bad
            mine = torch.arange(t, device="cuda") == 1
        c.run()
        assert torch.equal(c.out[~mine].view(torch.int16), clean[~mine].view(torch.int16)), what
        touched = mine & (c.ids >= 0) & (c.ids < 4) if what != "rows" else mine
        assert not c.out[touched].isfinite().any(), what


def test_repeated_calls_give_the_same_bits():
    for t in (64, 900):
        c = Case(mixed(t, 4), k=1000).run()
        first = c.out.clone()
        c.ws.fill_(0x7F)
        c.out.zero_()
        c.run()
        assert torch.equal(first.view(torch.int16), c.out.view(torch.int16))


def test_no_tokens_and_own_workspace():
    c = Case([0, 1, 2])
    c.run(workspace=None).check()
    e = Case([])
    e.run(workspace=None)


def test_other_stream_and_graph():
    """On a stream of its own behind the work that makes the rows; captured and replayed with other
    rows and other requests' adapters in the same tensors."""
    for t in (64, 500):
        c = Case(mixed(t, 4), k=512)
        s = torch.cuda.Stream()
        keep = c.rows.clone()
        for flags in (0, B.MSA_LAUNCH_PDL):
            c.rows.zero_()
            c.out.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)
                c.rows.copy_(keep)
                c.run(flags)
            s.synchronize()
            c.check()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                c.run(flags)
                c.run(flags)
            for ids in (mixed(t, 4, seed=8), [-1] * t, runs(t, 4), mixed(t, 4)):
                c.ids.copy_(torch.tensor(ids, dtype=torch.int32))
                g.replay()
                torch.cuda.synchronize()
                c.check()


def test_two_streams_with_their_own_workspaces():
    cases = [Case(runs(700, 4), k=1024, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_tensors_that_do_not_fit_are_refused():
    c = Case([0, 1, 2, 3])
    good = dict(cfg=c.cfg, hidden=c.hidden, down=c.down, up=c.up, adapter_ids=c.ids, rows=c.rows, out=c.out,
                hidden_scales=c.hidden_scales, adapter_scales=c.alpha, workspace=c.ws)
    B.adapter_tensors(**good)
    for bad in (dict(hidden=c.hidden[:, :-1]), dict(hidden=c.hidden.float()), dict(down=c.down[:3]), dict(down=c.down[:, ::2]),
                dict(up=c.up.transpose(1, 2)), dict(adapter_ids=c.ids.long()), dict(rows=c.rows[:3]), dict(out=c.out.cpu()),
                dict(hidden_scales=c.hidden_scales[:3]), dict(adapter_scales=c.alpha.double()), dict(workspace=c.ws.cpu()),
                dict(down=c.down[0])):
        with pytest.raises(ValueError):
            B.adapter_tensors(**dict(good, **bad))
    with pytest.raises(B.MsaError):
        B.adapter_tensors(**dict(good, workspace=c.ws[:256]))


def test_tiles_of_several_adapters_over_many_blocks():
    """Large batches of wide rows whose tiles of 128 tokens have one adapter, several or none: what
    the groups of warps that take blocks by turns must keep apart."""
    for seed in range(8):
        gen = torch.Generator().manual_seed(seed)
        edges = torch.cat([torch.tensor([0, 2048]), torch.randint(1, 2048, (4 + 5 * seed,), generator=gen)]).sort().values
        ids = []
        for i, n in enumerate(edges.diff().tolist()):
            ids += [i % 7 - 1] * n
        Case(ids, k=128, ends=PACKED, adapters=6, rank=(16, 32, 64, 96)[seed % 4], seed=seed).run().check()


@pytest.mark.parametrize("t", [3, 64, 700])
def test_a_chain_in_place(t):
    """Calls that each add to what the one before wrote, hidden states made by the kernel just ahead:
    the bits of the same calls with the device idle between them."""
    c = Case(mixed(t, 4), k=512)
    start, src = c.rows.clone(), c.hidden.clone()

    def steps(between):
        c.rows.copy_(start)
        for i in range(12):
            torch.mul(src, 1.0 + i / 8, out=c.hidden) if not between else c.hidden.copy_(src * (1.0 + i / 8))
            between and torch.cuda.synchronize()
            c.run(out=c.rows)
            between and torch.cuda.synchronize()
        return c.rows.clone()

    want = steps(True)
    for _ in range(3):
        assert torch.equal(steps(False).view(torch.int16), want.view(torch.int16))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = steps(False)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# Tiles of 128 tokens are taken from T^2 * rows of down * K of 5e11 and 56 tokens an adapter (up to 16
# of them) on.  Sizes below that are batches that tiles of 16 must hold as well.

def wide_case(order, t=1300, k=1000, rank=64, adapters=4, **kw):
    assert t * k >= 1200000 and rank > 24
    return Case(order(t, adapters), k=k, rank=rank, adapters=adapters, **kw)


@pytest.mark.parametrize("t,k", [(30001, 40), (19000, 64), (18500, 65), (6100, 200), (1300, 1000), (1201, 1001), (640, 2049),
                                 (200, 6144), (129, 9600), (128, 9600), (127, 9600), (80, 15500)])
@pytest.mark.parametrize("rank", [32, 40])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_wide_sizes(t, k, rank, fp8):
    wide_case(runs if t % 2 else mixed, t, k, rank, fp8=fp8, pad=1, seed=k).run().check()


@pytest.mark.parametrize("rank", [8, 16, 24, 48, 56, 64, 72, 96])
@pytest.mark.parametrize("order", [mixed, runs], ids=["mixed", "runs"])
def test_wide_ranks(rank, order):
    Case(order(1500, 3), k=1000, rank=rank, adapters=3, fp8=True).run().check()


@pytest.mark.parametrize("ends", [(8,), (72,), (64, 128, 192, 256, 320, 384, 448, 456), (1000,), (4096, 4104)], ids=str)
def test_wide_widths(ends):
    Case(mixed(1500, 4), k=1000, ends=ends, rank=56 if len(ends) > 4 else 128, fp8=True, pad=2).run().check()


def test_wide_without_scales_or_adapters():
    wide_case(mixed, scaled=False, alpha=False).run().check()
    for ids in (0, -1, 9):
        Case([ids] * 1300, k=1000, rank=64, adapters=1).run().check()


def test_wide_in_place_and_repeated():
    c = wide_case(mixed, pad=1).run().check()
    rows, want = c.rows.clone(), c.out.clone()
    c.ws.fill_(0x7F)
    c.out.zero_()
    c.run()
    assert torch.equal(c.out.view(torch.int16), want.view(torch.int16))
    c.run(out=c.rows)
    assert torch.equal(c.rows, want)
    c.check(out=c.rows, rows=rows)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_wide_requests_values_stay_their_own(bad, fp8):
    for what in ("down", "up", "alpha", "hidden", "hidden_scales", "rows"):
        if fp8 and what == "hidden" and bad == float("inf"):
            continue                                          # E4M3 has no infinity
        c = wide_case(mixed, pad=1, fp8=fp8).run()
        clean = c.out.clone()
        if what in ("down", "up", "alpha"):
            getattr(c, what)[2] = bad
            mine = c.ids == 2
        else:
            getattr(c, what)[1] = torch.tensor(bad).to(getattr(c, what).dtype)
            mine = torch.arange(c.n, device="cuda") == 1
        c.run()
        assert torch.equal(c.out[~mine].view(torch.int16), clean[~mine].view(torch.int16)), what
        touched = mine & (c.ids >= 0) & (c.ids < 4) if what != "rows" else mine
        assert not c.out[touched].isfinite().any(), what


def test_wide_chain_and_graph():
    """Calls in place one after another, other requests' adapters between them, eager and replayed."""
    c = wide_case(mixed)
    start = c.rows.clone()
    orders = [torch.tensor(o, dtype=torch.int32, device="cuda") for o in (mixed(1300, 4), runs(1300, 4), [-1] * 1300, [2] * 1300)]

    def steps(between):
        c.rows.copy_(start)
        for o in orders * 2:
            c.ids.copy_(o)
            between and torch.cuda.synchronize()
            c.run(out=c.rows)
            between and torch.cuda.synchronize()
        return c.rows.clone()

    want = steps(True)
    assert torch.equal(steps(False).view(torch.int16), want.view(torch.int16))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = steps(False)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("t", [17, 500, 3000])
def test_thousands_of_adapters(t):
    """Most of them unused; every token another one."""
    gen = torch.Generator().manual_seed(t)
    ids = torch.randint(-20, 16384 + 20, (t,), generator=gen).tolist()
    Case(ids, k=64, ends=(64,), rank=8, adapters=16384).run().check()
    Case([(i * 7) % 4099 for i in range(t)], k=512, ends=(64,), rank=32, adapters=4099, fp8=True).run().check()


def test_more_tokens_than_the_sort_keeps():
    """Tokens beyond those that the sorting threads hold in registers."""
    Case(mixed(20000, 5), k=24, ends=(64, 72), rank=8, adapters=5).run().check()
    wide_case(mixed, 40001, 32, adapters=3, ends=(128,)).run().check()


@pytest.mark.parametrize("t", [17, 31, 32, 33, 63, 65, 95, 96, 97, 128])
@pytest.mark.parametrize("order", [lambda t, n: [0] * t, lambda t, n: [-1] * t, lambda t, n: [n] * (t - 1) + [n - 1],
                                   lambda t, n: [i % 2 - 1 for i in range(t)], lambda t, n: [(5 * i) % n for i in range(t)],
                                   lambda t, n: [i * n // t for i in range(t)][::-1]],
                         ids=["one", "none", "last", "every other", "several", "chunks"])
def test_tiles_of_up_to_128_tokens(t, order):
    """Batches whose tiles every CTA makes by itself: one adapter's tiles over several warps' tokens."""
    for n in (3, 131):
        Case(order(t, n), k=40, ends=(64, 72), rank=8, adapters=n).run().check()


@pytest.mark.parametrize("t", [1, 20, 200, 1300])
def test_every_e4m3_value(t):
    """Every finite code, in every place of a word, through a down-projection that picks single elements
    out and an up-projection that passes them on: exact but for the output's rounding, none at all here
    (an E4M3 value times a power of two).  A NaN code makes its own element of the row NaN."""
    k, rank = 2048, 64
    cfg = B.make_adapter_cfg(k, (64, 128, 192), rank, 1, B.MSA_DTYPE_FP8_E4M3)
    at = torch.arange(t, device="cuda")[:, None] * 37 + torch.arange(k, device="cuda")
    codes = ((at + at // 256) % 256).to(torch.uint8)
    codes[codes & 0x7F == 0x7F] = 0
    values = codes.view(torch.float8_e4m3fn).double()
    up = torch.zeros(1, 192, rank, dtype=torch.bfloat16, device="cuda")
    up[0, torch.arange(192), torch.arange(192) % 64] = 4.0
    rows, out = torch.zeros(t, 192, dtype=torch.bfloat16, device="cuda"), torch.empty(t, 192, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(t, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.msa_adapter_workspace_bytes(cfg, t), dtype=torch.uint8, device="cuda")
    for first in (0, 192, 1024, k - 192):
        down = torch.zeros(1, 3 * rank, k, dtype=torch.bfloat16, device="cuda")
        down[0, torch.arange(192), first + torch.arange(192)] = 1.0
        B.adapter_tensors(cfg, codes, down, up, ids, rows, out, workspace=ws)
        assert torch.equal(out.double(), 4 * values[:, first:first + 192])
    codes[t // 2, 5] = 0xFF
    B.adapter_tensors(cfg, codes, down, up, ids, rows, out, workspace=ws)
    nan = out.isnan().any(1)
    assert nan[t // 2] and int(nan.sum()) == 1


def wide_tiles(order, t, k, ends=SMALL, rank=32, adapters=3, **kw):
    assert t * t * len(ends) * rank * k >= 5e11 and t >= 56 * min(adapters, 16)
    return Case(order(t, adapters), k=k, ends=ends, rank=rank, adapters=adapters, **kw)


@pytest.mark.parametrize("t,k", [(1400, 2049), (1801, 1001), (1800, 1000), (2200, 650), (700, 9000), (550, 15500)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_wide_tiles_of_other_sizes(t, k, fp8):
    wide_tiles(runs if t % 4 else mixed, t, k, fp8=fp8, pad=1, seed=k).run().check()


@pytest.mark.parametrize("rank", [8, 16, 24, 40])
@pytest.mark.parametrize("order", [mixed, runs], ids=["mixed", "runs"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_wide_tiles_of_small_ranks(rank, order, fp8):
    wide_tiles(order, 3600, 1000, rank=rank, fp8=fp8).run().check()


@pytest.mark.parametrize("ends", [(8,), (72,), (1000,), (4096, 4104)], ids=str)
def test_wide_tiles_of_few_slices(ends):
    wide_tiles(mixed, 2100, 1000, ends=ends, rank=128, fp8=True, pad=2).run().check()


@pytest.mark.parametrize("t", [895, 896, 897])
def test_many_adapters_at_the_step_to_wide_tiles(t):
    wide_tiles(mixed, 896, 4000, rank=40, adapters=40)
    Case(mixed(t, 40), k=4000, rank=40, adapters=40, fp8=True).run().check()


def from_rule(rows, k, adapters=1):
    """The tokens from which on a call takes tiles of 128."""
    return max(int((5e11 / (rows * k)) ** 0.5) + 1, 56 * min(adapters, 16))


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("t", [1, 20, 200, "wide"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_all_bits_of_u(rank, t, fp8):
    """u of 21 significant bits, put together from whole numbers of 7 bits (E4M3: 20 bits of 4), less
    another u of its upper bits: what is left, a number of 7 bits (4), is exact in every step."""
    k, bits = 2048, 4 if fp8 else 7
    pieces, pairs = 20 // bits if fp8 else 21 // bits, rank // 2
    t = from_rule(rank, k) if t == "wide" else t
    two = rank % 16 == 0                                 # two slices of half the rank each
    cfg = B.make_adapter_cfg(k, (64, 136) if two else (136,), rank // 2 if two else rank, 1,
                             B.MSA_DTYPE_FP8_E4M3 if fp8 else B.MSA_DTYPE_BF16)
    slices, per = cfg.num_slices, cfg.rank // 2          # pairs of rows of down in a slice
    gen = torch.Generator(device="cuda").manual_seed(rank)
    x = torch.zeros(t, k, device="cuda")
    x[:, :pieces * pairs] = torch.randint(1, 2 ** bits, (t, pieces * pairs), generator=gen, device="cuda").float()
    down = torch.zeros(1, slices * cfg.rank, k, device="cuda")
    for m in range(pairs):                               # rows 2 m and 2 m + 1: all pieces, and all but the last
        for i in range(pieces):
            down[0, 2 * m:2 * m + 1 + (i < pieces - 1), pieces * m + i] = 2.0 ** (-bits * i)
    col = torch.arange(136, device="cuda")
    pair = col % per
    up = torch.zeros(1, 136, cfg.rank, device="cuda")
    up[0, col, 2 * pair], up[0, col, 2 * pair + 1] = 1.0, -1.0
    rows = torch.zeros(t, 136, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(rows)
    hidden = x.to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
    assert torch.equal(hidden.float(), x)
    B.adapter_tensors(cfg, hidden, down.bfloat16(), up.bfloat16(), torch.zeros(t, dtype=torch.int32, device="cuda"), rows, out)
    last = pieces * (pair + (per * (col >= 64) if slices == 2 else 0)) + pieces - 1
    assert torch.equal(out.double(), x[:, last].double() * 2.0 ** (-bits * (pieces - 1)))


@pytest.mark.parametrize("t", [2, 64, 300, 1300])
@pytest.mark.parametrize("graph", [False, True])
def test_everything_made_by_the_kernel_just_ahead(t, graph):
    """Rows, ids, hidden states and the adapters themselves, written by copies right ahead of each call and
    other ones for each: the bits of the same calls with the device idle in between."""
    steps = 8
    c = Case(mixed(t, 4), k=1000, rank=64, adapters=4)
    gen = torch.Generator(device="cuda").manual_seed(t)
    pick = [torch.randint(-1, 5, (t,), generator=gen, device="cuda").int() for _ in range(steps)]
    turn = lambda x, i: x.roll(i + 1, 0)
    made = [(turn(c.rows, i).contiguous(), turn(c.hidden, i).contiguous(), turn(c.up, i).contiguous(),
             turn(c.down, i).contiguous()) for i in range(steps)]
    outs = [torch.zeros_like(c.rows) for _ in range(steps)]

    def run(idle):
        for i in range(steps):
            rows, hidden, up, down = made[i]
            # (the last copy ahead of the call is another one each time)
            copies = [(c.ids, pick[i]), (c.rows, rows), (c.up, up), (c.down, down), (c.hidden, hidden)]
            for j in range(len(copies)):
                to, of = copies[(j + i) % len(copies)]
                to.copy_(of)
            if idle:
                torch.cuda.synchronize()
            c.run(out=outs[i])
            if idle:
                torch.cuda.synchronize()

    run(True)
    want = [o.clone() for o in outs]
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(False)
    for _ in range(20):
        for o in outs:
            o.zero_()
        g.replay() if graph else run(False)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16))

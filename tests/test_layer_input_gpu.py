"""The input side of a layer as it is used (GPU): residual and norm, projection, adapters, producer,
one after another on a stream and in a graph.  Each step's output is checked against its formula in
64 bits, of the values that the step before gave it."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod
from paged_kv_cache_msa_gb300.device import LayerInput
from test_adapter_gpu import mixed, runs
from test_norm_gpu import F32, check_codes, expected
from test_rope_axes_gpu import BIG, TINY, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


class Layer:
    """A layer's weights, adapters and caches; the producer's part is a Case of the rotary tests."""

    def __init__(self, n, shape, k, rank, adapters=4, axes=True, with_adapters=True, order=mixed, seed=0, max_tokens=None):
        gen = torch.Generator(device="cuda").manual_seed(400 + seed)
        d = shape[-1]
        c = self.case = Case(n, shape, (d // 8, d // 8, d // 4), per_head=True, seed=seed, theta=5e6)
        if not axes:
            c.positions.copy_((torch.arange(n, device="cuda") % 64).to(torch.int32).expand(3, -1))
        W, sr = c.width, 5 * rank
        self.n, self.k = n, k
        self.x = (2 * torch.randn(n, k, generator=gen, device="cuda")).bfloat16()
        self.residual = (3 * torch.randn(n, k, generator=gen, device="cuda")).bfloat16()
        self.norm_w = (0.5 + torch.rand(k, generator=gen, device="cuda")).bfloat16()
        # (rows 16 bytes apart at least, as the projection wants them)
        padded = torch.zeros(W, -(-k // 16) * 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.weight = padded[:, :k]
        self.weight.view(torch.uint8).copy_(
            (8 * torch.randn(W, k, generator=gen, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8))
        self.weight_scales = (0.5 + torch.rand(W, generator=gen, device="cuda")) / 8 / k ** 0.5
        self.down = (torch.randn(adapters, sr, k, generator=gen, device="cuda") / k ** 0.5).bfloat16()
        self.up = torch.randn(adapters, W, rank, generator=gen, device="cuda").bfloat16()
        self.alpha = 0.5 + torch.rand(adapters, generator=gen, device="cuda")
        self.ids = torch.tensor(order(n, adapters), dtype=torch.int32, device="cuda") if with_adapters else None
        self.adapters = (self.down, self.up, self.alpha) if with_adapters else None
        self.desc = [B.cache_from_tensor(p) for p in c.pools]
        self.layer = LayerInput(c.cfg, max_tokens or n, self.weight.view(torch.uint8), self.weight_scales, self.norm_w,
                                c.weights, self.desc, c.scales, axes=c.axes if axes else None, adapters=self.adapters)
        self.axes = axes

    def run(self, flags=0, stream=None):
        c = self.case
        self.before = self.residual.clone()
        pos = c.positions if self.axes else c.positions[0].contiguous()
        self.layer.run(self.x, self.residual, pos, c.slots, c.table, self.ids, flags, stream)
        return self

    def check(self, before=None):
        c, layer, n = self.case, self.layer, self.n
        before = self.before if before is None else before
        assert int(layer.status) == 0
        assert torch.equal(self.residual, (self.x.float() + before.float()).bfloat16())
        codes = layer.codes[:n].view(torch.float8_e4m3fn)
        _, y, s = expected(self.x, before, self.norm_w, 1e-6)
        check_codes(codes, layer.hidden_scales[:n], y, s)
        if layer.rows is None:
            return self
        # rows: the projection of the codes, rounded to bf16 (2^-8), then the adapter's share, rounded
        # again; fp32 sums of K products are off by K 2^-24 of their magnitudes' sum at most
        h = codes.to(torch.float64) * layer.hidden_scales[:n, None].double()
        w = self.weight.to(torch.float64) * self.weight_scales[:, None].double()
        row = h @ w.T
        tol = 2.0 ** -8 * row.abs() + (self.k + 4) * 2.0 ** -24 * (h.abs() @ w.abs().T)
        if self.ids is not None:
            d, hq, hkv, hiq, hik = c.shape[-1], *c.shape[:4]
            ends, rank = [0], self.up.shape[2]
            for heads in (hq, hkv, hkv, hiq, hik):
                ends.append(ends[-1] + heads * d)
            for a in range(self.up.shape[0]):
                on = self.ids == a
                for i in range(5):
                    cols = slice(ends[i], ends[i + 1])
                    dn, up = self.down[a, i * rank:(i + 1) * rank].double(), self.up[a, cols].double()
                    row[on, cols] += float(self.alpha[a]) * (h[on] @ dn.T @ up.T)
                    size = float(self.alpha[a]) * (h[on].abs() @ dn.abs().T @ up.abs().T)
                    tol[on, cols] += size * ((self.k + rank + 8) * 2.0 ** -24 + 2.0 ** -16)
            tol += 2.0 ** -8 * row.abs() + 2.0 ** -8 * tol
        assert ((layer.rows[:n].double() - row).abs() <= tol).all()
        c.rows, c.q, c.iq = layer.rows[:n], layer.q_out[:n], layer.idx_q_out[:n]
        if self.axes:
            c.check()
        return self


@pytest.mark.parametrize("n", [1, 7, 64, 300])
@pytest.mark.parametrize("shape,k,rank", [(TINY, 320, 8), (TINY, 1000, 64), (BIG, 512, 16)], ids=["tiny", "tiny64", "big"])
@pytest.mark.parametrize("flags", [0, B.MSA_LAUNCH_PERSISTENT])
def test_steps(n, shape, k, rank, flags):
    Layer(n, shape, k, rank, seed=n).run(flags).check()


def test_prefill():
    """Chunks of requests with an adapter each; wide tiles of the adapters, the projection's 2-SM kernel."""
    Layer(1500, TINY, 2048, 32, order=runs).run(B.MSA_LAUNCH_PERSISTENT).check()


def test_longer_prefill():
    """Sizes of the adapters' wide tiles."""
    Layer(2000, TINY, 2048, 32, order=runs, seed=9).run(B.MSA_LAUNCH_PERSISTENT).check()


def test_axes_alone_and_adapters_alone():
    Layer(90, BIG, 512, 16, with_adapters=False).run().check()
    Layer(90, BIG, 512, 16, axes=False).run().check()


def test_neither_is_the_fused_projection():
    """Without adapters and axes the producer runs in the projection's epilogue: the same compact Q,
    up to a step of the rows' rounding, as through the rows."""
    a = Layer(40, TINY, 512, 8, axes=False, with_adapters=False).run().check()
    b = Layer(40, TINY, 512, 8, axes=False, order=lambda n, _: [-1] * n).run().check()
    assert a.layer.rows is None
    # rows a bf16 step apart (2^-7 of them) move a head's values by that, and by as much through its norm
    size = b.layer.q_out[:40].double().abs().amax(-1, keepdim=True)
    assert ((a.layer.q_out[:40].double() - b.layer.q_out[:40].double()).abs() <= 2.0 ** -5 * size).all()


def test_graph_of_two_layers():
    """Two layers one after another, the second on the first one's residual, on a side stream and in a
    graph that is replayed with other requests, positions and adapters."""
    one, two = Layer(64, TINY, 512, 16, seed=1, max_tokens=100), Layer(64, TINY, 512, 16, seed=2)
    two.residual = one.residual
    start = one.residual.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one.run(stream=s)
    two.run(stream=s)
    s.synchronize()
    two.check(before=(one.x.float() + start.float()).bfloat16())
    one.residual = (one.x.float() + start.float()).bfloat16()
    one.check(before=start)
    one.residual = two.residual
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one.run(B.MSA_LAUNCH_PERSISTENT | B.MSA_LAUNCH_PDL)
        two.run(B.MSA_LAUNCH_PERSISTENT | B.MSA_LAUNCH_PDL)
    for seed in (3, 4):
        for i, layer in enumerate((one, two)):
            new = Layer(64, TINY, 512, 16, seed=10 * seed + i)
            layer.x.copy_(new.x)
            layer.ids.copy_(new.ids)
            layer.case.positions.copy_(new.case.positions)
        one.residual.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        middle = (one.x.float() + start.float()).bfloat16()
        two.check(before=middle)
        one.residual = middle
        one.check(before=start)
        one.residual = two.residual


@pytest.mark.parametrize("n", [1, 16, 17, 33, 100, 500])
def test_fewer_tokens_than_the_layers(n):
    layer = Layer(n, TINY, 1000, 64, seed=n, max_tokens=1300)
    rows = layer.layer.rows
    rows.fill_(7.0)
    layer.run().check()
    assert (rows[n:] == 7.0).all(), "rows behind the last token"


def test_no_tokens():
    layer = Layer(5, TINY, 512, 16)
    c = layer.case
    before = [p.clone() for p in c.pools]
    layer.layer.run(layer.x[:0], layer.residual[:0], c.positions[:, :0].contiguous(), c.slots[:0], c.table,
                    layer.ids[:0])
    torch.cuda.synchronize()
    assert all(torch.equal(p.view(torch.uint8), b.view(torch.uint8)) for p, b in zip(c.pools, before))


@pytest.mark.parametrize("n", [3, 100, 700])
def test_streams_that_fork_and_join(n):
    """What a layer reads and writes is made and used by other streams around it: the input by a copy on
    one, the ids by a copy on another, the results read on the first, called one by one and in a graph."""
    layer = Layer(n, TINY, 2048, 32, seed=n)
    new = [Layer(n, TINY, 2048, 32, seed=n + s) for s in (1, 2)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    x, ids, residual = layer.x.clone(), layer.ids.clone(), layer.residual.clone()
    rows, q = torch.empty_like(layer.layer.rows), torch.empty_like(layer.layer.q_out)

    def step():
        here = torch.cuda.current_stream()
        a.wait_stream(here)
        b.wait_stream(here)
        with torch.cuda.stream(b):
            layer.ids.fill_(-7)
            layer.ids.copy_(ids)
            layer.residual.copy_(residual)
        with torch.cuda.stream(a):
            layer.x.zero_()
            layer.x.copy_(x)
            a.wait_stream(b)
            layer.run(stream=a)
        here.wait_stream(a)
        rows.copy_(layer.layer.rows)
        q.copy_(layer.layer.q_out)

    def check(before):
        torch.cuda.synchronize()
        layer.check(before=before)
        assert torch.equal(rows, layer.layer.rows) and torch.equal(q, layer.layer.q_out)

    torch.cuda.synchronize()
    step()
    check(residual)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for other in new:
        x.copy_(other.x)
        ids.copy_(other.ids)
        residual.copy_(other.residual)
        g.replay()
        check(residual)


def test_two_layers_at_once():
    """Two threads, a layer and a stream each."""
    import threading
    layers = [Layer(200, TINY, 1000, 64, seed=s) for s in (5, 6)]
    torch.cuda.synchronize()
    start = [layer.residual.clone() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    errors = []

    def work(layer, begin, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(20):
                    layer.residual.copy_(begin)
                    layer.run(stream=stream)
        except Exception as e:       # shown below
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(layers, start, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for layer, begin in zip(layers, start):
        layer.check(before=begin)


def test_refused_runs_leave_everything_as_it_was():
    layer = Layer(20, TINY, 512, 16)
    c = layer.case
    state = [layer.residual, layer.layer.codes, layer.layer.rows, layer.layer.q_out, *c.pools]
    before = [t.clone() for t in state]
    good = dict(x=layer.x, residual=layer.residual, positions=c.positions, slot_mapping=c.slots, page_table=c.table,
                adapter_ids=layer.ids)
    for bad in (dict(positions=c.positions.long()), dict(slot_mapping=c.slots.int()), dict(adapter_ids=layer.ids.long()),
                dict(page_table=c.table.long()), dict(adapter_ids=None), dict(x=layer.x[:19]), dict(residual=layer.residual.float())):
        with pytest.raises(ValueError):
            layer.layer.run(**dict(good, **bad))
    torch.cuda.synchronize()
    for t, b in zip(state, before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
    layer.run().check()


def test_a_projection_that_did_not_finish_is_reported():
    """In the starved test build no copy is issued and the projection's waits run out."""
    layer = Layer(20, TINY, 512, 16)
    normal = B._lib
    start = layer.residual.clone()
    B._lib = B.load(build_mod.build_starved())
    try:
        layer.run()
        with pytest.raises(RuntimeError, match="did not finish"):
            layer.layer.check_status()
    finally:
        B._lib = normal
    layer.residual.copy_(start)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.run(stream=s)
    layer.layer.check_status(s)
    layer.check()

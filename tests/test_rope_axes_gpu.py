"""The producer with rotary positions of several axes against its formula in 64 bits (GPU).

Tolerances.  The fp32 norm of 64 or 128 elements is off by less than 2^-19 of a value; an angle by
2^-25 of a turn, 2^-52 of itself (at most 2^-23 of a turn at 2^31) and its sine and cosine by 2^-23,
so that a rotated value is off by less than 2^-19 + 2^-20 of |u| + |v|, its pair: 2^-18 of that
covers both.  Then the rounding of the output: 2^-8 of it in bf16; in E4M3 2^-4 of it or half of
the smallest step, 2^-10, times the scale, whose reciprocal's rounding 2^-18 covers too."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -18
BIG, TINY = (64, 8, 8, 1, 128), (8, 2, 2, 1, 64)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def spread(gen, n, axes):
    """Positions of every kind: small, far, negative, the ends of int32."""
    p = torch.randint(-2**31, 2**31, (axes, n), generator=gen, device="cuda")
    p[:, ::3] = torch.randint(0, 500, p[:, ::3].shape, generator=gen, device="cuda")
    p[:, 1::7] = torch.randint(100000, 400000, p[:, 1::7].shape, generator=gen, device="cuda")
    ends = torch.tensor([0, -1, 2**31 - 1, -2**31], device="cuda")
    p[:, :4] = ends[:n] if n < 4 else ends
    return p.to(torch.int32)


class Case:
    def __init__(self, n, shape=BIG, pairs=(16, 24, 24), interleaved=False, restart=False, style=B.MSA_ROPE_NEOX, rd=None,
                 page=64, fp8=True, per_head=False, theta=1e4, seed=0, table=True, idx_k=True, row_pad=0, stride_pad=0,
                 nhd=False):
        self.n, self.shape, self.pairs, self.style, self.page, self.fp8 = n, shape, pairs, style, page, fp8
        hq, hkv, hiq, hik, d = shape
        self.rd = 2 * sum(pairs) if rd is None else rd
        gen = torch.Generator(device="cuda").manual_seed(31 + seed)
        self.cfg = B.make_cfg(hq, hkv, hiq, hik, d, self.rd, style, page, theta, 1e-6,
                              B.MSA_SCALE_PER_HEAD if per_head else B.MSA_SCALE_PER_TENSOR)
        self.axes = B.make_rope_axes(pairs, interleaved=interleaved, restart=restart)
        self.width = (hq + 2 * hkv + hiq + hik) * d
        wide = torch.full((n, self.width + row_pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :self.width] = 2 * torch.randn(n, self.width, generator=gen, device="cuda")
        self.rows = wide
        self.positions = torch.full((len(pairs), n + stride_pad), 77, dtype=torch.int32, device="cuda")[:, :n]
        self.positions.copy_(spread(gen, n, len(pairs)))
        pages = -(-n // page) + 2
        slots = torch.randperm(pages * page, generator=gen, device="cuda")[:n]
        slots[5::11] = -1
        if n > 8:
            slots[8] = (pages + 3) * page          # past the table, or past the caches
        self.slots = slots
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32) if table else None
        if table and pages > 2:
            self.table[1] = pages + 100            # a page outside the caches
        self.weights = [(0.5 + torch.rand(d, generator=gen, device="cuda")).bfloat16() for _ in range(4)]
        ns = (hkv, hkv, hik) if per_head else (1, 1, 1)
        self.scales = 0.03 + 0.05 * torch.rand(sum(ns), generator=gen, device="cuda")
        self.scale_of = [s if per_head else s.expand(h) for s, h in zip(self.scales.split(ns), (hkv, hkv, hik))]
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16

        def pool(h):
            x = torch.zeros((pages, page, h, d) if nhd else (pages, h, page, d), device="cuda").to(dt)
            x.view(torch.uint8).fill_(0x33)
            return x.transpose(1, 2) if nhd else x

        self.pools = [pool(h) for h in (hkv, hkv, hik)]
        if not idx_k:
            self.pools[2] = None
        self.q, self.iq = (torch.full((n, h, d), 9.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hiq))
        # formula
        axis = list(self.axes.pair_axis)[:self.rd // 2]
        theta = float(self.cfg.rope_theta)          # the configuration's, in fp32
        count, f = [axis.count(a) for a in range(len(pairs))], []
        for k, a in enumerate(axis):
            f.append(theta ** -(axis[:k].count(a) / count[a] if restart else k / len(axis)))
        self.axis, self.freq = axis, f

    def run(self, flags=0, stream=None):
        desc = [None if x is None else B.cache_from_tensor(x) for x in self.pools]
        B.forward_axes_tensors(self.cfg, self.axes, self.rows, self.positions, self.slots, self.table, self.weights,
                               self.q, self.iq, *desc, self.scales, launch_flags=flags, stream=stream)
        return self

    def turned(self, x, w):
        """x [n, h, d] after norm and rotation, and the sizes |u| + |v| that its tolerance goes by."""
        d = x.shape[-1]
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        half, size = self.rd // 2, x.abs()
        if half:
            angle = self.positions[self.axis].double() * torch.tensor(self.freq, dtype=torch.float64, device="cuda")[:, None]
            c, s = torch.cos(angle).T[:, None], torch.sin(angle).T[:, None]
            at = (slice(0, half), slice(half, 2 * half)) if self.style == B.MSA_ROPE_NEOX else \
                (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
            u, v = x[..., at[0]].clone(), x[..., at[1]].clone()
            x[..., at[0]], x[..., at[1]] = u * c - v * s, v * c + u * s
            size[..., at[0]] = size[..., at[1]] = u.abs() + v.abs()
        return x, size

    def check(self):
        hq, hkv, hiq, hik, d = self.shape
        x = self.rows[:, :self.width].double().reshape(self.n, -1, d)
        q, k, v, iq, ik = x.split([hq, hkv, hkv, hiq, hik], 1)
        for got, sec, w in ((self.q, q, self.weights[0]), (self.iq, iq, self.weights[2])):
            want, size = self.turned(sec, w)
            err = (got.double() - want).abs()
            assert (err <= 2.0 ** -8 * want.abs() + F32 * size).all(), float(err.max())
        ok = self.slots >= 0
        blk = torch.where(ok, self.slots, 0) // self.page
        if self.table is not None:
            ok &= blk < self.table.numel()
            blk = self.table.long()[blk.clamp(max=self.table.numel() - 1)]
        ok &= (blk >= 0) & (blk < self.pools[0].shape[0])
        pg, off = blk[ok], self.slots[ok] % self.page
        for pool, sec, w, sc in ((self.pools[0], k, self.weights[1], self.scale_of[0]), (self.pools[1], v, None, self.scale_of[1]),
                                 (self.pools[2], ik, self.weights[3], self.scale_of[2])):
            if pool is None:
                continue
            want, size = self.turned(sec, w) if w is not None else (sec, sec.abs())
            want, size = want[ok], size[ok]
            got = pool[pg, :, off] if not self.fp8 else pool.view(torch.uint8)[pg, :, off].view(torch.float8_e4m3fn)
            if self.fp8:
                s = sc.double()[:, None]
                want, size = (want / s).clamp(-448, 448), size / s
                tol = (2.0 ** -4 * want.abs()).clamp(min=2.0 ** -10) + F32 * size
            else:
                tol = 2.0 ** -8 * want.abs() + F32 * size
            assert ((got.double() - want).abs() <= tol).all()
            touched = torch.zeros(pool.shape[0], self.page, dtype=torch.bool, device="cuda")
            touched[pg, off] = True
            raw = pool.view(torch.uint8) if self.fp8 else pool.view(torch.int16)
            assert (raw.transpose(1, 2)[~touched] == (0x33 if self.fp8 else 0x3333)).all()
        return self


@pytest.mark.parametrize("flags", [0, B.MSA_LAUNCH_PERSISTENT, B.MSA_LAUNCH_PERSISTENT | B.MSA_LAUNCH_PDL])
@pytest.mark.parametrize("n", [1, 2, 9, 64, 700, 2500])
@pytest.mark.parametrize("shape,pairs", [(BIG, (16, 24, 24)), (TINY, (8, 12, 12))], ids=["big", "tiny"])
def test_batches(shape, pairs, n, flags):
    Case(n, shape, pairs, seed=n, row_pad=64, stride_pad=3).run(flags).check()


@pytest.mark.parametrize("style", [B.MSA_ROPE_NEOX, B.MSA_ROPE_GPTJ], ids=["neox", "gptj"])
@pytest.mark.parametrize("pairs", [(64,), (32, 32), (0, 64), (1, 2, 61), (16, 16, 16, 16), (8, 8), (2, 0, 6), (0, 0, 0)], ids=str)
@pytest.mark.parametrize("how", ["sections", "interleaved", "restart"])
def test_axes(pairs, how, style):
    """One to four axes, axes without a pair, part of the dims, none."""
    Case(150, BIG, pairs, interleaved=how == "interleaved", restart=how == "restart", style=style, theta=5e6).run().check()


@pytest.mark.parametrize("shape", [(1, 0, 0, 0, 64), (0, 1, 0, 0, 128), (0, 0, 1, 0, 64), (0, 0, 0, 1, 128), (3, 1, 0, 1, 128),
                                   (17, 5, 3, 2, 64), (128, 16, 4, 1, 128)], ids=str)
def test_heads(shape):
    """Every launch shape, sections without heads."""
    d = shape[-1]
    hq, hkv, hiq, hik, _ = shape
    c = Case(77, shape, (d // 8, d // 8, d // 4))
    desc = [B.cache_from_tensor(x) if h else None for x, h in zip(c.pools, (hkv, hkv, hik))]
    B.forward_axes_tensors(c.cfg, c.axes, c.rows, c.positions, c.slots, c.table, c.weights, c.q if hq else None,
                           c.iq if hiq else None, *desc, c.scales)
    c.check()


@pytest.mark.parametrize("kw", [dict(fp8=False), dict(per_head=True), dict(page=48), dict(page=1), dict(table=False),
                                dict(idx_k=False), dict(nhd=True), dict(page=7, fp8=False, nhd=True), dict(theta=1.0),
                                dict(theta=0.5), dict(theta=1e30)], ids=str)
def test_caches_and_bases(kw):
    Case(203, **kw).run(B.MSA_LAUNCH_PERSISTENT).check()


def test_one_axis_near_zero_agrees_with_the_producer():
    """Positions below 64 on every axis: angles that fp32 holds well, so both producers' codes and
    values agree to their rounding."""
    c = Case(300)
    c.positions.copy_((torch.arange(300, device="cuda") % 64).to(torch.int32).expand(3, -1))
    c.run().check()
    q, pools = c.q.clone(), [p.clone() for p in c.pools]
    desc = [B.cache_from_tensor(x) for x in c.pools]
    B.forward_tensors(c.cfg, c.rows, c.positions[0].contiguous(), c.slots, c.table, c.weights, c.q, c.iq, *desc, c.scales)
    size = c.turned(c.rows[:, :64 * 128].double().reshape(300, 64, 128), c.weights[0])[1]
    # both are within 2^-8 of the formula's value (a step apart where it lies between two), the
    # fp32 angles within 64 * 2^-24
    assert ((q.double() - c.q.double()).abs() <= 2.0 ** -7 * q.double().abs() + 2.0 ** -17 * size).all()
    assert torch.equal(pools[1].view(torch.uint8), c.pools[1].view(torch.uint8))      # V is not turned


def test_graph_and_stream():
    c = Case(64, seed=3)
    s = torch.cuda.Stream()
    keep = c.rows.clone()
    c.rows.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        c.rows.copy_(keep)
        c.run(B.MSA_LAUNCH_PERSISTENT)
    s.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(B.MSA_LAUNCH_PERSISTENT | B.MSA_LAUNCH_PDL)
    c.positions.copy_(c.positions.flip(1).clone())
    c.rows.copy_(keep.flip(0))
    c.q.zero_()
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_tensors_that_do_not_fit_are_refused():
    c = Case(16)
    desc = [B.cache_from_tensor(x) for x in c.pools]
    good = dict(cfg=c.cfg, axes=c.axes, qkv=c.rows, positions=c.positions, slot_mapping=c.slots, page_table=c.table,
                norm_weights=c.weights, q_out=c.q, idx_q_out=c.iq, k_cache=desc[0], v_cache=desc[1], idx_k_cache=desc[2],
                scales=c.scales)
    B.forward_axes_tensors(**good)
    for bad in (dict(qkv=c.rows[:, :-8]), dict(positions=c.positions[:2]), dict(positions=c.positions.long()),
                dict(positions=c.positions.cpu()), dict(slot_mapping=c.slots.int()), dict(q_out=c.q[:, :1]),
                dict(scales=c.scales[:2]), dict(norm_weights=[c.weights[0][:1]] * 4), dict(positions=c.positions.T)):
        with pytest.raises(ValueError):
            B.forward_axes_tensors(**dict(good, **bad))

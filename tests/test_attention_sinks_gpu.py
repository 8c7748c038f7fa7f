"""Concentrated attention over E4M3 caches (GPU): one token holds a large share of the
attention and thousands share the rest, each with a weight far below the first's.  What
the kernels may be off by does not grow with the number of tokens.

The tolerance follows from the arithmetic: half a bf16 step of the result (2^-8), a weight
off by at most 2^-8 of itself (a bf16 weight; an E4M3 cache's are nearer) and a score by
ds, which moves every weight by a factor within exp(+-ds): (2^-8 + 2 ds) times the mean of
|v|.  ds: fp32 accumulation (2^-16 of the products' magnitudes) and the query halves' floor
(2^-17 of the row's largest element for each element of a key)."""
import math

import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

P, SCALE = 64, 0.05


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


class Sink:
    """T queries over one sequence of n tokens, the first of which takes the share ``s`` of
    the attention among ``seen`` tokens; the other scores normal with deviation ``dev``, the
    values normal around ``mean``."""

    def __init__(self, seed, T, n, seen, s, heads=(16, 2), d=128, dev=1.0, mean=0.5, dtype="e4m3"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.d, self.n, self.T = *heads, d, n, T
        pages = -(-n // P)
        self.q = (dev * torch.randn(T, self.hq, d, generator=g, device="cuda")).bfloat16()
        self.q[:, :, 0] = 16.0
        k = torch.randn(self.hkv, pages * P, d, generator=g, device="cuda")
        k[:, :, 0] = 0.0
        k[:, 0] = 0.0
        k[:, 0, 0] = (math.log(s / (1 - s)) + math.log(seen) + dev * dev / 2) * d ** 0.5 / 16.0
        v = torch.randn(self.hkv, pages * P, d, generator=g, device="cuda") + mean
        self.scale = SCALE if dtype == "e4m3" else 1.0
        dt = torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16
        self.perm = torch.randperm(pages, generator=g, device="cuda")
        self.k, self.v = (self._pool(x / self.scale, dt) for x in (k, v))
        self.table = self.perm.int()
        self.scales = torch.tensor([SCALE, SCALE], device="cuda")
        self.toff = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.out = torch.empty_like(self.q)
        self.lse = torch.empty(T, self.hq, device="cuda")

    def _pool(self, x, dt):
        pool = torch.empty(self.perm.numel(), self.hkv, P, self.d, dtype=dt, device="cuda")
        raw = pool.view(torch.uint8 if dt == torch.float8_e4m3fn else torch.int16)
        raw[self.perm] = x.to(dt).view(raw.dtype).view(self.hkv, -1, P, self.d).transpose(0, 1).contiguous()
        return pool

    def rows(self, pool):
        raw = pool.view(torch.uint8 if pool.dtype == torch.float8_e4m3fn else torch.int16)
        x = raw[self.perm].transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :self.n].contiguous()
        return x.view(pool.dtype).double() * self.scale

    def check(self, seen=None):
        """``seen``: [T, n] truth values, or None for every token."""
        k, v = self.rows(self.k), self.rows(self.v)
        G, sc = self.hq // self.hkv, self.d ** -0.5
        for c in range(self.hkv):
            for t0 in range(0, self.T, 32):
                t = slice(t0, min(self.T, t0 + 32))
                h = slice(c * G, (c + 1) * G)
                q = self.q[t, h].double()
                z = (q @ k[c].T) * sc
                if seen is not None:
                    z = z.masked_fill(~seen[t, None, :], -math.inf)
                lse = torch.logsumexp(z, -1)
                a = torch.exp(z - lse[..., None])
                o, mean = a @ v[c], a @ v[c].abs()
                mag = (q.abs() @ k[c].abs().T).amax(-1) * sc
                ds = mag * 2.0 ** -16 + sc * 2.0 ** -17 * q.abs().amax(-1) * k[c].abs().sum(1).max()
                tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * ds[..., None]) * mean
                err = (self.out[t, h].double() - o).abs()
                assert (err <= tol).all(), f"{float((err / tol).max()):.2f} of the tolerance"
                assert ((self.lse[t, h].double() - lse).abs() <= ds + 2.0 ** -20 * (1 + lse.abs())).all()

    def sparse(self, topk, flags):
        g = torch.Generator(device="cuda").manual_seed(1)
        nb = -(-self.n // 128)
        pick = torch.rand(self.T, nb, generator=g, device="cuda")
        pick[:, 0] = 2.0
        ids = pick.topk(topk, dim=1).indices.int().contiguous()
        lens = (self.n - self.T + 1 + torch.arange(self.T, device="cuda")).int()
        cfg = B.make_attention_cfg(self.hq, self.hkv, self.d, P, 128, topk)
        B.sparse_attention_tensors(cfg, self.q, ids, lens, self.toff, self.table, B.cache_from_tensor(self.k),
                                   B.cache_from_tensor(self.v), self.scales, self.out, self.lse, launch_flags=flags)
        tok = torch.arange(self.n, device="cuda")
        seen = torch.zeros(self.T, nb, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)[:, tok // 128]
        self.check(seen & (tok < lens[:, None]))

    def dense(self, grouped):
        cfg = B.make_attention_cfg(self.hq, self.hkv, self.d, P)
        lens = torch.full((self.T,), 0 if grouped else self.n, dtype=torch.int32, device="cuda")
        groups = (torch.tensor([0, self.T], dtype=torch.int32, device="cuda"),
                  torch.tensor([self.n], dtype=torch.int32, device="cuda"), self.toff[:1]) if grouped else (None,) * 3
        B.prefix_attention_tensors(cfg, self.q, *groups, lens, self.toff, self.table, B.cache_from_tensor(self.k),
                                   B.cache_from_tensor(self.v), self.scales, self.out, self.lse)
        self.check()


# dev 0: the other tokens' weights are all alike, and so are their roundings
SHARES = [(0.3, 1.0), (0.5, 1.0), (0.8, 1.0), (0.5, 0.0), (0.8, 0.0)]


@pytest.mark.parametrize("s,dev", SHARES)
@pytest.mark.parametrize("topk,d,dtype", [(16, 128, "e4m3"), (64, 128, "e4m3"), (16, 64, "e4m3"), (64, 128, "bf16")])
def test_query_runs(topk, d, dtype, s, dev):
    n = 300 + 256 * topk
    Sink(81, 70, n, topk * 128, s, d=d, dev=dev, dtype=dtype).sparse(topk, B.MSA_LAUNCH_QUERY_RUNS)


@pytest.mark.parametrize("s,dev", SHARES)
@pytest.mark.parametrize("n,dtype", [(8192, "e4m3"), (16384, "e4m3"), (8192, "bf16")])
def test_behind_a_prefix(n, dtype, s, dev):
    Sink(82, 380, n, n, s, dev=dev, dtype=dtype).dense(True)


@pytest.mark.parametrize("s,dev", SHARES)
@pytest.mark.parametrize("heads,topk,dtype", [((16, 2), 16, "e4m3"), ((16, 1), 64, "e4m3"), ((16, 2), 64, "bf16")])
def test_single_queries(heads, topk, dtype, s, dev):
    Sink(83, 50, 300 + 256 * topk, topk * 128, s, heads=heads, dev=dev, dtype=dtype).sparse(topk, 0)


@pytest.mark.parametrize("s,dev", SHARES)
@pytest.mark.parametrize("heads,d", [((8, 1), 64), ((16, 1), 128)])
def test_long_histories(heads, d, s, dev):
    """Two lists of 65,536 tokens for each CTA, held whole or in two pieces."""
    Sink(84, 304, 65536, 65536, s, heads=heads, d=d, dev=dev).dense(False)

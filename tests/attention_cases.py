"""Problems for the attention operators and their definition in 64 bits.

``Problem`` holds one call's inputs on the CPU: queries, caches in any strided layout,
page tables, lengths, block ids or prefix groups.  Every cache cell that no history
covers holds NaN (E4M3 code 0x7F, bf16 0x7FC0), so that a kernel which lets a token
that is not visible into a result shows it.

``Problem.reference()`` evaluates the definition in float64, one query and head group
at a time, and with it the tolerance that follows from the arithmetic the header
states (nothing in it is fitted):

  out   half a bf16 step of the result (2^-8 relative), plus the weights' rounding
        (each weight off by at most 2^-8 of itself, and for E4M3 caches by 2^-14 of the
        largest weight), plus the scores' error ds, which moves every weight by a factor
        within exp(+-ds) and so the result by at most 2 ds times the mean of |v|;
  lse   ds, plus a few fp32 roundings of the logarithm and the sum (2^-20 (1 + |lse|));
  ds    fp32 accumulation of D products (2^-16 of the sum of their magnitudes, which is
        above D * 2^-24), plus for E4M3 caches the query halves' floor (2^-17 of the
        largest query element of the head group, per key element).
"""
import numpy as np
import torch

from paged_kv_cache_msa_gb300 import binding as B

NAN8 = 0x7F


class Problem:
    def __init__(self, seed, *, dtype="e4m3", v_dtype=None, heads=(8, 2), head_dim=128, page=64, block=128, topk=4,
                 lens=(300,), seq_of=None, prefixes=(), groups=None, layout="hnd", per_head=False, scale=None,
                 ids="random", spare_pages=3, bad_pages=0, q_gain=1.5):
        """``lens``: visible own tokens of each query; ``seq_of``: the sequence of each
        query (default: its own), whose history is the longest its queries see;
        ``prefixes``: lengths; ``groups``: group_start.  ``bad_pages``: table entries
        turned into -1 or past the pool."""
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hq, self.hkv = heads
        self.d, self.page, self.block, self.topk = head_dim, page, block, topk
        self.kd, self.vd = dtype, v_dtype or dtype
        T = len(lens)
        self.T = T
        self.q = (q_gain * torch.randn(T, self.hq, head_dim, generator=g)).to(torch.bfloat16)
        seq_of = list(range(T)) if seq_of is None else list(seq_of)
        nseq = max(seq_of, default=-1) + 1
        hist = [0] * nseq
        for n, s in zip(lens, seq_of):
            hist[s] = max(hist[s], n, 0)
        rows = list(prefixes) + hist
        need = [-(-max(n, 0) // page) for n in rows]
        width = max(need + [1])
        self.pages = sum(need) + spare_pages
        perm = torch.from_numpy(rng.permutation(self.pages).astype(np.int32))
        table = torch.full((len(rows) + 1, width), -1, dtype=torch.int32)
        k = 0
        for r, n in enumerate(need):
            table[r, :n] = perm[k:k + n]
            k += n
        for _ in range(bad_pages):
            r = int(rng.integers(0, len(rows)))
            if need[r]:
                table[r, int(rng.integers(0, need[r]))] = int(rng.choice([-1, -7, self.pages, 2**31 - 1]))
        self.table = table
        self.toff = torch.tensor([(len(prefixes) + s) * width for s in seq_of], dtype=torch.int64)
        self.lens = torch.tensor(list(lens), dtype=torch.int32)
        self.prefixes = torch.tensor(list(prefixes), dtype=torch.int32)
        self.poff = torch.arange(len(prefixes), dtype=torch.int64) * width
        self.groups = None if groups is None else torch.tensor(groups, dtype=torch.int32)
        self.softmax_scale = head_dim ** -0.5 if scale is None else scale
        ns = 2 * self.hkv if per_head else 2
        self.scales = torch.from_numpy(rng.uniform(0.02, 0.08, size=ns).astype(np.float32))
        self.per_head = per_head
        written = torch.zeros(self.pages, page, dtype=torch.bool)
        for r, n in enumerate(rows):
            for j in range(0, max(n, 0), page):
                pg = int(table[r, j // page])
                if 0 <= pg < self.pages:
                    written[pg, :min(page, n - j)] = True
        self.kpool, self.k = self._cache(g, dtype, layout, written, 0)
        self.vpool, self.v = self._cache(g, self.vd, layout, written, 1)
        if layout == "interleaved":      # one pool [pages, 2, Hkv, P, D] holding both
            raw = torch.stack([self._raw(self.k), self._raw(self.v)], 1).contiguous()
            raw = raw.view(self._dt(dtype))
            self.kpool = self.vpool = raw
            self.k, self.v = raw[:, 0], raw[:, 1]
        self.ids = None
        if ids is not None:
            self.ids = self._ids(rng, ids)

    @staticmethod
    def _dt(dtype):
        return torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16

    @staticmethod
    def _raw(t):
        return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16)

    def _cache(self, g, dtype, layout, written, which):
        n, h, p, d = self.pages, self.hkv, self.page, self.d
        x = torch.randn(n, h, p, d, generator=g)
        x[:, :, :, :3] *= 3.0
        x = (x / 0.05).to(torch.float8_e4m3fn).view(torch.uint8) if dtype == "e4m3" else x.to(torch.bfloat16).view(torch.int16)
        nan = NAN8 if dtype == "e4m3" else 0x7FC0
        x = torch.where(written[:, None, :, None], x, torch.full((), nan, dtype=x.dtype))
        es = 1 if dtype == "e4m3" else 2
        if layout in ("hnd", "interleaved"):
            st = (h * p * d, p * d, d, 1)
        elif layout == "padded":                   # 256 bytes after every page
            st = (h * p * d + 256 // es, p * d, d, 1)
        elif layout == "nhd":                      # tokens outside heads
            st = (h * p * d, d, h * d, 1)
        elif layout == "heads_outer":              # [heads, pages, P, D]
            st = (p * d, n * p * d, d, 1)
        elif layout == "odd":                      # rows 8 elements apart from a 16-byte grid
            st = (h * p * (d + 8), p * (d + 8), d + 8, 1)
        else:
            raise ValueError(layout)
        size = sum((a - 1) * b for a, b in zip((n, h, p, d), st)) + 1
        pool = torch.full((size,), nan, dtype=x.dtype)
        view = torch.as_strided(pool, (n, h, p, d), st)
        view.copy_(x)
        dt = self._dt(dtype)
        return pool.view(dt), torch.as_strided(pool.view(dt), (n, h, p, d), st)

    def _ids(self, rng, how):
        ids = np.full((self.T, self.topk), -1, dtype=np.int32)
        for t in range(self.T):
            n = max(int(self.lens[t]), 0)
            nb = -(-n // self.block)
            k = min(self.topk, nb)
            pick = rng.permutation(nb)[:k]
            if how == "near" and k:                # neighbours agree, the last block among them
                pick = np.unique(np.concatenate([[nb - 1], rng.permutation(min(nb, 2 * self.topk))[:k]]))[-k:]
                pick = rng.permutation(pick)
            ids[t, :len(pick)] = pick
            if how == "messy" and self.topk >= 4:  # gaps, repeats, ids outside the history
                ids[t, 0] = rng.choice([-1, -5, nb, nb + 3, 2**31 - 1])
                ids[t, 2] = ids[t, 1]
                ids[t, 3] = rng.choice([ids[t, 3], ids[t, 1], -2**31])
        return torch.from_numpy(ids)

    # -- the definition ----------------------------------------------------
    def group_of(self, t):
        if self.groups is None:
            return None
        gs = self.groups.tolist()
        for i, x in enumerate(gs):
            if x > t:
                return i - 1 if i >= 1 else None
        return None

    def _tokens(self, t):
        """(table start, token) of every visible token of query t, in order."""
        out = []
        g = self.group_of(t)
        spans = []
        if g is not None:
            spans.append((int(self.poff[g]), range(max(int(self.prefixes[g]), 0))))
        n = max(int(self.lens[t]), 0)
        if self.ids is None:
            own = range(n)
        else:
            blocks = sorted({b for b in self.ids[t].tolist() if 0 <= b < -(-n // self.block)})
            own = [j for b in blocks for j in range(b * self.block, min(n, (b + 1) * self.block))]
        spans.append((int(self.toff[t]), own))
        flat = self.table.reshape(-1)
        for off, js in spans:
            js = torch.as_tensor(list(js), dtype=torch.int64)
            if js.numel() == 0:
                continue
            i = off + js // self.page
            ok = (i >= 0) & (i < flat.numel())
            pg = torch.where(ok, flat[i.clamp(0, flat.numel() - 1)].long(), torch.tensor(-1))
            ok = (pg >= 0) & (pg < self.pages)
            out.append(torch.stack([pg[ok], (js % self.page)[ok]]))
        return torch.cat(out, 1) if out else torch.zeros(2, 0, dtype=torch.int64)

    def reference(self):
        """(out, lse, out tolerance, lse tolerance) in float64."""
        hq, hkv, d = self.hq, self.hkv, self.d
        G = hq // hkv
        out = torch.zeros(self.T, hq, d, dtype=torch.float64)
        lse = torch.full((self.T, hq), -np.inf, dtype=torch.float64)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        e8 = self.kd == "e4m3"
        for t in range(self.T):
            pg, row = self._tokens(t)
            if pg.numel() == 0:
                continue
            k = self._raw(self.k)[pg, :, row].view(self._dt(self.kd)).double()     # [L, Hkv, D]
            v = self._raw(self.v)[pg, :, row].view(self._dt(self.vd)).double()
            for c in range(hkv):
                ks = float(self.scales[c if self.per_head else 0]) if self.kd == "e4m3" else 1.0
                vs = float(self.scales[hkv + c if self.per_head else 1]) if self.vd == "e4m3" else 1.0
                q = self.q[t, c * G:(c + 1) * G].double()
                kc, vc = k[:, c] * ks, v[:, c] * vs
                s = q @ kc.T * self.softmax_scale
                mag = (q.abs() @ kc.abs().T).amax(1) * self.softmax_scale
                ds = mag * 2.0 ** -16
                if e8 or self.vd == "e4m3":
                    ds = ds + self.softmax_scale * 2.0 ** -17 * q.abs().max() * kc.abs().sum(1).max()
                m = s.amax(1, keepdim=True)
                p = torch.exp(s - m)
                l = p.sum(1, keepdim=True)
                o = p @ vc / l
                mean = p @ vc.abs() / l
                floor = vc.abs().sum(0)[None] / l * (2.0 ** -14 if self.vd == "e4m3" else 0.0)
                hs = slice(c * G, (c + 1) * G)
                out[t, hs] = o
                lse[t, hs] = (m + l.log())[:, 0]
                tol[t, hs] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * ds[:, None]) * mean + floor
                ltol[t, hs] = ds + 2.0 ** -20 * (1 + lse[t, hs].abs())
        return out, lse, tol, ltol

    # -- the call ----------------------------------------------------------
    def cfg(self):
        return B.make_attention_cfg(self.hq, self.hkv, self.d, self.page, self.block, self.topk, self.softmax_scale,
                                    B.MSA_SCALE_PER_HEAD if self.per_head else B.MSA_SCALE_PER_TENSOR)

    def device(self, dev="cuda"):
        return Device(self, dev)


class Device:
    """A problem's buffers on the GPU; ``run`` makes the call into fresh outputs."""

    def __init__(self, p, dev):
        self.p, self.cfg = p, p.cfg()
        self.kpool = p.kpool.to(dev)
        self.vpool = self.kpool if p.vpool is p.kpool else p.vpool.to(dev)

        def desc(pool, view):
            dt = B.MSA_DTYPE_FP8_E4M3 if view.dtype == torch.float8_e4m3fn else B.MSA_DTYPE_BF16
            return B.make_cache(pool.data_ptr() + view.storage_offset() * view.element_size(), dt, view.shape[0],
                                view.shape[1], view.stride(0), view.stride(1), view.stride(2))

        self.k, self.v = desc(self.kpool, p.k), desc(self.vpool, p.v)
        c = lambda t: None if t is None else t.to(dev)
        self.q, self.lens, self.toff, self.table = c(p.q), c(p.lens), c(p.toff), c(p.table.reshape(-1))
        self.ids, self.scales = c(p.ids), c(p.scales)
        self.groups = c(p.groups)
        self.prefixes, self.poff = (c(p.prefixes), c(p.poff)) if p.groups is not None else (None, None)
        self.out = torch.full((p.T, p.hq, p.d), float("nan"), dtype=torch.bfloat16, device=dev)
        self.lse = torch.full((p.T, p.hq), float("nan"), dtype=torch.float32, device=dev)
        n = B.msa_attention_workspace_bytes(self.cfg, p.T, 0 if p.groups is None else len(p.prefixes))
        self.ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=dev)   # NaN to start with

    def run(self, flags=0, stream=None, lse=True):
        l = self.lse if lse else None
        if self.ids is not None:
            B.sparse_attention_tensors(self.cfg, self.q, self.ids, self.lens, self.toff, self.table, self.k, self.v,
                                       self.scales, self.out, l, self.ws, flags, stream)
        else:
            B.prefix_attention_tensors(self.cfg, self.q, self.groups, self.prefixes, self.poff, self.lens, self.toff,
                                       self.table, self.k, self.v, self.scales, self.out, l, self.ws, flags, stream)
        return self

    def check(self, ref=None):
        out, lse, tol, ltol = ref if ref is not None else self.p.reference()
        o, s = self.out.double().cpu(), self.lse.double().cpu()
        assert torch.isfinite(o).all(), f"{int((~torch.isfinite(o)).sum())} outputs are not finite"
        bad = (o - out).abs() > tol
        assert not bad.any(), (f"out: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, "
                               f"worst {float(((o - out).abs() / tol.clamp_min(1e-30)).max()):.2f} of the tolerance")
        empty = torch.isinf(lse)
        assert torch.equal(empty, torch.isneginf(s)), "lse: -inf pattern"
        assert ((s - lse).abs()[~empty] <= ltol[~empty]).all(), "lse"
        return self

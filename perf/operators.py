"""The attention operators over the paged K/V caches, as cases to measure.

Two operators read the caches that the producer writes:

* sparse: each query attends the tokens of the blocks that the indexer selected for it
  (``topk_ids``), at most its own ``kv_len`` tokens of history;
* prefix: groups of queries attend a prefix that the group shares, then each its own tokens.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or with
``own`` set by the framework's kernels.  Outputs are (out, lse): bf16 [T, Hq, D], fp32 [T, Hq].
"""
import math

import torch

own = False

K_SCALE, V_SCALE = 0.05, 0.04      # dequantisation scales of the E4M3 caches
HEADS = {"big": (64, 8, 128), "tiny": (8, 2, 64), "wide": (32, 2, 128)}   # Hq, Hkv, D


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _sparse(**kw):
    d = dict(op="sparse", heads="big", dtype="e4m3", page=64, pad=0, topk=16, block=128, mode="decode",
             queries=1, lo=1, hi=8192, seqs=1, noise=0.3)
    d.update(kw)
    return d


def _prefix(**kw):
    d = dict(op="prefix", heads="big", dtype="e4m3", page=64, pad=0, queries=64, groups=1, prefix=8192,
             lo=1, hi=1024)
    d.update(kw)
    return d


def listed():
    return [
        # one sequence being decoded alone: latency counts
        _sparse(name="sparse_decode_1", queries=1, lo=8192, hi=8192),
        # the decode-batch-64 layer of the producer: contexts 1..9216, pages padded by 256 bytes
        _sparse(name="sparse_decode_64", queries=64, lo=1, hi=9216, pad=256),
        # the small-shape decode step, 256 sequences below 512 tokens
        _sparse(name="sparse_decode_256_tiny", heads="tiny", queries=256, lo=1, hi=512, topk=4),
        # bf16 caches, an odd batch, longer histories, groups of 16 heads
        _sparse(name="sparse_decode_37_bf16", heads="wide", dtype="bf16", queries=37, lo=2000, hi=16384),
        # one short prefill chunk of odd length after a history
        _sparse(name="sparse_prefill_333", mode="prefill", queries=333, seqs=1, hi=4500),
        # a chunked-prefill batch: 4 chunks of 2048 queries, the last of 8192-token prompts
        _sparse(name="sparse_prefill_4x2048", mode="prefill", queries=8192, seqs=4, hi=8192),
        # whole prompts, 2 of 8192 tokens
        _sparse(name="sparse_prefill_2x8192", mode="prefill", queries=16384, seqs=2, hi=8192),
        # bf16 caches, neighbouring queries that agree less on their blocks
        _sparse(name="sparse_prefill_4x1024_bf16", mode="prefill", dtype="bf16", queries=4096, seqs=4, hi=4096,
                noise=1.0),
        # three samples of one short prompt: latency counts
        _prefix(name="prefix_3x700", queries=3, prefix=700, lo=1, hi=60),
        # a batch of 64 requests behind one system prompt
        _prefix(name="prefix_64x8192", queries=64, prefix=8192, lo=1, hi=1024),
        # several prompts sampled many times each, bf16 caches, odd sizes
        _prefix(name="prefix_190_in_5_bf16", dtype="bf16", queries=190, groups=5, prefix=5001, lo=1, hi=777),
        # few requests over one long document
        _prefix(name="prefix_6x65536", queries=6, prefix=65536, lo=300, hi=2000, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, dtype = rng.choice(["big", "big", "tiny", "wide"]), rng.choice(["e4m3", "e4m3", "bf16"])
    page, pad = rng.choice([16, 32, 64, 64, 128]), rng.choice([0, 0, 256])
    kind = rng.randrange(3)
    if kind == 0:
        hi = _log(rng, 64, 16384)
        return _sparse(heads=heads, dtype=dtype, page=page, pad=pad, queries=_log(rng, 1, 128),
                       lo=rng.randint(1, hi), hi=hi, topk=rng.choice([4, 8, 16, 16, 20]))
    if kind == 1:
        seqs = rng.randint(1, 4)
        per = _log(rng, 40, 2048)
        return _sparse(heads=heads, dtype=dtype, page=page, pad=pad, mode="prefill", queries=seqs * per, seqs=seqs,
                       hi=max(per, _log(rng, 256, 8192)), noise=rng.choice([0.2, 0.3, 0.6, 1.0]))
    groups = rng.randint(1, 5)
    hi = _log(rng, 16, 1024)
    return _prefix(heads=heads, dtype=dtype, page=page, pad=pad, queries=groups + _log(rng, 2, 192), groups=groups,
                   prefix=_log(rng, 200, 16384), lo=rng.randint(1, hi), hi=hi)


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------

def _spread(n, lo, hi):
    """n lengths evenly over lo .. hi."""
    if n == 1:
        return [hi]
    return [lo + (i * (hi - lo)) // (n - 1) for i in range(n)]


def _sparse_lens(case):
    """(history of each sequence, [(sequence, visible tokens) of each query])"""
    if case["mode"] == "decode":
        lens = _spread(case["queries"], case["lo"], case["hi"])
        return lens, [(s, n) for s, n in enumerate(lens)]
    per = case["queries"] // case["seqs"]
    return [case["hi"]] * case["seqs"], [(s, case["hi"] - per + 1 + i) for s in range(case["seqs"])
                                         for i in range(per)]


def _selected(case, n):
    blk = case["block"]
    nb = -(-n // blk)
    return (min(case["topk"], nb) - 1) * blk + n - (nb - 1) * blk


def _group_sizes(case):
    g, t = case["groups"], case["queries"]
    w = [1 + (3 * i) % 5 for i in range(g)]
    sizes = [max(1, t * x // sum(w)) for x in w]
    sizes[-1] += t - sum(sizes)
    if sizes[-1] < 1:
        sizes = [t // g] * (g - 1) + [t - (g - 1) * (t // g)]
    return sizes


def _prefix_lens(case):
    g = case["groups"]
    return [max(1, case["prefix"] * (g + i) // (2 * g - 1)) if g > 1 else case["prefix"] for i in range(g)]


def work(case):
    hq, hkv, d = HEADS[case["heads"]]
    es = 1 if case["dtype"] == "e4m3" else 2
    t, page = case["queries"], case["page"]
    rows = t * hq * (2 * d + 2 * d + 4)                       # q, out, lse
    if case["op"] == "sparse":
        seqs, qs = _sparse_lens(case)
        sel = sum(_selected(case, n) for _, n in qs)
        kv = sel if case["mode"] == "decode" else min(sel, sum(seqs))   # chunks share their history
        meta = t * (4 + 8 + 4 * case["topk"]) + 4 * -(-kv // page)
        return {"bytes": rows + kv * hkv * d * 2 * es + meta, "flops": 4 * hq * d * sel}
    own_len = sum(_spread(t, case["lo"], case["hi"]))
    pre, sizes = _prefix_lens(case), _group_sizes(case)
    kv = own_len + sum(pre)
    dots = own_len + sum(a * b for a, b in zip(pre, sizes))
    return {"bytes": rows + kv * hkv * d * 2 * es + t * 12 + 4 * -(-kv // page), "flops": 4 * hq * d * dots}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pool(gen, case, pages):
    """A pool of `pages` HND pages, padded by case["pad"] bytes each, as a [pages, Hkv, P, D] view."""
    _, hkv, d = HEADS[case["heads"]]
    page = case["page"]
    es = 1 if case["dtype"] == "e4m3" else 2
    dt = torch.float8_e4m3fn if es == 1 else torch.bfloat16
    stride = hkv * page * d + case["pad"] // es
    pool = torch.empty(pages * stride, dtype=dt, device="cuda")
    step = 1 << 26
    for a in range(0, pool.numel(), step):
        x = torch.randn(min(step, pool.numel() - a), generator=gen, device="cuda")
        pool[a:a + step] = (x / K_SCALE).to(dt) if es == 1 else x.to(dt)
    return torch.as_strided(pool, (pages, hkv, page, d), (stride, page * d, d, 1))


def _tables(gen, case, lens):
    """A seeded permutation of the pages over rows of tokens: (flat table, row offsets, pages)."""
    need = [max(1, -(-n // case["page"])) for n in lens]
    width, total = max(need), sum(need)
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    n = torch.tensor(need, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < n[:, None]] = perm
    return table.reshape(-1), torch.arange(len(lens), device="cuda") * width, total


def _select(gen, case, qs):
    """Block ids as an indexer gives them: best first, padded with -1, the last block always among
    them; in a prefill the runs of 128 queries share most of their preferences."""
    blk, k, t = case["block"], case["topk"], len(qs)
    lens = torch.tensor([n for _, n in qs], device="cuda")
    nb = (lens + blk - 1) // blk
    width = max(int(nb.max()), k)
    score = torch.randn(t, width, generator=gen, device="cuda")
    if case["mode"] == "prefill":
        run = torch.tensor([s * 4096 + n // 128 for s, n in qs], device="cuda")
        _, run = torch.unique(run, return_inverse=True)
        base = torch.randn(int(run.max()) + 1, width, generator=gen, device="cuda")
        base[:, 0] += 3.0
        score = base[run] + case["noise"] * score
    col = torch.arange(width, device="cuda")[None, :]
    score[col == nb[:, None] - 1] += 100.0
    score[col >= nb[:, None]] = -math.inf
    val, ids = torch.topk(score, k, dim=1)
    ids[val == -math.inf] = -1
    return ids.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(7919 * seed + 13)
    hq, hkv, d = HEADS[case["heads"]]
    t = case["queries"]
    st = {"case": case}
    st["q"] = (1.5 * torch.randn(t, hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
    if case["op"] == "sparse":
        seqs, qs = _sparse_lens(case)
        if case["mode"] == "decode":   # lengths in no order
            order = torch.randperm(t, generator=gen, device="cuda").tolist()
            qs = [qs[i] for i in order]
        table, row, pages = _tables(gen, case, seqs)
        st["kv_len"] = torch.tensor([n for _, n in qs], dtype=torch.int32, device="cuda")
        st["table_offset"] = row[torch.tensor([s for s, _ in qs], device="cuda")].to(torch.int64)
        st["topk_ids"] = _select(gen, case, qs)
    else:
        own_len = _spread(t, case["lo"], case["hi"])
        order = torch.randperm(t, generator=gen, device="cuda").tolist()
        own_len = [own_len[i] for i in order]
        pre, sizes = _prefix_lens(case), _group_sizes(case)
        table, row, pages = _tables(gen, case, pre + own_len)
        starts = [0]
        for s in sizes:
            starts.append(starts[-1] + s)
        st["group_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["prefix_len"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
        st["prefix_offset"] = row[:len(pre)].to(torch.int64).contiguous()
        st["kv_len"] = torch.tensor(own_len, dtype=torch.int32, device="cuda")
        st["table_offset"] = row[len(pre):].to(torch.int64).contiguous()
        # what the plain form loops over: a scheduler has these on the host
        st["host"] = (starts, pre, own_len)
    st["page_table"] = table
    st["k"], st["v"] = _pool(gen, case, pages), _pool(gen, case, pages)
    st["scales"] = torch.tensor([K_SCALE, V_SCALE, 1.0], device="cuda")
    if own:
        from paged_kv_cache_msa_gb300 import binding as B
        st["B"] = B
        st["cfg"] = B.make_attention_cfg(hq, hkv, d, page_size=case["page"],
                                         block_tokens=case.get("block", 128), topk=case.get("topk", 16))
        st["k_desc"], st["v_desc"] = B.cache_from_tensor(st["k"]), B.cache_from_tensor(st["v"])
        st["out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(t, hq, dtype=torch.float32, device="cuda")
        nbytes = B.msa_attention_workspace_bytes(st["cfg"], t, case.get("groups", 0))
        st["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _rows(pool, page, off, scale):
    """Cache rows as fp32 [..., Hkv, D] for pages and in-page offsets of any shape."""
    if pool.dtype == torch.bfloat16:
        return pool[page, :, off].float()
    return pool.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float() * scale


def _attend(q, k, v, mask):
    """q [n, Hq, D]; k, v [n, L, Hkv, D] (or n = 1: shared); mask [n, L] or None."""
    n, hq, d = q.shape
    hkv = k.shape[2]
    qg = q.float().reshape(n, hkv, hq // hkv, d)
    if k.shape[0] == 1 and n > 1:
        a = qg.transpose(0, 1).reshape(1, hkv, -1, d) @ k.permute(0, 2, 3, 1)
        s = a.reshape(hkv, n, hq // hkv, -1).transpose(0, 1) / math.sqrt(d)
    else:
        s = qg @ k.permute(0, 2, 3, 1) / math.sqrt(d)
    if mask is not None:
        s = s.masked_fill(~mask[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    if v.shape[0] == 1 and n > 1:
        o = (p.transpose(0, 1).reshape(1, hkv, -1, p.shape[-1]) @ v.permute(0, 2, 1, 3))
        o = o.reshape(hkv, n, hq // hkv, d).transpose(0, 1)
    else:
        o = p @ v.permute(0, 2, 1, 3)
    return o, m, l


def _finish(o, m, l):
    n, hkv, g, d = o.shape
    out = o / torch.where(l == 0, torch.ones_like(l), l)
    return out.reshape(n, hkv * g, d), (m + torch.log(l)).reshape(n, hkv * g)


def _plain_sparse(st):
    case = st["case"]
    blk, page = case["block"], case["page"]
    t, hq, d = st["q"].shape
    hkv = HEADS[case["heads"]][1]
    out, lse = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hq, device="cuda")
    step = max(1, (1 << 28) // (case["topk"] * blk * hkv * d))
    within = torch.arange(blk, device="cuda")
    for a in range(0, t, step):
        sl = slice(a, min(t, a + step))
        ids = st["topk_ids"][sl].long()
        tok = (ids[:, :, None] * blk + within).reshape(ids.shape[0], -1)
        ok = (tok >= 0) & (tok < st["kv_len"][sl, None])
        tok = torch.where(ok, tok, torch.zeros_like(tok))
        pg = st["page_table"][st["table_offset"][sl, None] + tok // page].long()
        k, v = _rows(st["k"], pg, tok % page, K_SCALE), _rows(st["v"], pg, tok % page, V_SCALE)
        o, s = _finish(*_attend(st["q"][sl], k, v, ok))
        out[sl], lse[sl] = o.to(torch.bfloat16), s
    return out, lse


def _plain_prefix(st):
    case = st["case"]
    page = case["page"]
    t, hq, d = st["q"].shape
    hkv = HEADS[case["heads"]][1]
    starts, pre, own_len = st["host"]
    out, lse = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hq, device="cuda")
    for g, n in enumerate(pre):
        tok = torch.arange(n, device="cuda")
        pg = st["page_table"][st["prefix_offset"][g] + tok // page].long()
        kp = _rows(st["k"], pg, tok % page, K_SCALE)[None]
        vp = _rows(st["v"], pg, tok % page, V_SCALE)[None]
        step = max(1, min((1 << 28) // (max(own_len) * hkv * d), (1 << 29) // (n * hq)))
        for a in range(starts[g], starts[g + 1], step):
            sl = slice(a, min(starts[g + 1], a + step))
            tok = torch.arange(max(own_len[sl]), device="cuda")[None, :].expand(sl.stop - a, -1)
            ok = tok < st["kv_len"][sl, None]
            tok = torch.where(ok, tok, torch.zeros_like(tok))
            pg = st["page_table"][st["table_offset"][sl, None] + tok // page].long()
            k, v = _rows(st["k"], pg, tok % page, K_SCALE), _rows(st["v"], pg, tok % page, V_SCALE)
            o1, m1, l1 = _attend(st["q"][sl], kp, vp, None)
            o2, m2, l2 = _attend(st["q"][sl], k, v, ok)
            m = torch.maximum(m1, m2)
            e1, e2 = torch.exp(m1 - m), torch.exp(m2 - m)
            o, s = _finish(o1 * e1 + o2 * e2, m, l1 * e1 + l2 * e2)
            out[sl], lse[sl] = o.to(torch.bfloat16), s
    return out, lse


def run(state):
    if not own:
        return _plain_sparse(state) if state["case"]["op"] == "sparse" else _plain_prefix(state)
    B, st = state["B"], state
    if st["case"]["op"] == "sparse":
        flags = B.MSA_LAUNCH_QUERY_RUNS if st["case"]["mode"] == "prefill" else 0
        B.sparse_attention_tensors(st["cfg"], st["q"], st["topk_ids"], st["kv_len"], st["table_offset"],
                                   st["page_table"], st["k_desc"], st["v_desc"], st["scales"], st["out"],
                                   lse=st["lse"], workspace=st["workspace"], launch_flags=flags)
    else:
        B.prefix_attention_tensors(st["cfg"], st["q"], st["group_start"], st["prefix_len"], st["prefix_offset"],
                                   st["kv_len"], st["table_offset"], st["page_table"], st["k_desc"],
                                   st["v_desc"], st["scales"], st["out"], lse=st["lse"],
                                   workspace=st["workspace"])
    return st["out"], st["lse"]


# ---------------------------------------------------------------------------
# the definition in 64 bits, one query at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv, d = HEADS[case["heads"]]
    page, t = case["page"], case["queries"]
    es8 = case["dtype"] == "e4m3"
    ks, vs = float(st["scales"][0]) if es8 else 1.0, float(st["scales"][1]) if es8 else 1.0
    table, kv_len, toff = st["page_table"].long(), st["kv_len"].tolist(), st["table_offset"].tolist()

    def gather(pool, base, tokens):
        pg = table[base + torch.div(tokens, page, rounding_mode="floor")]
        flat = pg * pool.stride(0) + (tokens % page) * pool.stride(2)
        idx = flat[:, None] + (torch.arange(hkv, device="cuda") * pool.stride(1))[None, :]
        raw = torch.as_strided(pool, ((pool.shape[0] - 1) * pool.stride(0) + hkv * page * d,), (1,))
        raw = raw.view(torch.uint8) if es8 else raw
        x = raw[idx[:, :, None] + torch.arange(d, device="cuda")]
        return (x.view(torch.float8_e4m3fn) if es8 else x).double().transpose(0, 1)     # [Hkv, L, D]

    prefix = {}
    if case["op"] == "prefix":
        starts, pre, _ = st["host"]
        for g, n in enumerate(pre):
            tokens = torch.arange(n, device="cuda")
            base = int(st["prefix_offset"][g])
            kv = gather(st["k"], base, tokens), gather(st["v"], base, tokens)
            for i in range(starts[g], starts[g + 1]):
                prefix[i] = kv
    out = torch.zeros(t, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(t, hq, dtype=torch.float64, device="cuda")
    ids = st["topk_ids"].tolist() if case["op"] == "sparse" else None
    for i in range(t):
        n = kv_len[i]
        if ids is None:
            tokens = torch.arange(n, device="cuda")
        else:
            starts_ = torch.tensor(sorted({b for b in ids[i] if b >= 0}), device="cuda") * case["block"]
            tokens = (starts_[:, None] + torch.arange(case["block"], device="cuda")).flatten()
            tokens = tokens[:tokens.numel() - max(0, int(max(ids[i])) * case["block"] + case["block"] - n)]
        k, v = gather(st["k"], toff[i], tokens), gather(st["v"], toff[i], tokens)
        if i in prefix:
            k, v = torch.cat([prefix[i][0], k], 1), torch.cat([prefix[i][1], v], 1)
        z = torch.bmm(st["q"][i].double().view(hkv, hq // hkv, d), k.transpose(1, 2)) * (ks / math.sqrt(d))
        lse[i] = torch.logsumexp(z, -1).flatten()
        out[i] = (torch.bmm(torch.softmax(z, -1), v) * vs).reshape(hq, d)
    return out, lse

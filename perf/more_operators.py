"""The operators on the input side of an MSA layer, as cases to measure.

Three operators, in the order in which a layer runs them around its packed projection:

* norm: RMSNorm of the hidden states with the residual's addition, and an output in E4M3 with one
  scale for each token (the projection's operand), in bf16, or both;
* adapters: low-rank adapters of many requests at once, added to the packed projection's rows
  [Q | K | V | index-Q | index-K], each section with a down-projection of its own;
* axes: the producer (per-head norm, rotation, paged cache write) with rotary positions of several
  axes (time, height, width).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, angles in
64), or with ``own`` set by the framework's kernels.
"""
import math

import torch

own = False

# query, K/V, index-query, index-key heads and head size of the packed row; hidden size
SHAPES = {"big": (64, 8, 8, 1, 128, 6144), "tiny": (8, 2, 2, 1, 64, 1000)}
SCALES = (0.05, 0.04, 0.06)          # dequantisation scales of the E4M3 caches: K, V, index-K
THETA = 5e6
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(**kw):
    d = dict(op="norm", tokens=64, hidden=6144, residual=True, out="e4m3", pad=0)
    d.update(kw)
    return d


def _adapters(**kw):
    d = dict(op="adapters", shape="big", dtype="bf16", tokens=64, adapters=8, rank=16, order="mixed")
    d.update(kw)
    return d


def _axes(**kw):
    d = dict(op="axes", shape="big", cache="e4m3", per_head=False, style="neox", rotary=128, layout="sections",
             tokens=64, page=64, pad=0, mode="prefill")
    d.update(kw)
    return d


def listed():
    return [
        # one sequence being decoded alone: latency counts
        _norm(name="norm_1", tokens=1),
        # the decode batch of 64; another consumer (a router, an adapter) reads the bf16 rows as well
        _norm(name="norm_64_both", tokens=64, out="both"),
        # the first norm of a model, no residual yet, rows that are not whole vectors
        _norm(name="norm_777_odd", tokens=777, hidden=1001, residual=False, out="bf16", pad=7),
        # a chunked-prefill batch of 4 x 2048 tokens
        _norm(name="norm_8192", tokens=8192),
        # one request with its adapter
        _adapters(name="adapters_1", tokens=1),
        # a decode batch of 64 requests over 48 adapters, some without any
        _adapters(name="adapters_64_in_48", tokens=64, adapters=48),
        # a short ragged prefill on the small shapes, tokens of several requests mixed
        _adapters(name="adapters_333_tiny", shape="tiny", tokens=333, adapters=5, rank=8),
        # a chunked-prefill batch: 4 chunks of 2048 tokens, each its own adapter or none, 8-bit hidden states
        _adapters(name="adapters_4x2048_e4m3", dtype="e4m3", tokens=8192, adapters=3, rank=32, order="runs"),
        # a step of text decoding behind images: all axes equal, far positions
        _axes(name="axes_decode_64", mode="decode", tokens=64, pad=256),
        # the small decode batch
        _axes(name="axes_decode_4_tiny", mode="decode", shape="tiny", rotary=64, tokens=4),
        # images in a prompt: bf16 caches, interleaved axes, half the dims rotated, odd length
        _axes(name="axes_1999_bf16", cache="bf16", tokens=1999, rotary=64, layout="interleaved", style="gptj"),
        # video prefill: 16,384 tokens of frames, frequencies that restart in each axis, scales per head
        _axes(name="axes_16384", tokens=16384, layout="restart", per_head=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.randrange(3)
    if kind == 0:
        return _norm(tokens=_log(rng, 1, 8192), hidden=_log(rng, 64, 8192), residual=rng.random() < 0.7,
                     out=rng.choice(["e4m3", "e4m3", "bf16", "both"]), pad=rng.choice([0, 0, 5, 16]))
    if kind == 1:
        order = rng.choice(["mixed", "runs"])
        return _adapters(shape=rng.choice(["big", "big", "tiny"]), dtype=rng.choice(["bf16", "e4m3"]),
                         tokens=_log(rng, 1, 6000 if order == "runs" else 512), adapters=_log(rng, 1, 48),
                         rank=rng.choice([8, 16, 16, 32, 64]), order=order)
    shape = rng.choice(["big", "big", "tiny"])
    d = SHAPES[shape][4]
    return _axes(shape=shape, cache=rng.choice(["e4m3", "e4m3", "bf16"]), per_head=rng.random() < 0.3,
                 style=rng.choice(["neox", "neox", "gptj"]), rotary=rng.choice([d, d // 2]),
                 layout=rng.choice(["sections", "interleaved", "restart"]), tokens=_log(rng, 1, 8192),
                 page=rng.choice([16, 64, 128]), pad=rng.choice([0, 256]), mode=rng.choice(["decode", "prefill"]))


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------

def _sections(shape):
    """Heads of Q, K, V, index-Q, index-K, the head size, the hidden size."""
    hq, hkv, hiq, hik, d, k = SHAPES[shape]
    return [hq, hkv, hkv, hiq, hik], d, k


def _ends(shape):
    heads, d, _ = _sections(shape)
    return [sum(heads[:i + 1]) * d for i in range(len(heads))]


def _axis_pairs(case):
    """How many of the rotary pairs turn with time, height and width."""
    half = case["rotary"] // 2
    t = half // 4
    h = (half - t + 1) // 2
    return t, h, half - t - h


def _adapter_of(case):
    """The adapter of each token, -1 without one."""
    n, t = case["adapters"], case["tokens"]
    if case["order"] == "runs":                 # one more request than adapters, without one
        return [(i * (n + 1)) // t - 1 if n > 1 else 0 for i in range(t)]
    return [(7 * i) % n if i % 9 != 8 else -1 for i in range(t)]


def work(case):
    t = case["tokens"]
    if case["op"] == "norm":
        k = case["hidden"]
        b = 2 * t * k * (3 if case["residual"] else 1) + 2 * k
        b += t * k * {"e4m3": 1, "bf16": 2, "both": 3}[case["out"]] + (0 if case["out"] == "bf16" else 4 * t)
        return {"bytes": b, "flops": 6 * t * k}
    heads, d, k = _sections(case["shape"])
    w = sum(heads) * d
    if case["op"] == "adapters":
        ids = _adapter_of(case)
        used, on, r = len({a for a in ids if a >= 0}), sum(a >= 0 for a in ids), case["rank"]
        b = used * 2 * r * (len(heads) * k + w) + t * (4 + 4 * w) + on * k * (2 if case["dtype"] == "bf16" else 1)
        return {"bytes": b, "flops": 2 * on * r * (len(heads) * k + w)}
    es = 1 if case["cache"] == "e4m3" else 2
    live = sum(1 for i in range(t) if i % 61 != 60)
    b = t * (2 * w + 3 * 4 + 8 + 4) + 2 * t * d * (heads[0] + heads[3]) + live * d * es * (heads[1] + heads[2] + heads[4])
    return {"bytes": b, "flops": 10 * t * w}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _padded(x, pad):
    """The same rows, a multiple of 16 elements and `pad` whole vectors of 16 apart."""
    t, k = x.shape
    wide = torch.zeros(t, -(-k // 16) * 16 + 16 * pad, dtype=x.dtype, device="cuda")
    wide[:, :k] = x
    return wide[:, :k]


def _stream(gen, t, k):
    """Hidden states: a few strong channels among ordinary ones."""
    x = torch.randn(t, k, generator=gen, device="cuda")
    return (x * torch.where(torch.arange(k, device="cuda") % 97 == 13, 20.0, 1.0)).to(torch.bfloat16)


def _prepare_norm(case, gen):
    t, k = case["tokens"], case["hidden"]
    st = {"x": _padded(_stream(gen, t, k), case["pad"]),
          "weight": (0.5 + torch.rand(k, generator=gen, device="cuda")).to(torch.bfloat16), "residual": None}
    if case["residual"]:
        st["residual"] = _padded(3 * _stream(gen, t, k), case["pad"])
    empty = torch.empty(t, k, dtype=torch.bfloat16, device="cuda")
    st["residual_out"] = _padded(empty, case["pad"]) if case["residual"] else None
    st["out"] = _padded(empty, case["pad"]) if case["out"] != "e4m3" else None
    st["codes"] = _padded(empty.to(torch.float8_e4m3fn), case["pad"]) if case["out"] != "bf16" else None
    st["scales"] = torch.empty(t, device="cuda") if case["out"] != "bf16" else None
    return st


def _prepare_adapters(case, gen):
    heads, d, k = _sections(case["shape"])
    t, n, r, w, s = case["tokens"], case["adapters"], case["rank"], sum(heads) * d, len(heads)
    x = _padded(_stream(gen, t, k), 0)
    st = {"hidden": x, "hidden_scales": None}
    if case["dtype"] == "e4m3":
        scales = x.float().abs().amax(1) / 448
        st["hidden_scales"] = scales
        st["hidden"] = _padded((x.float() / scales[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), 0)
    st["down"] = (torch.randn(n, s * r, k, generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
    st["up"] = (0.3 * torch.randn(n, w, r, generator=gen, device="cuda")).to(torch.bfloat16)
    st["ids"] = torch.tensor(_adapter_of(case), dtype=torch.int32, device="cuda")
    st["alpha"] = 0.5 + torch.rand(n, generator=gen, device="cuda")
    st["rows"] = torch.randn(t, w, generator=gen, device="cuda").to(torch.bfloat16)
    st["out"] = torch.empty_like(st["rows"])
    return st


def _positions(case, gen):
    """Positions [3, T]: in decoding all axes equal and far; in a prefill runs of text and grids of
    patches by turns, whose tokens share a time (images) or a time for each frame."""
    t = case["tokens"]
    if case["mode"] == "decode":
        p = torch.randint(0, 200000, (t,), generator=gen, device="cuda")
        return p.expand(3, t).to(torch.int32).contiguous()
    i = torch.arange(t, device="cuda")
    start = int(torch.randint(0, 50000, (1,), generator=gen, device="cuda"))
    run, at = i // 600, i % 600
    base = start + 150 * run
    grid = torch.stack([at // 200, (at % 200) // 20, at % 20])
    return torch.where(run % 2 == 1, base + grid, base + at).to(torch.int32).contiguous()


def _pool(case, pages, heads, d):
    """A zeroed pool of HND pages, padded by case["pad"] bytes each, as [pages, heads, P, D]."""
    dt, es = (torch.float8_e4m3fn, 1) if case["cache"] == "e4m3" else (torch.bfloat16, 2)
    stride = heads * case["page"] * d + case["pad"] // es
    pool = torch.zeros(pages * stride, dtype=dt, device="cuda")
    return torch.as_strided(pool, (pages, heads, case["page"], d), (stride, case["page"] * d, d, 1))


def _prepare_axes(case, gen):
    heads, d, _ = _sections(case["shape"])
    hq, hkv, _, hiq, hik = heads
    t, page, w = case["tokens"], case["page"], sum(heads) * d
    st = {"rows": _stream(gen, t, w), "positions": _positions(case, gen)}
    if case["mode"] == "decode":               # each token in a page of its own, somewhere in it
        pages = t
        block = torch.arange(t, device="cuda")
        off = torch.randint(0, page, (t,), generator=gen, device="cuda")
    else:
        pages = -(-t // page)
        i = torch.arange(t, device="cuda")
        block, off = i // page, i % page
    slots = block * page + off
    slots[torch.arange(t, device="cuda") % 61 == 60] = -1          # padded tokens
    st["slots"] = slots
    st["table"] = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    st["weights"] = [(0.5 + torch.rand(d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(4)]
    ns = [hkv, hkv, hik] if case["per_head"] else [1, 1, 1]
    st["scales"] = torch.cat([x * (1 + 0.5 * torch.rand(n, generator=gen, device="cuda")) for x, n in zip(SCALES, ns)])
    st["k"], st["v"], st["idx_k"] = (_pool(case, pages, n, d) for n in (hkv, hkv, hik))
    st["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
    st["idx_q_out"] = torch.empty(t, hiq, d, dtype=torch.bfloat16, device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(104729 * seed + 7)
    st = {"norm": _prepare_norm, "adapters": _prepare_adapters, "axes": _prepare_axes}[case["op"]](case, gen)
    st["case"] = case
    if own:
        # the handles and workspaces that a program makes once for a layer
        from paged_kv_cache_msa_gb300 import binding as B
        st["B"] = B
        if case["op"] == "norm":
            st["cfg"] = B.make_norm_cfg(case["hidden"], rms_eps=EPS)
        elif case["op"] == "adapters":
            _, _, k = _sections(case["shape"])
            st["cfg"] = B.make_adapter_cfg(k, _ends(case["shape"]), case["rank"], case["adapters"],
                                           hidden_dtype=B.MSA_DTYPE_BF16 if case["dtype"] == "bf16"
                                           else B.MSA_DTYPE_FP8_E4M3)
            st["workspace"] = torch.empty(B.msa_adapter_workspace_bytes(st["cfg"], case["tokens"]),
                                          dtype=torch.uint8, device="cuda")
        else:
            heads, d, _ = _sections(case["shape"])
            style = B.MSA_ROPE_NEOX if case["style"] == "neox" else B.MSA_ROPE_GPTJ
            st["cfg"] = B.make_cfg(heads[0], heads[1], heads[3], heads[4], d, case["rotary"], style, case["page"],
                                   THETA, EPS, B.MSA_SCALE_PER_HEAD if case["per_head"] else B.MSA_SCALE_PER_TENSOR)
            st["axes"] = B.make_rope_axes(_axis_pairs(case), interleaved=case["layout"] == "interleaved",
                                          restart=case["layout"] == "restart")
            st["descs"] = [B.cache_from_tensor(st[x]) for x in ("k", "v", "idx_k")]
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_norm(st):
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
        st["residual_out"].copy_(h)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["weight"].float()
    if st["out"] is not None:
        st["out"].copy_(y)
    if st["codes"] is not None:
        scales = y.abs().amax(1).clamp(min=2.0 ** -100) / 448
        st["scales"].copy_(scales)
        st["codes"].copy_((y / scales[:, None]).clamp(-448, 448))


def _plain_adapters(st):
    case = st["case"]
    heads, d, k = _sections(case["shape"])
    t, n, r, s = case["tokens"], case["adapters"], case["rank"], len(heads)
    x = st["hidden"].float()
    if st["hidden_scales"] is not None:
        x = x * st["hidden_scales"][:, None]
    on = torch.arange(n, device="cuda") == st["ids"].long()[:, None]                 # [T, n]
    u = (x @ st["down"].float().reshape(n * s * r, k).T).reshape(t, n, s, r)
    u = torch.where(on[:, :, None, None], u * st["alpha"][:, None, None], torch.zeros_like(u))
    owner = torch.repeat_interleave(torch.arange(s, device="cuda"), torch.tensor(heads, device="cuda") * d)
    up = st["up"].float()                                                            # [n, W, r]
    up = torch.where((owner[:, None] == torch.arange(s, device="cuda"))[None, :, :, None], up[:, :, None, :],
                     torch.zeros((), device="cuda"))                                 # [n, W, s, r]
    out = torch.einsum("tk,kw->tw", u.reshape(t, -1), up.permute(0, 2, 3, 1).reshape(n * s * r, -1))
    st["out"].copy_(st["rows"].float() + out)


def _axis_of_pair(case):
    """The axis of each rotary pair, and its place among the pairs of that axis."""
    counts = _axis_pairs(case)
    if case["layout"] == "interleaved":       # t h w t h w ..., an axis that is used up falling out
        axis, left = [], list(counts)
        while sum(left):
            for a in range(3):
                if left[a]:
                    axis.append(a)
                    left[a] -= 1
    else:
        axis = [a for a in range(3) for _ in range(counts[a])]
    return axis, [axis[:i].count(a) for i, a in enumerate(axis)], counts


def _frequencies(case):
    axis, place, counts = _axis_of_pair(case)
    if case["layout"] == "restart":
        return [THETA ** (-place[i] / counts[a]) for i, a in enumerate(axis)]
    return [THETA ** (-i / len(axis)) for i in range(len(axis))]


def _plain_axes(st):
    case = st["case"]
    heads, d, _ = _sections(case["shape"])
    t, rd, page = case["tokens"], case["rotary"], case["page"]
    axis = torch.tensor(_axis_of_pair(case)[0], device="cuda")
    angle = st["positions"].double()[axis] * torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")[:, None]
    cos, sin = (f(angle).float().T[:, None, :] for f in (torch.cos, torch.sin))      # [T, 1, rd/2]

    def normed(x, w):
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = (x[..., :rd // 2], x[..., rd // 2:rd]) if case["style"] == "neox" else (x[..., 0:rd:2], x[..., 1:rd:2])
        a, b = a * cos - b * sin, b * cos + a * sin
        rot = torch.cat([a, b], -1) if case["style"] == "neox" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([rot, x[..., rd:]], -1)

    q, k, v, iq, ik = st["rows"].reshape(t, -1, d).float().split(heads, 1)
    wq, wk, wiq, wik = st["weights"]
    st["q_out"].copy_(normed(q, wq))
    st["idx_q_out"].copy_(normed(iq, wiq))
    live = st["slots"] >= 0
    slot = st["slots"][live]
    pg, off = st["table"][slot // page].long(), slot % page
    counts = (heads[1], heads[1], heads[4]) if case["per_head"] else (1, 1, 1)
    for name, x, s in zip(("k", "v", "idx_k"), (normed(k, wk), v, normed(ik, wik)), st["scales"].split(counts)):
        if case["cache"] == "e4m3":
            code = (x[live] / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            st[name].view(torch.uint8)[pg, :, off] = code.view(torch.uint8)
        else:
            st[name][pg, :, off] = x[live].to(torch.bfloat16)


def _outputs(st):
    if st["case"]["op"] == "norm":
        return {n: st[n] for n in ("residual_out", "out", "codes", "scales")}
    if st["case"]["op"] == "adapters":
        return {"out": st["out"]}
    return {n: st[n] for n in ("q_out", "idx_q_out", "k", "v", "idx_k")}


def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        {"norm": _plain_norm, "adapters": _plain_adapters, "axes": _plain_axes}[op](st)
    elif op == "norm":
        st["B"].norm_tensors(st["cfg"], st["x"], st["weight"], residual=st["residual"],
                             residual_out=st["residual_out"], out=st["out"], codes=st["codes"], scales=st["scales"])
    elif op == "adapters":
        st["B"].adapter_tensors(st["cfg"], st["hidden"], st["down"], st["up"], st["ids"], st["rows"], st["out"],
                                hidden_scales=st["hidden_scales"], adapter_scales=st["alpha"],
                                workspace=st["workspace"])
    else:
        st["B"].forward_axes_tensors(st["cfg"], st["axes"], st["rows"], st["positions"], st["slots"], st["table"],
                                     st["weights"], st["q_out"], st["idx_q_out"], *st["descs"], st["scales"],
                                     launch_flags=st["B"].MSA_LAUNCH_PERSISTENT)
    return _outputs(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(st):
    h = st["x"].double() if st["residual"] is None else st["x"].double() + st["residual"].double()
    rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / h.shape[1] + EPS)
    y = st["weight"].double() * (h / rms[:, None])
    big = torch.maximum(y.max(1).values, -y.min(1).values) / 448
    return {"residual_out": h if st["residual"] is not None else None, "out": y if st["out"] is not None else None,
            "codes": y / big[:, None] if st["codes"] is not None else None,
            "scales": big if st["scales"] is not None else None}


def _exact_adapters(st):
    case = st["case"]
    r, ids, starts = case["rank"], st["ids"].tolist(), [0] + _ends(case["shape"])
    out = st["rows"].double()
    for a in sorted(set(ids) - {-1}):
        tok = torch.tensor([i for i, b in enumerate(ids) if b == a], device="cuda")
        x = st["hidden"][tok].to(torch.float64)
        if st["hidden_scales"] is not None:
            x = x * st["hidden_scales"].double()[tok, None]
        for s in range(len(starts) - 1):
            u = x @ st["down"][a, s * r:(s + 1) * r].double().T
            out[tok, starts[s]:starts[s + 1]] += float(st["alpha"][a]) * (u @ st["up"][a, starts[s]:starts[s + 1]].double().T)
    return {"out": out}


def _exact_axes(st):
    case = st["case"]
    heads, d, _ = _sections(case["shape"])
    page, half = case["page"], case["rotary"] // 2
    axis, place, counts = _axis_of_pair(case)
    turn = torch.empty(case["tokens"], half, dtype=torch.complex128, device="cuda")
    for i, a in enumerate(axis):
        power = place[i] / counts[a] if case["layout"] == "restart" else i / half
        turn[:, i] = torch.polar(torch.ones(case["tokens"], dtype=torch.float64, device="cuda"),
                                 st["positions"][a].double() / THETA ** power)
    parts, at = [], 0
    for sec, n in enumerate(heads):
        x = st["rows"][:, at:at + n * d].double().reshape(-1, n, d)
        at += n * d
        if sec != 2:
            w = st["weights"][[0, 1, None, 2, 3][sec]].double()
            x = w * x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
            if case["style"] == "neox":
                z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn[:, None]
                x[..., :half], x[..., half:2 * half] = z.real, z.imag
            else:
                z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:2], half, 2).contiguous()) * turn[:, None]
                x[..., :2 * half] = torch.view_as_real(z).flatten(-2)
        parts.append(x)
    out = {"q_out": parts[0], "idx_q_out": parts[3]}
    slots = st["slots"]
    tok = torch.nonzero(slots >= 0).flatten()
    pages, rows = st["table"].long()[torch.div(slots[tok], page, rounding_mode="floor")], slots[tok] % page
    first = 0
    for name, x in (("k", parts[1]), ("v", parts[2]), ("idx_k", parts[4])):
        pool = torch.zeros(st[name].shape, dtype=torch.float64, device="cuda")
        n = x.shape[1] if case["per_head"] else 1
        for h in range(x.shape[1]):
            scale = float(st["scales"][first + (h if n > 1 else 0)]) if case["cache"] == "e4m3" else 1.0
            pool[pages, h, rows] = (x[tok, h] / scale).clamp(-448, 448) if case["cache"] == "e4m3" else x[tok, h]
        first += n
        out[name] = pool
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "adapters": _exact_adapters, "axes": _exact_axes}[case["op"]](st)

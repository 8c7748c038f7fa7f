"""Device-resident buffers for a workload, and the C-ABI call on them.

``DeviceWorkload`` copies a ``workloads.Workload`` (rows, positions, slots, page
table, weights, scales and sentinel-filled cache pools) into CUDA memory with
torch, builds the cache descriptors, and calls ``msa_producer_forward`` through
the binding.  torch is used for memory and streams only.
"""
from __future__ import annotations

import numpy as np

from . import binding as B
from . import workloads as wl


def _t(a: np.ndarray, device):
    import torch
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


class DeviceWorkload:
    def __init__(self, w: wl.Workload, device="cuda", host_pools: dict | None = None,
                 pools_on_device: dict | None = None):
        import torch
        self.w = w
        self.device = torch.device(device)
        s = w.shape
        self.cfg = B.make_cfg(s["num_q_heads"], s["num_kv_heads"], s["num_idx_q_heads"],
                              s["num_idx_k_heads"], s["head_dim"], s["rotary_dim"], s["rope_style"],
                              s["page_size"], s["rope_theta"], s["rms_eps"], s.get("scale_mode", 0))
        self.qkv = _t(w.qkv, self.device)
        self.positions = _t(w.positions, self.device)
        self.slots = _t(w.slot_mapping, self.device)
        self.page_table = None if w.page_table is None else _t(w.page_table.reshape(-1), self.device)
        self.weights = {k: (None if v is None else _t(v, self.device)) for k, v in w.weights.items()}
        self.scales = _t(w.scales, self.device)
        T, D = w.num_tokens, s["head_dim"]
        self.q_out = torch.zeros((T, s["num_q_heads"], D), dtype=torch.int16, device=self.device)
        self.idx_q_out = torch.zeros((T, s["num_idx_q_heads"], D), dtype=torch.int16,
                                     device=self.device)
        if pools_on_device is not None:
            self.pools = pools_on_device
        else:
            if host_pools is None:
                host_pools = wl.host_pools(w)
            self.pools = {k: _t(v, self.device) for k, v in host_pools.items()}
        self.caches = {}
        for key in ("k", "v", "idx_k"):
            c = w.caches.get(key)
            self.caches[key] = None if c is None else B.make_cache(
                self.pools[c.pool].data_ptr() + c.offset, c.dtype, c.num_pages, c.num_heads,
                c.stride_page, c.stride_head, c.stride_token)

    def args(self, launch_flags=0, num_tokens=None, qkv_ptr=None):
        """Positional arguments of msa_producer_forward minus the stream."""
        w = self.w
        p = lambda t: None if t is None else int(t.data_ptr())
        T = w.num_tokens if num_tokens is None else int(num_tokens)
        return (self.cfg, T, p(self.qkv) if qkv_ptr is None else qkv_ptr, w.row_stride,
                p(self.positions), p(self.slots), p(self.page_table),
                0 if self.page_table is None else self.page_table.numel(),
                p(self.weights.get("q")), p(self.weights.get("k")), p(self.weights.get("idx_q")),
                p(self.weights.get("idx_k")), p(self.q_out), p(self.idx_q_out),
                self.caches["k"], self.caches["v"], self.caches["idx_k"], p(self.scales),
                launch_flags)

    def run(self, launch_flags=0, stream=None, num_tokens=None):
        import torch
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        with B.on_device(self.device):
            return B.msa_producer_forward(*self.args(launch_flags, num_tokens), stream=stream.cuda_stream)

    def outputs_to_host(self):
        q = self.q_out.cpu().numpy().view(np.uint16)
        iq = self.idx_q_out.cpu().numpy().view(np.uint16)
        return q, iq

    def pools_to_host(self):
        return {k: v.cpu().numpy() for k, v in self.pools.items()}


class DeviceIndexer:
    """Device copies of an indexer workload (queries, lengths, table, the index-K
    history pool) and the C-ABI call on them."""

    def __init__(self, w: wl.IndexerWorkload, device="cuda", pool=None):
        import torch
        self.w = w
        self.device = torch.device(device)
        T, H, D = w.idx_q.shape
        self.cfg = B.make_indexer_cfg(H, D, w.page_size, w.block_tokens, w.topk, w.max_blocks)
        self.idx_q = _t(w.idx_q, self.device)
        self.kv_len = _t(w.kv_len, self.device)
        self.table_offset = _t(w.table_offset, self.device)
        self.page_table = _t(w.page_table.reshape(-1), self.device)
        self.pool = _t(w.pool_fill if pool is None else pool, self.device)
        self.k_scale = torch.tensor([w.k_scale], dtype=torch.float32, device=self.device)
        self.block_scores = torch.empty((T, w.max_blocks), dtype=torch.float32, device=self.device)
        self.topk_ids = torch.empty((T, w.topk), dtype=torch.int32, device=self.device)
        self.counters = torch.zeros((T,), dtype=torch.int32, device=self.device)
        c = w.cache
        self.cache = B.make_cache(self.pool.data_ptr() + c.offset, c.dtype, c.num_pages, 1,
                                  c.stride_page, c.stride_head, c.stride_token)

    def run(self, stream=None, launch_flags=0, fused=False):
        """msa_indexer_forward, or with ``fused`` msa_indexer_forward_fused on this
        indexer's zeroed per-query counters."""
        import torch
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        p = lambda t: int(t.data_ptr())
        args = (self.cfg, self.w.idx_q.shape[0], p(self.idx_q), p(self.kv_len),
                p(self.table_offset), p(self.page_table), self.page_table.numel(), self.cache,
                p(self.k_scale), p(self.block_scores), p(self.topk_ids))
        with B.on_device(self.device):
            if fused:
                return B.msa_indexer_forward_fused(*args, p(self.counters), launch_flags,
                                                   stream=stream.cuda_stream)
            return B.msa_indexer_forward(*args, launch_flags, stream=stream.cuda_stream)


class DeviceProjection:
    """Device copies of a projection workload: hidden states, the packed weight and,
    through a ``DeviceWorkload`` of the producer part, everything the epilogue
    writes; ``run`` calls msa_projection_forward on them."""

    def __init__(self, pw: wl.ProjectionWorkload, device="cuda", pools_on_device: dict | None = None,
                 rows_out: bool = False):
        import torch
        self.pw = pw
        self.dw = DeviceWorkload(pw.producer, device, pools_on_device=pools_on_device)
        self.device = self.dw.device
        self.hidden = _t(pw.hidden, self.device)
        self.weight = _t(pw.weight, self.device)
        self.hidden_scales = None if pw.hidden_scales is None else _t(pw.hidden_scales, self.device)
        self.weight_scales = None if pw.weight_scales is None else _t(pw.weight_scales, self.device)
        self.rows_out = (torch.zeros((pw.num_tokens, pw.width), dtype=torch.int16, device=self.device)
                         if rows_out else None)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    @property
    def pools(self):
        return self.dw.pools

    def args(self):
        """Positional arguments of msa_projection_forward minus the stream."""
        dw, pw = self.dw, self.pw
        p = lambda t: None if t is None else int(t.data_ptr())
        return (dw.cfg, pw.num_tokens, p(self.hidden), pw.hidden_size, pw.hidden.shape[1],
                p(self.weight), pw.weight.shape[1], pw.operand_dtype, p(self.hidden_scales),
                p(self.weight_scales), p(dw.positions), p(dw.slots), p(dw.page_table),
                0 if dw.page_table is None else dw.page_table.numel(),
                p(dw.weights.get("q")), p(dw.weights.get("k")), p(dw.weights.get("idx_q")),
                p(dw.weights.get("idx_k")), p(dw.q_out), p(dw.idx_q_out), dw.caches["k"],
                dw.caches["v"], dw.caches["idx_k"], p(dw.scales), p(self.rows_out),
                0 if self.rows_out is None else pw.width, p(self.status))

    def run(self, stream=None):
        import torch
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        with B.on_device(self.device):
            return B.msa_projection_forward(*self.args(), stream=stream.cuda_stream)

    def outputs_to_host(self):
        return self.dw.outputs_to_host()

    def rows_to_host(self):
        return self.rows_out.cpu().numpy().view(np.uint16)


def _checked(name, t, shape, kinds, dev, contiguous=True, optional=False):
    """``t``, if it is a tensor of one of the dtypes ``kinds`` and of ``shape`` on ``dev`` (rows any
    stride apart unless ``contiguous``), else a ValueError."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    rows = t.is_contiguous() if contiguous else t.dim() < 2 or t.stride(-1 % t.dim()) == 1 or t.shape[-1] < 2
    if t.dtype not in kinds or tuple(t.shape) != tuple(shape) or not rows:
        raise ValueError(f"{name}: expected a {'contiguous' if contiguous else 'unit column stride'} {kinds[0]} tensor of "
                         f"shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}")
    return t


class LayerInput:
    """The input side of an MSA layer for up to ``max_tokens`` tokens: the residual's addition and
    the norm, which makes the projection's E4M3 operand with a scale for each token; the packed
    projection; the requests' low-rank adapters on its rows; and the producer, with rotary
    positions of one axis or several.

    ``weight`` E4M3 [W, K] and ``weight_scales`` fp32 [W] are the projection's, ``norm_w`` bf16 [K]
    the layer's norm, ``head_norms`` the producer's four, ``caches`` its (k, v, idx_k) MsaCacheDesc,
    ``scales`` theirs.  ``axes``: an MsaRopeAxes for positions [num_axes, T], else positions are [T].
    ``adapters``: (down, up, adapter_scales) tensors as ``binding.adapter_tensors`` takes them, the
    slices being the row's sections.  ``adapter_hidden``: the MSA_DTYPE of the hidden states that the
    adapters read, the projection's E4M3 operand or bf16 rows, which the norm then writes beside it (2
    bytes an element more; the layer's ``hidden``).  Without adapters and axes the producer runs in the
    projection's epilogue and the rows never leave the chip.

    A layer keeps one set of buffers: its runs (and replays of graphs of them) follow one another.
    Tensors that do not fit are a ValueError, before anything is enqueued."""

    def __init__(self, cfg: B.MsaProducerCfg, max_tokens: int, weight, weight_scales, norm_w, head_norms, caches, scales,
                 axes=None, adapters=None, rms_eps: float = 1e-6, adapter_hidden: int = B.MSA_DTYPE_FP8_E4M3):
        import torch
        bf16, e4m3, f32 = (torch.bfloat16, torch.int16), (torch.float8_e4m3fn, torch.uint8), (torch.float32,)
        dev, D = weight.device, cfg.head_dim
        sections = [cfg.num_q_heads, cfg.num_kv_heads, cfg.num_kv_heads, cfg.num_idx_q_heads, cfg.num_idx_k_heads]
        if dev.type != "cuda":
            raise ValueError(f"weight is on {dev}; a layer takes CUDA tensors")
        if weight.dim() != 2:
            raise ValueError(f"weight: expected [W, K], got {tuple(weight.shape)}")
        W, K = sum(sections) * D, weight.shape[1]
        _checked("weight", weight, (W, K), e4m3, dev, contiguous=False)
        if weight.data_ptr() % 16 or weight.stride(0) % 16 or weight.stride(0) < K:
            raise ValueError(f"weight: 16-byte aligned rows, a stride that is a multiple of 16, got strides {weight.stride()}")
        _checked("weight_scales", weight_scales, (W,), f32, dev, optional=True)
        _checked("norm_w", norm_w, (K,), bf16, dev)
        for name, w in zip(("q", "k", "idx_q", "idx_k"), head_norms, strict=True):
            _checked(f"head_norms ({name})", w, (D,), bf16, dev, optional=True)
        if scales is not None:
            ns = 2 * cfg.num_kv_heads + cfg.num_idx_k_heads if cfg.scale_mode == B.MSA_SCALE_PER_HEAD else 3
            if scales.dim() != 1 or scales.shape[0] < ns:
                raise ValueError(f"scales: expected at least {ns} values, got shape {tuple(scales.shape)}")
            _checked("scales", scales, scales.shape, f32, dev)
        if adapters is not None:
            down, up, adapter_scales = adapters
            if up.dim() != 3 or down.dim() != 3:
                raise ValueError(f"adapters: expected down [n, slices * rank, K] and up [n, W, rank], got "
                                 f"{tuple(down.shape)} and {tuple(up.shape)}")
            n, rank, slices = up.shape[0], up.shape[2], sum(heads > 0 for heads in sections)
            _checked("adapters (up)", up, (n, W, rank), bf16, dev)
            _checked("adapters (down)", down, (n, slices * rank, K), bf16, dev, contiguous=False)
            if n > 1 and down.stride(0) != slices * rank * down.stride(1) or down.stride(1) % 8 or down.stride(1) < K or \
                    down.data_ptr() % 16:
                raise ValueError(f"adapters (down): 16-byte aligned rows one stride apart, a multiple of 8, got strides "
                                 f"{down.stride()}")
            _checked("adapters (scales)", adapter_scales, (n,), f32, dev, optional=True)
        if adapter_hidden not in (B.MSA_DTYPE_FP8_E4M3, B.MSA_DTYPE_BF16):
            raise ValueError(f"adapter_hidden: {adapter_hidden}")
        self.max_tokens = max_tokens
        self.cfg, self.weight, self.weight_scales, self.norm_w = cfg, weight, weight_scales, norm_w
        self.head_norms, self.caches, self.scales, self.axes, self.adapters = head_norms, caches, scales, axes, adapters
        self.norm_cfg = B.make_norm_cfg(K, rms_eps)
        self.codes = torch.empty((max_tokens, -(-K // 16) * 16), dtype=torch.uint8, device=dev)[:, :K]
        self.hidden_scales = torch.empty(max_tokens, dtype=torch.float32, device=dev)
        self.q_out = torch.empty((max_tokens, cfg.num_q_heads, D), dtype=torch.bfloat16, device=dev)
        self.idx_q_out = torch.empty((max_tokens, cfg.num_idx_q_heads, D), dtype=torch.bfloat16, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.hidden = None
        if adapters is not None and adapter_hidden == B.MSA_DTYPE_BF16:
            self.hidden = torch.empty((max_tokens, -(-K // 8) * 8), dtype=torch.bfloat16, device=dev)[:, :K]
        self.rows = None
        if axes is not None or adapters is not None:
            self.rows = torch.empty((max_tokens, W), dtype=torch.bfloat16, device=dev)
            # rows alone: index-K heads whose cache is absent, so that nothing else is written
            self.rows_cfg = B.make_cfg(0, 0, 0, W // D, D, 0, cfg.rope_style, cfg.page_size)
        if adapters is not None:
            down, up, _ = adapters
            ends = [sum(sections[:i + 1]) * D for i, n in enumerate(sections) if n > 0]
            self.adapter_cfg = B.make_adapter_cfg(K, ends, up.shape[2], up.shape[0], adapter_hidden)
            nbytes = B.msa_adapter_workspace_bytes(self.adapter_cfg, max_tokens)
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)

    def _project(self, cfg, n, positions, slots, page_table, norms, q, iq, caches, scales, rows, stream):
        p = lambda t: None if t is None else int(t.data_ptr())
        with B.on_device(self.weight.device):
            B.msa_projection_forward(
                cfg, n, p(self.codes), self.codes.shape[1], self.codes.stride(0), p(self.weight), self.weight.stride(0),
                B.MSA_DTYPE_FP8_E4M3, p(self.hidden_scales), p(self.weight_scales), p(positions), p(slots),
                p(page_table), 0 if page_table is None else page_table.numel(), *(p(w) for w in norms), p(q), p(iq),
                *caches, p(scales), p(rows), 0 if rows is None else rows.stride(0), p(self.status),
                stream=stream.cuda_stream)

    def run(self, x, residual, positions, slot_mapping, page_table, adapter_ids=None, launch_flags=0, stream=None):
        """For x and residual bf16 [T, K], T at most max_tokens: residual becomes their sum; q_out and
        idx_q_out [:T] and the caches are written.  positions int32, slot_mapping int64 [T],
        page_table int32 or None; adapter_ids int32 [T] with adapters, else None; launch_flags: the
        producer's, where it is a launch of its own (with axes or adapters)."""
        import torch
        if x.dim() != 2:
            raise ValueError(f"x: expected [T, K], got {tuple(x.shape)}")
        n, dev, i32 = x.shape[0], self.weight.device, (torch.int32,)
        if n > self.max_tokens:
            raise ValueError(f"{n} tokens; the layer was made for {self.max_tokens}")
        if self.axes is None:
            _checked("positions", positions, (n,), i32, dev)
        else:
            axes = self.axes.num_axes
            _checked("positions", positions, (axes, n), i32, dev, contiguous=False)
            if axes > 1 and n > 0 and positions.stride(0) < n:
                raise ValueError(f"positions: {n} tokens an axis, axes {positions.stride(0)} apart")
        _checked("slot_mapping", slot_mapping, (n,), (torch.int64,), dev)
        if page_table is not None:
            _checked("page_table", page_table, page_table.shape, i32, dev)
        if self.adapters is not None:
            _checked("adapter_ids", adapter_ids, (n,), i32, dev)
        elif adapter_ids is not None:
            raise ValueError("adapter_ids for a layer without adapters")
        if stream is not None and stream.device != dev:
            raise ValueError(f"a stream of {stream.device}, tensors on {dev}")
        if stream is None:
            stream = torch.cuda.current_stream(x.device)
        codes, hidden_scales = self.codes[:n], self.hidden_scales[:n]
        q, iq = self.q_out[:n], self.idx_q_out[:n]
        hidden = None if self.hidden is None else self.hidden[:n]
        B.norm_tensors(self.norm_cfg, x, self.norm_w, residual=residual, residual_out=residual, out=hidden, codes=codes,
                       scales=hidden_scales, stream=stream)
        if self.rows is None:
            self._project(self.cfg, n, positions, slot_mapping, page_table, self.head_norms, q, iq, self.caches,
                          self.scales, None, stream)
            return
        rows = self.rows[:n]
        # (nothing is turned or placed: any positions and slots will do)
        self._project(self.rows_cfg, n, positions, slot_mapping, None, (None,) * 4, None, None, (None,) * 3, None, rows,
                      stream)
        if self.adapters is not None:
            down, up, adapter_scales = self.adapters
            of, of_scales = (codes, hidden_scales) if hidden is None else (hidden, None)
            B.adapter_tensors(self.adapter_cfg, of, down, up, adapter_ids, rows, rows, hidden_scales=of_scales,
                              adapter_scales=adapter_scales, workspace=self.workspace, stream=stream)
        args = (rows, positions, slot_mapping, page_table, self.head_norms, q, iq, *self.caches, self.scales,
                launch_flags, stream)
        if self.axes is None:
            B.forward_tensors(self.cfg, *args)
        else:
            B.forward_axes_tensors(self.cfg, self.axes, *args)

    def check_status(self, stream=None):
        """Waits for the runs on ``stream`` (the current one) and raises a RuntimeError if a wait inside
        their projections has run out since the last call of this (a failure of the hardware, never
        expected): what those runs wrote is then incomplete."""
        import torch
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.weight.device)):
            bits = int(self.status.item())
            self.status.zero_()
        if bits:
            raise RuntimeError(f"a projection did not finish (status {bits:#x})")


class DecodeLayer:
    """One MSA decode layer's hot path on the device: the producer (rows -> compact
    Q / index-Q, K/V/index-K into the caches) followed by the indexer on what the
    producer wrote (its compact index-Q and index-K cache), each token's visible
    history being its position + 1 tokens in its sequence's page-table row.  With
    ``attention``, the sparse attention of the compact Q over the K/V caches and the
    blocks the indexer selected comes last (``attn_out``, ``attn_lse``).  Its workspace
    holds nothing between calls: layers that run one after another on a stream may share
    one (``attn_workspace=`` another layer's), layers that may run at once may not."""

    def __init__(self, dw: DeviceWorkload, max_blocks_per_seq: int, block_tokens: int = 128,
                 topk: int = 16, attention: bool = False, attn_workspace=None):
        import torch
        self.dw = dw
        w = dw.w
        s = w.shape
        assert w.page_table is not None and dw.caches.get("idx_k") is not None
        P = s["page_size"]
        self.cfg = B.make_indexer_cfg(s["num_idx_q_heads"], s["head_dim"], P, block_tokens, topk,
                                      -(-max_blocks_per_seq * P // block_tokens))
        T = w.num_tokens
        pt = w.page_table.reshape(w.page_table.shape[0], -1)
        # the sequence of each token is its slot's table row (logical slots); a padded
        # token keeps the row of its position in the batch
        seq = np.where(w.slot_mapping >= 0, w.slot_mapping // (pt.shape[1] * P),
                       np.arange(T) % pt.shape[0])
        self.kv_len = _t((w.positions.astype(np.int64) + 1).astype(np.int32), dw.device)
        self.table_offset = _t((seq * pt.shape[1]).astype(np.int64), dw.device)
        self.k_scale = dw.scales[2:3] if s.get("scale_mode", 0) == 0 else dw.scales[-1:]
        self.block_scores = torch.empty((T, self.cfg.max_blocks), dtype=torch.float32,
                                        device=dw.device)
        self.topk_ids = torch.empty((T, topk), dtype=torch.int32, device=dw.device)
        self.counters = torch.zeros((T,), dtype=torch.int32, device=dw.device)
        self.attn_cfg = None
        if attention:
            self.attn_cfg = B.make_attention_cfg(s["num_q_heads"], s["num_kv_heads"], s["head_dim"], P,
                                                 block_tokens, topk, scale_mode=s.get("scale_mode", 0))
            self.attn_out = torch.empty_like(dw.q_out)
            self.attn_lse = torch.empty(dw.q_out.shape[:2], dtype=torch.float32, device=dw.device)
            self.attn_workspace = attn_workspace
            if attn_workspace is None:
                self.attn_workspace = torch.empty(B.msa_attention_workspace_bytes(self.attn_cfg, T),
                                                  dtype=torch.uint8, device=dw.device)

    def run(self, stream, flags=0, fused=False):
        """The producer, then the indexer on what it wrote (with ``fused``, the
        single-launch indexer on this layer's zeroed counters), then the attention of a
        layer that has it."""
        dw = self.dw
        p = lambda t: int(t.data_ptr())
        dw.run(B.MSA_LAUNCH_PERSISTENT | (flags & B.MSA_LAUNCH_PDL), stream=stream)
        args = (self.cfg, dw.w.num_tokens, p(dw.idx_q_out), p(self.kv_len), p(self.table_offset),
                p(dw.page_table), dw.page_table.numel(), dw.caches["idx_k"], p(self.k_scale),
                p(self.block_scores), p(self.topk_ids))
        with B.on_device(dw.device):
            if fused:
                B.msa_indexer_forward_fused(*args, p(self.counters), flags & B.MSA_LAUNCH_PDL,
                                            stream=stream.cuda_stream)
            else:
                B.msa_indexer_forward(*args, flags & B.MSA_LAUNCH_PDL, stream=stream.cuda_stream)
            if self.attn_cfg is not None:
                B.msa_sparse_attention_forward(
                    self.attn_cfg, dw.w.num_tokens, p(dw.q_out), p(self.kv_len), p(self.table_offset),
                    p(dw.page_table), dw.page_table.numel(), p(self.topk_ids), dw.caches["k"], dw.caches["v"],
                    p(dw.scales), p(self.attn_out), p(self.attn_lse), p(self.attn_workspace),
                    self.attn_workspace.nbytes, flags & B.MSA_LAUNCH_PDL, stream=stream.cuda_stream)

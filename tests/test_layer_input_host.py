"""The layer's input side on the host, with no GPU: on which device its calls run, and what it
refuses.  The C entry points are stand-ins, and so are the tensors: they have a device, a shape
and strides, and no memory."""
import contextlib

import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300.device import LayerInput

DEV = torch.device("cuda", 1)


class Tensor:
    """A row-major tensor on a device that this machine need not have."""

    def __init__(self, shape, dtype, device=DEV, strides=None, address=1 << 20):
        self.shape, self.dtype, self.device, self.address = torch.Size(shape), dtype, torch.device(device), address
        if strides is None:
            strides = [1]
            for n in reversed(shape[1:]):
                strides.insert(0, strides[0] * n)
            strides = strides[:len(shape)]
        self.strides = tuple(strides)
        self.is_cuda = self.device.type == "cuda"

    def data_ptr(self):
        return self.address

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def numel(self):
        return self.shape.numel()

    def size(self, i):
        return self.shape[i]

    def is_contiguous(self):
        return self.strides == Tensor(self.shape, self.dtype).strides or self.numel() == 0

    def __getitem__(self, at):
        at = at if isinstance(at, tuple) else (at,)
        shape = [len(range(n)[s]) for n, s in zip(self.shape, at)] + list(self.shape[len(at):])
        return Tensor(shape, self.dtype, self.device, self.strides, self.address)


class Stream:
    cuda_stream, device = 0, DEV


@pytest.fixture
def gpu(monkeypatch):
    """Two devices, of which 0 is current: the calls made, each with the device that was current."""
    state = {"current": 0, "calls": []}

    @contextlib.contextmanager
    def device(d):
        before, state["current"] = state["current"], torch.device(d).index
        yield
        state["current"] = before

    def record(name):
        def call(*a, **k):
            state["calls"].append((name, state["current"]))
            return B.MSA_OK
        return call

    make = lambda shape, dtype=torch.float32, device=None: Tensor(
        (shape,) if isinstance(shape, int) else tuple(shape), dtype, device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream())
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch, "zeros", make)
    for name in ("msa_projection_forward", "msa_producer_forward"):
        monkeypatch.setattr(B, name, record(name))
    # (these set the device themselves, in the extension)
    for name in ("norm_tensors", "adapter_tensors", "forward_axes_tensors"):
        monkeypatch.setattr(B, name, record(name))
    monkeypatch.setattr(B, "msa_adapter_workspace_bytes", lambda cfg, n: 4096)
    return state


BF16, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
D, K, T, RANK = 64, 256, 6, 16
HEADS = (8, 2, 2, 2, 1)
W = sum(HEADS) * D


def cfg():
    return B.make_cfg(8, 2, 2, 1, D, D // 2, B.MSA_ROPE_NEOX, 64)


def layer(max_tokens=16, with_adapters=False, with_axes=False, **over):
    a = dict(weight=Tensor((W, K), U8), weight_scales=Tensor((W,), F32), norm_w=Tensor((K,), BF16),
             head_norms=[Tensor((D,), BF16)] * 4, caches=(None, None, None), scales=Tensor((3,), F32),
             axes=B.make_rope_axes((4, 4, 8)) if with_axes else None,
             adapters=(Tensor((3, 5 * RANK, K), BF16), Tensor((3, W, RANK), BF16), Tensor((3,), F32)) if with_adapters else None)
    a.update(over)
    return LayerInput(cfg(), max_tokens, **a)


def run(lay, n=T, **over):
    a = dict(x=Tensor((n, K), BF16), residual=Tensor((n, K), BF16),
             positions=Tensor((3, n) if lay.axes is not None else (n,), I32), slot_mapping=Tensor((n,), I64),
             page_table=Tensor((12,), I32), adapter_ids=Tensor((n,), I32) if lay.adapters is not None else None)
    a.update(over)
    lay.run(**a)


@pytest.mark.parametrize("adapters", [False, True])
@pytest.mark.parametrize("axes", [False, True])
@pytest.mark.parametrize("stream", [None, Stream()], ids=["current", "given"])
def test_calls_run_on_the_tensors_device(gpu, adapters, axes, stream):
    run(layer(with_adapters=adapters, with_axes=axes), stream=stream)
    raw = [c for c in gpu["calls"] if c[0] in ("msa_projection_forward", "msa_producer_forward")]
    assert len(raw) == (1 if axes or not adapters else 2)
    assert all(dev == 1 for _, dev in raw), raw
    assert gpu["current"] == 0


def test_producer_runs_on_the_rows_device(gpu):
    q = Tensor((T, 8, D), BF16)
    B.forward_tensors(cfg(), Tensor((T, W), BF16), Tensor((T,), I32), Tensor((T,), I64), None, (None,) * 4, q, q, None,
                      None, None, None)
    assert gpu["calls"] == [("msa_producer_forward", 1)] and gpu["current"] == 0


@pytest.mark.parametrize("over", [
    dict(weight=Tensor((W, K), BF16)), dict(weight=Tensor((W - D, K), U8)), dict(weight=Tensor((W, K), U8, "cpu")),
    dict(weight=Tensor((W * K,), U8)), dict(weight=Tensor((W, K), U8, strides=(1, W))),
    dict(weight=Tensor((W, K), U8, strides=(K + 8, 1))), dict(weight=Tensor((W, K), U8, address=(1 << 20) + 8)),
    dict(weight_scales=Tensor((W,), BF16)), dict(weight_scales=Tensor((W - 1,), F32)),
    dict(weight_scales=Tensor((W,), F32, "cuda:0")), dict(weight_scales=Tensor((W,), F32, strides=(2,))),
    dict(norm_w=Tensor((K + 1,), BF16)), dict(norm_w=Tensor((K,), F32)), dict(norm_w=None),
    dict(head_norms=[Tensor((D,), BF16)] * 3), dict(head_norms=[Tensor((D,), F32)] * 4),
    dict(head_norms=[None, None, None, Tensor((D // 2,), BF16)]), dict(scales=Tensor((2,), F32)),
    dict(scales=Tensor((3,), torch.float64)), dict(scales=Tensor((1, 3), F32)), dict(scales=Tensor((3,), F32, "cpu")),
    dict(adapters=(Tensor((3, 5 * RANK, K), BF16), Tensor((3, W, RANK), F32), None)),
    dict(adapters=(Tensor((3, 4 * RANK, K), BF16), Tensor((3, W, RANK), BF16), None)),
    dict(adapters=(Tensor((2, 5 * RANK, K), BF16), Tensor((3, W, RANK), BF16), None)),
    dict(adapters=(Tensor((3, 5 * RANK, K), BF16), Tensor((3, W, RANK), BF16), Tensor((2,), F32))),
    dict(adapters=(Tensor((3, 5 * RANK, K), BF16, strides=(5 * RANK * K + 8, K, 1)), Tensor((3, W, RANK), BF16), None)),
    dict(adapters=(Tensor((3, 5 * RANK, K), BF16, strides=(5 * RANK * (K + 4), K + 4, 1)), Tensor((3, W, RANK), BF16), None)),
    dict(adapters=(Tensor((5 * RANK, K), BF16), Tensor((W, RANK), BF16), None)),
], ids=lambda o: next(iter(o)))
def test_a_layers_tensors_that_do_not_fit(gpu, over):
    with pytest.raises(ValueError):
        layer(**over)


@pytest.mark.parametrize("axes", [False, True])
@pytest.mark.parametrize("over", [
    dict(positions=Tensor((T,), I64)), dict(positions=Tensor((3, T), I64)), dict(positions=Tensor((T - 1,), I32)),
    dict(positions=Tensor((2, T), I32)), dict(positions=Tensor((3, T), I32, strides=(1, 3))),
    dict(positions=Tensor((3, T), I32, strides=(0, 1))), dict(positions=Tensor((T,), I32, strides=(2,))),
    dict(positions=Tensor((T,), I32, "cpu")), dict(positions=None), dict(slot_mapping=Tensor((T,), I32)),
    dict(slot_mapping=Tensor((T + 1,), I64)), dict(slot_mapping=Tensor((T,), I64, "cuda:0")), dict(slot_mapping=None),
    dict(slot_mapping=Tensor((T,), I64, strides=(2,))), dict(page_table=Tensor((12,), I64)),
    dict(page_table=Tensor((12,), I32, strides=(2,))), dict(page_table=Tensor((12,), I32, "cpu")),
    dict(adapter_ids=Tensor((T,), I64)), dict(adapter_ids=Tensor((T - 1,), I32)), dict(adapter_ids=None),
    dict(x=Tensor((K,), BF16)), dict(stream=type("Other", (), dict(cuda_stream=0, device=torch.device("cuda", 0)))()),
], ids=lambda o: next(iter(o)))
def test_a_runs_tensors_that_do_not_fit(gpu, axes, over):
    """Refused before the first call, which adds to the residual where it is."""
    lay = layer(with_adapters=True, with_axes=axes)
    with pytest.raises(ValueError):
        run(lay, **over)
    assert gpu["calls"] == []


def test_more_tokens_than_the_layers(gpu):
    with pytest.raises(ValueError):
        run(layer(max_tokens=5))
    with pytest.raises(ValueError):
        run(layer(), adapter_ids=Tensor((T,), I32))         # no adapters
    assert gpu["calls"] == []


def test_tensors_that_do_fit(gpu):
    """Raw words in the place of 8- and 16-bit floats, rows and axes further apart, optional tensors left out."""
    run(layer(with_adapters=True, with_axes=True, weight=Tensor((W, K), torch.float8_e4m3fn, strides=(K + 16, 1)), weight_scales=None,
              norm_w=Tensor((K,), torch.int16), head_norms=[None] * 4, scales=Tensor((9,), F32)),
        positions=Tensor((3, T), I32, strides=(T + 5, 1)), page_table=None)
    run(layer(scales=None), n=1, page_table=Tensor((3, 4), I32))
    run(layer(with_axes=True), n=0)


def made(cls, **attributes):
    """An object of a class without its constructor, which copies to the GPU."""
    obj = cls.__new__(cls)
    for name, value in attributes.items():
        setattr(obj, name, value)
    return obj


def test_the_other_helpers_run_on_their_device(gpu, monkeypatch):
    from paged_kv_cache_msa_gb300 import device as dev_mod
    from paged_kv_cache_msa_gb300.pipeline import HostPipeline
    names = ("msa_producer_forward", "msa_projection_forward", "msa_indexer_forward", "msa_indexer_forward_fused",
             "msa_sparse_attention_forward")
    for name in names:
        monkeypatch.setattr(B, name, lambda *a, _n=name, **k: gpu["calls"].append((_n, gpu["current"])))
    monkeypatch.setattr(B, "msa_host_buffer_device_address", lambda p: p)
    t, s = Tensor((T,), I32), Stream()
    work = type("Work", (), dict(num_tokens=T, idx_q=t))()
    dw = made(dev_mod.DeviceWorkload, w=work, device=DEV, args=lambda *a: (), idx_q_out=t, q_out=t, page_table=t,
              scales=t, caches=dict(k=None, v=None, idx_k=None))
    dw.run()
    made(dev_mod.DeviceProjection, device=DEV, args=lambda: ()).run()
    own = dict(device=DEV, cfg=None, idx_q=t, kv_len=t, table_offset=t, page_table=t, cache=None, k_scale=t, block_scores=t,
               topk_ids=t, counters=t)
    for fused in (False, True):
        made(dev_mod.DeviceIndexer, w=work, **own).run(fused=fused)
        lse = type("Bytes", (Tensor,), dict(nbytes=64))((T,), U8)
        made(dev_mod.DecodeLayer, dw=dw, attn_cfg=cfg(), attn_out=t, attn_lse=t, attn_workspace=lse, **own).run(s, fused=fused)
    stream = type("S", (Stream,), dict(synchronize=lambda self: None))()
    made(HostPipeline, device=DEV, cfg=None, row_stride=W, weights=(None,) * 4, caches=(None,) * 3, scales=t, page_table=None,
         flags=0, s_comp=stream).run_zero_copy(t, t, t, t, t)
    assert len(gpu["calls"]) == 1 + 1 + 2 + 2 * 3 + 1 and {n for n, _ in gpu["calls"]} == set(names)
    assert all(d == 1 for _, d in gpu["calls"]), gpu["calls"]

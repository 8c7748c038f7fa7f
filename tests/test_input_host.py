"""The norm, the adapters and the producer with several rotary axes on the host, with no GPU:
what their argument checks accept and refuse.  Pointers are made-up addresses: the checks never
look behind them, and a refused call launches nothing."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

BASE = 0x7F0000000000
INVALID, UNSUPPORTED, MISALIGNED, OVERFLOW = (B.MSA_ERR_INVALID_ARGUMENT, B.MSA_ERR_UNSUPPORTED,
                                              B.MSA_ERR_MISALIGNED, B.MSA_ERR_OFFSET_OVERFLOW)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def at(i):
    return BASE + i * 2**34


def with_field(cfg, name, value):
    if isinstance(value, tuple):
        getattr(cfg, name)[value[0]] = value[1]
    else:
        setattr(cfg, name, value)
    return cfg


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def norm(**over):
    a = dict(cfg=B.make_norm_cfg(6144), num_tokens=16, x=at(0), x_stride=6144, residual=at(1), residual_stride=6144,
             weight=at(2), residual_out=at(3), residual_out_stride=6144, out=at(4), out_stride=6144, codes=at(5),
             codes_stride=6144, scales=at(6))
    a.update(over)
    return B.msa_norm_forward(**a, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(cfg=None), INVALID),
    (dict(num_tokens=-1), INVALID),
    (dict(num_tokens=2**31), UNSUPPORTED),
    (dict(x=None), INVALID),
    (dict(weight=None), INVALID),
    (dict(residual=None), INVALID),                      # residual_out without a residual
    (dict(out=None, codes=None, scales=None), INVALID),
    (dict(codes=None), INVALID),                         # scales alone
    (dict(scales=None), INVALID),
    (dict(x_stride=6143), INVALID),
    (dict(codes_stride=6136), INVALID),
    (dict(x_stride=6148), MISALIGNED),
    (dict(codes_stride=6152), MISALIGNED),
    (dict(x=at(0) + 8), MISALIGNED),
    (dict(weight=at(2) + 2), MISALIGNED),
    (dict(codes=at(5) + 8), MISALIGNED),
    (dict(scales=at(6) + 2), MISALIGNED),
    (dict(out_stride=2**62), OVERFLOW),
    (dict(residual_out=at(1), residual_out_stride=6152), INVALID),   # in place, another stride
    (dict(out=at(0), out_stride=6152), INVALID),
    (dict(launch_flags=B.MSA_LAUNCH_PERSISTENT), INVALID),
], ids=str)
def test_norm_refuses(over, status):
    assert norm(**over) == status, B.last_error_detail()
    assert B.last_error_detail()


@pytest.mark.parametrize("name,value,status", [
    ("hidden_size", 0, INVALID), ("hidden_size", 16385, UNSUPPORTED), ("rms_eps", -1e-6, INVALID),
    ("rms_eps", float("nan"), INVALID), ("rms_eps", float("inf"), INVALID), ("reserved", (0, 1), INVALID),
    ("reserved", (1, 1), INVALID),
])
def test_norm_cfg_refuses(name, value, status):
    wide = dict.fromkeys(("x_stride", "residual_stride", "residual_out_stride", "out_stride", "codes_stride"), 32768)
    assert norm(cfg=with_field(B.make_norm_cfg(6144), name, value), **wide) == status


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------

def adapter_cfg(**kw):
    d = dict(hidden_size=6144, slice_ends=[8192, 9216, 10240, 11264, 11392], rank=16, num_adapters=4)
    d.update(kw)
    return B.make_adapter_cfg(**d)


def adapter(**over):
    a = dict(cfg=adapter_cfg(), num_tokens=16, hidden=at(0), hidden_stride=6144, hidden_scales=at(1), down=at(2),
             down_stride=6144, up=at(3), adapter_ids=at(4), adapter_scales=at(5), rows=at(6), rows_stride=11392,
             out=at(7), out_stride=11392, workspace=at(8), workspace_bytes=1 << 30)
    a.update(over)
    return B.msa_adapter_forward(**a, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(cfg=None), INVALID),
    (dict(num_tokens=-1), INVALID),
    (dict(num_tokens=2**24 + 1), UNSUPPORTED),
    (dict(hidden=None), INVALID),
    (dict(down=None), INVALID),
    (dict(up=None), INVALID),
    (dict(adapter_ids=None), INVALID),
    (dict(rows=None), INVALID),
    (dict(out=None), INVALID),
    (dict(hidden_stride=6136), INVALID),
    (dict(down_stride=6136), INVALID),
    (dict(rows_stride=11384), INVALID),
    (dict(out_stride=11384), INVALID),
    (dict(out=at(6), out_stride=11400), INVALID),
    (dict(hidden_stride=6148), MISALIGNED),
    (dict(cfg=adapter_cfg(hidden_dtype=B.MSA_DTYPE_FP8_E4M3), hidden_stride=6152), MISALIGNED),
    (dict(down_stride=6148), MISALIGNED),
    (dict(rows_stride=11396), MISALIGNED),
    (dict(hidden=at(0) + 8), MISALIGNED),
    (dict(up=at(3) + 8), MISALIGNED),
    (dict(adapter_ids=at(4) + 2), MISALIGNED),
    (dict(adapter_scales=at(5) + 2), MISALIGNED),
    (dict(workspace=at(8) + 16), MISALIGNED),
    (dict(rows_stride=2**62), OVERFLOW),
    (dict(down_stride=2**62), OVERFLOW),
    (dict(down_stride=2**39), UNSUPPORTED),
    (dict(workspace=None), INVALID),
    (dict(workspace_bytes=16), INVALID),
    (dict(launch_flags=B.MSA_LAUNCH_QUERY_RUNS), INVALID),
], ids=str)
def test_adapter_refuses(over, status):
    assert adapter(**over) == status, B.last_error_detail()
    assert B.last_error_detail()


@pytest.mark.parametrize("name,value,status", [
    ("hidden_size", 0, INVALID), ("rank", 0, INVALID), ("rank", 12, UNSUPPORTED), ("rank", 136, UNSUPPORTED),
    ("rank", 128, UNSUPPORTED), ("num_adapters", 0, INVALID), ("num_adapters", 16385, UNSUPPORTED), ("hidden_dtype", 2, UNSUPPORTED),
    ("num_slices", 0, INVALID), ("num_slices", 9, INVALID), ("num_slices", 4, INVALID),
    ("slice_end", (1, 8192), INVALID), ("slice_end", (0, 8200), UNSUPPORTED), ("slice_end", (4, 11390), UNSUPPORTED),
    ("slice_end", (0, 0), INVALID), ("slice_end", (7, 64), INVALID), ("reserved", (2, 1), INVALID),
])
def test_adapter_cfg_refuses(name, value, status):
    assert adapter(cfg=with_field(adapter_cfg(), name, value)) == status, B.last_error_detail()
    with pytest.raises(B.MsaError):
        B.msa_adapter_workspace_bytes(with_field(adapter_cfg(), name, value), 16)


@pytest.mark.parametrize("rank,slices", [(8, 1), (16, 5), (64, 8), (128, 4)])
@pytest.mark.parametrize("t", [0, 1, 63, 64, 65, 1000, 8192, 2**24])
def test_adapter_workspace_bounds(rank, slices, t):
    """What the header promises: less than 2 MB and 512 bytes an adapter, and at most 32 * num_slices *
    rank + 80 bytes a token."""
    for adapters in (1, 48, 16384):
        cfg = adapter_cfg(rank=rank, slice_ends=[64 * (i + 1) for i in range(slices)], num_adapters=adapters)
        n = B.msa_adapter_workspace_bytes(cfg, t)
        assert 0 <= n < 2 * 2**20 + 512 * adapters + (32 * slices * rank + 80) * t


@pytest.mark.parametrize("rank,slices", [(8, 1), (16, 5), (64, 5), (128, 4)])
@pytest.mark.parametrize("k", [64, 6144, 40000])
@pytest.mark.parametrize("dtype", [B.MSA_DTYPE_BF16, B.MSA_DTYPE_FP8_E4M3])
def test_adapter_workspace_serves_fewer_tokens(rank, slices, k, dtype):
    """A workspace for n tokens serves every call of fewer: never fewer bytes for more tokens, across
    the step to wide tiles and the counts at which a tile more leaves fewer pieces of K."""
    cfg = adapter_cfg(hidden_size=k, rank=rank, hidden_dtype=dtype, num_adapters=3,
                      slice_ends=[64 * (i + 1) for i in range(slices)])
    sizes = [B.msa_adapter_workspace_bytes(cfg, t) for t in range(0, 2600)]
    assert sizes == sorted(sizes)
    sizes = [B.msa_adapter_workspace_bytes(cfg, t) for t in range(0, 400_000, 977)]
    assert sizes == sorted(sizes)


# ---------------------------------------------------------------------------
# the producer with several axes
# ---------------------------------------------------------------------------

def axes_call(axes=None, **over):
    hq, hkv, hiq, hik, d, p = 64, 8, 8, 1, 128, 64
    cfg = B.make_cfg(hq, hkv, hiq, hik, d, 128, B.MSA_ROPE_NEOX, p)

    def cache(i, heads):
        return B.make_cache(at(i), B.MSA_DTYPE_FP8_E4M3, 1024, heads, heads * p * d, p * d, d)

    a = dict(cfg=cfg, axes=B.make_rope_axes((16, 24, 24)) if axes is None else axes, num_tokens=16, qkv=at(0),
             qkv_row_stride=(hq + 2 * hkv + hiq + hik) * d, positions=at(1), positions_stride=16, slot_mapping=at(2),
             page_table=at(3), page_table_len=1024, q_norm_w=at(4), k_norm_w=at(4) + 256, idx_q_norm_w=at(4) + 512,
             idx_k_norm_w=at(4) + 768, q_out=at(5), idx_q_out=at(6), k_cache=cache(7, hkv), v_cache=cache(8, hkv),
             idx_k_cache=cache(9, hik), scales=at(10))
    a.update(over)
    return B.msa_producer_axes_forward(**a, check=False)


def good_axes():
    return B.make_rope_axes((16, 24, 24))


@pytest.mark.parametrize("axes,status", [
    (with_field(good_axes(), "num_axes", 0), INVALID), (with_field(good_axes(), "num_axes", 2), INVALID),
    (with_field(good_axes(), "num_axes", 5), UNSUPPORTED), (with_field(good_axes(), "restart", 2), INVALID),
    (with_field(good_axes(), "pair_axis", (0, 3)), INVALID), (with_field(good_axes(), "reserved", (0, 1)), INVALID),
    (with_field(good_axes(), "reserved", (1, 1)), INVALID),
])
def test_axes_refuse(axes, status):
    assert axes_call(axes) == status, B.last_error_detail()


def test_axes_call_refuses():
    assert axes_call(positions_stride=15) == INVALID
    assert axes_call(positions_stride=2**61) == OVERFLOW
    a = dict(cfg=B.make_cfg(64, 8, 8, 1, 128, 64, B.MSA_ROPE_NEOX, 64))     # 32 pairs, an axis for the 33rd
    assert axes_call(**a) == INVALID
    for over, status in ((dict(cfg=None), INVALID), (dict(qkv=None), INVALID), (dict(positions=None), INVALID),
                         (dict(qkv=at(0) + 2), MISALIGNED), (dict(num_tokens=-1), INVALID), (dict(scales=None), INVALID),
                         (dict(launch_flags=B.MSA_LAUNCH_QUERY_RUNS), INVALID), (dict(k_cache=None), INVALID)):
        assert axes_call(**over) == status, over
    assert B.msa_producer_axes_forward(B.make_cfg(1, 0, 0, 0, 64), None, 1, at(0), 64, at(1), 1, at(2), None, 0, at(3),
                                       None, None, None, at(4), None, None, None, None, None, check=False) == INVALID


def test_axis_arrangements():
    assert list(B.make_rope_axes((2, 3, 1)).pair_axis)[:6] == [0, 0, 1, 1, 1, 2]
    assert list(B.make_rope_axes((2, 3, 1), interleaved=True).pair_axis)[:6] == [0, 1, 2, 0, 1, 1]
    assert B.make_rope_axes((64,), restart=True).restart == 1
    for bad in ((), (1, 1, 1, 1, 1), (65,), (-1, 3)):
        with pytest.raises(ValueError):
            B.make_rope_axes(bad)
    with pytest.raises(ValueError):
        B.make_adapter_cfg(64, [], 8, 1)


# ---------------------------------------------------------------------------
# all three
# ---------------------------------------------------------------------------

def test_no_tokens_is_ok_without_launch():
    assert norm(num_tokens=0, x=None) == B.MSA_OK
    assert adapter(num_tokens=0, hidden=None, workspace=None) == B.MSA_OK
    assert axes_call(num_tokens=0) == B.MSA_OK
    assert B.msa_adapter_workspace_bytes(adapter_cfg(), 0) == 0


def test_tensor_functions_take_cuda_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.norm_tensors(B.make_norm_cfg(64), x, x[0], out=x)
    with pytest.raises(ValueError, match="CUDA"):
        B.adapter_tensors(adapter_cfg(), x, x, x, ids, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        B.forward_axes_tensors(B.make_cfg(1, 0, 0, 0, 64), good_axes(), x, ids, ids, None, (None,) * 4, x, None, None,
                               None, None, None)


def test_adapter_sizes_are_bounded():
    """Sizes up to 2^30 are taken (here up to the workspace, which is too small), larger ones refused:
    a tile of K or a chunk of W more would pass 32 bits."""
    most, wide = 2**30, dict.fromkeys(("hidden_stride", "down_stride", "rows_stride", "out_stride"), 2**31)
    for cfg in (adapter_cfg(hidden_size=most), adapter_cfg(slice_ends=[64, most]), adapter_cfg(slice_ends=[most])):
        assert B.msa_adapter_workspace_bytes(cfg, 16) > 0
        assert adapter(cfg=cfg, workspace_bytes=16, **wide) == INVALID and "workspace" in B.last_error_detail()
    for cfg in (adapter_cfg(hidden_size=most + 1), adapter_cfg(hidden_size=2**31 - 1), adapter_cfg(slice_ends=[64, most + 8]),
                adapter_cfg(slice_ends=[2**31 - 8]), adapter_cfg(slice_ends=[most + 64, most + 128])):
        assert adapter(cfg=cfg, **wide) == UNSUPPORTED, B.last_error_detail()
        with pytest.raises(B.MsaError):
            B.msa_adapter_workspace_bytes(cfg, 16)

"""Host checks of the attention entry points: well-formed arguments pass the checks of
malformed ones, which return their status with nothing launched (no GPU needed: the
pointers are made-up aligned addresses, and every call here is refused or empty)."""
import pytest

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

BASE = 0x7F0000000000
INV, UNS, MIS, OVF = (B.MSA_ERR_INVALID_ARGUMENT, B.MSA_ERR_UNSUPPORTED, B.MSA_ERR_MISALIGNED,
                      B.MSA_ERR_OFFSET_OVERFLOW)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def cfg(**kw):
    base = dict(num_q_heads=64, num_kv_heads=8, head_dim=128)
    base.update(kw)
    c = B.make_attention_cfg(**base)
    return c


def cache(i=0, **kw):
    a = dict(data_ptr=BASE + (20 + i) * 2**34, dtype=B.MSA_DTYPE_FP8_E4M3, num_pages=1024, num_heads=8,
             stride_page=8 * 64 * 128, stride_head=64 * 128, stride_token=128)
    a.update(kw)
    return B.make_cache(**a)


def common(**over):
    a = dict(cfg=cfg(), num_queries=4, q=BASE, kv_len=BASE + 2**32, table_offset=BASE + 2 * 2**32,
             page_table=BASE + 3 * 2**32, page_table_len=4096, k_cache=cache(0), v_cache=cache(1),
             scales=BASE + 5 * 2**32, out=BASE + 6 * 2**32, lse=BASE + 7 * 2**32, workspace=BASE + 8 * 2**32,
             workspace_bytes=2**32, launch_flags=0)
    a.update(over)
    return a


def sparse(**over):
    return B.msa_sparse_attention_forward(**{**common(topk_ids=BASE + 9 * 2**32), **over}, stream=0, check=False)


def prefix(**over):
    return B.msa_prefix_attention_forward(**{**common(num_groups=2, group_start=BASE + 10 * 2**32,
                                                      prefix_len=BASE + 11 * 2**32,
                                                      prefix_offset=BASE + 12 * 2**32), **over},
                                          stream=0, check=False)


REFUSED = [
    (dict(cfg=None), INV),
    (dict(cfg=cfg(num_q_heads=0)), INV),
    (dict(cfg=cfg(num_kv_heads=0)), INV),
    (dict(cfg=cfg(num_q_heads=60)), INV),
    (dict(cfg=cfg(num_q_heads=8 * 129)), UNS),
    (dict(cfg=cfg(num_q_heads=1025, num_kv_heads=1025)), UNS),
    (dict(cfg=cfg(head_dim=96)), UNS),
    (dict(cfg=cfg(page_size=0)), INV),
    (dict(cfg=cfg(softmax_scale=0.0)), INV),
    (dict(cfg=cfg(softmax_scale=-1.0)), INV),
    (dict(cfg=cfg(softmax_scale=float("nan"))), INV),
    (dict(cfg=cfg(softmax_scale=float("inf"))), INV),
    (dict(cfg=cfg(scale_mode=2)), UNS),
    (dict(num_queries=-1), INV),
    (dict(num_queries=2**31), UNS),
    (dict(q=None), INV),
    (dict(q=BASE + 8), MIS),
    (dict(kv_len=None), INV),
    (dict(kv_len=BASE + 2), MIS),
    (dict(table_offset=None), INV),
    (dict(table_offset=BASE + 4), MIS),
    (dict(page_table=None), INV),
    (dict(page_table=BASE + 2), MIS),
    (dict(page_table_len=0), INV),
    (dict(k_cache=None), INV),
    (dict(v_cache=None), INV),
    (dict(k_cache=cache(num_heads=4)), INV),
    (dict(v_cache=cache(num_heads=9)), INV),
    (dict(k_cache=cache(stride_token=124)), MIS),
    (dict(v_cache=cache(data_ptr=BASE + 8)), MIS),
    (dict(v_cache=cache(dtype=3)), UNS),
    (dict(k_cache=cache(stride_token=64)), INV),
    (dict(k_cache=cache(stride_page=2**62)), OVF),
    (dict(scales=None), INV),
    (dict(scales=BASE + 2), MIS),
    (dict(out=None), INV),
    (dict(out=BASE + 8), MIS),
    (dict(lse=BASE + 2), MIS),
    (dict(launch_flags=B.MSA_LAUNCH_PERSISTENT), INV),
    (dict(launch_flags=8), INV),
]


@pytest.mark.parametrize("over,status", REFUSED)
def test_both_refuse(over, status):
    for fn in (sparse, prefix):
        assert fn(**over) == status, B.last_error_detail()
        assert B.last_error_detail()


def test_reserved_fields():
    for i in range(2):
        c = cfg()
        c.reserved[i] = 1
        assert sparse(cfg=c) == INV and prefix(cfg=c) == INV


@pytest.mark.parametrize("over,status", [
    (dict(cfg=cfg(block_tokens=16)), UNS),
    (dict(cfg=cfg(block_tokens=100)), UNS),
    (dict(cfg=cfg(block_tokens=1056)), UNS),
    (dict(cfg=cfg(topk=0)), UNS),
    (dict(cfg=cfg(topk=65)), UNS),
    (dict(topk_ids=None), INV),
    (dict(topk_ids=BASE + 2), MIS),
])
def test_sparse_refuses(over, status):
    assert sparse(**over) == status, B.last_error_detail()


@pytest.mark.parametrize("over,status", [
    (dict(num_groups=-1), UNS),
    (dict(num_groups=513), UNS),
    (dict(group_start=None), INV),
    (dict(prefix_len=None), INV),
    (dict(prefix_offset=None), INV),
    (dict(group_start=BASE + 2), MIS),
    (dict(prefix_len=BASE + 1), MIS),
    (dict(prefix_offset=BASE + 4), MIS),
    (dict(launch_flags=B.MSA_LAUNCH_QUERY_RUNS), INV),
])
def test_prefix_refuses(over, status):
    assert prefix(**over) == status, B.last_error_detail()


def test_no_queries_is_ok_without_launch():
    assert sparse(num_queries=0, q=None, out=None, topk_ids=None, workspace=None, workspace_bytes=0) == B.MSA_OK
    assert prefix(num_queries=0, q=None, out=None, group_start=None, workspace=None, workspace_bytes=0) == B.MSA_OK


def test_workspace_size_and_refusals():
    n1 = B.msa_attention_workspace_bytes(cfg(), 64)
    assert 0 <= n1 <= 2**28
    # bounded however many queries, and never less with groups
    assert B.msa_attention_workspace_bytes(cfg(), 2**20) <= 2**29
    assert B.msa_attention_workspace_bytes(cfg(), 64, 5) >= 0
    assert B.msa_attention_workspace_bytes(cfg(), 0) >= 0
    for bad in (dict(cfg=cfg(head_dim=32), num_queries=1), dict(cfg=cfg(), num_queries=-1),
                dict(cfg=cfg(), num_queries=1, num_groups=513), dict(cfg=None, num_queries=1)):
        with pytest.raises(B.MsaError):
            B.msa_attention_workspace_bytes(**bad)
    if n1 > 0:
        assert sparse(num_queries=64, workspace_bytes=n1 - 1) == INV
        assert sparse(num_queries=64, workspace=None) == INV
        assert sparse(num_queries=64, workspace=BASE + 8) == MIS
    n2 = B.msa_attention_workspace_bytes(cfg(), 64, 2)
    if n2 > 0:
        assert prefix(num_queries=64, workspace_bytes=n2 - 1) == INV


def test_bf16_caches_need_no_scales_to_pass_the_checks():
    # the next check refuses, so that nothing is launched
    kw = dict(k_cache=cache(0, dtype=B.MSA_DTYPE_BF16), v_cache=cache(1, dtype=B.MSA_DTYPE_BF16), scales=None)
    assert sparse(**kw, workspace=BASE + 8) == MIS
    assert "workspace" in B.last_error_detail()


def test_tensor_functions_check_their_tensors():
    import torch
    q = torch.zeros(2, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attention_tensors(cfg(), q, None, None, None, None, None, None, None, None)


MB = 10**6


@pytest.mark.parametrize("heads", [(64, 8, 128), (8, 2, 64), (1, 1, 128), (128, 1, 64), (1024, 8, 128), (8192, 64, 128),
                                   (65536, 512, 128), (131072, 1024, 128)], ids=str)
def test_workspace_bounds(heads):
    """The sizes that the header states, at few and many heads and queries."""
    hq, hkv, d = heads
    c = cfg(num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    dense = cfg(num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    dense.topk = 0
    assert B.msa_attention_workspace_bytes(c, 0) == 0 and B.msa_attention_workspace_bytes(c, 0, 3) == 0
    for T in (1, 2, 7, 16, 33, 64, 100, 190, 256, 384, 385, 1000, 2**14):
        if T * hkv * -(-hq // hkv // 8) > 2**31 - 1:
            continue
        n = B.msa_attention_workspace_bytes(c, T)
        assert 0 < n < 30 * MB
        assert n < 4 * MB or T * hkv < 2**12, "tiles that are not split need no pieces"
        assert 0 < B.msa_attention_workspace_bytes(dense, T) < 4 * MB
        g = B.msa_attention_workspace_bytes(c, T, 3)
        rows = min(T, 384, max(1, 65536 // hq))
        assert n <= g
        assert g < 55 * MB + 2 * (rows * hq * (d + 4) * 4 + 256)
        assert g < 125 * MB or hq > 65536


def test_one_query_takes_little_workspace():
    assert B.msa_attention_workspace_bytes(cfg(), 1) < 3 * MB
    assert B.msa_attention_workspace_bytes(cfg(), 1, 1) < 6 * MB
    assert B.msa_attention_workspace_bytes(cfg(), 500) < 4 * MB


@pytest.mark.parametrize("T", [1, 5, 64, 400, 5000])
def test_workspace_too_small(T):
    n, g = B.msa_attention_workspace_bytes(cfg(), T), B.msa_attention_workspace_bytes(cfg(), T, 2)
    assert 0 < n and 0 < g
    for flags in (0, B.MSA_LAUNCH_QUERY_RUNS):
        assert sparse(num_queries=T, workspace_bytes=n - 1, launch_flags=flags) == INV
        assert sparse(num_queries=T, workspace=None, launch_flags=flags) == INV
        assert sparse(num_queries=T, workspace=BASE + 8, launch_flags=flags) == MIS
    assert prefix(num_queries=T, workspace_bytes=g - 1) == INV
    assert prefix(num_queries=T, workspace=None) == INV
    assert prefix(num_queries=T, workspace=BASE + 8) == MIS

"""The attention operators in workspaces of exactly the bytes they ask for (GPU): pieces of
tiles that few queries fill in part, many heads, windows of fewer queries."""
import pytest
import torch

from attention_cases import Problem
from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

RUNS = B.MSA_LAUNCH_QUERY_RUNS


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def guarded(p, flags, nbytes=None):
    """Runs and checks ``p`` with its workspace between guard bands, filled with NaN."""
    d = p.device()
    n = nbytes or B.msa_attention_workspace_bytes(d.cfg, p.T, 0 if p.groups is None else len(p.prefixes))
    raw = torch.full((n + 2 * 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    raw[4096:4096 + n] = 0xFF
    d.ws = raw[4096:4096 + n]
    d.run(flags).check()
    assert (raw[:4096] == 0xA5).all() and (raw[4096 + n:] == 0xA5).all()
    return d


@pytest.mark.parametrize("dtype,d", [("e4m3", 128), ("bf16", 128), ("e4m3", 64)])
@pytest.mark.parametrize("heads", [(8, 8), (3, 1), (64, 8), (40, 2), (128, 1)], ids=str)
@pytest.mark.parametrize("n", [1, 2, 3, 17])
@pytest.mark.parametrize("kind", ["runs", "prefix"])
def test_few_queries(kind, n, heads, dtype, d):
    if kind == "runs":
        p = Problem(111, lens=list(range(1500, 1500 + n)), seq_of=[0] * n, topk=8, heads=heads, dtype=dtype, head_dim=d)
    else:
        p = Problem(112, lens=[(50 * i) % 170 for i in range(n)], prefixes=(900,), groups=(0, n), ids=None, heads=heads,
                    dtype=dtype, head_dim=d)
    guarded(p, RUNS if kind == "runs" else 0)


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_windows_of_many_heads(dtype):
    """512 heads: windows of 128 queries behind prefixes, which cut groups."""
    p = Problem(113, lens=[(37 * i) % 140 for i in range(300)], prefixes=(300, 150, 70), groups=(3, 120, 131, 290), ids=None,
                heads=(512, 4), head_dim=64, dtype=dtype)
    guarded(p, 0)


def test_a_size_without_blocks():
    """A cfg with topk 0, for prefix attention alone, asks for less; so much is enough."""
    p = Problem(114, lens=(700, 0, 64, 3000, 5), ids=None, heads=(64, 8))
    cfg = p.cfg()
    cfg.topk = 0
    n = B.msa_attention_workspace_bytes(cfg, p.T)
    p.cfg = lambda: cfg
    guarded(p, 0, n)


def test_layers_share_a_workspace():
    """Two decode layers that run one after another in one workspace: the same bits as each
    in its own."""
    from paged_kv_cache_msa_gb300 import workloads as wl
    from paged_kv_cache_msa_gb300.device import DecodeLayer, DeviceWorkload
    w = wl.config2_decode64()
    pools = {k: torch.randint(0, 120, (n,), dtype=torch.uint8, device="cuda") for k, n in w.pools.items()}
    own = [DecodeLayer(DeviceWorkload(w, pools_on_device=pools), 144, topk=k, attention=True) for k in (16, 8)]
    first = DecodeLayer(DeviceWorkload(w, pools_on_device=pools), 144, attention=True)
    shared = [first, DecodeLayer(DeviceWorkload(w, pools_on_device=pools), 144, topk=8, attention=True,
                                 attn_workspace=first.attn_workspace)]
    s = torch.cuda.current_stream()
    for flags in (0, B.MSA_LAUNCH_PDL):
        for layers in (own, shared):
            for _ in range(3):
                for layer in layers:
                    layer.run(s, flags)
        torch.cuda.synchronize()
        for a, b in zip(own, shared):
            assert torch.equal(a.attn_out, b.attn_out) and torch.equal(a.attn_lse, b.attn_lse)

"""Calls from a host thread that has made no CUDA call before (GPU): the same outputs as from the
main thread.  Such a thread has no context of its own until a runtime call binds one."""
import threading

import pytest
import torch

import attention_cases
from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod
from paged_kv_cache_msa_gb300 import workloads as wl
from paged_kv_cache_msa_gb300.device import DeviceIndexer, DeviceProjection
from test_adapter_gpu import Case, runs
from test_projection_gpu import _batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def in_a_fresh_thread(call):
    errors = []

    def work():
        try:
            call()
        except Exception as e:       # raised below
            errors.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    if errors:
        raise errors[0]
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [5, 300])
def test_projection(tokens):
    pw = _batch(46, wl.TINY, tokens, 256)
    main, other = DeviceProjection(pw, rows_out=True), DeviceProjection(pw, rows_out=True)
    main.run()
    stream = torch.cuda.current_stream().cuda_stream
    in_a_fresh_thread(lambda: B.msa_projection_forward(*other.args(), stream=stream))
    assert torch.equal(main.rows_out, other.rows_out) and torch.equal(main.dw.q_out, other.dw.q_out)


@pytest.mark.parametrize("flags", [0, B.MSA_LAUNCH_QUERY_RUNS])
def test_indexer(flags):
    w = wl.indexer_decode64()
    main, other = DeviceIndexer(w), DeviceIndexer(w)
    main.run(launch_flags=flags)
    stream = torch.cuda.current_stream()
    in_a_fresh_thread(lambda: other.run(stream, launch_flags=flags))
    assert torch.equal(main.topk_ids, other.topk_ids)


@pytest.mark.parametrize("flags", [0, B.MSA_LAUNCH_QUERY_RUNS])
def test_attention(flags):
    d = attention_cases.Problem(3).device()
    stream = torch.cuda.current_stream()
    in_a_fresh_thread(lambda: d.run(flags, stream))
    d.check()


@pytest.mark.parametrize("tokens", [5, 300, 2600])
def test_adapters(tokens):
    c = Case(runs(tokens, 3), k=1000, adapters=3, rank=64)
    stream = torch.cuda.current_stream()
    in_a_fresh_thread(lambda: c.run(stream=stream))
    c.check()

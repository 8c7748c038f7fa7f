"""A layer's input side with adapters (GPU): the hidden states that they read, and everything that the
producer writes of their rows, with positions of one axis as well."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod
from paged_kv_cache_msa_gb300.device import LayerInput
from test_adapter_gpu import mixed, runs
from test_layer_input_gpu import Layer
from test_norm_gpu import F32, check_codes, close, expected
from test_rope_axes_gpu import BIG, TINY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def with_bf16_rows(layer, axes):
    c = layer.case
    layer.layer = LayerInput(c.cfg, layer.n, layer.weight, layer.weight_scales, layer.norm_w, c.weights, layer.desc, c.scales,
                             axes=c.axes if axes else None, adapters=layer.adapters, adapter_hidden=B.MSA_DTYPE_BF16)
    return layer


@pytest.mark.parametrize("n,order", [(1, mixed), (20, mixed), (300, mixed), (1500, runs)])
@pytest.mark.parametrize("k,rank", [(1000, 32), (2048, 64)])
def test_adapters_of_bf16_rows(n, order, k, rank):
    """The norm's bf16 rows go to the adapters, its codes to the projection: the rows are the
    projection of the one and the adapters' share of the other.  Tolerances as for codes (see
    Layer.check): the projection's rounding to bf16, the sums, u's parts, the sum's rounding."""
    layer = with_bf16_rows(Layer(n, TINY, k, rank, order=order, seed=n), axes=True)
    layer.run()
    own, c = layer.layer, layer.case
    assert torch.equal(layer.residual, (layer.x.float() + layer.before.float()).bfloat16())
    _, y, s = expected(layer.x, layer.before, layer.norm_w, 1e-6)
    codes = own.codes[:n].view(torch.float8_e4m3fn)
    check_codes(codes, own.hidden_scales[:n], y, s)
    close(own.hidden[:n], y, 2.0 ** -8 + F32)
    h = codes.to(torch.float64) * own.hidden_scales[:n, None].double()
    w = layer.weight.to(torch.float64) * layer.weight_scales[:, None].double()
    row = h @ w.T
    tol = 2.0 ** -8 * row.abs() + (k + 4) * 2.0 ** -24 * (h.abs() @ w.abs().T)
    d, hq, hkv, hiq, hik = c.shape[-1], *c.shape[:4]
    ends, rows16 = [0], own.hidden[:n].double()
    for heads in (hq, hkv, hkv, hiq, hik):
        ends.append(ends[-1] + heads * d)
    for a in range(layer.up.shape[0]):
        on = layer.ids == a
        for i in range(5):
            cols = slice(ends[i], ends[i + 1])
            dn, up = layer.down[a, i * rank:(i + 1) * rank].double(), layer.up[a, cols].double()
            row[on, cols] += float(layer.alpha[a]) * (rows16[on] @ dn.T @ up.T)
            size = float(layer.alpha[a]) * (rows16[on].abs() @ dn.abs().T @ up.abs().T)
            tol[on, cols] += size * ((k + rank + 8) * 2.0 ** -24 + 2.0 ** -16)
    tol += 2.0 ** -8 * row.abs() + 2.0 ** -8 * tol
    assert ((own.rows[:n].double() - row).abs() <= tol).all()
    c.rows, c.q, c.iq = own.rows[:n], own.q_out[:n], own.idx_q_out[:n]
    c.check()


def test_bf16_rows_are_nearer():
    """Than E4M3 codes: the adapters' share alone (a projection of zeros) against the unrounded norm."""
    off = []
    for bf16 in (False, True):
        layer = Layer(40, TINY, 1000, 16, seed=3, order=lambda n, _: [0] * n)
        layer.weight.view(torch.uint8).zero_()
        layer = with_bf16_rows(layer, axes=True) if bf16 else layer
        layer.run()
        _, y, _ = expected(layer.x, layer.before, layer.norm_w, 1e-6)
        d, rank = layer.case.shape[-1], 16
        q = slice(0, layer.case.shape[0] * d)
        want = float(layer.alpha[0]) * (y @ layer.down[0, :rank].double().T @ layer.up[0, q].double().T)
        off.append(float((layer.layer.rows[:40, q].double() - want).norm() / want.norm()))
    # a code is off by up to 2^-4 of itself, a bf16 value by 2^-8 (and the rows by 2^-8 in both)
    assert off[1] < 2.0 ** -7 < off[0]


@pytest.mark.parametrize("bf16", [False, True], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("n,shape", [(1, TINY), (90, BIG), (700, TINY)])
def test_one_axis(n, shape, bf16):
    """Without several axes the producer of one axis runs on the adapters' rows: compact Q and index-Q and
    every cache.  (Positions below 8: the angles' fp32 product and frequency are off by less than
    2^-21, within the tolerance of the norm and the sines.)"""
    layer = Layer(n, shape, 512, 16, axes=False, seed=n)
    layer.case.positions.copy_((torch.arange(n, device="cuda") % 8).to(torch.int32).expand(3, -1))
    if bf16:
        layer = with_bf16_rows(layer, axes=False)
    layer.run()
    if not bf16:
        layer.check()
    c, own = layer.case, layer.layer
    c.rows, c.q, c.iq = own.rows[:n], own.q_out[:n], own.idx_q_out[:n]
    c.check()


def test_hidden_types_that_are_none():
    with pytest.raises(ValueError):
        layer = Layer(3, TINY, 512, 16)
        c = layer.case
        LayerInput(c.cfg, 3, layer.weight, layer.weight_scales, layer.norm_w, c.weights, layer.desc, c.scales,
                   adapters=layer.adapters, adapter_hidden=7)

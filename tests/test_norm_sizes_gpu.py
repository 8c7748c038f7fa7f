"""The norm of as many rows as take each of its kernels (GPU): threads of two to seven vectors of 8
elements, rows of one warp of which eight share a CTA, last CTAs and last vectors that are short.

Tolerances as for smaller batches: a thread adds up to 56 squares, five shuffles follow, then up to 8
warps of such threads (a thread of two vectors adds 16, and 32 warps follow): fewer than 70 roundings
of 2^-24 in the sum, which the square root halves, and ten more: below 2^-18 of a value."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod
from test_norm_gpu import F32, check_codes, close, expected, guarded, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def rows_from(k):
    """The rows from which on a thread has more vectors than one (the GPU's warps filled twice)."""
    warps = -(-(-(-k // 8)) // 32)
    return 2 * 152 * 32 // warps + 1


# vectors a thread:              2    2    3    3    4     4     4     5     5     7     7     7     5     5
@pytest.mark.parametrize("k", [264, 509, 520, 768, 1000, 1021, 1024, 1280, 1279, 1544, 1790, 1792, 2560, 5120,
                               # and rows of several warps with   3     7     4     7     2      3      2
                               6144, 7168, 8192, 8200, 12280, 12288, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_of_each_kernel(k, residual):
    for t in (rows_from(k), rows_from(k) + (5 - rows_from(k)) % 8 + 8):       # at the step, and 5 rows in the last eight
        x, w = make(t, k, pad=1), make(1, k, seed=2)[0].contiguous()
        res = make(t, k, seed=3, scale=4.0) if residual else None
        out, out_ok = guarded(t, k, torch.bfloat16)
        codes, codes_ok = guarded(t, k, torch.float8_e4m3fn, pad=2)
        res_out, res_ok = guarded(t, k, torch.bfloat16, pad=3) if residual else (None, lambda: True)
        scales = torch.full((t,), -1.0, device="cuda")
        B.norm_tensors(B.make_norm_cfg(k, rms_eps=1e-6), x, w, residual=res, residual_out=res_out, out=out, codes=codes,
                       scales=scales)
        _, y, s = expected(x, res, w, 1e-6)
        close(out, y, 2.0 ** -8 + F32)
        check_codes(codes, scales, y, s)
        if residual:
            assert torch.equal(res_out, (x.float() + res.float()).bfloat16())
        assert out_ok() and codes_ok() and res_ok()


@pytest.mark.parametrize("k", [264, 520, 1024, 1280, 1544, 2560])
def test_the_same_bits_in_either_kernel(k):
    """A batch with few rows takes one vector a thread, the same rows among many several: the outputs of
    both are within a step of each other, and equal where the sum is exact (rows of powers of two)."""
    t = rows_from(k) + 3
    gen = torch.Generator(device="cuda").manual_seed(k)
    x = torch.exp2(torch.randint(-3, 4, (t, k), generator=gen, device="cuda").float()).bfloat16()
    w = torch.exp2(torch.randint(-2, 3, (k,), generator=gen, device="cuda").float()).bfloat16()
    cfg = B.make_norm_cfg(k, rms_eps=1e-6)

    def run(rows):
        out, codes = torch.empty_like(rows), torch.empty(rows.shape[0], -(-k // 16) * 16, dtype=torch.uint8, device="cuda")[:, :k]
        scales = torch.empty(rows.shape[0], device="cuda")
        B.norm_tensors(cfg, rows, w, out=out, codes=codes, scales=scales)
        return out, codes, scales

    many, few = run(x), run(x[:50].contiguous())
    for a, b in zip(many, few):
        assert torch.equal(a[:50], b)


@pytest.mark.parametrize("k", [264, 1280, 1792, 7168])
def test_far_magnitudes_and_values_that_are_not_finite(k):
    """Rows whose squares leave the range of fp32, zeros and rows with a NaN or an infinity among many others."""
    t = rows_from(k) + 6
    x, w = make(t, k).contiguous(), (0.5 + torch.rand(k, device="cuda")).bfloat16()
    for i, size in ((1, 1e-37), (2, 1e30), (t - 1, 2e38), (t - 2, 1e-19)):
        x[i] = (x[i].double() / x[i].double().abs().max() * size).bfloat16()
    x[7], x[8, k - 1], x[9, 0] = 0, float("nan"), float("-inf")
    codes = torch.empty(t, -(-k // 16) * 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :k]
    out, scales = torch.empty_like(x), torch.empty(t, device="cuda")
    B.norm_tensors(B.make_norm_cfg(k, rms_eps=0.0), x, w, out=out, codes=codes, scales=scales)
    assert out[7].isnan().all() and scales[7].isnan()            # eps 0: 0 / 0
    assert scales[8].isnan() and out[8].isnan().all() and scales[9].isnan() and (out[9, 1:] == 0).all()
    rest = torch.ones(t, dtype=torch.bool, device="cuda")
    rest[7:10] = False
    _, y, s = expected(x[rest], None, w, 0.0)
    close(out[rest], y, 2.0 ** -8 + F32)
    check_codes(codes[rest], scales[rest], y, s)

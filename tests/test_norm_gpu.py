"""The norm with the residual's addition and 8-bit output against its formula in 64 bits (GPU).

Tolerances.  fp32 arithmetic: the sum of K squares is added in runs of at most 32 products a
thread, five shuffles and at most 32 warps, so it is off by less than 70 roundings of 2^-24; the
square root halves that, rsqrtf and the products add ten more roundings: 2^-18 of a value covers
them.  Then each output's own rounding: 2^-8 of it in bf16; 2^-4 in E4M3, or half of the smallest
step 2^-9 where a code is below 2^-6.  A code also moves with its scale, by 2^-18 of itself."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def make(t, k, pad=0, seed=1, scale=1.0):
    """Rows of k values in a wider tensor whose other elements are NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000 + k)
    wide = torch.full((t, -(-k // 16) * 16 + 16 * pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = torch.randn(t, k, generator=gen, device="cuda") * scale
    x[:, 3 % k] *= 30.0
    wide[:, :k] = x
    return wide[:, :k]


def guarded(t, k, dtype, pad=0):
    """An output of rows between guard values, and a check that those stayed."""
    width = -(-k // 16) * 16 + 16 * pad
    raw = torch.full(((t + 2) * width * dtype.itemsize,), 0x5B, dtype=torch.uint8, device="cuda")
    view = raw.view(dtype).view(t + 2, width)

    def untouched():
        r = raw.view(t + 2, -1)
        return bool((r[0] == 0x5B).all() and (r[-1] == 0x5B).all() and (r[1:-1, k * dtype.itemsize:] == 0x5B).all())

    return view[1:-1, :k], untouched


def expected(x, res, w, eps):
    h = x.double() if res is None else x.double() + res.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w.double()
    return h, y, y.abs().amax(1).clamp(min=2.0 ** -100) / 448


def close(got, want, rel, absolute=0.0):
    err = (got.double() - want).abs()
    assert (err <= rel * want.abs() + absolute).all(), float((err - rel * want.abs()).max())


def check_codes(codes, scales, y, s):
    close(scales, s, F32)
    want = y / s[:, None]
    close(codes, want, 2.0 ** -4 + F32, 2.0 ** -10)
    assert (codes.double().abs().amax(1) >= 416).all()          # the largest uses the whole range


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 64, 100, 255, 256, 1001, 2048, 2049, 6144, 8192, 8200, 12288, 16383, 16384])
@pytest.mark.parametrize("t", [1, 3, 305])
@pytest.mark.parametrize("residual", [False, True])
def test_sizes(k, t, residual):
    """Every number of vectors a thread, rows that share a CTA, short last vectors."""
    x, w = make(t, k, pad=1), make(1, k, seed=2)[0].contiguous()
    res = make(t, k, seed=3, scale=4.0) if residual else None
    out, out_ok = guarded(t, k, torch.bfloat16)
    codes, codes_ok = guarded(t, k, torch.float8_e4m3fn, pad=2)
    res_out, res_ok = guarded(t, k, torch.bfloat16, pad=3) if residual else (None, lambda: True)
    scales = torch.full((t,), -1.0, device="cuda")
    B.norm_tensors(B.make_norm_cfg(k, rms_eps=1e-6), x, w, residual=res, residual_out=res_out, out=out, codes=codes,
                   scales=scales)
    h, y, s = expected(x, res, w, 1e-6)
    close(out, y, 2.0 ** -8 + F32)
    check_codes(codes, scales, y, s)
    if residual:
        assert torch.equal(res_out, (x.float() + res.float()).bfloat16())
    assert out_ok() and codes_ok() and res_ok()


@pytest.mark.parametrize("outs", ["out", "codes", "both"])
@pytest.mark.parametrize("t", [1, 1000])
def test_each_output_alone(outs, t):
    x, w, res = make(t, 640), make(1, 640, seed=2)[0].contiguous(), make(t, 640, seed=3)
    _, y, s = expected(x, res, w, 1e-5)
    out = torch.empty(t, 640, dtype=torch.bfloat16, device="cuda") if outs != "codes" else None
    codes = torch.empty(t, 640, dtype=torch.uint8, device="cuda") if outs != "out" else None
    scales = torch.empty(t, device="cuda") if outs != "out" else None
    B.norm_tensors(B.make_norm_cfg(640, rms_eps=1e-5), x, w, residual=res, out=out, codes=codes, scales=scales)
    if out is not None:
        close(out, y, 2.0 ** -8 + F32)
    if codes is not None:
        check_codes(codes.view(torch.float8_e4m3fn), scales, y, s)


@pytest.mark.parametrize("k", [72, 6144])
def test_in_place(k):
    """The residual updated where it is, the norm in the place of x: the bits of separate outputs."""
    x, w, res = make(37, k), make(1, k, seed=2)[0].contiguous(), make(37, k, seed=3)
    cfg = B.make_norm_cfg(k)
    a, b = torch.empty(37, k, dtype=torch.bfloat16, device="cuda"), torch.empty(37, k, dtype=torch.bfloat16, device="cuda")
    B.norm_tensors(cfg, x, w, residual=res, residual_out=a, out=b)
    x2, res2 = x.clone(), res.clone()
    B.norm_tensors(cfg, x2, w, residual=res2, residual_out=res2, out=x2)
    assert torch.equal(a, res2) and torch.equal(b, x2)
    x3, res3 = x.clone(), res.clone()
    B.norm_tensors(cfg, x3, w, residual=res3, residual_out=x3, out=res3)
    assert torch.equal(a, x3) and torch.equal(b, res3)


@pytest.mark.parametrize("k", [64, 6144])
@pytest.mark.parametrize("size", [1e-37, 1e-30, 1e-19, 1e19, 1e30, 2e38])
def test_far_magnitudes(size, k):
    """Rows whose squares leave the range of fp32, beside ordinary ones.  (Inputs below 2^-126 are
    not normal numbers: the tolerance is theirs, of the bf16 input, not of the norm.)"""
    x, w = make(5, k), (0.5 + torch.rand(k, device="cuda")).bfloat16()
    x = x.contiguous()
    x[1] = (x[1].double() / x[1].double().abs().max() * size).bfloat16()
    x[3] = (x[3].double() / x[3].double().abs().max() * size).bfloat16()
    out, codes, scales = torch.empty_like(x), torch.empty_like(x, dtype=torch.float8_e4m3fn), torch.empty(5, device="cuda")
    B.norm_tensors(B.make_norm_cfg(k, rms_eps=0.0), x, w, out=out, codes=codes, scales=scales)
    _, y, s = expected(x, None, w, 0.0)
    close(out, y, 2.0 ** -8 + F32)
    check_codes(codes, scales, y, s)


@pytest.mark.parametrize("k", [48, 6144])
def test_zeros_and_values_that_are_not_finite(k):
    x, w = make(6, k).contiguous(), make(1, k, seed=2)[0].contiguous()
    good = x.clone()
    x[0] = 0
    x[2, k - 1] = float("nan")
    x[4, 0] = float("inf")
    out, codes, scales = torch.empty_like(x), torch.empty_like(x, dtype=torch.float8_e4m3fn), torch.empty(6, device="cuda")
    B.norm_tensors(B.make_norm_cfg(k), x, w, out=out, codes=codes, scales=scales)
    assert (out[0] == 0).all() and (codes[0].float() == 0).all() and scales[0] > 0 and scales[0] <= 2.0 ** -108
    assert scales[2].isnan() and scales[4].isnan()
    assert out[2].isnan().all() and out[4, 0].isnan() and (out[4, 1:] == 0).all()
    _, y, s = expected(good, None, w, 1e-6)
    for i in (1, 3, 5):
        close(out[i], y[i], 2.0 ** -8 + F32)
        check_codes(codes[i:i + 1], scales[i:i + 1], y[i:i + 1], s[i:i + 1])


def test_no_tokens_and_repeated_calls():
    cfg, w = B.make_norm_cfg(512), make(1, 512)[0].contiguous()
    empty = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    B.norm_tensors(cfg, empty, w, out=empty)
    x = make(2000, 512)
    a, b = (torch.empty(2000, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.norm_tensors(cfg, x, w, out=a)
    B.norm_tensors(cfg, x, w, out=b)
    assert torch.equal(a, b)


def test_other_stream_and_graph():
    """On a stream of its own behind the work that makes its input; captured and replayed with
    new values in the same tensors, with and without programmatic dependent launch."""
    cfg, w = B.make_norm_cfg(6144), make(1, 6144, seed=2)[0].contiguous()
    x, src = torch.zeros(64, 6144, dtype=torch.bfloat16, device="cuda"), make(64, 6144, seed=5)
    res, res_out, out = make(64, 6144, seed=6), torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    for flags in (0, B.MSA_LAUNCH_PDL):
        x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
            x.copy_(src)
            B.norm_tensors(cfg, x, w, residual=res, residual_out=res_out, out=out, launch_flags=flags)
        s.synchronize()
        _, y, _ = expected(src, res, w, 1e-6)
        close(out, y, 2.0 ** -8 + F32)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.norm_tensors(cfg, x, w, residual=res, residual_out=res_out, out=out, launch_flags=flags)
            # the next layer's norm, of what this one wrote
            B.norm_tensors(cfg, out, w, residual=res_out, residual_out=x, launch_flags=flags, out=out)
        for seed in (7, 8):
            new = make(64, 6144, seed=seed)
            x.copy_(new)
            g.replay()
            torch.cuda.synchronize()
            _, y, _ = expected(new, res, w, 1e-6)
            h = (new.float() + res.float()).bfloat16()
            _, y2, _ = expected(y.bfloat16(), h, w, 1e-6)
            # the first norm's own rounding, 2^-8 of it, may fall the other way (a step, 2^-7); the
            # second adds the residual to it, normalises (no more than the largest |w| over the row's
            # rms, which is over 1 here) and rounds
            assert ((out.double() - y2).abs() <= 2.0 ** -8 * y2.abs() + 2.0 ** -6 * y.abs() * w.double().abs()
                    + 2.0 ** -14 * y2.abs()).all()


def test_tensors_that_do_not_fit_are_refused():
    cfg, x, w = B.make_norm_cfg(64), make(4, 64), make(1, 64)[0].contiguous()
    good = dict(out=torch.empty(4, 64, dtype=torch.bfloat16, device="cuda"))
    for bad in (dict(residual=x[:3]), dict(out=x.float()), dict(residual=x.cpu()), dict(out=torch.empty_like(x.T)),
                dict(codes=torch.empty_like(x, dtype=torch.uint8), scales=torch.empty(3, device="cuda"))):
        with pytest.raises(ValueError):
            B.norm_tensors(cfg, x, w, **dict(good, **bad))
    with pytest.raises(ValueError):
        B.norm_tensors(cfg, x, w[:63], **good)
    with pytest.raises(B.MsaError):
        B.norm_tensors(cfg, x, w)


def test_flags_that_are_no_flags():
    """Also those whose low 32 bits are."""
    cfg, x, w = B.make_norm_cfg(64), make(4, 64), make(1, 64)[0].contiguous()
    out = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for flags in (2**32, 2**32 + B.MSA_LAUNCH_PDL, 2**31, -2**32, 2**40):
        with pytest.raises(ValueError):
            B.norm_tensors(cfg, x, w, out=out, launch_flags=flags)
    for flags in (64, -1):
        with pytest.raises(B.MsaError):
            B.norm_tensors(cfg, x, w, out=out, launch_flags=flags)
    assert (out == 0).all()

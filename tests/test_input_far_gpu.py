"""The layer's input side where offsets pass 32 bits (GPU): rows, tables of adapters and batches of
more than 2^31 elements, of which some rows are checked against the formula in 64 bits (tolerances as
for small ones)."""
import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod
from test_norm_gpu import F32, check_codes, close, expected

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    yield B.load()
    torch.cuda.empty_cache()


def check_rows(got, rows, x, down, up, alpha, ids, some):
    """Tokens `some` of one slice's adapters."""
    k, rank = x.shape[1], up.shape[2]
    for t in some:
        a = int(ids[t])
        want, size = rows[t].double(), torch.zeros(up.shape[1], dtype=torch.float64, device="cuda")
        if 0 <= a < up.shape[0]:
            c = float(alpha[a])
            want = want + c * (up[a].double() @ (down[a].double() @ x[t].double()))
            size = abs(c) * (up[a].double().abs() @ (down[a].double().abs() @ x[t].double().abs()))
        err = (got[t].double() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + size * ((k + rank + 8) * 2.0 ** -24 + 2.0 ** -16)).all(), t


def adapters(n, w, rank, k, gen):
    down = torch.empty(n, rank, k, dtype=torch.bfloat16, device="cuda").normal_(generator=gen).mul_(k ** -0.5)
    up = torch.empty(n, w, rank, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return down, up, 0.5 + torch.rand(n, generator=gen, device="cuda")


@pytest.mark.parametrize("in_place", [False, True])
def test_most_tokens(in_place):
    """2^24 tokens of 136 columns: 2.3e9 elements of rows, 2^17 tiles and more."""
    t, w, k, rank, n = 2**24, 136, 64, 8, 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(t, k, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    rows = torch.empty(t, w, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    down, up, alpha = adapters(n, w, rank, k, gen)
    ids = torch.randint(-1, n, (t,), generator=gen, device="cuda", dtype=torch.int32)
    cfg = B.make_adapter_cfg(k, (w,), rank, n)
    some = [0, 1, 127, 128, 2**23 - 1, 15_790_320, 15_790_321, 2**24 - 129, 2**24 - 2, 2**24 - 1]
    before = {i: rows[i].clone() for i in some}
    out = rows if in_place else torch.empty_like(rows)
    B.adapter_tensors(cfg, x, down, up, ids, rows, out, adapter_scales=alpha)
    check_rows(out, before, x, down, up, alpha, ids, some)
    none = (ids < 0).nonzero().flatten()[-50_000:]
    if not in_place:
        assert torch.equal(out[none].view(torch.int16), rows[none].view(torch.int16))


@pytest.mark.parametrize("t", [5, 40, 300])
def test_rows_far_apart(t):
    """Rows of a wide tensor: the last ones lie past 2^32 bytes and 2^31 elements of each."""
    k, w, rank, n = 256, 136, 16, 4
    stride = -(-(2**31 + 2**20) // (t - 1)) // 16 * 16 + 16
    gen = torch.Generator(device="cuda").manual_seed(t)
    far = lambda width: torch.empty(stride * (t - 1) + width, dtype=torch.bfloat16, device="cuda").as_strided((t, width), (stride, 1))
    x, rows, out = far(k), far(w), far(w)
    assert (t - 1) * stride > 2**31
    x.copy_(torch.randn(t, k, generator=gen, device="cuda"))
    rows.copy_(torch.randn(t, w, generator=gen, device="cuda"))
    down, up, alpha = adapters(n, w, rank, k, gen)
    ids = torch.tensor([i % (n + 1) - 1 for i in range(t)], dtype=torch.int32, device="cuda")
    B.adapter_tensors(B.make_adapter_cfg(k, (w,), rank, n), x, down, up, ids, rows, out, adapter_scales=alpha)
    check_rows(out, rows, x, down, up, alpha, ids, range(t))
    norm_w = torch.rand(k, generator=gen, device="cuda").bfloat16()
    res = far(k)
    res.copy_(torch.randn(t, k, generator=gen, device="cuda"))
    before = res.clone()
    src = x.clone()
    codes = torch.empty(stride * (t - 1) + k, dtype=torch.uint8, device="cuda").as_strided((t, k), (stride, 1))
    scales = torch.empty(t, device="cuda")
    B.norm_tensors(B.make_norm_cfg(k), x, norm_w, residual=res, residual_out=res, out=x, codes=codes, scales=scales)
    _, want, s = expected(src, before, norm_w, 1e-6)
    close(x, want, 2.0 ** -8 + F32)
    check_codes(codes.contiguous().view(torch.float8_e4m3fn), scales, want, s)
    assert torch.equal(res, (src.float() + before.float()).bfloat16())


@pytest.mark.parametrize("t", [1, 12, 100, 400, 3500])
@pytest.mark.parametrize("which", ["down", "up"])
def test_tables_of_adapters(t, which):
    """16,384 adapters, of which the last lie past 2^31 elements of down or up."""
    n, rank = 16384, 8
    k, w = (17000, 64) if which == "down" else (64, 17000)
    gen = torch.Generator(device="cuda").manual_seed(t)
    down, up, alpha = adapters(n, w, rank, k, gen)
    assert max(down.numel(), up.numel()) > 2**31
    x = torch.randn(t, k, generator=gen, device="cuda").bfloat16()
    rows = torch.randn(t, w, generator=gen, device="cuda").bfloat16()
    ids = torch.tensor([n - 1 - (i * i) % 7 * 1000 if i % 5 != 4 else (0, n, -1)[i // 5 % 3] for i in range(t)], dtype=torch.int32,
                       device="cuda")
    out = torch.empty_like(rows)
    B.adapter_tensors(B.make_adapter_cfg(k, (w,), rank, n), x, down, up, ids, rows, out, adapter_scales=alpha)
    check_rows(out, rows, x, down, up, alpha, ids, range(0, t, -(-t // 120)))


def test_norm_of_more_than_2_to_the_31():
    t, k = 262_149, 8208
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(t, k, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.rand(k, generator=gen, device="cuda").bfloat16()
    out = torch.empty_like(x)
    codes, scales = torch.empty(t, k, dtype=torch.uint8, device="cuda"), torch.empty(t, device="cuda")
    B.norm_tensors(B.make_norm_cfg(k), x, w, out=out, codes=codes, scales=scales)
    some = torch.tensor([0, 1, 131_070, 131_075, 261_630, 261_633, t - 2, t - 1], device="cuda")
    _, y, s = expected(x[some], None, w, 1e-6)
    close(out[some], y, 2.0 ** -8 + F32)
    check_codes(codes[some].view(torch.float8_e4m3fn), scales[some], y, s)

"""Every kernel of the FP8 product in each of its forms, by the rule that chooses them; rows that depend on nothing but
themselves; the value tests of the product again, with comparisons that NaN cannot pass."""
import pytest
import torch

import strict_checks as strict
import test_gpu_fp8 as fp8
from test_host_fp8_tiles import STREAM, T64X32, T64X64, T64X128, T128X128, T256X256, choose  # noqa: F401

pytestmark = pytest.mark.gpu
# K of each form: whole K-blocks or a last one that is cut, and their number a multiple of four (the scales' copies) or not
FORMS = {"four": 512, "four, cut": 400, "one": 384, "one, cut": 272, "many": 2816, "many, cut": 2000}
SIZES = {STREAM: [(1, 4096), (7, 1001)], T64X32: [(9, 4096), (33, 2001), (64, 8192)], T64X64: [(128, 8192), (100, 5003)],
         T64X128: [(400, 5000), (333, 4999)], T128X128: [(2048, 4096), (1901, 3333)], T256X256: [(4096, 3200), (4000, 3333)]}
CASES = [(kernel, b, n) for kernel, sizes in SIZES.items() for b, n in sizes]


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kernel,b,n", CASES)
def test_every_form_of_every_kernel(nv, choose, kernel, b, n, form):  # noqa: F811
    K = FORMS[form]
    assert choose([(b, n)])[0][0] == kernel
    ops = fp8.exact_operands(b, n, K, seed=b + n + K)
    want, _ = fp8.binary64(*ops)
    for dtype in (torch.float16, torch.bfloat16):
        assert torch.equal(nv.fp8_gemm(*ops, out_dtype=dtype), want.to(dtype))
    ops = fp8.operands(b, n, K, seed=b + n)
    strict.fp8_check(nv.fp8_gemm(*ops), *fp8.binary64(*ops), K)


@pytest.mark.parametrize("K", [512, 400])
@pytest.mark.parametrize("kernel,b,n", CASES)
def test_scales_at_any_four_bytes(nv, choose, kernel, b, n, K):  # noqa: F811
    a, sa, w, sw = fp8.exact_operands(b, n, K, seed=b)
    want = fp8.binary64(a, sa, w, sw)[0].half()
    for da, dw in ((1, 0), (0, 1), (2, 3)):
        xa, xw = (torch.zeros(s.numel() + d, device="cuda")[d:].view(s.shape).copy_(s) for s, d in ((sa, da), (sw, dw)))
        assert torch.equal(nv.fp8_gemm(a, xa, w, xw), want), (da, dw)


@pytest.mark.parametrize("K", [384, 400])
@pytest.mark.parametrize("kernel,b,n", CASES)
def test_a_row_depends_on_itself_alone(nv, choose, kernel, b, n, K):  # noqa: F811
    """All other rows of a and their scales are replaced: the bits of a row stay.  The same of the columns and w, whose
    scales a column shares with its 128."""
    a, sa, w, sw = fp8.operands(b, n, K, seed=1)
    oa, osa, ow, osw = fp8.operands(b, n, K, seed=2)
    y = nv.fp8_gemm(a, sa, w, sw)
    for row in {0, b // 2, b - 1}:
        xa, xs = oa.clone(), osa * 3
        xa.view(torch.uint8)[row], xs[row] = a.view(torch.uint8)[row], sa[row]
        z = nv.fp8_gemm(xa, xs, w, sw)
        assert torch.equal(z[row], y[row]), row
        assert b == 1 or not torch.equal(z, y)
    for col in {0, n // 2, n - 1}:
        xw, xs = ow.clone(), osw * 3
        xw.view(torch.uint8)[col], xs[col // 128] = w.view(torch.uint8)[col], sw[col // 128]
        z = nv.fp8_gemm(a, sa, xw, xs)
        assert torch.equal(z[:, col], y[:, col]), col


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", fp8.SIZES)
def test_product_strictly(nv, monkeypatch, size, dtype):
    monkeypatch.setattr(fp8, "check", strict.fp8_check)
    fp8.test_product(nv, size, dtype)


@pytest.mark.parametrize("size", [(4096, 3200, 400), (4000, 3333, 272), (2048, 8192, 1024)])
def test_many_tiles_strictly(nv, monkeypatch, size):
    monkeypatch.setattr(fp8, "check", strict.fp8_check)
    fp8.test_product_of_many_tiles(nv, size)


def test_the_most_rows(nv, choose):  # noqa: F811
    """2^29 rows of one column: offsets beyond 2^33, and more workgroups of 64 x 64 than a launch takes."""
    B, period = 1 << 29, (1 << 20) - 3
    assert choose([(B, 1)])[0][0] == T128X128
    a, sa, w, sw = fp8.exact_operands(period, 1, 16, seed=5)
    want = fp8.binary64(a, sa, w, sw)[0].half().view(-1)
    times = -(-B // period)
    many = a.view(torch.uint8).repeat(times, 1)[:B].view(fp8.FP8)
    y = nv.fp8_gemm(many, sa.repeat(times, 1)[:B], w, sw).view(-1)
    for at in range(0, B, period):
        part = y[at:at + period]
        assert torch.equal(part, want[:len(part)]), at

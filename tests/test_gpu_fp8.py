"""E4M3 quantization with a scale per 128 values and the product of such operands."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
TINY = np.float32(2.0 ** -126)


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def blocks_amax(y, block_rows):
    rows, k = y.shape
    p = np.zeros((-(-rows // block_rows) * block_rows, -(-k // 128) * 128), y.dtype)
    p[:rows, :k] = np.abs(y)
    return p.reshape(-1, block_rows, p.shape[1] // 128, 128).max((1, 3))


def spread(scale, block_rows, rows, k):
    return np.repeat(np.repeat(scale, block_rows, 0), 128, 1)[:rows, :k]


def quantize_ref(x, block_rows):
    """Codes and scales by the written binary32 steps (numpy rounds each of them once)."""
    y = x.float().numpy()
    scale = np.maximum(blocks_amax(y, block_rows) / np.float32(448), TINY)
    inv = spread(np.float32(1) / scale, block_rows, *y.shape)
    return torch.from_numpy(y * inv).to(FP8), scale


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 16), (3, 128), (5, 144), (130, 2064), (257, 112), (64, 4096), (1000, 1040)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_equals_the_definition(nv, shape, block_rows, dtype):
    g = torch.Generator().manual_seed(sum(shape) + block_rows)
    x = torch.randn(shape, generator=g)
    x[:, ::37] *= 40
    x[0] *= 1e-3
    x[-1, : shape[1] // 2] = 0
    x = x.to(dtype)
    got = nv.fp8_quantize(x.cuda(), block_rows=block_rows)
    codes, scale = quantize_ref(x, block_rows)
    assert np.array_equal(got["scale"].cpu().numpy(), scale)
    assert torch.equal(got["codes"].cpu().view(torch.uint8), codes.view(torch.uint8))


def test_quantize_unaligned_is_the_same(nv):
    x = torch.randn(3 * 272 + 1).bfloat16().cuda()
    for block_rows in (1, 128):
        out = {"codes": torch.zeros(3 * 272 + 3, dtype=torch.uint8, device="cuda")[3:].view(3, 272).view(FP8),
               "scale": torch.zeros((3 if block_rows == 1 else 1, 3), device="cuda")}
        got = nv.fp8_quantize(x[1:].view(3, 272), block_rows=block_rows, out=out)
        codes, scale = quantize_ref(x[1:].view(3, 272).cpu(), block_rows)
        assert np.array_equal(got["scale"].cpu().numpy(), scale)
        assert torch.equal(got["codes"].cpu().view(torch.uint8), codes.view(torch.uint8))


def test_quantize_ends_of_the_range(nv):
    """Blocks of zeros, of the smallest and largest numbers, with infinities and NaN."""
    x = torch.zeros((8, 128), dtype=torch.bfloat16)
    x[1] = 2.0 ** -133                     # the smallest bf16
    x[2, 5] = torch.finfo(torch.bfloat16).max
    x[3] = 448 * 2.0 ** -126
    x[4], x[4, 7] = 1.0, float("inf")
    x[5], x[5, 9] = 2.0, float("nan")
    x[6] = torch.arange(128).bfloat16() * -3.5
    x[7, 0], x[7, 1] = -0.0, 2.0 ** -126
    got = nv.fp8_quantize(x.cuda())
    codes, scale = got["codes"].float().cpu(), got["scale"].cpu()[:, 0]
    ref, ref_scale = quantize_ref(x[[0, 1, 2, 3, 6, 7]], 1)
    rows = [0, 1, 2, 3, 6, 7]
    assert torch.equal(got["codes"].cpu()[rows].view(torch.uint8), ref.view(torch.uint8))
    assert np.array_equal(scale[rows].numpy(), ref_scale[:, 0])
    assert scale[4] == float("inf") and codes[4, 7].isnan() and (codes[4, :7] == 0).all()
    assert scale[5] == np.float32(2) / np.float32(448) and codes[5, 9].isnan() and (codes[5, :9] == 448).all()


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_with_activation(nv, act, dtype, block_rows):
    """Values within half a step of E4M3 of the binary64 activation (2^-4 of the value, 2^-10 scales below the
    normal range), with 2^-18 for the activation and the scale in binary32 (|gate| <= 120: the exponent's
    argument is rounded to 2^-17.2 at most there, where the activation is below 2^-160; up to |gate| = 30 it is
    2^-19)."""
    rows, k = 200, 656
    g = torch.Generator().manual_seed(7)
    x = torch.randn((rows, 2 * k if act == "swiglu" else k), generator=g) * 4
    x[3] *= 30
    x[:, 40:60] *= 1e-4
    x = x.to(dtype)
    y = x.double().numpy()
    if act == "swiglu":
        gate, up = y[:, :k], y[:, k:]
        y = gate / (1 + np.exp(-gate)) * up
    else:
        y = np.maximum(y, 0) ** 2
    got = nv.fp8_quantize(x.cuda(), block_rows=block_rows, act=act)
    scale = got["scale"].cpu().double().numpy()
    want = np.maximum(blocks_amax(y, block_rows) / 448, float(TINY))
    assert (np.abs(scale - want) <= want * 2.0 ** -18).all()
    s = spread(scale, block_rows, rows, k)
    off = np.abs(got["codes"].float().cpu().double().numpy() * s - y)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) * (1 + 2.0 ** -14) + 2.0 ** -18 * np.abs(y)).all()


# ---------------------------------------------------------------- the product

def operands(B, N, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nkb = -(-K // 128)
    a = (torch.randn((B, K), generator=g, device="cuda") * 100).clamp(-448, 448).to(FP8)
    w = (torch.randn((N, K), generator=g, device="cuda") * 100).clamp(-448, 448).to(FP8)
    sa = torch.rand((B, nkb), generator=g, device="cuda") * 2.0 ** -8 + 2.0 ** -12
    sw = torch.rand((-(-N // 128), nkb), generator=g, device="cuda") * 2.0 ** -9 + 2.0 ** -13
    return a, sa, w, sw


def binary64(a, sa, w, sw):
    """(product, sum of the terms' sizes) in binary64."""
    K, N = a.shape[1], w.shape[0]
    x = a.float().double() * sa.double().repeat_interleave(128, 1)[:, :K]
    y = w.float().double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x @ y.t(), x.abs() @ y.abs().t()


def check(y, want, size, K):
    """Half a step of the type, and what the sums may add to the terms' sizes.  The matrix instruction joins eight
    neighbouring products at a time, each cut to a multiple of 2^(ea + eb - 13) where 2^(ea + eb) is the power of
    two in the largest of the eight (measured: beside 256 * 256 a product of 8 stays, of 12 becomes 8, of 4
    vanishes).  2^(ea + eb) is at most that product, so seven others lose less than 7 * 2^-13 of the eight's
    sizes.  Beyond that binary32: 16 sums of eight, one addition per K-block, the scale's two roundings, each
    off by at most 2^-23 of the sizes."""
    eps = torch.finfo(y.dtype).eps / 2
    room = (7 * 2.0 ** -13 + (16 + -(-K // 128) + 3) * 2.0 ** -23) * size
    off = (y.double() - want).abs()
    bad = off > eps * want.abs() * (1 + 2.0 ** -8) + room * (1 + eps) + (2.0 ** -25 if y.dtype is torch.float16 else 0)
    assert not bad.any(), (bad.nonzero()[:4].tolist(), float(off.max()))


def exact_operands(B, N, K, seed=0):
    """Codes 0, +-0.5, +-1, +-1.5, +-2 and scales that are powers of two: every product and every sum is a multiple
    of 2^-14 below 2^9 (K <= 8208 in blocks of scale at most 2^-4), so all of them are exact and only y is rounded."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nkb = -(-K // 128)
    few = torch.tensor([0, 0.5, 1, 1.5, 2, -0.5, -1, -1.5, -2], device="cuda")
    a, w = (few[torch.randint(0, 9, (r, K), generator=g, device="cuda")].to(FP8) for r in (B, N))
    sa = torch.exp2(-2.0 - torch.randint(0, 5, (B, nkb), generator=g, device="cuda"))
    sw = torch.exp2(-2.0 - torch.randint(0, 5, (-(-N // 128), nkb), generator=g, device="cuda"))
    return a, sa, w, sw


SIZES = [(1, 1, 16), (1, 8192, 4096), (2, 5, 48), (16, 576, 1040), (17, 130, 128), (32, 64, 2064), (33, 200, 400),
         (64, 1000, 1152), (65, 131, 144), (100, 576, 4096), (128, 128, 128), (200, 257, 272), (257, 300, 16),
         (512, 640, 1296), (300, 2120, 7184), (5, 33, 8208), (40, 96, 20000)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_product(nv, size, dtype):
    B, N, K = size
    ops = operands(B, N, K, seed=B + N + K)
    y = nv.fp8_gemm(*ops, out_dtype=dtype)
    assert y.dtype is dtype and y.shape == (B, N)
    check(y, *binary64(*ops), K)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", [s for s in SIZES if s[2] <= 8208] + [(4096, 3200, 400), (4000, 3333, 272)])
def test_exact_product(nv, size, dtype):
    ops = exact_operands(*size, seed=sum(size))
    want, _ = binary64(*ops)
    assert torch.equal(nv.fp8_gemm(*ops, out_dtype=dtype), want.to(dtype))


@pytest.mark.parametrize("size", [(4096, 3200, 400), (4000, 3333, 272), (2048, 8192, 1024)])
def test_product_of_many_tiles(nv, size):
    ops = operands(*size, seed=3)
    check(nv.fp8_gemm(*ops, out_dtype=torch.bfloat16), *binary64(*ops), size[2])


@pytest.mark.parametrize("B", [1, 16, 30, 64, 100, 300])
def test_nan_stays_in_its_row_and_column(nv, B):
    a, sa, w, sw = operands(B, 260, 272, seed=B)
    a, w = a.clone(), w.clone()
    a.view(torch.uint8)[B - 1, 271] = 0x7F
    w.view(torch.uint8)[259, 3] = 0x7F
    y = nv.fp8_gemm(a, sa, w, sw).isnan().cpu()
    want = torch.zeros_like(y)
    want[B - 1], want[:, 259] = True, True
    assert torch.equal(y, want)


@pytest.mark.parametrize("B", [1, 20, 64, 90, 400])
def test_output_bounds(nv, B):
    """Nothing is written outside y, at any alignment of y."""
    N, K = 134, 144
    ops = operands(B, N, K, seed=1)
    want = nv.fp8_gemm(*ops)
    flat = torch.full((B * N + 16,), 7.0, dtype=torch.float16, device="cuda")
    out = flat[5:5 + B * N].view(B, N)
    assert nv.fp8_gemm(*ops, out=out) is out
    assert torch.equal(out, want) and (flat[:5] == 7).all() and (flat[5 + B * N:] == 7).all()


@pytest.mark.parametrize("size", [(1, 512, 2048), (50, 300, 1040), (300, 512, 528)])
def test_rows_do_not_depend_on_each_other_and_calls_repeat(nv, size):
    ops = operands(*size, seed=2)
    y = nv.fp8_gemm(*ops)
    for _ in range(3):
        assert torch.equal(nv.fp8_gemm(*ops), y)


def test_streams_and_replays(nv):
    x = torch.randn((40, 1040), device="cuda").half()
    wq = nv.fp8_quantize(torch.randn((264, 1040), device="cuda").half(), block_rows=128)

    def step(stream=None):
        a = nv.fp8_quantize(x, stream=stream)
        return nv.fp8_gemm(a["codes"], a["scale"], wq["codes"], wq["scale"], stream=stream)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = step(s)
    s.synchronize()
    assert torch.equal(y, step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        x.normal_()
        want = step()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), turn


def test_no_rows(nv):
    q = nv.fp8_quantize(torch.zeros((0, 256), dtype=torch.float16, device="cuda"))
    assert q["codes"].shape == (0, 256) and q["scale"].shape == (0, 2)
    ops = operands(1, 64, 256)
    assert nv.fp8_gemm(q["codes"], q["scale"], ops[2], ops[3]).shape == (0, 64)


def test_quantized_product_is_near_the_product(nv):
    """x W^T through both quantizers: the errors of the codes are independent, at most 2^-4 and 2^-4 / sqrt(3) of
    each value's size on average, so the product's relative error stays below 2^-4 sqrt(2 / 3) (1 + 2^-4)."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((96, 1040), generator=g, device="cuda").bfloat16()
    w = torch.randn((200, 1040), generator=g, device="cuda").bfloat16()
    a, q = nv.fp8_quantize(x), nv.fp8_quantize(w, block_rows=128)
    y = nv.fp8_gemm(a["codes"], a["scale"], q["codes"], q["scale"]).double()
    want = x.double() @ w.double().t()
    assert float((y - want).norm() / want.norm()) < 2.0 ** -4 * (2 / 3) ** 0.5 * (1 + 2.0 ** -4)


@pytest.mark.parametrize("size", [(20, 4100, 528), (64, 8192, 400), (70, 6000, 272), (130, 5000, 1040), (128, 8192, 128),
                                  (200, 7000, 272), (400, 5000, 656), (64, 9000, 48)])
def test_every_tile_size(nv, size):
    """Sizes around the limits between the kernels for a few rows, K not a multiple of 128 and fewer blocks than groups of waves."""
    a, sa, w, sw = exact_operands(*size, seed=sum(size))
    want, _ = binary64(a, sa, w, sw)
    y = nv.fp8_gemm(a, sa, w, sw)
    assert torch.equal(y, want.to(torch.float16))
    b = operands(*size, seed=1)
    check(nv.fp8_gemm(*b, out_dtype=torch.bfloat16), *binary64(*b), size[2])


@pytest.mark.parametrize("B", [3, 70, 300, 1500])
@pytest.mark.parametrize("N", [257, 514, 1027])
def test_rows_at_any_alignment(nv, N, B):
    """Rows that start at any two bytes, the output itself too: exact results, and nothing beside them is touched."""
    a, sa, w, sw = exact_operands(B, N, 400, seed=N + B)
    want = binary64(a, sa, w, sw)[0].to(torch.float16)
    for shift in (0, 1, 2, 3):
        room = torch.full((B * N + 8,), 7.0, dtype=torch.float16, device="cuda")
        y = room[shift:shift + B * N].view(B, N)
        nv.fp8_gemm(a, sa, w, sw, out=y)
        assert torch.equal(y, want)
        assert (room[:shift] == 7).all() and (room[shift + B * N:] == 7).all()

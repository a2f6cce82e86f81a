"""Comparisons that NaN cannot pass: `abs(nan) > bound` is False, so a test that collects what is too far off finds
nothing in a result, a reference or a bound of NaN."""
import torch

# half of a type's smallest number: what a rounding may take where the value has left the normal range
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def within(got, want, bound):
    got, want, bound = got.double(), want.double(), torch.as_tensor(bound, dtype=torch.float64, device=want.device)
    assert torch.isfinite(want).all() and torch.isfinite(bound).all(), "nothing to compare with"
    off = (got.to(want.device) - want).abs()
    good = off <= bound
    assert good.all(), ((~good).nonzero()[:4].tolist(), float(off[~good][0]))


def fp8_check(y, want, size, K):
    """The bound of test_gpu_fp8.check."""
    eps = torch.finfo(y.dtype).eps / 2
    room = (7 * 2.0 ** -13 + (16 + -(-K // 128) + 3) * 2.0 ** -23) * size
    within(y, want, eps * want.abs() * (1 + 2.0 ** -8) + room * (1 + eps) + SMALLEST[y.dtype])


def moe_check(got, want, room, kind):
    """The bound of test_gpu_moe_decode.check."""
    dtype = {"fp16": torch.float16, "bf16": torch.bfloat16}[kind]
    assert got.dtype is dtype
    within(got, want, torch.finfo(dtype).eps / 2 * want.abs() * (1 + 2.0 ** -8) + room + SMALLEST[dtype])

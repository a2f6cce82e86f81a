"""What the strict comparisons accept and refuse (no GPU)."""
import pytest
import torch

import strict_checks as strict

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("check", [lambda y, w, r: strict.fp8_check(y, w, r, 128), lambda y, w, r: strict.moe_check(y, w, r, "bf16")])
def test_what_is_accepted(check):
    want, room = torch.tensor([[1.0, -2.0, 0.0]]).double(), torch.zeros((1, 3)).double()
    y = want.bfloat16()
    check(y, want, room)
    check(y, want * (1 + 2.0 ** -10), room)
    for bad in (NAN, INF, 1.02):
        z = y.clone()
        z[0, 0] = bad
        with pytest.raises(AssertionError):
            check(z, want, room)
    for bad in (NAN, INF):
        w, r = want.clone(), room.clone()
        w[0, 2] = r[0, 2] = bad
        for a, b in ((w, room), (want, r), (w, r)):
            with pytest.raises(AssertionError):
                check(y, a, b)
            with pytest.raises(AssertionError):
                check(torch.full_like(y, 123), a, b)

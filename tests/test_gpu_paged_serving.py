"""The serving example: every attention call it makes is compared with binary64 attention over the keys
and values that were written, request by request."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import attention_checks as ac

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("paged_serving", EXAMPLE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def spied(nv, monkeypatch):
    """Records q, k, v and the outputs of the attention calls."""
    seen = {}

    def wrap(name, keep):
        f = getattr(nv, name)

        def call(*args, **kw):
            r = f(*args, **kw)
            keep(args, r)
            return r
        monkeypatch.setattr(nv, name, call)

    wrap("kv_write", lambda a, r: seen.update(k=a[0].detach().clone(), v=a[1].detach().clone()))
    for name in ("prompt_attn", "paged_attn"):
        wrap(name, lambda a, r, n=name: seen.update(q=a[0].detach().clone(), out=r.detach().clone(), name=n))
    return seen


@pytest.mark.parametrize("window", [0, 50])
def test_every_step_is_right(ex, monkeypatch, window):
    hq, hk, d = 8, 2, 64
    seen = spied(ex.nv, monkeypatch)
    s = ex.Server(512, hq, hk, d, seqs=4, page_size=8, pages=128, max_pages=40, window=window)
    gen = torch.Generator().manual_seed(3)
    ks, vs = [np.zeros((0, hk, d))] * 4, [np.zeros((0, hk, d))] * 4
    for new, name in [([90, 7, 0, 1], "prompt_attn"), ([1, 70, 33, 1], "paged_attn"), ([1, 1, 1, 1], "paged_attn"),
                      ([0, 3, 0, 5], "paged_attn"), ([1, 1, 1, 1], "paged_attn")]:
        y = s.step(torch.randn((sum(new), 512), generator=gen).half().cuda(), new)
        assert seen["name"] == name and y.shape == (sum(new), 512) and torch.isfinite(y).all()
        k, v, q = (seen[n].cpu().double().numpy() for n in "kvq")
        refs, at = [], 0
        for i, m in enumerate(new):
            ks[i], vs[i] = np.concatenate([ks[i], k[at:at + m]]), np.concatenate([vs[i], v[at:at + m]])
            if m:
                refs.append(ac.attend(q[at:at + m], ks[i], vs[i], d ** -0.5, window))
            at += m
        longest = max(len(x) for x in ks)
        ac.check(seen["out"].cpu(), None, refs, torch.float16, longest, max(np.abs(x).max(initial=0.0) for x in vs))
        assert s.lens.tolist() == s.held == [len(x) for x in ks]


def test_recorded_decode_equals_eager(ex):
    a, b = (ex.Server(512, 8, 2, 64, seqs=3, page_size=4, pages=64, max_pages=20) for _ in range(2))
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((13, 512), generator=gen).half().cuda()
    for s in (a, b):
        s.step(x, [9, 1, 3])
    g = ex.DecodeGraph(a)
    for n in range(10):
        x = torch.randn((3, 512), generator=gen).half().cuda()
        got = g.step(x).clone()
        want = b.step(x, [1, 1, 1])
        torch.cuda.synchronize()
        assert torch.equal(got, want), n
        assert torch.equal(a.table, b.table) and a.lens.tolist() == b.lens.tolist() == a.held


def test_refusals(ex):
    s = ex.Server(512, 8, 2, 64, seqs=2, page_size=4, pages=4, max_pages=8)
    x = torch.zeros((20, 512), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="new"):
        s.step(x, [10, 5])
    with pytest.raises(RuntimeError, match="free"):
        s.step(x, [10, 10])
    with pytest.raises(ValueError, match="exceeds"):
        s.step(torch.zeros((33, 512), dtype=torch.float16, device="cuda"), [33, 0])

"""The layer of the serving example: FP8 projections, rotation with the cache write, attention over the cache, routed
experts.  Every operator is held against the formula on the inputs that it was given in the run, with the bounds of
its own tests; what leads from one to the next is torch's."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import attention_checks as ac
import test_gpu_fp8 as fp8
import test_gpu_moe_decode as moe
import test_gpu_rope_kv as rope

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")
OPERATORS = ("page_maps", "fp8_quantize", "fp8_gemm", "rope_kv_write", "prompt_attn", "paged_attn", "moe_decode")
HIDDEN, HQ, HK, D, EXPERTS, TOP_K, INTER = 512, 8, 2, 64, 16, 3, 192


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("paged_serving", EXAMPLE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def layer(ex, seqs, page_size, window=0):
    return ex.Layer(HIDDEN, HQ, HK, D, seqs=seqs, page_size=page_size, pages=128, max_pages=40, window=window,
                    experts=EXPERTS, top_k=TOP_K, inter=INTER)


def copies(x):
    if isinstance(x, torch.Tensor):
        return x.detach().clone()
    return {k: copies(v) for k, v in x.items()} if isinstance(x, dict) else x


def spied(nv, monkeypatch):
    """The calls in order: (operator, arguments as they were, arguments afterwards, options, result)."""
    calls = []

    def wrap(name):
        f = getattr(nv, name)

        def call(*args, **kw):
            before = [copies(a) for a in args]
            r = f(*args, **kw)
            calls.append((name, before, [copies(a) for a in args], kw, copies(r)))
            return r
        monkeypatch.setattr(nv, name, call)

    for name in OPERATORS:
        wrap(name)
    return calls


def check_quantize(call):
    (x,), got = call[1], call[4]
    codes, scale = fp8.quantize_ref(x.cpu(), 1)
    assert np.array_equal(got["scale"].cpu().numpy(), scale)
    assert torch.equal(got["codes"].cpu().view(torch.uint8), codes.view(torch.uint8))


def check_gemm(call):
    a, sa, w, sw = call[1]
    fp8.check(call[4], *fp8.binary64(a, sa, w, sw), a.shape[1])


def check_rope(call):
    before, after = call[1], call[2]
    q, k, v, positions, freq, slots = [t.cpu() for t in before[:6]]
    for x, got in ((q, after[0].cpu()), (k, after[1].cpu())):
        want, room = rope.turned(x, positions, freq, False, 1.0)
        rope.near(got, want, room, x.dtype)
    for cache, rows in ((after[6], after[1]), (after[7], after[2])):
        at = cache.transpose(1, 2).reshape(-1, HK, D)[slots.cuda()]
        assert torch.equal(at, rows)


def sum_of_terms(run, ids, wts):
    """Sum over a token's experts of |weight times its output|, binary64."""
    total = torch.zeros(run.x.shape, dtype=torch.float64)
    for t in range(len(ids)):
        for e, w in zip(ids[t], wts[t]):
            total[t:t + 1] += moe.reference(one(run, t), [[e]], [[w]])[0].abs()
    return total


def one(run, t):
    part = moe.Layer.__new__(moe.Layer)
    part.__dict__.update(run.__dict__, x=run.x[t:t + 1])
    return part


def check_moe(call):
    x, router, bias, w1, w1_sf, w1_g, w2, w2_sf, w2_g, top_k = call[1]
    run = moe.Layer("fp16", x.shape[0], EXPERTS, HIDDEN, INTER, "swiglu")
    run.x, run.router, run.bias = x.cpu(), router.cpu(), bias.cpu()
    run.w1, run.w2 = [t.cpu() for t in (w1, w1_sf, w1_g)], [t.cpu() for t in (w2, w2_sf, w2_g)]
    logits = (run.x.double() @ run.router.double().t()).numpy()
    ids, wts = zip(*(moe.choose(row, run.bias.double().numpy(), top_k, 1, 1, True, 1.0) for row in logits))
    out, room = moe.reference(run, ids, wts)
    # the operator's selection is its own, in binary32: its weights are held to 2e-5 in its tests, which is that much of
    # every |w o|
    size = sum_of_terms(run, ids, wts)
    moe.check(call[4], out, room + 2e-5 * size, "fp16")


@pytest.mark.parametrize("window", [0, 50])
def test_every_step_is_right(ex, monkeypatch, window):
    calls = spied(ex.nv, monkeypatch)
    s = layer(ex, 4, 8, window)
    calls.clear()
    gen = torch.Generator().manual_seed(3)
    ks, vs = [np.zeros((0, HK, D))] * 4, [np.zeros((0, HK, D))] * 4
    for new, attention in [([40, 7, 0, 1], "prompt_attn"), ([1, 34, 20, 1], "paged_attn"), ([1, 1, 1, 1], "paged_attn"),
                           ([0, 3, 0, 5], "paged_attn"), ([0, 0, 1, 0], "paged_attn")]:
        x = torch.randn((sum(new), HIDDEN), generator=gen).half().cuda()
        y = s.step(x, new)
        assert y.shape == x.shape and torch.isfinite(y).all()
        assert [c[0] for c in calls] == ["page_maps", "fp8_quantize", "fp8_gemm", "rope_kv_write", attention,
                                         "fp8_quantize", "fp8_gemm"] + ["moe_decode"] * -(-sum(new) // 32)
        for c in calls:
            {"fp8_quantize": check_quantize, "fp8_gemm": check_gemm, "rope_kv_write": check_rope,
             "moe_decode": check_moe}.get(c[0], lambda c: None)(c)
        q, k, v = (t.cpu().double().numpy() for t in calls[3][2][:3])
        refs, at = [], 0
        for i, m in enumerate(new):
            ks[i], vs[i] = np.concatenate([ks[i], k[at:at + m]]), np.concatenate([vs[i], v[at:at + m]])
            if m:
                refs.append(ac.attend(q[at:at + m], ks[i], vs[i], D ** -0.5, window))
            at += m
        ac.check(calls[4][4].cpu(), None, refs, torch.float16, max(len(x) for x in ks),
                 max(np.abs(x).max(initial=0.0) for x in vs))
        total = x + calls[6][4]
        assert torch.equal(y, total + torch.cat([c[4] for c in calls[7:]]))
        calls.clear()


def test_recorded_decode_equals_eager(ex):
    a, b = (layer(ex, 3, 4) for _ in range(2))
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((13, HIDDEN), generator=gen).half().cuda()
    for s in (a, b):
        s.step(x, [9, 1, 3])
    g = ex.DecodeGraph(a)
    for n in range(10):
        x = torch.randn((3, HIDDEN), generator=gen).half().cuda()
        got = g.step(x).clone()
        want = b.step(x, [1, 1, 1])
        torch.cuda.synchronize()
        assert torch.equal(got, want), n
        assert torch.equal(a.table, b.table) and a.lens.tolist() == b.lens.tolist() == a.held


def test_two_recorded_layers_on_two_streams(ex):
    """Each graph has buffers of its own: replayed side by side they give what they give alone."""
    pair = [layer(ex, 2, 4) for _ in range(2)]
    alone = [layer(ex, 2, 4) for _ in range(2)]
    gen = torch.Generator().manual_seed(5)
    for s, t in zip(pair, alone):
        x = torch.randn((5, HIDDEN), generator=gen).half().cuda()
        s.step(x, [2, 3])
        t.step(x, [2, 3])
    graphs = [ex.DecodeGraph(s) for s in pair]
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for n in range(6):
        xs = [torch.randn((2, HIDDEN), generator=gen).half().cuda() for _ in pair]
        got = []
        torch.cuda.synchronize()
        for g, stream, x in zip(graphs, streams, xs):
            with torch.cuda.stream(stream):
                got.append(g.step(x).clone())
        torch.cuda.synchronize()
        for t, x, y in zip(alone, xs, got):
            assert torch.equal(t.step(x, [1, 1]), y), n

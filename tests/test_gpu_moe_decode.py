"""The MoE layer for a few tokens against binary64, with the selection of moe_w4a16 by plain loops.

Tolerance.  Sums of K terms in binary32, each term's two factors exact (x) or to 22 bits (h): with S the sum of the
terms' sizes, fc1 is off by at most (K + 4) 2^-23 S1; a relative error d of a ReLU^2 or SwiGLU input is at most
2 d (1 + |gate|) of its output's size; fc2 adds (inter + 8) 2^-22 of its terms' sizes, the weighted sum top_k 2^-23, and
the output half a step of its type.  The matrix instruction's own sums are given twice that room."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E2M1 = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def weights(experts, rows, k, g, spread=6):
    codes = torch.randint(0, 256, (experts, rows, k // 2), generator=g, dtype=torch.uint8)
    sf = (0.5 + torch.rand((experts, rows, k // 16), generator=g)) * torch.exp2(
        -torch.randint(0, spread, (experts, rows, k // 16), generator=g).float())
    glob = (0.5 + torch.rand(experts, generator=g)) * k ** -0.5
    return codes, sf.to(FP8).view(torch.uint8), glob


def values(codes, sf, glob):
    w = torch.stack((E2M1[(codes & 15).long()], E2M1[(codes >> 4).long()]), -1).flatten(-2)
    return w * sf.view(FP8).double().repeat_interleave(16, -1) * glob.double()


class Layer:
    def __init__(self, kind, tokens, experts, hidden, inter, act, seed=0, x_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.act, self.inter, self.kind = act, inter, kind
        self.x = (torch.randn((tokens, hidden), generator=g) * x_scale).to(TYPES[kind])
        self.router = (torch.randn((experts, hidden), generator=g) * hidden ** -0.5).to(TYPES[kind])
        self.bias = torch.randn(experts, generator=g) * 0.1
        self.w1 = weights(experts, 2 * inter if act == "swiglu" else inter, hidden, g)
        self.w2 = weights(experts, hidden, inter, g)

    def args(self):
        return [t.cuda() for t in (self.x, self.router, self.bias, *self.w1, *self.w2)]


def choose(logits, bias, top_k, n_group, topk_group, norm, scaling):
    """(experts, weights) of one token by the definition; NaN ranks below every number."""
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-logits))
    b = s + bias
    b[np.isnan(b)] = -np.inf
    per = len(b) // n_group
    score = [sum(sorted(b[i * per:(i + 1) * per])[-2:]) for i in range(n_group)]
    kept = sorted(range(n_group), key=lambda i: (-score[i], i))[:topk_group]
    inside = [e for i in kept for e in range(i * per, (i + 1) * per)]
    ids = sorted(inside, key=lambda e: (-b[e], e))[:top_k]
    w = s[ids]
    return ids, (w / w.sum() if norm else w) * scaling


def reference(layer, ids, wts):
    """(out, room) in binary64 for a given selection."""
    x = layer.x.double()
    out, room = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    cache = {}
    hidden, inter = x.shape[1], layer.inter
    for t in range(x.shape[0]):
        for e, w in zip(ids[t], wts[t]):
            if e not in cache:
                cache[e] = [values(m[0][e], m[1][e], m[2][e]) for m in (layer.w1, layer.w2)]
            w1, w2 = cache[e]
            y, size = w1 @ x[t], w1.abs() @ x[t].abs()
            off = 2 * (hidden + 4) * 2.0 ** -23 * size
            if layer.act == "swiglu":
                gate, up = y[:inter], y[inter:]
                sig = torch.sigmoid(gate)
                h = gate * sig * up
                # d(silu) <= 1.1 d(gate); silu itself to 2^-20
                dh = 1.1 * off[:inter] * (up.abs() + off[inter:]) + (gate * sig).abs() * off[inter:] + h.abs() * 2.0 ** -20
            else:
                h = torch.clamp(y, min=0) ** 2
                dh = 2 * torch.clamp(y, min=0) * off + off ** 2 + h * 2.0 ** -22
            o = w2 @ h
            out[t] += w * o
            room[t] += abs(w) * (w2.abs() @ (dh + 2 * (inter + 8 + len(ids[t])) * 2.0 ** -23 * h.abs()))
    return out, room


def check(got, want, room, kind):
    eps = torch.finfo(TYPES[kind]).eps / 2
    off = (got.double().cpu() - want).abs()
    bad = off > eps * want.abs() * (1 + 2.0 ** -8) + room + (2.0 ** -25 if kind == "fp16" else 0)
    assert not bad.any(), (bad.nonzero()[:4].tolist(), float((off / want.abs().clamp(min=1e-9)).max()))


def run(nv, layer, top_k, n_group, topk_group, norm=True, scaling=1.0, tiled=False, **kw):
    args = layer.args()
    if tiled:
        args[3], args[4] = nv.moe_pretile_weights(args[3], args[4])
        args[6], args[7] = nv.moe_pretile_weights(args[6], args[7])
    out, ids, wts = nv.moe_decode(*args, top_k, n_group, topk_group, norm_topk_prob=norm, routed_scaling=scaling,
                                  act=layer.act, tiled=tiled, want_routing=True, **kw)
    return out, ids.cpu(), wts.cpu()


def full(nv, layer, top_k, n_group, topk_group, norm=True, scaling=1.0, tiled=False):
    out, ids, wts = run(nv, layer, top_k, n_group, topk_group, norm, scaling, tiled)
    logits = (layer.x.double() @ layer.router.double().t()).numpy()
    for t in range(len(logits)):
        want_ids, want_w = choose(logits[t], layer.bias.double().numpy(), top_k, n_group, topk_group, norm, scaling)
        assert ids[t].tolist() == want_ids, t
        assert np.allclose(wts[t].numpy(), want_w, rtol=2e-5, atol=0)
    check(out, *reference(layer, ids.tolist(), wts.double().tolist()), layer.kind)
    return out


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ["relu2", "swiglu"])
@pytest.mark.parametrize("size", [(1, 64, 8, 8, 4, 512, 256), (2, 8, 2, 1, 1, 64, 64), (5, 16, 4, 4, 2, 320, 192),
                                  (16, 32, 6, 1, 1, 256, 128), (17, 16, 3, 8, 3, 192, 320), (32, 12, 4, 2, 1, 128, 64),
                                  (31, 256, 16, 8, 4, 128, 64), (3, 100, 1, 10, 10, 1088, 64), (4, 1, 1, 1, 1, 2048, 128),
                                  (1, 128, 6, 8, 3, 1280, 192), (1, 256, 8, 16, 4, 64, 64), (1, 96, 5, 4, 2, 192, 64),
                                  (2, 128, 8, 2, 1, 1088, 64), (32, 64, 8, 64, 20, 512, 512), (8, 250, 3, 5, 2, 64, 1088)])
def test_against_binary64(nv, size, act, kind):
    tokens, experts, top_k, n_group, topk_group, hidden, inter = size
    full(nv, Layer(kind, tokens, experts, hidden, inter, act, seed=sum(size)), top_k, n_group, topk_group)


@pytest.mark.parametrize("act", ["relu2", "swiglu"])
@pytest.mark.parametrize("size", [(1, 384, 256), (9, 384, 256), (20, 256, 128), (3, 128, 640)])
def test_tiled_weights(nv, act, size):
    """The pre-tiled layout has the same values; the sums' order over k differs, so it is held against binary64 too."""
    tokens, hidden, inter = size
    layer = Layer("fp16", tokens, 16, hidden, inter, act, seed=tokens)
    _, ids, wts = run(nv, layer, 4, 4, 2, scaling=2.5)
    _, tids, twts = run(nv, layer, 4, 4, 2, scaling=2.5, tiled=True)
    assert torch.equal(ids, tids) and torch.equal(wts, twts)
    full(nv, layer, 4, 4, 2, norm=False, scaling=2.5, tiled=True)


def test_the_layer_of_the_batch_operator(nv):
    """The same weights and routing through moe_w4a16 (FP16, ReLU^2): equal selection, results within the
    two operators' roundings (moe_w4a16 carries h in FP16: 2^-11 of each h, 2^-11 of the output)."""
    layer = Layer("fp16", 8, 64, 512, 256, "relu2", seed=3)
    out, ids, wts = run(nv, layer, 8, 8, 4)
    x, router, bias, *w = layer.args()
    logits = (x.double() @ router.double().t()).float()
    ref, rids, rw = nv.moe_w4a16(logits, bias, x, *w, 8, 8, 4, want_routing=True)
    assert torch.equal(rids.cpu(), ids) and torch.allclose(rw.cpu(), wts, rtol=1e-5)
    off = (out.double() - ref.double()).norm() / ref.double().norm()
    assert float(off) < 3 * 2.0 ** -11


@pytest.mark.parametrize("kind,scale", [("fp16", 1e-4), ("fp16", 30.0), ("bf16", 1e-4), ("bf16", 30.0), ("bf16", 1e-20),
                                        ("bf16", 1e15)])
def test_sizes_of_values(nv, kind, scale):
    """Large and small activations: h far outside FP16's range.  The results are brought back by the globals of fc2."""
    layer = Layer(kind, 6, 8, 256, 128, "relu2", seed=9, x_scale=scale)
    layer.w2 = (layer.w2[0], layer.w2[1], layer.w2[2] / np.float32(scale) ** 2)
    full(nv, layer, 3, 1, 1)


def test_all_tokens_choose_the_same_experts(nv):
    layer = Layer("bf16", 32, 64, 256, 128, "swiglu", seed=11)
    layer.x = layer.x[:1].expand(32, -1).contiguous()
    out = full(nv, layer, 5, 8, 4)
    assert torch.equal(out, out[:1].expand_as(out))


def test_ties_and_values_that_are_not_finite(nv):
    layer = Layer("fp16", 4, 16, 128, 64, "relu2", seed=12)
    layer.router = torch.zeros_like(layer.router)
    layer.bias = torch.zeros(16)
    out, ids, wts = run(nv, layer, 4, 4, 2)
    assert (ids == torch.tensor([0, 1, 2, 3], dtype=torch.int32)).all()      # all scores equal: lowest indexes
    assert torch.equal(wts, torch.full((4, 4), 0.25))
    # a NaN token: every logit NaN, the lowest indexes, a row of NaN; the other rows as they were
    x = layer.x.clone()
    x[2, 5] = float("nan")
    layer.x, old = x, layer.x
    got, ids, _ = run(nv, layer, 4, 4, 2)
    assert got[2].isnan().all() and torch.equal(got[[0, 1, 3]], out[[0, 1, 3]]) and ids[2].tolist() == [0, 1, 2, 3]
    layer.x = old
    layer.bias[7], layer.bias[9] = float("nan"), float("-inf")                # ranked below everything
    _, ids, _ = run(nv, layer, 8, 4, 2)
    assert not (ids == 9).any()
    layer.bias[:] = float("nan")
    _, ids, _ = run(nv, layer, 3, 1, 1)
    assert (ids == torch.tensor([0, 1, 2], dtype=torch.int32)).all()


@pytest.mark.parametrize("tokens", [2, 13, 32])
def test_tokens_do_not_depend_on_each_other(nv, tokens):
    layer = Layer("bf16", tokens, 32, 320, 192, "swiglu", seed=tokens)
    out, ids, wts = run(nv, layer, 4, 4, 2)
    x = layer.x
    for t in (0, tokens - 1):
        layer.x = torch.randn(x.shape, generator=torch.Generator().manual_seed(t)).to(x.dtype)
        layer.x[t] = x[t]
        other, i1, w1 = run(nv, layer, 4, 4, 2)
        assert torch.equal(i1[t], ids[t]) and torch.equal(w1[t], wts[t]) and torch.equal(other[t], out[t])


def test_workspace_streams_and_replays(nv):
    layer = Layer("fp16", 7, 32, 512, 256, "relu2", seed=4)
    args = layer.args()
    ws = torch.full((nv.moe_decode_workspace_size(7, 32, 4, 512, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    a = nv.moe_decode(*args, 4, 4, 2, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = nv.moe_decode(*args, 4, 4, 2, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    out = torch.zeros_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.moe_decode(*args, 4, 4, 2, out=out, workspace=ws)
    for turn in range(5):
        args[0].normal_()
        want = nv.moe_decode(*args, 4, 4, 2)
        ws.fill_(turn * 37)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), turn


def test_no_tokens(nv):
    args = Layer("fp16", 1, 8, 64, 64, "relu2").args()
    args[0] = args[0][:0]
    assert nv.moe_decode(*args, 2).shape == (0, 64)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("size", [(2, 8, 3, 4, 2, 2112, 192, "relu2"), (5, 6, 2, 1, 1, 192, 2112, "swiglu"),
                                  (1, 16, 5, 4, 2, 2112, 4160, "relu2"), (1, 70, 16, 7, 3, 64, 2112, "swiglu"),
                                  (16, 64, 8, 8, 4, 1024, 1024, "relu2"), (3, 40, 8, 4, 4, 1088, 1536, "swiglu")])
def test_long_rows_and_many_units(nv, size, kind):
    """Rows of more blocks than waves, and more units than workgroups, so that a workgroup crosses into the next expert."""
    tokens, experts, top_k, n_group, topk_group, hidden, inter, act = size
    full(nv, Layer(kind, tokens, experts, hidden, inter, act, seed=sum(size[:7])), top_k, n_group, topk_group)


@pytest.mark.parametrize("tokens,experts,top_k", [(17, 4, 4), (32, 2, 1), (32, 3, 2), (31, 16, 16), (32, 40, 16)])
def test_experts_of_more_than_sixteen_tokens(nv, tokens, experts, top_k):
    """Such an expert is worked on in two parts; with an expert of exactly 16 beside it, and of one."""
    layer = Layer("fp16", tokens, experts, 320, 192, "swiglu", seed=tokens + experts)
    layer.bias[0] += 0.3
    full(nv, layer, top_k, 1, 1)
    # by hand: token t to expert 0 below 16, to expert 1 from there on, and so on
    layer = Layer("bf16", 32, 8, 64, 64, "relu2", seed=1)
    layer.x[:] = layer.x.abs() * 0.01
    layer.router[:] = 0
    for e, members in enumerate((range(0, 16), range(16, 31), range(31, 32))):
        for t in members:
            layer.x[t, e] = 8
        layer.router[e, e] = 1
    _, ids, _ = run(nv, layer, 1, 1, 1)
    assert ids[:, 0].tolist() == [0] * 16 + [1] * 15 + [2]
    full(nv, layer, 1, 1, 1)


@pytest.mark.parametrize("tokens", [1, 2])
@pytest.mark.parametrize("experts,n_group,topk_group", [(16, 4, 2), (64, 1, 1), (64, 8, 3), (200, 10, 4), (256, 256, 100)])
def test_ties(nv, tokens, experts, n_group, topk_group):
    """Equal scores: the lower index first, within an order of a few different biases."""
    layer = Layer("fp16", tokens, experts, 64, 64, "relu2", seed=experts)
    layer.router[:] = 0
    g = torch.Generator().manual_seed(experts + tokens)
    for few in (1, 2, 3, 8):
        layer.bias = torch.tensor([0.0, 0.5, -0.25, 1.0, 2.0, -3.0, 0.125, 4.0])[torch.randint(0, few, (experts,), generator=g)]
        for top_k in (1, 3, 8):
            full(nv, layer, top_k, n_group, topk_group)


def test_one_token_that_is_not_finite(nv):
    layer = Layer("fp16", 1, 64, 128, 64, "relu2", seed=2)
    layer.x[0, 3] = float("nan")
    out, ids, wts = run(nv, layer, 4, 8, 2)
    assert out.isnan().all() and ids.tolist() == [[0, 1, 2, 3]] and wts.isnan().all()
    layer = Layer("bf16", 1, 64, 128, 64, "relu2", seed=2)
    layer.bias[:32], layer.bias[40] = float("nan"), float("-inf")
    _, ids, _ = run(nv, layer, 16, 1, 1)
    assert (ids >= 32).all() and not (ids == 40).any()
    # weights times globals far outside binary16: the sum's own scale takes them
    layer = Layer("bf16", 1, 16, 128, 64, "relu2", seed=3)
    layer.w2 = (layer.w2[0], layer.w2[1], layer.w2[2] * 2.0 ** 60)
    full(nv, layer, 4, 1, 1, scaling=2.0 ** 30)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 9])
def test_in_place(nv, tokens, kind):
    layer = Layer(kind, tokens, 16, 256, 128, "relu2", seed=tokens)
    want, _, _ = run(nv, layer, 4, 1, 1)
    args = layer.args()
    got = nv.moe_decode(*args, 4, act="relu2", out=args[0])
    assert got is args[0] and torch.equal(got, want)

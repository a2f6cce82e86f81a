"""Every instance of the expert rows' kernel, by the rules that choose them, against binary64 on the GPU; comparisons that
NaN cannot pass.

Tolerance: that of test_gpu_moe_decode (sums of K terms in binary32, the matrix instructions' given twice the room, the
activation, h in two parts), and what those two parts leave of a small h beside a large one: less than 2^-38 of the
row's largest (of one token: of the largest h times its factor)."""
import pytest
import torch

import strict_checks as strict
import test_gpu_moe_decode as moe

pytestmark = pytest.mark.gpu
E2M1 = moe.E2M1


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def routing(layer, ids, wts, n_group, topk_group, norm, scaling):
    """The selection holds by the definition, but for scores that binary32 cannot tell apart (2e-6); weights to 2e-5."""
    logits = layer.x.double() @ layer.router.double().t()
    for t in range(len(ids)):
        b = torch.sigmoid(logits[t]) + layer.bias.double()
        want, w = moe.choose(logits[t].numpy(), layer.bias.double().numpy(), len(ids[t]), n_group, topk_group, norm, scaling)
        assert len(set(ids[t])) == len(want)
        if list(ids[t]) == want:
            assert torch.allclose(torch.tensor(wts[t]).double(), torch.tensor(w.tolist()).double(), rtol=2e-5, atol=0), t
        else:
            assert n_group == 1 and (b[list(ids[t])] - b[want]).abs().max() < 2e-6, (t, ids[t], want)


def expert(w, e):
    codes, sf, glob = (t[e].cuda() for t in w)
    v = E2M1.cuda()[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    return v * sf.view(moe.FP8).double().repeat_interleave(16, -1) * glob.double()


def reference(layer, ids, wts):
    """(out, room) in binary64 on the GPU, an expert at a time."""
    x = layer.x.double().cuda()
    T, hidden = x.shape
    inter, k = layer.inter, len(ids[0])
    out, room, floor = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    takers, top = {}, 0.0
    for t in range(T):
        for e, w in zip(ids[t], wts[t]):
            takers.setdefault(e, []).append((t, w))
    for e, who in takers.items():
        rows = torch.tensor([t for t, _ in who]).cuda()
        share = torch.tensor([w for _, w in who], dtype=torch.float64).cuda()[:, None]
        w1, w2 = expert(layer.w1, e), expert(layer.w2, e)
        y = x[rows] @ w1.t().contiguous()
        off = 2 * (hidden + 4) * 2.0 ** -23 * (x[rows].abs() @ w1.abs().t().contiguous())
        if layer.act == "swiglu":
            gate, up = y[:, :inter], y[:, inter:]
            sig = torch.sigmoid(gate)
            h = gate * sig * up
            dh = (1.1 * off[:, :inter] * (up.abs() + off[:, inter:]) + (gate * sig).abs() * off[:, inter:] +
                  h.abs() * 2.0 ** -20)
        else:
            h = torch.clamp(y, min=0) ** 2
            dh = 2 * torch.clamp(y, min=0) * off + off ** 2 + h * 2.0 ** -22
        dh = dh + 2.0 ** -149   # h may be subnormal
        out[rows] += share * (h @ w2.t().contiguous())
        each = dh + 2 * (inter + 8 + k) * 2.0 ** -23 * h.abs()
        if T > 1:
            each = each + 2.0 ** -38 * h.abs().amax(1, keepdim=True)
        else:   # one scale for all experts, of the largest h times its factor: w2 without its global has the factor's share
            glob = layer.w2[2][e].double().cuda().abs()
            top = max(top, float(h.abs().max() * share[0, 0].abs() * glob))
            floor += (w2.abs() / glob).sum(1)
        room[rows] += share.abs() * (each @ w2.abs().t().contiguous())
    return out, room + 2.0 ** -38 * top * floor


def full(nv, layer, top_k, n_group=1, topk_group=1, norm=True, scaling=1.0, tiled=False):
    out, ids, wts = moe.run(nv, layer, top_k, n_group, topk_group, norm, scaling, tiled)
    ids, wts = ids.tolist(), wts.double().tolist()
    routing(layer, ids, wts, n_group, topk_group, norm, scaling)
    strict.moe_check(out, *reference(layer, ids, wts), layer.kind)
    return out


# (tokens, experts, hidden, inter): the chosen experts are all of them or nearly.  A row has up to four, up to eight, or
# more blocks of 256; units have 32 weight rows, of rows of more than eight blocks 64 where that leaves three units to each of
# 256 workgroups.  There are more units than workgroups (256, of rows of up to four blocks 512), so that they cross experts.
UNITS = {"64 rows, more blocks": (8, 64, 2176, 2304), "32 rows, more blocks": (2, 10, 2176, 2304),
         "many, eight blocks": (10, 80, 1408, 1664), "eight blocks": (2, 16, 1408, 1664),
         "many, four blocks": (32, 256, 896, 896), "four blocks": (4, 32, 896, 896)}


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("act", ["relu2", "swiglu"])
@pytest.mark.parametrize("case", UNITS)
def test_every_instance(nv, case, act, tiled):
    tokens, experts, hidden, inter = UNITS[case]
    at_once = min(8 * tokens, experts)
    for rows, k in ((inter, hidden), (2 * inter, hidden), (hidden, inter)):
        blocks = -(-k // 256)
        assert blocks <= 8 or (rows // 64 * at_once >= 3 * 256) == case.startswith("64")
        assert rows // 32 * at_once > (512 if blocks <= 4 else 256)
    full(nv, moe.Layer("bf16" if tiled else "fp16", tokens, experts, hidden, inter, act, seed=hidden + tokens), 8, tiled=tiled)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("size", [(2, 4, 2, 2112, 4160, "swiglu"), (1, 8, 4, 2304, 2304, "swiglu"), (32, 8, 8, 4224, 128, "swiglu"),
                                  (1, 12, 8, 7168, 2048, "swiglu"), (6, 10, 8, 7168, 2048, "swiglu")])
def test_long_rows(nv, size, kind):
    tokens, experts, top_k, hidden, inter, act = size
    layer = moe.Layer(kind, tokens, experts, hidden, inter, act, seed=sum(size[:5]))
    full(nv, layer, top_k)
    if hidden % 128 == 0 and inter % 128 == 0:
        full(nv, layer, top_k, tiled=True)


@pytest.mark.parametrize("act", ["relu2", "swiglu"])
@pytest.mark.parametrize("tokens", [1, 6])
@pytest.mark.parametrize("scale", [1e-15, 1e-12, 1e-6, 1e-3, 1.0, 1e3, 1e12, 1e15])
def test_sizes_of_values(nv, scale, tokens, act):
    """Small and large activations in BF16, h far outside FP16's range; the globals of fc2, all of them finite, bring the
    results back."""
    layer = moe.Layer("bf16", tokens, 8, 256, 128, act, seed=9, x_scale=scale)
    if act == "swiglu" and scale > 1:   # a gate and its up rows
        layer.w1 = (*layer.w1[:2], layer.w1[2] / scale ** 0.5)
        scale = scale ** 0.5
    layer.w2 = (*layer.w2[:2], (layer.w2[2].double() / scale ** 2).float())
    assert torch.isfinite(layer.w2[2]).all() and (layer.w2[2] > 2.0 ** -126).all()
    full(nv, layer, 3)


@pytest.mark.parametrize("size", [(1, 64, 8, 8, 4, 512, 256), (2, 8, 2, 1, 1, 64, 64), (17, 16, 3, 8, 3, 192, 320),
                                  (31, 256, 16, 8, 4, 128, 64), (1, 256, 8, 16, 4, 64, 64), (8, 250, 3, 5, 2, 64, 1088)])
@pytest.mark.parametrize("act", ["relu2", "swiglu"])
def test_groups_strictly(nv, size, act):
    tokens, experts, top_k, n_group, topk_group, hidden, inter = size
    for kind in ("fp16", "bf16"):
        full(nv, moe.Layer(kind, tokens, experts, hidden, inter, act, seed=sum(size)), top_k, n_group, topk_group,
             scaling=2.5)

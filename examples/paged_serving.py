"""An attention block served from a paged cache: NVFP4 projections around the serving attention
operators.

    python examples/paged_serving.py [--hidden 4096 --q-heads 32 --kv-heads 8 --head-dim 128]

A step takes the new tokens of all requests, packed: whole prompts, a chunk of a long prompt, single
tokens, in any mixture.

    page_maps   lengths -> page table, slots and positions, on the GPU
    act_quant + gemm_pretiled      q, k, v of the new tokens (FP16), then rotary embedding (torch)
    kv_write    k, v -> their slots in the cache
    prompt_attn where no request has cached tokens, else paged_attn
    act_quant + gemm_pretiled      output projection

The host knows how many tokens it sends, so it follows the free pages without asking the GPU.  Decode
steps read their lengths from device memory only: `DecodeGraph` records one and replays it.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_quantize_amd as nv  # noqa: E402


class Linear:
    """NVFP4 weights [n, k], pre-tiled once."""

    def __init__(self, n, k, gen):
        w = (torch.randn((n, k), generator=gen) * k ** -0.5).to(torch.bfloat16).cuda()
        q = nv.quantize(w, group_rows=n, want_scale=False)
        self.tiles, self.g = nv.pretile_weight(q["codes"], q["sf"]), q["g_dec"]

    def __call__(self, x):
        a = nv.act_quant(x)
        return nv.gemm_pretiled(a["codes"], a["scale"], self.tiles, self.g)


def rotate(x, positions, base=10000.0):
    """Rotary embedding of x [tokens, heads, dim], in place, in binary32."""
    half = x.shape[2] // 2
    freq = base ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = positions.float()[:, None, None] * freq
    c, s = angle.cos(), angle.sin()
    a, b = x[..., :half].float(), x[..., half:].float()
    x[..., :half], x[..., half:] = a * c - b * s, a * s + b * c


class Server:
    """Cache, page table and the block's weights; requests are rows 0 .. seqs - 1."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, seqs=4, page_size=16, pages=2048,
                 max_pages=512, window=0, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        self.window, self.page_size, self.seqs = window, page_size, seqs
        self.qkv = Linear((q_heads + 2 * kv_heads) * head_dim, hidden, gen)
        self.proj = Linear(hidden, q_heads * head_dim, gen)
        shape = (pages, kv_heads, page_size, head_dim)
        self.k_cache = torch.empty(shape, dtype=torch.float16, device="cuda")
        self.v_cache = torch.empty(shape, dtype=torch.float16, device="cuda")
        self.table = torch.full((seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=gen).to(torch.int32).cuda()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")   # cached tokens
        self.held = [0] * seqs                                            # the same on the host

    def pages_for(self, new):
        """Pages a step with new[i] tokens takes."""
        p, width = self.page_size, self.table.shape[1]
        if any(h + m > width * p for h, m in zip(self.held, new)):
            raise ValueError("a request exceeds %d tokens" % (width * p))
        return sum(-(-(h + m) // p) + -h // p for h, m in zip(self.held, new))

    def attend(self, x, new_lens, free, fresh):
        """Block output for the packed new tokens x [tokens, hidden]; device work only."""
        m = nv.page_maps(self.lens, new_lens, self.table, free, self.page_size, x.shape[0])
        hq, hk, d = self.q_heads, self.kv_heads, self.head_dim
        q, k, v = self.qkv(x).view(x.shape[0], hq + 2 * hk, d).split([hq, hk, hk], dim=1)
        rotate(q, m["positions"])
        rotate(k, m["positions"])
        nv.kv_write(k, v, m["slot_map"], self.k_cache, self.v_cache)
        if fresh:
            out = nv.prompt_attn(q, k, v, m["cu_new"], window=self.window)
        else:
            out = nv.paged_attn(q, self.k_cache, self.v_cache, self.table, m["cu_new"], m["kv_lens"],
                                window=self.window)
        self.lens.copy_(m["kv_lens"])
        return self.proj(out.view(x.shape[0], hq * d))

    def step(self, x, new):
        """x [sum(new), hidden] FP16 or BF16, new[i] tokens of request i (0 for a request that waits)."""
        if len(new) != self.seqs or sum(new) != x.shape[0]:
            raise ValueError("new must hold a number for each request and sum to the rows of x")
        take = self.pages_for(new)
        if take > self.free.shape[0]:
            raise RuntimeError("%d pages needed, %d free" % (take, self.free.shape[0]))
        fresh = not any(h for h, m in zip(self.held, new) if m)
        y = self.attend(x, torch.tensor(new, dtype=torch.int32).cuda(), self.free, fresh)
        self.free = self.free[take:]
        self.held = [h + m for h, m in zip(self.held, new)]
        return y


class DecodeGraph:
    """One token per request and step, recorded once.  Every replay takes its pages from the front of
    `free`, a buffer as long as a step can need."""

    def __init__(self, server):
        self.server = s = server
        self.x = torch.zeros((s.seqs, s.hidden), dtype=torch.float16, device="cuda")
        self.new = torch.zeros(s.seqs, dtype=torch.int32, device="cuda")
        self.free = torch.zeros(s.seqs, dtype=torch.int32, device="cuda")
        # the rehearsal sends no token, so it leaves the cache and the table as they are
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            s.attend(self.x, self.new, self.free, False)
        torch.cuda.current_stream().wait_stream(stream)
        self.new.fill_(1)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            self.y = s.attend(self.x, self.new, self.free, False)

    def step(self, x):
        s = self.server
        take = s.pages_for([1] * s.seqs)
        if take > s.free.shape[0]:
            raise RuntimeError("%d pages needed, %d free" % (take, s.free.shape[0]))
        self.free[:take].copy_(s.free[:take])
        self.x.copy_(x)
        self.graph.replay()
        s.free = s.free[take:]
        s.held = [h + 1 for h in s.held]
        return self.y


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("hidden", 4096), ("q-heads", 32), ("kv-heads", 8), ("head-dim", 128), ("page-size", 16),
                        ("steps", 200)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    s = Server(a.hidden, a.q_heads, a.kv_heads, a.head_dim, seqs=4, page_size=a.page_size, pages=40960 // a.page_size,
               max_pages=16384 // a.page_size)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def tokens(n):
        return torch.randn((n, a.hidden), generator=gen, device="cuda").half()

    def timed(what, n, f):
        torch.cuda.synchronize()
        t = time.perf_counter()
        f()
        torch.cuda.synchronize()
        t = time.perf_counter() - t
        print("%-44s %8d tokens  %9.3f ms  %10.0f tokens/s" % (what, n, t * 1e3, n / t), flush=True)

    prompts = [1900, 37, 800, 1]
    warm = Server(a.hidden, a.q_heads, a.kv_heads, a.head_dim, seqs=4, pages=512, max_pages=256)
    warm.step(tokens(sum(prompts)), prompts)   # loads the kernels
    warm.step(tokens(4), [1, 1, 1, 1])
    del warm
    timed("four prompts", sum(prompts), lambda: s.step(tokens(sum(prompts)), prompts))
    timed("a chunk beside decoding requests", 1003, lambda: s.step(tokens(1003), [1, 1, 1000, 1]))
    timed("decode steps", 4 * a.steps, lambda: [s.step(tokens(4), [1] * 4) for _ in range(a.steps)])
    g = DecodeGraph(s)
    timed("decode steps, recorded", 4 * a.steps, lambda: [g.step(tokens(4)) for _ in range(a.steps)])


if __name__ == "__main__":
    main()

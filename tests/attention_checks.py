"""Binary64 references and error bounds of the serving attention operators (test helpers).

Bounds.  With u the unit roundoff of the inputs' type (2^-8 bf16, 2^-11 fp16) and A the attention of
|v| with the exact weights:
  * the output is rounded once                        u |out|
  * every weight is rounded once before the product   u A
    (fp16 weights below 2^-14 of a maximum that is at least 1: 2^-25 each, n 2^-25 max|v|)
  * binary32 scores: a dot product of head_dim terms, its scaling and the exponent's argument, each
    with relative roundoff 2^-24, move the argument by at most
    d = 2^-24 (head_dim + 4) scale sum|q||k| (largest of the row's keys) + 2^-23 |s|; every weight
    and the sum of the weights move by that factor: 2 d A (plus 2^-21 for exp2 and log2 themselves)
  * binary32 sums over n keys: 2 n 2^-24 A at the most
Beyond a factor of 1.05 for second-order terms nothing is added.
"""
import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend(q, k, v, scale, window=0):
    """One request in binary64: q [m, Hq, D], k and v [L, Hk, D] (numpy, any values) -> out
    [m, Hq, D], lse [m, Hq], and the error bounds' parts A (attention of |v|) and d (see above)."""
    m, hq, dim = q.shape
    length, hk, _ = k.shape
    out, big = np.zeros((m, hq, dim)), np.zeros((m, hq, dim))
    lse, d = np.full((m, hq), -np.inf), np.zeros((m, hq))
    for i in range(m):
        p = length - m + i
        lo = max(0, p - window + 1) if window > 0 else 0
        if p < lo:
            continue
        for h in range(hq):
            kk, vv = k[lo:p + 1, h * hk // hq], v[lo:p + 1, h * hk // hq]
            with np.errstate(all="ignore"):
                s = scale * (kk @ q[i, h])
                top = s.max()
                if top == -np.inf:
                    continue
                w = np.exp(s - top)
                out[i, h] = (w[:, None] * vv).sum(0) / w.sum()
                big[i, h] = (w[:, None] * np.abs(vv)).sum(0) / w.sum()
                lse[i, h] = top + np.log(w.sum())
                d[i, h] = 2.0 ** -24 * (dim + 4) * scale * (np.abs(kk) @ np.abs(q[i, h])).max() + \
                    2.0 ** -23 * np.abs(s).max()
    return out, lse, big, d


def check(got, lse, refs, dtype, keys, vmax):
    """got [T, Hq, D], lse [T, Hq] (CPU tensors) against the list of attend()'s results in order."""
    out, want_lse, big, d = (np.concatenate([r[i] for r in refs]) for i in range(4))
    u = UNIT[dtype]
    g, n = got.double().numpy(), max(keys, 1)
    assert np.array_equal(np.isnan(g), np.isnan(out)), "NaN in other places"
    fine = np.isfinite(out)
    assert np.array_equal(g[~fine & ~np.isnan(out)], out[~fine & ~np.isnan(out)])
    sub = n * 2.0 ** -25 * vmax if dtype == torch.float16 else 0.0
    tol = 1.05 * (u * np.abs(out) + (u + 2 * d[..., None] + 2.0 ** -21 + 2 * n * 2.0 ** -24) * big) + sub + \
        (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133)
    err = np.abs(g - out)
    bad = fine & ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / np.maximum(tol, 1e-300))[fine].max()))
    if lse is not None:
        x = lse.double().numpy()
        known = np.isfinite(want_lse)
        assert np.array_equal(x[~known & ~np.isnan(want_lse)], want_lse[~known & ~np.isnan(want_lse)])
        assert np.array_equal(np.isnan(x), np.isnan(want_lse))
        tol = 1.05 * (2 * d + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(want_lse))
        assert np.all(np.abs(x - want_lse)[known] <= tol[known]), float(np.abs(x - want_lse)[known].max())


def rounding_only(got, refs, dtype):
    """Frobenius error in units of the roundoff: two independent roundings of relative size at most u
    have a root mean square of at most sqrt(2 / 3) u."""
    out = np.concatenate([r[0] for r in refs])
    off = np.linalg.norm(got.double().numpy() - out) / max(np.linalg.norm(out), 1e-300)
    return off / UNIT[dtype]


def starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def pages_of(lens, page, extra, rng):
    """A block table for requests of these lengths with shuffled pages, and the number of pages."""
    each = [-(-n // page) for n in lens]
    total = sum(each) + extra
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(max(each, default=0), 1)), -1, np.int32)
    at = 0
    for i, e in enumerate(each):
        table[i, :e] = order[at:at + e]
        at += e
    return torch.from_numpy(table), total


def fill_cache(rows, table, page, total, fill):
    """A cache [total, H, page, D] (CPU) with rows[i] [L_i, H, D] in request i's pages and `fill`
    everywhere else."""
    h, dim = rows[0].shape[1:]
    cache = torch.full((total, h, page, dim), fill, dtype=rows[0].dtype)
    for i, r in enumerate(rows):
        for p in range(r.shape[0]):
            cache[int(table[i, p // page]), :, p % page] = r[p]
    return cache

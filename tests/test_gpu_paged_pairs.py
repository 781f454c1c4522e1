"""Paged attention where rows and weights are carried as fp16 pairs hi + lo
(fp16 outputs, and up to 4 rows a KV head): the pairs' accuracy, which a
tolerance for operands rounded once does not see.

The 16 levels are made exact in fp16, so the tables add no error.  What is
left, relative to |q| |k_j| scale for logit j: the pair's 2^-22, and 2^-25 of
the row's largest coordinate for those below fp16's normal range (sqrt(d) 2^-25
in all); the turned row's fp32 stages, at most 2^-21; 2 d products, each cut
below 2^-24 of the sum it goes into.  For the output: the logits' errors, 2^-21
for a weight (its pair, ex2 and the product with the norm), 2 products a token
cut likewise, 2^-21 for the fp32 stages behind, and the output's half step.
Every test also forms what one rounding to fp16 would give and checks that the
bar rejects it."""

import math

import numpy as np
import pytest
import torch

from helpers import host, oracle_twin
from kv_cache_vector_13_b200 import api
from test_gpu_paged import DEV, paged_problem, rotate64, unpacked64

pytestmark = pytest.mark.gpu


def exact_levels(*qs):
    for z in qs:
        z.centroids.copy_(z.centroids.half().float())


def twin(z):
    o = oracle_twin(z)
    o.centroids = host(z.centroids)
    return o


def once(x):
    return x.astype(np.float16).astype(np.float64)


def reference(p, scale):
    """out, lse, their bars, and both with rows (lse) or weights (out) rounded once."""
    kq, vq, q, kc, vc, table, kv_lens, cu = p
    ok, ov = twin(kq), twin(vq)
    (T, Hq, d), (_, Hkv, P) = q.shape, kc.norms.shape
    q = host(q).astype(np.float64)
    table, kv_lens, cu, kcodes, knorms, vcodes, vnorms = (
        host(x) for x in (table, kv_lens, cu, kc.codes, kc.norms, vc.codes, vc.norms))
    out, bar, lse, lse_bar = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, Hq)), np.zeros((T, Hq))
    out1, lse1 = np.zeros(q.shape), np.zeros((T, Hq))
    rel = 2.0 ** -22 + math.sqrt(d) * 2.0 ** -25 + 2.0 ** -21 + 2 * d * 2.0 ** -24
    for r, m in enumerate(kv_lens):
        j = np.arange(m)
        pages = table[r][j // P]
        for hq in range(Hq):
            h = hq // (Hq // Hkv)
            K = unpacked64(ok, kcodes[pages, h, j % P], knorms[pages, h, j % P])
            V = unpacked64(ov, vcodes[pages, h, j % P], vnorms[pages, h, j % P])
            vn = vnorms[pages, h, j % P].astype(np.float64)
            Vo = np.abs(rotate64(V, 1.0))
            for t in range(cu[r], cu[r + 1]):
                x = rotate64(q[t, hq], ok.signs.astype(np.float64))
                z = scale * (K @ x)
                e = np.exp(z - z.max())
                w = e / e.sum()
                lse[t, hq] = z.max() + math.log(e.sum())
                out[t, hq] = rotate64(w @ V, 1.0) * ov.signs
                delta = rel * scale * np.linalg.norm(x) * np.linalg.norm(K, axis=1)
                lse_bar[t, hq] = delta.max() + 2.0 ** -21 * (1 + np.abs(z).max())
                bar[t, hq] = ((w * (delta + w @ delta + 2.0 ** -21)) @ Vo + 2.0 ** -21 * np.linalg.norm(w @ V)
                              + 2 * m * 2.0 ** -24 * np.linalg.norm(w @ np.abs(V)))
                f = 2.0 ** -math.floor(math.log2(np.abs(x).max()))
                z1 = scale * (K @ (once(x * f) / f))
                lse1[t, hq] = z1.max() + math.log(np.exp(z1 - z1.max()).sum())
                g = e * vn / (e * vn).max()
                out1[t, hq] = rotate64((once(g) * (e * vn).max() / e.sum()) @ (V / vn[:, None]), 1.0) * ov.signs
    return out, bar, lse, lse_bar, out1, lse1


@pytest.mark.parametrize("d,G,n,dtype", [
    (64, 1, 1, torch.float16), (128, 1, 1, torch.bfloat16), (128, 4, 1, torch.float16), (128, 2, 2, torch.bfloat16),
    (256, 4, 1, torch.bfloat16), (128, 8, 1, torch.float16), (64, 2, 4, torch.float16), (256, 8, 1, torch.float16),
    (128, 4, 4, torch.float16), (128, 8, 4, torch.float16), (64, 16, 3, torch.float16), (256, 4, 6, torch.float16),
    (64, 1, 60, torch.float16), (128, 4, 20, torch.float16), (128, 1, 140, torch.float16),
])
def test_rows_and_weights_as_pairs(d, G, n, dtype):
    kv = [1, 2, 2, 1, 40] if n * G > 40 else [1, 2] * 24 + [33, 40]
    p = paged_problem(d + n, [n] * len(kv), kv, 2 * G, 2, d, 16, dtype)
    kq, vq, q, kc, vc, table, kv_lens, cu = p
    exact_levels(kq, vq)
    scale = 1.0 / math.sqrt(d)
    op = api.PagedAttention(kq, vq, 2 * G, 2, len(kv), q.shape[0], device=DEV)

    def run():
        lse = torch.empty(q.shape[:2], device=DEV)
        out = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=n, causal=False, lse=lse)
        api.check()
        return host(out).astype(np.float64), host(lse)

    _, lse = run()
    _, _, want, bar, _, rounded = reference(p, scale)
    assert np.all(np.abs(lse - want) <= bar), (np.abs(lse - want) / bar).max()
    assert np.any(np.abs(rounded - want) > bar)  # rows without their lo half would show
    # values that nearly cancel, two by two: small logits, every other value the opposite of the one before
    kc.norms.mul_(0.01)
    vc.codes[:, :, 1::2] = ~vc.codes[:, :, 0::2]
    vc.norms[:, :, 1::2] = vc.norms[:, :, 0::2]
    out, _ = run()
    want, bar, _, _, rounded, _ = reference(p, scale)
    bar = bar + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.01 + torch.finfo(dtype).tiny
    assert np.all(np.abs(out - want) <= bar), (np.abs(out - want) / bar).max()
    assert np.any(np.abs(rounded - want) > bar)  # weights without theirs

"""Paged calls at the ends of their ranges on the GPU: values without a norm,
overflowed rows, windows and lengths near 2^31, weights far below the largest
one, slots that do not exist.  Plain 64-bit forms and tolerances as in
test_gpu_paged.py unless a test says otherwise."""

import math

import numpy as np
import pytest
import torch

from kv_cache_vector_13_b200 import api
from kv_cache_vector_13_b200 import _lib as L

from helpers import host, oracle_twin
from test_gpu_paged import DEV, attention_ref, check_attention, gen, paged_problem, quantizers, rotate64, unpacked64

pytestmark = pytest.mark.gpu


def repeated(problem, R):
    """A request R times: its rows and its table row again and again, so that
    units lie whole in a CTA's range, and are cut, at many places."""
    kq, vq, q, kc, vc, table, kv_lens, cu = problem
    n = q.shape[0]
    many = torch.arange(R + 1, device=DEV, dtype=torch.int32) * n
    return kq, vq, q.repeat(R, 1, 1), kc, vc, table.repeat(R, 1), kv_lens.repeat(R), many


def check_repeated(problem, R, finite=None, causal=True, window=0, least=0.0):
    """check_attention's bars for one request, held by each of its R copies.
    finite [T, Hq]: rows that have to be NaN throughout where it is False.
    least: what any output may be off besides."""
    kq, vq, q, kc, vc, table, kv_lens, cu = problem
    (n, Hq, d), Hkv = q.shape, kc.norms.shape[1]
    scale = 1.0 / math.sqrt(d)
    with np.errstate(all="ignore"):
        want, want_lse, tol, lse_tol = attention_ref(kq, vq, q, kc, vc, table, kv_lens, cu, scale, causal, window)
    many = repeated(problem, R)
    op = api.PagedAttention(kq, vq, Hq, Hkv, R, R * n, device=DEV)
    lse = torch.empty((R * n, Hq), device=DEV)
    out = op(many[2], kc, vc, many[5], many[6], cu_q=many[7], max_q=n, causal=causal, window=window, lse=lse)
    api.check()
    got, lse = host(out).astype(np.float64).reshape(R, n, Hq, d), host(lse).reshape(R, n, Hq)
    assert np.all(np.abs(lse - want_lse) <= lse_tol), np.abs(lse - want_lse).max()
    ok = np.ones((n, Hq), bool) if finite is None else finite
    assert np.all(np.isnan(got[:, ~ok])) and np.all(np.isnan(want[~ok]))
    want, tol, got = want[ok], tol[ok], got[:, ok]
    step = torch.finfo(q.dtype).eps / 2 * np.abs(want) * 1.01 + torch.finfo(q.dtype).tiny
    off = np.abs(got - want)
    assert np.all(off <= tol + step + least), np.nanmax(off - tol - step)


@pytest.mark.parametrize("R", [1, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,n", [(128, 1), (128, 8), (128, 24), (128, 45), (128, 100), (64, 100), (256, 20)])
@pytest.mark.parametrize("size,zeros", [(12.0, 1), (7.8, 64), (12.0, 64)])
def test_large_logits_of_values_without_a_norm(d, n, dtype, R, size, zeros):
    """Keys along the rows' common direction in the third block of 128 tokens,
    with logits of about 11 size above the others (85 and 135: weights of 2^122
    and beyond fp32 relative to the blocks before), whose values are zeros.

    A value without a norm counts as one of 2^-64 where the reference is
    chosen, and fp16 weights end at 2^-25 (half their smallest step) of it, so
    each of the other tokens may lose 2^-89 of its value."""
    p = paged_problem(n + d, [n], [460], 2, 1, d, 16, dtype)
    kq, vq, q, kc, vc, table, kv_lens, cu = p
    g = gen(3)
    base = torch.randn((1, 1, d), generator=g, device=DEV)
    base *= math.sqrt(d) / base.norm()
    q.copy_(base + 0.1 * torch.randn(q.shape, generator=g, device=DEV))
    key = api.encode(kq, (size * math.sqrt(128.0 / d) * base)[None])  # logits size sqrt(128) for any d
    for j in range(300, 300 + zeros):
        page = table[0, j // 16].long()
        kc.codes[page, 0, j % 16] = key.codes[0, 0, 0]
        kc.norms[page, 0, j % 16] = key.norms[0, 0, 0]
        vc.norms[page, 0, j % 16] = 0
    check_repeated(p, R, least=460 * 2.0 ** -89 * float(vc.norms.max()))


@pytest.mark.parametrize("R", [1, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,n", [(128, 1), (128, 8), (128, 24), (128, 45), (128, 100), (64, 100), (256, 20)])
@pytest.mark.parametrize("at", [3, 290, 459])
def test_an_infinite_value_norm_reaches_its_rows_only(d, n, dtype, R, at):
    """A value row that overflowed before it was stored: NaN in every row that
    sees it, as the definition has it, and their lse as it would be without."""
    p = paged_problem(n + d, [n], [460], 4, 2, d, 16, dtype)
    p[4].norms[p[5][0, at // 16].long(), 1, at % 16] = float("inf")
    finite = np.ones((n, 4), bool)
    finite[:, 2:] = (460 - n + np.arange(n) < at)[:, None]
    check_repeated(p, R, finite)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 6])
@pytest.mark.parametrize("d,qs,kv", [(128, [8, 1], [3, 40]), (128, [70, 5], [20, 300]), (64, [300], [7]), (256, [30], [5])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_window_wider_than_any_cache(d, qs, kv, dtype, window):
    """More query rows than cached tokens: their positions start below 0."""
    check_attention(paged_problem(d, qs, kv, 4, 2, d, 16, dtype), window=window)

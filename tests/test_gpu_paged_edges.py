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


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,n", [(128, 1), (128, 8), (128, 16), (128, 40), (128, 60), (128, 160), (64, 1), (64, 60), (256, 8)])
def test_many_small_weights_beside_a_large_one(d, n, dtype, apart):
    """Tokens in the first runs of 32 (small tiles: 12, one a run; else one a
    block of 128 in two) whose weight is 2^25.2 times that of each of the many
    others, which together carry about a fiftieth of the output (apart: their
    value's coordinates are of the largest level, the large token's of the
    smallest) or a hundredth (values of one kind, up to three million tokens).
    148 equal requests, so a CTA has a whole one.

    The relative 2-norm error: the levels' rounding 2^-11; for bf16 rows and
    weights 2^-11 each, rows behind the weights' logit of 17.5 for the share s
    of the small ones alone (the large ones are alike); the output's half step;
    half of fp16's smallest step, 2^-25, a weight of 2^-25.2 of the largest:
    that is kept at 2^8, so 2^-7.8 of s (were it kept at 1, all of s would be
    lost; for bf16 on the large tiles it is kept at 2, and the small weights,
    0.87 of the smallest step, round to it: 0.15 of s).  The products are summed in 32 bits: each may be cut
    below 2^-24 of the sum it goes into, which takes the products of a warp's
    tokens (one of 12, or 6 or 8) or a set's (all, or every other block's),
    two a token where weights are pairs."""
    kq, vq = quantizers(d)
    pairs, large = dtype == torch.float16, n > (48 if dtype == torch.float16 else 40)
    g, R, P, pages = gen(d + n), 148, 384, (200 if large else 1000) if apart else 8000
    x = torch.randn((2, 2, 1, 1, d), generator=g, device=DEV)
    q = torch.randn((1, 1, d), generator=g, device=DEV).to(dtype)
    # the large token's key lies along the query; the others' have no norm, so their logit is 0
    kc = api.encode(kq, q.float()[None].expand(2, 1, P, d).contiguous())
    vc = api.encode(vq, x[1].expand(2, 1, P, d).contiguous())
    big = api.encode(vq, x[0, :1])
    if apart:  # levels 7 and 8 are the two next to 0, 0 and 15 the outermost
        sign = torch.randint(0, 2, (d,), generator=g, device=DEV).to(torch.uint8)
        pack = lambda c: (c[0::2] | c[1::2] << 4)  # noqa: E731
        big.codes[:], vc.codes[:] = pack(7 + sign), pack(15 * sign.flip(0))
        big.norms.fill_(3.0)
        vc.norms.fill_(3.0)
    kc.norms.zero_()
    ok, ov = oracle_twin(kq), oracle_twin(vq)
    qr = rotate64(host(q)[0, 0].astype(np.float64), ok.signs.astype(np.float64))
    unit = unpacked64(ok, host(kc.codes[0, 0, :1]), np.ones(1))[0] @ qr / math.sqrt(d)
    norm = np.float32(25.2 * math.log(2) / unit)
    at = torch.tensor([0, 128] if large and apart else range(0, P, 32), device=DEV)
    kc.norms[0, 0, at] = float(norm)
    vc.codes[0, 0, at] = big.codes[0, 0, 0]
    vc.norms[0, 0, at] = big.norms[0, 0, 0]
    big_v = unpacked64(ov, host(big.codes)[0, 0], host(big.norms)[0, 0])[0]
    small_v = unpacked64(ov, host(vc.codes[1, 0, :1]), host(vc.norms[1, 0, :1]))[0]
    count, w = P * pages - len(at), len(at) * math.exp(float(norm) * unit)
    want = rotate64((w * big_v + count * small_v) / (w + count), 1.0) * ov.signs
    s = count * np.linalg.norm(small_v) / np.linalg.norm(w * big_v + count * small_v)
    table = torch.ones((1, pages), dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    lens = torch.full((R,), P * pages, dtype=torch.int32, device=DEV)
    cu = torch.arange(R + 1, dtype=torch.int32, device=DEV) * n
    op = api.PagedAttention(kq, vq, 1, 1, R, R * n, device=DEV)
    out = op(q.repeat(R * n, 1, 1), kc, vc, table.expand(R, pages).contiguous(), lens, cu_q=cu, max_q=n, causal=False)
    api.check()
    off = np.linalg.norm(host(out)[:, 0].astype(np.float64) - want, axis=-1) / np.linalg.norm(want)
    once = 0 if pairs or n <= 4 else 2.0 ** -11
    sets = (1 if n > 128 and not pairs else 2) if large else 8 if d == 256 else 6 if n > 16 else 12
    sums = P * pages / sets * (2 if pairs and n > 4 else 1) * 2.0 ** -24
    step = 2.0 ** 0.2 - 0.999 if large and not pairs else 2.0 ** -7.8
    bar = 2.0 ** -11 + torch.finfo(dtype).eps / 2 + once + s * (2 * 17.5 * 2.0 ** -10 + step) + sums
    assert off.max() <= bar, (off.max(), bar, s)
    assert not apart or bar < 0.98 * s  # a bar that the loss of the small ones would not pass


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 1), (torch.float16, 20), (torch.bfloat16, 60), (torch.float16, 60),
                                     (torch.bfloat16, 150)])
def test_the_longest_request(dtype, n):
    """2^31 - 16 tokens: 262657 times the same page of 8176, so the output is
    the page's own and its lse the page's plus log 262657.  The tensor cores'
    32-bit sums cut each product below 2^-24 of the sum it goes into, so the
    output may lose that for each of a warp's tokens (2^31 / 1776) or of a set's
    (2^31 / 296, or / 148 where the sets split the rows), twice where weights
    are pairs; the scalar sums of the weights lose at most 2^-24 in each of a
    lane's 2^17.3 additions.  A length that wraps leaves an output several times
    its own norm away."""
    P, m = 8176, 262657
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(n, [n], [P], 1, 1, 64, P, dtype, spare=0)
    op = api.PagedAttention(kq, vq, 1, 1, 1, n, device=DEV)
    lse, one_lse = torch.empty((n, 1), device=DEV), torch.empty((n, 1), device=DEV)
    one = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=n, lse=one_lse, causal=False)
    long = torch.full((1, m), int(table[0, 0]), dtype=torch.int32, device=DEV)
    out = op(q, kc, vc, long, torch.full_like(kv_lens, P * m), cu_q=cu, max_q=n, lse=lse, causal=False)
    api.check()
    off = (out.float() - one.float()).norm(dim=-1) / one.float().norm(dim=-1)
    tokens = 2 ** 31 / (888 if n == 20 else 1776 if n == 1 else 148 if n == 150 else 296)
    bar = tokens * 2.0 ** -24 * (2 if dtype == torch.float16 and n > 4 else 1) + 2.0 ** -6
    assert bool((off <= bar).all()), (off.max(), bar)
    assert bool(((lse - one_lse - math.log(m)).abs() <= 2.0 ** -6).all())


def refused(match="outside its cache"):
    with pytest.raises(L.TqError, match=match):
        api.check()
    api.check()  # the word is cleared


@pytest.mark.parametrize("slot", [-2, -2 ** 31, -2 ** 63])
def test_negative_slots_other_than_none_are_reported(slot):
    kq, vq = quantizers(64)
    kc, vc = (api.empty_cache(z, 2, 3, 16, device=DEV) for z in (kq, vq))
    for c in (kc, vc):
        c.codes.fill_(5)
        c.norms.fill_(2.0)
    k = torch.randn((3, 3, 64), generator=gen(1), device=DEV)
    none, bad = (torch.tensor([7, s, 9], device=DEV) for s in (-1, slot))
    api.paged_append(kq, vq, k, k, kc, vc, none)
    want = api.paged_dequant(kq, kc, none)
    api.check()
    api.paged_append(kq, vq, k, k, kc, vc, bad)
    refused()
    got = api.paged_dequant(kq, kc, bad)
    refused()
    assert torch.equal(got, want) and bool((got[1] == 0).all())
    touched = kc.norms != 2.0
    assert int(touched.sum()) == 6 and bool(touched.view(-1, 16)[:3, [7, 9]].all())  # page 0, three heads


def test_a_plan_over_a_missing_page_is_reported():
    """A request whose last page is begun but not in its table row: its tokens
    there have no slot."""
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    for missing, slots in ((-1, [-1, -1, 16 * 9]), (3, [16 * 3 + 14, 16 * 3 + 15, 16 * 9])):
        table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
        table[0, 0] = missing
        p = api.PagePlanner(2, 16, 4, device=DEV)(i32(14, 0), i32(3, 1), i32(8, 9), i32(2), table)
        if missing < 0:
            refused()
        else:
            api.check()
        assert p.slots.tolist() == slots + [16 * 8] and p.status.tolist() == [0, 0]
    # a request that is refused, or adds nothing, reads no page
    p = api.PagePlanner(2, 16, 40, device=DEV)(i32(14, 5), i32(40, 0), i32(8), i32(1), torch.full_like(table, -1))
    api.check()
    assert p.status.tolist() == [1, 0] and p.slots.tolist() == [-1] * 40


@pytest.mark.parametrize("call", ["append", "dequant", "attend", "encode", "dequant all", "search"])
def test_outputs_belong_to_the_stream_of_their_call(call):
    """The memory of what a call on another stream returns: none that the
    current stream has just let go of, and none that it gets next."""
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(40, [64, 64], [300, 90], 8, 2, 128, 16, torch.bfloat16)
    rope = api.Rope(torch.ones(64, device=DEV))
    op = api.PagedAttention(kq, vq, 8, 2, 2, 128, device=DEV)
    slots = torch.arange(128, device=DEV)
    places, queries = slots.int(), q[:, 0].contiguous()
    find = api.Search(kq, 128, 2048, device=DEV)
    db = api.encode(kq, torch.randn((2048, 128), generator=gen(1), device=DEV))
    rows = q.permute(1, 0, 2)[None].contiguous()
    run = {
        "append": lambda s: api.paged_append(kq, vq, q[:, :2], q[:, :2], *caches, slots, q=q, rope=rope,
                                             positions=places, stream=s),
        "dequant": lambda s: api.paged_dequant(kq, kc, slots, stream=s),
        "attend": lambda s: op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=64, stream=s),
        "encode": lambda s: api.encode(kq, rows, stream=s).codes,
        "dequant all": lambda s: api.dequant(kq, kc, stream=s),
        "search": lambda s: find(queries, db, 10, stream=s)[1],
    }[call]
    caches = [api.empty_cache(z, 8, 2, 16, device=DEV) for z in (kq, vq)]
    side = torch.cuda.Stream()
    for s in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        want = run(None)
        torch.cuda.synchronize()
        gone = torch.empty_like(want)
        before = gone.data_ptr()
        del gone
        got = run(s)
        at = got.data_ptr()
        s.synchronize()
        assert torch.equal(got, want) and at != before
        torch.cuda.synchronize()
        del got
        assert torch.empty_like(want).data_ptr() != at
    assert torch.equal(run(torch.cuda.current_stream()), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_named_too_often_are_refused(dtype):
    """Forty requests of the same 300 rows make more tiles than the call's 300
    rows have, which the workspace has no room for: none is worked on."""
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(41, [300], [350], 4, 2, 128, 16, dtype)
    many = torch.tensor([0, 300] * 40 + [0], dtype=torch.int32, device=DEV)
    op = api.PagedAttention(kq, vq, 4, 2, 80, 300, device=DEV)
    out, lse = torch.full_like(q, 5.0), torch.full((300, 4), 7.0, device=DEV)
    op(q, kc, vc, table.repeat(80, 1), kv_lens.repeat(80), cu_q=many, max_q=300, out=out, lse=lse)
    refused()
    assert bool((out == 5.0).all()) and bool((lse == 7.0).all())
    check_attention((kq, vq, q, kc, vc, table, kv_lens, cu), op=op)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("qs", [[3, 1], [70, 1]])
def test_large_scales(qs, dtype):
    """Logits of a few tens and more: one or two tokens carry a row."""
    for scale in (5.0 / math.sqrt(128), -20.0 / math.sqrt(128)):
        kq, vq, q, kc, vc, table, kv_lens, cu = p = paged_problem(9, qs, [90, 70], 4, 2, 128, 16, dtype)
        want, want_lse, tol, lse_tol = attention_ref(*p, scale, True, 0)
        lse = torch.empty(q.shape[:2], device=DEV)
        out = api.PagedAttention(kq, vq, 4, 2, 2, sum(qs), device=DEV)(
            q, kc, vc, table, kv_lens, cu_q=cu, max_q=max(qs), scale=scale, lse=lse)
        api.check()
        off = np.abs(host(out).astype(np.float64) - want)
        assert np.all(np.abs(host(lse) - want_lse) <= lse_tol)
        # a logit off by delta moves its weight by a factor exp(delta): to first order what tol holds, and beyond it
        # by exp(2 delta) - 1 over 2 delta at most
        grow = np.expm1(2 * lse_tol) / (2 * lse_tol)
        assert np.all(off <= tol * grow[..., None] + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.01
                      + torch.finfo(dtype).tiny)

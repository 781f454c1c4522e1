"""Serving on a paged 4-bit cache on the GPU: page plan, rotary append,
read-back and ragged attention, each against a plain 64-bit implementation in
this file, and a serving loop that chains them.

Tolerances.  Integers are equal.  Records without positions are bit-identical
to tq_encode's (and so to the oracle's).  Turned rows: an output rounds by at
most half a step (finfo.eps / 2), and the fp32 steps before it (sin and cos to
2^-22 of a unit vector, two products and a sum) stay below 2^-20 of the pair's
length.

Attention.  The kernels' operands are fp16, each off by at most 2^-11 of
itself (half a step): q and the 16 levels move logit j by at most
  delta_j = (2^-11 + 2^-11) scale sum_i |q_i k_ji| <= 2^-10 scale ||q|| ||k_j||,
so, to first order, softmax weight p_j by p_j (delta_j + sum_k p_k delta_k)
and the output by sum_j of that times |v_j|; the rounded weights add 2^-11
sum_j p_j |v_j|, the levels of the values 2^-11 || sum_j p_j |v'_j| || (v' in
the rotated basis, the error rotated back), weights below fp16's normal range
2^-24 of the largest term each; 5% on top for the second order, and the
output's half step.  lse moves by at most the largest delta_j.  Over a whole
output the errors average: its relative 2-norm error stays within the
framework's 2e-3 (and the output's rounding).  Up to 8 query rows a KV head
every row holds the framework's decode bar, 2e-3 of its largest output (up to
4, and for fp16 outputs, rows and weights are carried as hi + lo pairs)."""

import math

import numpy as np
import pytest
import torch

from kv_cache_vector_13_b200 import api
from kv_cache_vector_13_b200 import _lib as L
from oracle import quantizer as OQ

from helpers import host, oracle_twin

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def quantizers(d):
    return (api.Quantizer(d, 4, "mse", seed_rot=21, device=DEV), api.Quantizer(d, 4, "mse", seed_rot=22, device=DEV))


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# --------------------------------------------------------------------- plan

def plan_ref(lens, new, free, n_free, table, P, rows):
    """Plain loops over requests and tokens."""
    table, R = table.copy(), len(lens)
    n_free = min(max(n_free, 0), len(free))
    slots, pos = np.full(rows, -1, np.int64), np.zeros(rows, np.int32)
    cu, seq, status = [0], [], []
    want = left = 0
    left = n_free
    for r in range(R):
        l, n = max(int(lens[r]), 0), max(int(new[r]), 0)
        begin = cu[-1]
        cu.append(begin + n)
        had, has = -(-l // P), -(-(l + n) // P)
        st = 0
        if has > table.shape[1] or begin + n > rows:
            st = 2
        elif has > had:
            if want + has - had > n_free:
                st = 1
            else:
                for j in range(had, has):
                    table[r, j] = free[n_free - 1 - want - (j - had)]
                left -= has - had
            want += has - had
        status.append(st)
        seq.append(l if st else l + n)
        for i in range(n):
            t = begin + i
            if t < rows:
                pos[t] = l + i
                if st == 0:
                    slots[t] = int(table[r, (l + i) // P]) * P + (l + i) % P
    return slots, pos, np.array(cu), np.array(seq), np.array(status), left, table


@pytest.mark.parametrize("R,P,most_len,most_new,pool,spare", [
    (1, 16, 0, 1, 1.0, 0), (1, 1, 5, 3, 1.0, 2), (7, 16, 100, 40, 1.0, 3), (16, 64, 1000, 1, 1.0, 0),
    (40, 16, 300, 100, 0.5, 0), (513, 16, 50, 9, 0.7, 11), (1500, 3, 20, 5, 1.2, 0), (300, 48, 4000, 700, 1.0, 1),
    (9, 16, 64, 16, 0.0, 0), (5, 7, 30, 0, 1.0, 4),
])
def test_plan_matches_loops(R, P, most_len, most_new, pool, spare):
    rng = np.random.default_rng(R * 1000 + P)
    lens = rng.integers(0, most_len + 1, R).astype(np.int32)
    new = rng.integers(0, most_new + 1, R).astype(np.int32)
    lens[rng.random(R) < 0.2] = 0
    new[rng.random(R) < 0.2] = 0
    if R > 4:
        lens[1], new[1] = -3, 2      # a negative length counts as 0
        new[2] = -1
        lens[3] = lens[3] // P * P   # a full last page
    width = int((np.maximum(lens, 0) + np.maximum(new, 0)).max() // P + 1)
    if R > 4:
        width = max(1, width - 1)    # the longest do not fit their row
    had = -(-np.maximum(lens, 0) // P)
    need = int((-(-(np.maximum(lens, 0) + np.maximum(new, 0)) // P) - had).sum())
    n_free = int(need * pool)
    ids = rng.permutation(int(had.sum()) + n_free + 5).astype(np.int32)
    table = np.full((R, width), -7, np.int32)
    at = 0
    for r in range(R):
        k = min(int(had[r]), width)
        table[r, :k] = ids[at:at + k]
        at += k
    free = ids[int(had.sum()):]
    rows = int(np.maximum(new, 0).sum()) + spare - (2 if R == 40 else 0)  # too few rows once
    ref = plan_ref(lens, new, free, n_free, table, P, rows)
    dt = torch.from_numpy(table).to(DEV)
    planner = api.PagePlanner(R, P, rows, device=DEV)
    args = [torch.from_numpy(x).to(DEV) for x in (lens, new, free)]
    for _ in range(2):  # the same step planned twice: nothing it reads has changed
        p = planner(*args, torch.tensor([n_free], dtype=torch.int32, device=DEV), dt)
        for got, want in zip((p.slots, p.positions, p.cu_new, p.seq_lens, p.status, p.n_free, dt), ref):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(np.shape(want)), want)


def test_plan_strided_table_and_clamped_free_count():
    table = torch.full((3, 20), -1, dtype=torch.int32, device=DEV)
    sub = table[:, :4]
    planner = api.PagePlanner(3, 16, 60, device=DEV)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    new = torch.tensor([20, 20, 20], dtype=torch.int32, device=DEV)
    free = torch.tensor([5, 6, 7, 8], dtype=torch.int32, device=DEV)
    p = planner(lens, new, free, torch.tensor([99], dtype=torch.int32, device=DEV), sub)  # 99 of 4
    assert p.status.tolist() == [0, 0, 1] and p.n_free.tolist() == [0]
    assert table[:2, :2].tolist() == [[8, 7], [6, 5]] and int((table >= 0).sum()) == 4
    p = planner(lens, new, free, torch.tensor([-2], dtype=torch.int32, device=DEV), sub)
    assert p.status.tolist() == [1, 1, 1] and p.n_free.tolist() == [0]
    p = api.PagePlanner(0, 16, 3, device=DEV)(lens[:0], new[:0], free, torch.tensor([2], dtype=torch.int32, device=DEV),
                                            table[:0])
    assert p.slots.tolist() == [-1] * 3 and p.cu_new.tolist() == [0] and p.n_free.tolist() == [2]


# ---------------------------------------------------------- append, read-back

def rope_ref(x, pos, inv_freq, axis, pairing):
    """x [T, H, d] in 64 bits, turned by plain complex products."""
    x = x.astype(np.float64).copy()
    half = len(inv_freq)
    theta = pos.astype(np.float64)[axis].T * inv_freq.astype(np.float64)  # [T, half]
    e = np.exp(1j * theta)[:, None]
    a = slice(0, half) if pairing == "half" else slice(0, 2 * half, 2)
    b = slice(half, 2 * half) if pairing == "half" else slice(1, 2 * half, 2)
    z = (x[..., a] + 1j * x[..., b]) * e
    x[..., a], x[..., b] = z.real, z.imag
    return x


def flat_records(cache, slots):
    """Host (codes, norms) at slots, [T, H, ...]."""
    P = cache.norms.shape[2]
    s = slots.cpu()
    return (cache.codes.cpu()[s // P, :, s % P].numpy(), cache.norms.cpu()[s // P, :, s % P].numpy())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,H,P", [(1, 1, 16), (5, 3, 7), (67, 8, 48), (1300, 2, 16)])
def test_append_without_positions_equals_encode(d, T, H, P, dtype):
    g = gen(T * d + H)
    kq, vq = quantizers(d)
    rows = torch.randn((T, 2 * H + 1, d), generator=g, device=DEV).to(dtype)  # strided rows
    k, v = rows[:, 1:1 + H], rows[:, 1 + H:]
    k[T // 2, 0] = 0  # a zero vector
    n_pages = -(-T // P) + 2
    slots = torch.randperm(n_pages * P, generator=g, device=DEV)[:T]
    skip = torch.arange(T, device=DEV) % 5 == 3
    slots = torch.where(skip, -1, slots).contiguous()
    kc, vc = (api.empty_cache(z, n_pages, H, P, device=DEV) for z in (kq, vq))
    for c in (kc, vc):
        c.codes.fill_(0xAB)
        c.norms.fill_(-1.0)
    assert api.paged_append(kq, vq, k, v, kc, vc, slots) is None
    api.check()
    live = slots[~skip]
    touched = torch.zeros(n_pages * P, dtype=torch.bool, device=DEV)
    touched[live] = True
    for z, x, c in ((kq, k, kc), (vq, v, vc)):
        want = api.encode(z, x.permute(1, 0, 2)[None].contiguous())
        codes, norms = flat_records(c, live)
        keep = (~skip).cpu()
        np.testing.assert_array_equal(codes, want.codes[0].permute(1, 0, 2).cpu()[keep].numpy())
        np.testing.assert_array_equal(norms.view(np.uint32), want.norms[0].permute(1, 0).cpu()[keep].contiguous().numpy().view(np.uint32))
        enc = OQ.encode(oracle_twin(z), host(x[~skip].reshape(-1, d)), aux=False)
        np.testing.assert_array_equal(codes.reshape(-1, d // 2), enc["codes"])
        # no other record was written
        rest = (~touched).view(n_pages, P)
        assert bool((c.norms.permute(0, 2, 1)[rest] == -1).all()) and bool((c.codes.permute(0, 2, 1, 3)[rest] == 0xAB).all())


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("d,rot,sections,dtype", [
    (128, 128, None, torch.bfloat16), (128, 96, (20, 14, 14), torch.float16), (128, 48, (8, 16), torch.float32),
    (64, 64, (16, 8, 8), torch.bfloat16), (64, 16, None, torch.float32), (256, 256, (64, 32, 32), torch.float16),
    (256, 80, (0, 40), torch.float32),
])
def test_append_with_positions(d, rot, sections, dtype, pairing):
    T, Hq, Hkv, P = 53, 6, 2, 16
    g = gen(d + rot)
    kq, vq = quantizers(d)
    half = rot // 2
    inv_freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float()
    rope = api.Rope(inv_freq.to(DEV), sections=sections, pairing=pairing)
    pos = torch.randint(0, 1 << 20, (rope.n_axes, T), generator=g, device=DEV, dtype=torch.int32)
    pos[:, 0] = 0
    pos[:, 1] = 2 ** 31 - 1
    pos[:, 2] = -77
    q = torch.randn((T, Hq, d), generator=g, device=DEV).to(dtype)
    k, v = (torch.randn((T, Hkv, d), generator=g, device=DEV).to(dtype) for _ in range(2))
    if rot < d:
        q[5, 0, d - 1] = float("inf")  # a coordinate that is not turned keeps what it holds
        q[6, 0, d - 1] = float("nan")
    slots = torch.randperm(5 * P, generator=g, device=DEV)[:T].contiguous()
    kc, vc = (api.empty_cache(z, 5, Hkv, P, device=DEV) for z in (kq, vq))
    qo = api.paged_append(kq, vq, k, v, kc, vc, slots, q=q, rope=rope, positions=pos)
    axis = np.zeros(half, int) if rope.axis is None else rope.axis.cpu().numpy()
    want = rope_ref(host(q), pos.cpu().numpy(), inv_freq.numpy(), axis, pairing)
    got = host(qo).astype(np.float64)
    a, b = (slice(0, half), slice(half, rot)) if pairing == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    length = np.zeros_like(want)
    length[..., a] = length[..., b] = np.hypot(want[..., a], want[..., b])
    eps = torch.finfo(dtype).eps / 2
    with np.errstate(invalid="ignore"):
        tol = np.abs(want) * eps + length * 2.0 ** -20 + torch.finfo(dtype).tiny
        np.testing.assert_array_equal(np.isfinite(got), np.isfinite(want))
        ok = np.isfinite(want)
        assert np.all(np.abs(got - want)[ok] <= tol[ok])
        np.testing.assert_array_equal(got[..., rot:], host(q).astype(np.float64)[..., rot:])
    # K: the record of the exactly turned row, but for coordinates that the fp32 turn moves over a threshold
    turned = rope_ref(host(k), pos.cpu().numpy(), inv_freq.numpy(), axis, pairing).reshape(-1, d)
    oq = oracle_twin(kq)
    n = np.linalg.norm(turned, axis=1)
    codes, norms = flat_records(kc, slots)
    assert np.all(np.abs(norms.reshape(-1) - n) <= n * 2.0 ** -20)
    H = oq.signs[None].astype(np.float64) * turned
    h = 1
    while h < d:
        H = H.reshape(-1, d // (2 * h), 2, h)
        H = np.stack([H[:, :, 0] + H[:, :, 1], H[:, :, 0] - H[:, :, 1]], 2).reshape(-1, d)
        h *= 2
    u = H / (n[:, None] * math.sqrt(d))
    idx = OQ.unpack_bits(codes.reshape(-1, d // 2), d, 4)
    thr = oq.thresholds.astype(np.float64)
    # a coordinate of the unit vector is off by at most the turned row's relative error, 2^-20, and the
    # transform's own fp32 steps, log2(d) + 3 roundings of values up to sum |x_i| / (n sqrt d) <= 1
    band = 2.0 ** -20 + (math.log2(d) + 3) * 2.0 ** -24
    lo = (u[..., None] > thr + band).sum(-1)
    hi = (u[..., None] > thr - band).sum(-1)
    assert np.all((idx >= lo) & (idx <= hi))
    # V is not turned
    np.testing.assert_array_equal(flat_records(vc, slots)[0].reshape(-1, d // 2),
                                  OQ.encode(oracle_twin(vq), host(v).reshape(-1, d), aux=False)["codes"])


def test_append_only_queries_or_only_keys():
    kq, vq = quantizers(128)
    rope = api.Rope(torch.ones(64, device=DEV))
    g = gen(5)
    k = torch.randn((4, 1, 128), generator=g, device=DEV)
    q = torch.randn((4, 2, 128), generator=g, device=DEV)
    kc, vc = (api.empty_cache(z, 1, 1, 16, device=DEV) for z in (kq, vq))
    slots = torch.arange(4, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert api.paged_append(kq, vq, k, k, kc, vc, slots, rope=rope, positions=pos) is None
    codes = kc.codes.clone()
    no = torch.full((4,), -1, device=DEV, dtype=torch.int64)
    kc.codes.fill_(1)
    qo = api.paged_append(kq, vq, k, k, kc, vc, no, q=q, rope=rope, positions=pos)
    assert torch.equal(qo, q) and bool((kc.codes == 1).all())  # position 0 turns nothing, no slot writes nothing
    np.testing.assert_array_equal(codes[0, :, :4].cpu().numpy().reshape(4, 64),
                                  OQ.encode(oracle_twin(kq), host(k).reshape(4, 128), aux=False)["codes"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,T,H,P", [(64, 1, 1, 16), (64, 333, 5, 48), (128, 77, 3, 7), (128, 2000, 8, 64), (256, 19, 2, 16)])
def test_dequant_matches_definition(d, T, H, P, dtype):
    g = gen(d + T)
    kq, _ = quantizers(d)
    oq = oracle_twin(kq)
    n_pages = -(-T // P) + 1
    c = api.encode(kq, torch.randn((n_pages, H, P, d), generator=g, device=DEV) * 3)
    slots = torch.randperm(n_pages * P, generator=g, device=DEV)[:T].contiguous()
    if T > 4:
        slots[3] = -1
        slots[4] = slots[0]  # reading one slot twice is fine
    x = api.paged_dequant(kq, c, slots, dtype=dtype)
    codes, norms = flat_records(c, slots.clamp(min=0))
    cent = oq.centroids.astype(np.float64)[OQ.unpack_bits(codes.reshape(-1, d // 2), d, 4)]
    h = 1
    y = cent
    while h < d:
        y = y.reshape(-1, d // (2 * h), 2, h)
        y = np.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2).reshape(-1, d)
        h *= 2
    want = (y / math.sqrt(d) * oq.signs * norms.reshape(-1, 1).astype(np.float64)).reshape(T, H, d)
    if T > 4:
        want[3] = 0
    # log2(d) + 4 fp32 roundings of partial sums below sum |c_i|, then the output's half step
    size = (np.abs(cent).sum(1) / math.sqrt(d) * norms.reshape(-1)).reshape(T, H, 1)
    tol = size * (math.log2(d) + 4) * 2.0 ** -24 + np.abs(want) * torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -10)
    assert np.all(np.abs(host(x).astype(np.float64) - want) <= tol + torch.finfo(dtype).tiny)



# ---------------------------------------------------------------- attention

def unpacked64(oq, codes, norms):
    d = oq.d
    c = oq.centroids.astype(np.float64)[OQ.unpack_bits(codes.reshape(-1, d // 2), d, 4)]
    return c.reshape(codes.shape[:-1] + (d,)) * norms[..., None].astype(np.float64)


def rotate64(x, signs):
    """H (signs x) / sqrt d over the last axis."""
    d = x.shape[-1]
    i = np.arange(d)
    pop = np.array([bin(v).count("1") & 1 for v in range(d)])
    Hm = 1.0 - 2.0 * pop[i[:, None] & i[None]]
    return (x * signs) @ Hm / math.sqrt(d)


def attention_ref(kq, vq, q, kc, vc, table, kv_lens, cu, scale, causal, window):
    """(out, lse, tolerance of out, of lse) in 64 bits, request by request; rows behind cu[-1] NaN."""
    ok, ov = oracle_twin(kq), oracle_twin(vq)
    T, Hq, d = q.shape
    P, Hkv = kc.norms.shape[2], kc.norms.shape[1]
    q = host(q).astype(np.float64)
    out, lse = np.full(q.shape, np.nan), np.full((T, Hq), np.nan)
    tol, lse_tol = np.zeros(q.shape), np.zeros((T, Hq))
    table, kv_lens, cu = (host(x) for x in (table, kv_lens, cu))
    kcodes, knorms, vcodes, vnorms = (host(x) for x in (kc.codes, kc.norms, vc.codes, vc.norms))
    ov_signs = ov.signs.astype(np.float64)
    for r in range(len(kv_lens)):
        n, m = int(cu[r + 1] - cu[r]), int(kv_lens[r])
        j = np.arange(m)
        pages = table[r][j // P]
        for h in range(Hkv):
            K = unpacked64(ok, kcodes[pages, h, j % P], knorms[pages, h, j % P])
            V = unpacked64(ov, vcodes[pages, h, j % P], vnorms[pages, h, j % P])
            Vo = np.abs(rotate64(V, 1.0))
            kn = np.linalg.norm(K, axis=1)
            for i in range(n):
                p = m - n + i
                seen = np.ones(m, bool)
                if causal:
                    seen = j <= p
                if window:
                    seen &= j > p - window
                for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    t = cu[r] + i
                    if not seen.any():
                        out[t, hq], lse[t, hq] = 0.0, -np.inf
                        continue
                    z = scale * (K[seen] @ rotate64(q[t, hq], ok.signs.astype(np.float64)))
                    p = np.exp(z - z.max())
                    lse[t, hq] = z.max() + math.log(p.sum())
                    p /= p.sum()
                    out[t, hq] = rotate64(p @ V[seen], 1.0) * ov_signs
                    delta = 2.0 ** -10 * abs(scale) * np.linalg.norm(q[t, hq]) * kn[seen]
                    lse_tol[t, hq] = 1e-5 + delta.max()
                    tol[t, hq] = 1.05 * ((p * (delta + p @ delta + 2.0 ** -11)) @ Vo[seen]
                                         + 2.0 ** -11 * np.linalg.norm(p @ np.abs(V[seen]))
                                         + len(z) * 2.0 ** -24 * (p[:, None] * Vo[seen]).max())
    return out, lse, tol, lse_tol


def paged_problem(seed, qs, kv, Hq, Hkv, d, P, dtype, sigma=0.5, spare=1):
    g = gen(seed)
    kq, vq = quantizers(d)
    R, T = len(qs), sum(qs)
    width = max(1, max(-(-m // P) for m in kv)) + spare
    held = sum(-(-m // P) for m in kv)
    n_pages = held + 2
    x = torch.randn((2, n_pages, Hkv, P, d), generator=g, device=DEV) * torch.exp(
        sigma * torch.randn((2, n_pages, Hkv, P, 1), generator=g, device=DEV))
    kc, vc = api.encode(kq, x[0]), api.encode(vq, x[1])
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    ids = torch.randperm(n_pages, generator=g, device=DEV).int()
    at = 0
    for r, m in enumerate(kv):
        k = -(-m // P)
        table[r, :k] = ids[at:at + k]
        at += k
    q = torch.randn((T, Hq, d), generator=g, device=DEV).to(dtype)
    kv_lens = torch.tensor(kv, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32, device=DEV)
    return kq, vq, q, kc, vc, table, kv_lens, cu


def poison_unseen(kc, vc, table, kv_lens):
    """NaN and infinite norms in every record that no request holds."""
    P = kc.norms.shape[2]
    held = torch.zeros((kc.norms.shape[0], P), dtype=torch.bool, device=DEV)
    for r, m in enumerate(kv_lens.tolist()):
        for j in range(-(-m // P)):
            held[int(table[r, j]), :min(P, m - j * P)] = True
    for c, bad in ((kc, float("nan")), (vc, float("inf"))):
        c.norms.copy_(torch.where(held[:, None, :], c.norms, bad))


def check_attention(problem, causal=True, window=0, max_q=None, scale=None, use_cu=True, op=None):
    kq, vq, q, kc, vc, table, kv_lens, cu = problem
    T, Hq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    op = op or api.PagedAttention(kq, vq, Hq, kc.norms.shape[1], len(kv_lens), T, device=DEV)
    lse = torch.full((T, Hq), 7.0, device=DEV)
    out = torch.full((T, Hq, d), 5.0, dtype=q.dtype, device=DEV)
    qs = cu.diff().tolist()
    o = op(q, kc, vc, table, kv_lens, cu_q=cu if use_cu else None, max_q=max_q or max(max(qs), 1), causal=causal,
           window=window, scale=scale, out=out, lse=lse)
    assert o is out
    api.check()
    want, want_lse, tol, lse_tol = attention_ref(kq, vq, q, kc, vc, table, kv_lens, cu, scale, causal, window)
    n = int(cu[-1])
    got = host(out).astype(np.float64)
    assert np.all(got[n:] == 5.0) and bool((lse[n:] == 7.0).all())  # rows behind the last sequence
    want, got, want_lse = want[:n], got[:n], want_lse[:n]
    step = torch.finfo(q.dtype).eps / 2 * np.abs(want) * 1.01 + torch.finfo(q.dtype).tiny
    off = np.abs(got - want)
    assert np.all(off <= tol[:n] + step), (off / (tol[:n] + step)).max()
    assert np.linalg.norm(off) <= 2e-3 * np.linalg.norm(want) + np.linalg.norm(step)
    if max(max(qs), 1) * (Hq // kc.norms.shape[1]) <= 8 and max_q is None:
        assert np.all(off <= 2e-3 * np.abs(want).max(-1, keepdims=True) + step)
    fl = host(lse)[:n]
    empty = np.isinf(want_lse)
    np.testing.assert_array_equal(np.isneginf(fl), empty)
    assert np.all(np.abs(fl[~empty] - want_lse[~empty]) <= lse_tol[:n][~empty])
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,Hkv", [(1, 1), (4, 2), (7, 1), (8, 2), (16, 1), (3, 3)])
def test_decode_rows(d, G, Hkv, dtype):
    kv = [1, 15, 16, 17, 0, 33, 200, 64]
    check_attention(paged_problem(d + G, [1] * len(kv), kv, G * Hkv, Hkv, d, 16, dtype), use_cu=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 48, 64, 256])
def test_long_and_ragged_decode(d, P):
    kv = [3000, 1, 777, 2048]
    p = paged_problem(P + d, [1] * 4, kv, 8, 2, d, P, torch.bfloat16)
    poison_unseen(p[3], p[4], p[5], p[6])
    check_attention(p)
    check_attention(p, window=100)
    check_attention(p, causal=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qs,kv", [
    ([4, 2, 5], [100, 2, 37]), ([3, 0, 1, 7], [40, 9, 0, 3]), ([16], [16]), ([17, 1], [17, 500]), ([33, 40], [33, 139]),
    ([130, 3], [130, 700]), ([70, 300], [250, 300]),
])
@pytest.mark.parametrize("window", [0, 29])
def test_ragged_rows_with_causal_mask(d, qs, kv, window):
    p = paged_problem(sum(qs) + d, qs, kv, 4, 2, d, 16, torch.bfloat16)
    poison_unseen(p[3], p[4], p[5], p[6])
    check_attention(p, window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G", [1, 5, 8])
def test_prefill_rows(G, dtype):
    p = paged_problem(G, [200, 1, 64], [456, 300, 64], G * 2, 2, 128, 32, dtype)
    poison_unseen(p[3], p[4], p[5], p[6])
    check_attention(p)
    check_attention(p, causal=False)


def test_rows_behind_the_last_sequence_and_strided_rows():
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(3, [2, 9], [50, 9], 8, 2, 128, 16, torch.bfloat16)
    wide = torch.randn((14, 12, 128), device=DEV, generator=gen(4)).to(torch.bfloat16)
    wide[:11, 2:10] = q
    check_attention((kq, vq, wide[:, 2:10], kc, vc, table, kv_lens, cu))


def test_scale_sign_and_large_logits():
    p = paged_problem(9, [3, 1], [90, 70], 4, 2, 128, 16, torch.float16)
    # logits of a few tens: the fp16 operands' 2^-11 moves them by up to some 1e-2, and each weight as much;
    # 5 / sqrt(d) keeps |logit| <= 5 * 11.3 * a few and the row's error inside the bar by the weights' averaging
    check_attention(p, scale=0.0)
    check_attention(p, scale=-1.0 / math.sqrt(128))


def test_query_rows_of_any_size():
    # rows of 1e4 and 1e-4: the fp16 operands are scaled by the row
    for f in (1e4, 1e-4):
        kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(10, [3, 1, 40], [90, 70, 60], 4, 2, 128, 16, torch.bfloat16)
        check_attention((kq, vq, (q.float() * f).to(torch.bfloat16), kc, vc, table, kv_lens, cu), scale=0.088 / f)


def test_value_norms_of_any_size():
    for f in (1e-6, 1e5):
        p = paged_problem(12, [1, 2, 130], [90, 70, 260], 4, 2, 128, 16, torch.bfloat16)
        p[4].norms.mul_(f)
        p[4].norms[:, :, 5] = 0
        check_attention(p)


def test_pages_in_another_layout():
    # [n_pages, P, H] records (stride_n = H) next to [n_pages, H, P]
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(13, [1, 5], [90, 70], 4, 2, 128, 16, torch.bfloat16)
    t = lambda c: api.PackedCache(c.codes.transpose(1, 2).contiguous().transpose(1, 2),
                                  c.norms.transpose(1, 2).contiguous().transpose(1, 2))
    check_attention((kq, vq, q, t(kc), vc, table, kv_lens, cu))
    check_attention((kq, vq, q, kc, t(vc), table, kv_lens, cu))


def other_layout(c, order):
    """The cache with pages, heads and tokens in another order in memory."""
    back = [order.index(i) for i in range(3)]
    return api.PackedCache(c.codes.permute(*order, 3).contiguous().permute(*back, 3),
                           c.norms.permute(*order).contiguous().permute(*back))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,qs", [(1, [3, 1, 1]), (2, [4, 0, 1]), (4, [4, 1, 3]), (8, [4, 1, 2])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_a_unit_in_another_layout(d, G, qs, dtype):
    """3 to 32 rows a request and head, caches whose tokens do not lie side by side, K and V laid out apart."""
    p = list(paged_problem(d + G, qs, [600, 47, 1], 2 * G, 2, d, 48, dtype))
    poison_unseen(p[3], p[4], p[5], p[6])
    p[3] = other_layout(p[3], (0, 2, 1))
    check_attention(p)
    p[4] = other_layout(p[4], (2, 1, 0))
    check_attention(p, window=40)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,qs,kv", [(4, [5, 1, 9], [300, 33, 9]), (8, [3, 40, 1], [129, 40, 2000]), (1, [130, 16], [700, 16])])
@pytest.mark.parametrize("window", [0, 29])
def test_ragged_rows_of_256(G, qs, kv, window, dtype):
    p = paged_problem(G, qs, kv, G * 2, 2, 256, 16, dtype)
    poison_unseen(p[3], p[4], p[5], p[6])
    check_attention(p, window=window)
    if not window:
        check_attention(p, causal=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,qs", [(1, [40, 33, 1]), (4, [10, 1, 9]), (8, [5, 5, 2]), (6, [8, 7, 0])])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_two_units(d, G, qs, dtype):
    """Around the most rows that the small tiles take: more than one unit a request and head, and just beyond."""
    p = paged_problem(d + G, qs, [300, 1000, 41], 2 * G, 2, d, 16, dtype)
    poison_unseen(p[3], p[4], p[5], p[6])
    check_attention(p)
    check_attention(p, window=29)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("qs,kv", [([1], [1]), ([1], [40]), ([70], [70]), ([1] * 300, [(17 * i) % 90 for i in range(300)]),
                                   ([40] + [1] * 20, [40] + [3000] + [5] * 19)])
def test_short_units_beside_long_ones(d, qs, kv):
    """Units of a step or none beside long ones, and fewer steps than there are SMs."""
    check_attention(paged_problem(len(qs) + d, qs, kv, 1, 1, d, 16, torch.bfloat16))



def test_a_nan_in_a_seen_record_reaches_its_rows_only():
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(14, [1, 3], [40, 70], 4, 2, 128, 16, torch.bfloat16)
    vc.norms[table[0, 1].long(), 1, 3] = float("nan")
    out = api.PagedAttention(kq, vq, 4, 2, 2, 4, device=DEV)(q, kc, vc, table, kv_lens, cu_q=cu, max_q=3)
    assert bool(out[0, 2:].isnan().all()) and not bool(out[0, :2].isnan().any()) and not bool(out[1:].isnan().any())


def test_bad_pages_slots_and_lengths_are_reported_and_skipped():
    p = paged_problem(15, [1, 3, 100], [40, 70, 150], 4, 2, 128, 16, torch.bfloat16, spare=0)
    kq, vq, q, kc, vc, table, kv_lens, cu = p
    ref = check_attention(p)
    op = api.PagedAttention(kq, vq, 4, 2, 3, 104, device=DEV)
    for bad in (-1, kc.norms.shape[0], 2 ** 30):
        t = table.clone()
        t[0, 1] = bad
        out = op(q, kc, vc, t, kv_lens, cu_q=cu, max_q=100)
        with pytest.raises(L.TqError, match="outside its cache"):
            api.check()
        assert torch.equal(out[1:], ref[1:]) and bool(out[0].isfinite().all())
    long = kv_lens.clone()
    long[2] = 10 ** 6  # longer than its table row
    out = op(q, kc, vc, table, long, cu_q=cu, max_q=100)
    with pytest.raises(L.TqError):
        api.check()
    assert torch.equal(out[:4], ref[:4])
    slots = torch.tensor([0, 10 ** 9, -1], device=DEV)
    x = api.paged_dequant(kq, kc, slots)
    with pytest.raises(L.TqError):
        api.check()
    assert bool((x[1:] == 0).all())
    k = torch.randn((3, 2, 128), device=DEV)
    before = kc.codes.clone()
    api.paged_append(kq, vq, k, k, kc, vc, slots)
    with pytest.raises(L.TqError):
        api.check()
    assert bool((kc.codes[0, :, 0] != before[0, :, 0]).any())
    before[0, :, 0] = kc.codes[0, :, 0]
    assert torch.equal(kc.codes, before)
    api.check()  # the word is cleared


def test_two_calls_agree_bit_for_bit_and_a_graph_replays():
    p = paged_problem(16, [1, 3, 60, 1], [900, 70, 400, 2000], 8, 2, 128, 16, torch.bfloat16)
    kq, vq, q, kc, vc, table, kv_lens, cu = p
    op = api.PagedAttention(kq, vq, 8, 2, 4, 65, device=DEV)
    a = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=60)
    assert torch.equal(a, op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=60))
    out = torch.empty_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=60, out=out)
    g.replay()
    assert torch.equal(out, a)
    kv_lens[0] = 450  # a replay follows the lengths of the moment
    kv_lens[3] = 1
    g.replay()
    b = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=60)
    assert torch.equal(out, b) and not torch.equal(a, b)
    check_attention(p)


def test_max_q_does_not_change_which_rows_are_computed():
    p = paged_problem(17, [1, 30, 2], [64, 90, 33], 8, 2, 128, 16, torch.bfloat16)
    check_attention(p, max_q=1)
    check_attention(p, max_q=1000)


def test_another_stream():
    p = paged_problem(18, [1, 4], [640, 90], 8, 2, 128, 16, torch.bfloat16)
    kq, vq, q, kc, vc, table, kv_lens, cu = p
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    op = api.PagedAttention(kq, vq, 8, 2, 2, 5, device=DEV)
    ref = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=4)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        a = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=4)
    s.synchronize()
    b = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=4, stream=s)
    s.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)


def test_many_requests():
    # more requests than a block has threads, some without rows, some without tokens
    rng = np.random.default_rng(1)
    qs = rng.integers(0, 3, 900).tolist()
    kv = rng.integers(0, 40, 900).tolist()
    check_attention(paged_problem(19, qs, kv, 4, 2, 64, 16, torch.bfloat16))
    qs = (rng.integers(0, 3, 600) * (rng.random(600) < 0.5)).tolist()
    qs[7], kv = 40, rng.integers(0, 40, 600).tolist()
    kv[7] = 50
    check_attention(paged_problem(20, qs, kv, 4, 2, 64, 16, torch.float16))


@pytest.mark.parametrize("G,qs", [(8, [2, 1, 2]), (8, [3, 3, 1]), (5, [6, 4, 2]), (16, [2, 1, 2]), (4, [1, 8, 9])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_several_rows_a_head(G, qs, dtype):
    # 16, 24, 32 and just above 32 rows of a request and KV head
    p = paged_problem(G + sum(qs), qs, [300, 1030, 33], 2 * G, 2, 128, 16, dtype)
    poison_unseen(p[3], p[4], p[5], p[6])
    check_attention(p)
    check_attention(p, window=70)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_fp16(d):
    p = paged_problem(d, [140, 300, 2], [700, 300, 1000], 4, 2, d, 16, torch.float16)
    poison_unseen(p[3], p[4], p[5], p[6])
    check_attention(p)
    check_attention(p, window=150)


@pytest.mark.parametrize("qs", [[1, 1], [3, 60]])
def test_a_nan_query_row_stays_alone(qs):
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(21, qs, [200, 100], 8, 2, 128, 16, torch.bfloat16)
    op = api.PagedAttention(kq, vq, 8, 2, 2, sum(qs), device=DEV)
    ref = op(q, kc, vc, table, kv_lens, cu_q=cu, max_q=max(qs))
    bad = q.clone()
    bad[0, 1, 5] = float("nan")
    bad[1, 6, 9] = float("inf")
    out = op(bad, kc, vc, table, kv_lens, cu_q=cu, max_q=max(qs))
    hit = torch.zeros(sum(qs), 8, dtype=torch.bool, device=DEV)
    hit[0, 1] = hit[1, 6] = True
    assert torch.equal(out[~hit], ref[~hit]) and bool(out[0, 1].isnan().all()) and not bool(out[1, 6].isfinite().any())


@pytest.mark.parametrize("qs", [[1, 1, 1], [2, 70, 1]])
def test_caches_beyond_32_bit_offsets(qs):
    # 1.25 million pages of 64 records: code offsets pass 2^32 bytes, record offsets 2^26; the pages in use lie at
    # both ends
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(22, qs, [70, 130, 17], 8, 4, 128, 16, torch.bfloat16)
    ref = api.PagedAttention(kq, vq, 8, 4, 3, sum(qs), device=DEV)(q, kc, vc, table, kv_lens, cu_q=cu, max_q=max(qs))
    n, big = kc.norms.shape[0], 1_250_000
    far = torch.arange(n, device=DEV)
    far = torch.where(far % 2 == 0, far, big - 1 - far)
    caches = []
    for c, z in ((kc, kq), (vc, vq)):
        b = api.empty_cache(z, big, 4, 16, device=DEV)
        b.codes[far], b.norms[far] = c.codes, c.norms
        caches.append(b)
    t = torch.where(table >= 0, far[table.clamp(min=0).long()].int(), table)
    out = api.PagedAttention(kq, vq, 8, 4, 3, sum(qs), device=DEV)(q, *caches, t, kv_lens, cu_q=cu, max_q=max(qs))
    api.check()
    assert torch.equal(out, ref)
    slots = torch.tensor([big * 16 - 1, 5, big * 16 - 16], device=DEV)
    k = torch.randn((3, 4, 128), device=DEV, generator=gen(23))
    api.paged_append(kq, vq, k, k, *caches, slots)
    x = api.paged_dequant(kq, caches[0], slots)
    api.check()
    small = api.empty_cache(kq, 1, 4, 16, device=DEV)
    api.paged_append(kq, vq, k, k, small, api.empty_cache(vq, 1, 4, 16, device=DEV), torch.arange(3, device=DEV))
    assert torch.equal(x, api.paged_dequant(kq, small, torch.arange(3, device=DEV)))


def test_two_objects_on_two_streams():
    ps = [paged_problem(30 + i, [1, 40], [900, 300 + i], 8, 2, 128, 16, torch.bfloat16) for i in range(2)]
    ops = [api.PagedAttention(p[0], p[1], 8, 2, 2, 41, device=DEV) for p in ps]
    run = lambda i, m: ops[i](ps[i][2][:m], *ps[i][3:6], ps[i][6], cu_q=torch.clamp(ps[i][7], max=m), max_q=m)  # noqa: E731
    for m in (2, 41):  # the small tiles and the large ones
        refs = [run(i, m) for i in range(2)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [[], []]
        for _ in range(10):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    outs[i].append(run(i, m))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(o, refs[i]) for o in outs[i])


def test_a_table_without_entries_and_rows_named_twice():
    kq, vq, q, kc, vc, table, kv_lens, cu = paged_problem(24, [1, 60], [40, 70], 4, 2, 128, 16, torch.bfloat16)
    op = api.PagedAttention(kq, vq, 4, 2, 2, 61, device=DEV)
    for m in (1, 60):
        out = op(q, kc, vc, table[:, :0], kv_lens, cu_q=cu, max_q=m)
        with pytest.raises(L.TqError):
            api.check()
        assert bool((out == 0).all())
    many = torch.tensor([0, 61] * 40 + [0], dtype=torch.int32, device=DEV)  # 40 times the same rows
    t, lens = table[:1].repeat(80, 1), kv_lens[:1].repeat(80)
    big = api.PagedAttention(kq, vq, 4, 2, 80, 61, device=DEV)
    big(q, kc, vc, t, lens, cu_q=many, max_q=61)
    try:
        api.check()
    except L.TqError:
        pass
    api.check()


# ------------------------------------------------------------ a serving loop

@pytest.mark.parametrize("d,Hq,Hkv,P", [(128, 8, 2, 16), (64, 6, 3, 32)])
def test_serving_loop(d, Hq, Hkv, P):
    """Prompts of different lengths, chunked, then decode steps: plan, append
    with positions and attend, each step captured by nothing but the calls;
    the outputs equal 64-bit attention over what was encoded."""
    g = gen(77 + d)
    kq, vq = quantizers(d)
    rope = api.Rope((10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().to(DEV))
    R, n_pages = 3, 24
    kc, vc = (api.empty_cache(z, n_pages, Hkv, P, device=DEV) for z in (kq, vq))
    for c in (kc, vc):
        c.norms.fill_(float("nan"))
        c.codes.zero_()
    table = torch.full((R, 10), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(n_pages, generator=g, device=DEV).int()
    n_free = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
    lens = torch.zeros(R, dtype=torch.int32, device=DEV)
    held = 0
    for step in ([20, 5, 0], [17, 1, 33], [1, 1, 1], [1, 4, 1], [1, 1, 1]):
        T = sum(step) + 2  # a padded batch
        planner = api.PagePlanner(R, P, T, device=DEV)
        p = planner(lens, torch.tensor(step, dtype=torch.int32, device=DEV), free, n_free, table)
        q, k, v = (torch.randn((T, h, d), generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        qt = api.paged_append(kq, vq, k, v, kc, vc, p.slots, q=q, rope=rope, positions=p.positions)
        check_attention((kq, vq, qt, kc, vc, table, p.seq_lens, p.cu_new), max_q=max(step))
        lens, n_free = p.seq_lens.clone(), p.n_free.clone()
        assert p.status.tolist() == [0] * R
        held += sum(step)
    assert lens.sum().item() == held
    used = sorted(table[table >= 0].tolist())
    assert len(set(used)) == len(used) and sorted(used + free[:int(n_free)].tolist()) == list(range(n_pages))
    # a cached prefix read back equals the encoder's vectors
    j = torch.arange(20, device=DEV)
    slots = table[0, j // P].long() * P + j % P
    x = api.paged_dequant(vq, vc, slots, dtype=torch.float32)
    assert bool(x.isfinite().all())

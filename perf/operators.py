"""Serving on a paged 4-bit TurboQuant cache: what is timed, and its plain form.

A pass is one of four operators: the page plan of a batch (block tables and
slot maps from request lengths), the append of a batch's K and V rows (rotary
positions on several axes, then the 4-bit records written at their slots), the
read-back of cached rows, and attention of ragged query rows over the pages.
``own`` selects the library's calls; otherwise the same is computed with
elementary torch operations in 32 bits (angles in 64).

Codes are held in 4 bits, so the append's pass reads the records it wrote back
and returns the vectors they stand for.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# the positive half of the 16-level Lloyd-Max quantizer of N(0, 1)
LEVELS = (0.12839502985114504, 0.3880482994902857, 0.6567591185324552, 0.9423404564869502,
          1.2562311973471636, 1.6180463860218683, 2.0690172265313693, 2.7325895709951453)

SEED_K, SEED_V = 11, 12  # the rotations of the key and of the value quantizer


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of a batch of 16: one new token each, latency only
        dict(name="plan decode 16", op="plan", R=16, new=1, len=131072, P=16, pool=1.0),
        # a mixed batch: long prompts admitted next to decoding requests, not enough free pages for the last ones
        dict(name="plan mixed 257", op="plan", R=257, new=700, len=8191, P=32, pool=0.9),
        # a whole offline batch planned at once
        dict(name="plan prompts 2048", op="plan", R=2048, new=512, len=2048, P=16, pool=1.1),
        # the append of one decode step, 32 / 8 heads, plain positions
        dict(name="append decode 16", op="append", T=16, Hq=32, Hkv=8, d=128, P=16, axes=1, pairing="half", rot=128, dtype="bf16"),
        # an image prompt of a 64 / 8 head model: three axes, adjacent pairs, part of the head rotated, odd length
        dict(name="append image 1531", op="append", T=1531, Hq=64, Hkv=8, d=128, P=48, axes=3, pairing="adjacent", rot=96, dtype="fp16"),
        # a prefill step of 16384 tokens with time, height and width positions
        dict(name="append prefill 16384", op="append", T=16384, Hq=32, Hkv=8, d=128, P=64, axes=3, pairing="half", rot=128, dtype="bf16"),
        # a short prefix read back (d = 64)
        dict(name="dequant 333", op="dequant", T=333, H=8, d=64, P=16, dtype="fp16"),
        # a shared prompt's rows read back for a dense consumer
        dict(name="dequant 65536", op="dequant", T=65536, H=8, d=128, P=64, dtype="bf16"),
        # decode of one sequence: 32 / 8 heads over 32768 cached tokens
        dict(name="decode 1 x 32768", op="attend", R=1, q=1, kv=32768, Hq=32, Hkv=8, d=128, P=64, window=0, dtype="bf16"),
        # ragged decode of a batch of 16 over up to 65536 tokens each
        dict(name="decode 16 x 65536", op="attend", R=16, q=1, kv=65536, Hq=32, Hkv=8, d=128, P=64, window=0, dtype="bf16"),
        # several draft tokens verified per sequence, many short sequences, 64 / 8 heads
        dict(name="verify 128 x 4", op="attend", R=128, q=4, kv=4001, Hq=64, Hkv=8, d=128, P=16, window=0, dtype="fp16"),
        # chunked prefill: ragged prompts of up to 2048 new tokens on up to 16384 cached ones
        dict(name="prefill 3 x 2048", op="attend", R=3, q=2048, kv=16384, Hq=32, Hkv=8, d=128, P=64, window=0, dtype="bf16"),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "dequant", "attend", "attend", "attend"])
    P = rng.choice([16, 32, 48, 64, 128, 256])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "plan":
        R = log_int(rng, 1, 2048)
        return dict(op=op, R=R, new=log_int(rng, 1, max(1, 1000000 // R)), len=log_int(rng, 1, 131072), P=P,
                    pool=rng.choice([0.5, 1.0, 1.5]))
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 3, 4, 8])
        T = log_int(rng, 1, min(16384, 524288 // (Hkv * G)))
        rot = rng.choice([d, d, d // 2, d // 2 + 16])
        return dict(op=op, T=T, Hq=Hkv * G, Hkv=Hkv, d=d, P=P, axes=rng.choice([1, 2, 3]),
                    pairing=rng.choice(["half", "adjacent"]), rot=rot, dtype=dtype)
    if op == "dequant":
        return dict(op=op, T=log_int(rng, 1, 65536), H=rng.choice([1, 2, 5, 8]), d=d, P=P, dtype=dtype)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8, 16])
    q = rng.choice([1, 1, log_int(rng, 2, 16), log_int(rng, 17, 2048)])
    R = log_int(rng, 1, 128) if q <= 16 else log_int(rng, 1, 4)
    kv = log_int(rng, 1, min(65536, max(1, 8388608 // (R * Hkv)), max(1, 1 << 30) // (R * q * Hkv * G)))
    return dict(op=op, R=R, q=q, kv=kv, Hq=Hkv * G, Hkv=Hkv, d=d, P=P, window=rng.choice([0, 0, 0, log_int(rng, 1, 4096)]),
                dtype=dtype)


# ------------------------------------------------- sizes that a case fixes

def spread(n, most):
    """n lengths in 1..most, the first one `most`, the others spread over the range."""
    return [most] + [1 + int(most * math.fmod((r + 1) * 0.6180339887498949, 1.0)) % most for r in range(1, n)]


def plan_lengths(c):
    """Cached and new tokens: every fourth request only decodes, every seventh is new."""
    old = [0 if r % 7 == 5 else n for r, n in enumerate(spread(c["R"], c["len"]))]
    new = [1 if r % 4 == 1 else n for r, n in enumerate(spread(c["R"], c["new"])[::-1])]
    return old, new


def attend_lengths(c):
    """Query and cached tokens of each request; one of a larger batch has an empty cache."""
    qs = [n if c["q"] > 1 else 1 for n in spread(c["R"], c["q"])]
    kv = [n for n in spread(c["R"], c["kv"])]
    if c["R"] >= 8:
        kv[5] = 0
    return qs, kv


def pages_of(n, P):
    return -(-n // P)


def work(case):
    c = case
    if c["op"] == "plan":
        old, new = plan_lengths(c)
        pages = sum(pages_of(o + n, c["P"]) - pages_of(o, c["P"]) for o, n in zip(old, new))
        return {"bytes": sum(new) * 12 + 8 * pages + 24 * c["R"], "flops": 0}
    if c["op"] == "append":
        d, rec = c["d"], c["d"] // 2 + 4
        heads = c["Hq"] + 2 * c["Hkv"]
        # q, k and v read, rotated q and the records written, then read back into K and V
        per = 2 * d * heads + 2 * d * c["Hq"] + 2 * c["Hkv"] * (2 * rec + 2 * d) + 8 + 4 * c["axes"]
        return {"bytes": c["T"] * per, "flops": c["T"] * heads * d * 14}
    if c["op"] == "dequant":
        return {"bytes": c["T"] * (8 + c["H"] * (c["d"] // 2 + 4 + 2 * c["d"])), "flops": c["T"] * c["H"] * c["d"] * 8}
    qs, kv = attend_lengths(c)
    G, d, w = c["Hq"] // c["Hkv"], c["d"], c["window"] or (1 << 40)
    pairs = sum(_pairs(n, m, w) for n, m in zip(qs, kv))
    reach = sum(min(m, w + n - 1) for n, m in zip(qs, kv))
    return {"bytes": reach * c["Hkv"] * 2 * (d // 2 + 4) + 4 * sum(qs) * c["Hq"] * d, "flops": 4 * d * pairs * c["Hkv"] * G}


def _pairs(n, m, w):
    """Attended (query, key) pairs of n queries at the end of m cached tokens, each seeing at most the last w."""
    first = max(0, m - n)          # tokens seen by all queries, were there no window
    short = max(0, n - m)          # queries before the first token
    lo, hi = first + 1, m          # the counts of the others run from lo to hi
    k = n - short
    if k <= 0:
        return 0
    if w >= hi:
        return (lo + hi) * k // 2
    below = max(0, min(k, w - lo))  # counts lo .. w-1
    return (lo + lo + below - 1) * below // 2 + w * (k - below)


# ------------------------------------------------------------------- inputs

def seeded_signs(seed, d):
    """The framework's rotation signs: -1 where bit 63 of SplitMix64's output i is set."""
    k = (np.arange(1, d + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)) + np.uint64(seed)
    k = (k ^ (k >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    k = (k ^ (k >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return np.where((k ^ (k >> np.uint64(31))) >> np.uint64(63), -1.0, 1.0)


def codebook(d):
    """Centroids and thresholds of coordinates N(0, 1/d), 32 bits."""
    c = np.array([-v for v in LEVELS[::-1]] + list(LEVELS)) / math.sqrt(d)
    return (torch.tensor(c, dtype=torch.float32, device=DEV),
            torch.tensor(0.5 * (c[:-1] + c[1:]), dtype=torch.float32, device=DEV))


def hadamard(d, dtype=torch.float32):
    """The Sylvester Hadamard matrix over sqrt(d)."""
    i = torch.arange(d, device=DEV)
    x = i[:, None] & i[None, :]
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = x ^ (x >> 1)
    return (1.0 - 2.0 * (x & 1).to(dtype)) / math.sqrt(d)


def quantizers(s, d):
    s["centroids"], s["thresholds"] = codebook(d)
    s["H"] = hadamard(d)
    s["signs_k"] = torch.tensor(seeded_signs(SEED_K, d), dtype=torch.float32, device=DEV)
    s["signs_v"] = torch.tensor(seeded_signs(SEED_V, d), dtype=torch.float32, device=DEV)
    if own:
        from kv_cache_vector_13_b200 import api
        s["kq"] = api.Quantizer(d, 4, "mse", seed_rot=SEED_K, device=DEV)
        s["vq"] = api.Quantizer(d, 4, "mse", seed_rot=SEED_V, device=DEV)


def random_cache(g, n_pages, H, P, d, thresholds, sigma):
    """Records as encoding Gaussian vectors leaves them: packed codes and norms."""
    codes = torch.empty((n_pages, H, P, d // 2), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (H * P * d))
    for p in range(0, n_pages, step):
        n = min(step, n_pages - p)
        u = torch.randn((n, H, P, d // 2, 2), generator=g, device=DEV) / math.sqrt(d)
        i = torch.bucketize(u, thresholds, out_int32=True)
        codes[p:p + n] = (i[..., 0] | (i[..., 1] << 4)).to(torch.uint8)
    norms = math.sqrt(d) * torch.exp(sigma * torch.randn((n_pages, H, P), generator=g, device=DEV))
    return codes, norms


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": dict(c)}
    if c["op"] == "plan":
        old, new = plan_lengths(c)
        R, P = c["R"], c["P"]
        # the same lengths in another order: other requests, the same work
        at = torch.randperm(R, generator=g, device=DEV)
        s["lens"] = torch.tensor(old, dtype=torch.int32, device=DEV)[at]
        s["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)[at]
        s["max_pages"] = max(pages_of(o + n, P) for o, n in zip(old, new)) + 3
        held = sum(pages_of(o, P) for o in old)
        need = sum(pages_of(o + n, P) - pages_of(o, P) for o, n in zip(old, new))
        n_free = int(need * c["pool"])
        ids = torch.randperm(held + n_free + 8, generator=g, device=DEV, dtype=torch.int32)
        s["free"] = ids[held:].contiguous()
        s["n_free"] = torch.tensor([n_free], dtype=torch.int32, device=DEV)
        s["tokens"] = sum(new)
        s["rows"] = s["tokens"] + 5  # a padded batch
        table = torch.full((R, s["max_pages"]), -1, dtype=torch.int32, device=DEV)
        has = (s["lens"].long() + P - 1) // P
        mine = torch.arange(s["max_pages"], device=DEV)[None] < has[:, None]
        table[mine] = ids[:held]
        s["table"] = table
        if own:
            from kv_cache_vector_13_b200 import api
            s["planner"] = api.PagePlanner(R, P, s["rows"], device=DEV)
        return s
    dt = TYPES[c["dtype"]]
    quantizers(s, c["d"])
    d, P = c["d"], c["P"]
    if c["op"] == "append":
        T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
        # the rows of a fused projection: q, k and v side by side
        s["qkv"] = torch.randn((T, Hq + 2 * Hkv, d), generator=g, device=DEV).to(dt)
        n_pages = pages_of(T, P) + 3
        s["slots"] = torch.randperm(n_pages * P, generator=g, device=DEV)[:T].contiguous()
        half = c["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        # the first frequencies turn with the time, the next ones with height and width
        cut = [half - (c["axes"] - 1) * (half // 3)] + [half // 3] * (c["axes"] - 1)
        s["axis"] = torch.repeat_interleave(torch.arange(c["axes"], device=DEV), torch.tensor(cut, device=DEV))
        start = torch.randint(0, 1 << 20, (1,), generator=g, device=DEV, dtype=torch.int32)
        t = torch.arange(T, device=DEV, dtype=torch.int32)
        s["positions"] = torch.stack([start + t, start + t // 37, start + t % 37][:c["axes"]]).contiguous()
        if own:
            from kv_cache_vector_13_b200 import api
            s["rope"] = api.Rope(s["inv_freq"], sections=cut, pairing=c["pairing"])
            s["kcache"] = api.empty_cache(s["kq"], n_pages, Hkv, P, device=DEV)
            s["vcache"] = api.empty_cache(s["vq"], n_pages, Hkv, P, device=DEV)
        return s
    if c["op"] == "dequant":
        n_pages = pages_of(c["T"], P) + 3
        codes, norms = random_cache(g, n_pages, c["H"], P, d, s["thresholds"], 0.5)
        s["codes"], s["norms"] = codes, norms
        s["slots"] = torch.randperm(n_pages * P, generator=g, device=DEV)[:c["T"]].contiguous()
        if own:
            from kv_cache_vector_13_b200 import api
            s["cache"] = api.PackedCache(codes, norms)
        return s
    qs, kv = attend_lengths(c)
    R, T = c["R"], sum(qs)
    s["q"] = torch.randn((T, c["Hq"], d), generator=g, device=DEV).to(dt)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["cu_q"] = torch.tensor([0] + qs, device=DEV).cumsum(0).to(torch.int32)
    width = max(pages_of(m, P) for m in kv)
    held = sum(pages_of(m, P) for m in kv)
    n_pages = held + 1
    s["kcodes"], s["knorms"] = random_cache(g, n_pages, c["Hkv"], P, d, s["thresholds"], 0.5)
    s["vcodes"], s["vnorms"] = random_cache(g, n_pages, c["Hkv"], P, d, s["thresholds"], 0.5)
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    mine = torch.arange(width, device=DEV)[None] * P < s["kv_lens"][:, None]
    table[mine] = torch.randperm(n_pages, generator=g, device=DEV, dtype=torch.int32)[:held]
    s["table"], s["max_q"] = table, max(qs)
    if own:
        from kv_cache_vector_13_b200 import api
        s["kcache"] = api.PackedCache(s["kcodes"], s["knorms"])
        s["vcache"] = api.PackedCache(s["vcodes"], s["vnorms"])
        s["op"] = api.PagedAttention(s["kq"], s["vq"], c["Hq"], c["Hkv"], max_requests=R, max_tokens=T, device=DEV)
    return s


# ----------------------------------------------------------------- one pass

def run(state):
    return {"plan": plan, "append": append, "dequant": dequant, "attend": attend}[state["case"]["op"]](state)


def plan(s):
    P = s["case"]["P"]
    if own:
        p = s["planner"](s["lens"], s["new"], s["free"], s["n_free"], s["table"])
        return {"slots": p.slots, "positions": p.positions, "cu_new": p.cu_new, "seq_lens": p.seq_lens,
                "status": p.status, "n_free": p.n_free, "table": s["table"]}
    lens, new, table, R = s["lens"].long(), s["new"].long(), s["table"], s["case"]["R"]
    total = lens + new
    end = new.cumsum(0)
    begin = end - new
    had, has = (lens + P - 1) // P, (total + P - 1) // P
    fits = (has <= s["max_pages"]) & (end <= s["rows"])
    need = torch.where(fits, has - had, 0)
    before = need.cumsum(0) - need
    paid = (need == 0) | (before + need <= s["n_free"])
    ok = fits & paid
    # the new pages come off the end of the free list
    top = s["n_free"].long() - 1
    col = torch.arange(s["max_pages"], device=DEV)[None]
    fresh = (col >= had[:, None]) & (col < has[:, None]) & ok[:, None]
    pick = (top - before[:, None] - (col - had[:, None])).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][pick], table)
    t = torch.arange(s["rows"], device=DEV)
    r = torch.searchsorted(end, t, right=True).clamp(max=R - 1)
    live = t < end[-1]
    pos = torch.where(live, lens[r] + t - begin[r], 0)
    slot = table[r, (pos // P).clamp(max=s["max_pages"] - 1)].long() * P + pos % P
    return {"slots": torch.where(live & ok[r], slot, -1), "positions": pos.int(),
            "cu_new": torch.cat([torch.zeros_like(end[:1]), end]).int(),
            "seq_lens": torch.where(ok, total, lens).int(),
            "status": torch.where(fits, torch.where(paid, 0, 1), 2).int(),
            "n_free": (s["n_free"] - torch.where(ok, need, 0).sum()).int(), "table": table}


def append(s):
    c = s["case"]
    Hq, Hkv, dt = c["Hq"], c["Hkv"], TYPES[c["dtype"]]
    q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
    if own:
        from kv_cache_vector_13_b200 import api
        q_out = api.paged_append(s["kq"], s["vq"], k, v, s["kcache"], s["vcache"], s["slots"], q=q, rope=s["rope"],
                                 positions=s["positions"])
        return {"q": q_out, "k": api.paged_dequant(s["kq"], s["kcache"], s["slots"], dtype=dt),
                "v": api.paged_dequant(s["vq"], s["vcache"], s["slots"], dtype=dt)}
    angle = (s["positions"][s["axis"]].double() * s["inv_freq"].double()[:, None]).t()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    turn = lambda x: torch.cat([rotated(x[..., :c["rot"]], cos, sin, c["pairing"]), x[..., c["rot"]:]], -1)  # noqa: E731
    return {"q": turn(q.float()).to(dt),
            "k": reread(turn(k.float()), s["signs_k"], s).to(dt),
            "v": reread(v.float(), s["signs_v"], s).to(dt)}


def rotated(x, cos, sin, pairing):
    if pairing == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def reread(x, signs, s):
    """Each row through its 4-bit record: norm, rotation, nearest centroids, and back."""
    norm = (x * x).sum(-1, keepdim=True).sqrt()
    u = torch.where(norm > 0, ((x * signs) @ s["H"]) / norm, 0.0)
    i = torch.bucketize(u, s["thresholds"], out_int32=True)
    return ((s["centroids"][i] * norm) @ s["H"]) * signs


def unpacked(codes, centroids):
    """The centroids of packed codes, two to a byte, the low half first."""
    i = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return centroids.index_select(0, i.flatten().int()).view(i.shape)


def dequant(s):
    c = s["case"]
    if own:
        from kv_cache_vector_13_b200 import api
        return api.paged_dequant(s["kq"], s["cache"], s["slots"], dtype=TYPES[c["dtype"]])
    page, at = s["slots"] // c["P"], s["slots"] % c["P"]
    x = unpacked(s["codes"][page, :, at], s["centroids"]) * s["norms"][page, :, at][..., None]
    return ((x @ s["H"]) * s["signs_k"]).to(TYPES[c["dtype"]])


def attend(s):
    c = s["case"]
    if own:
        return s["op"](s["q"], s["kcache"], s["vcache"], s["table"], s["kv_lens"], cu_q=s["cu_q"], max_q=s["max_q"],
                       window=c["window"])
    R, Hq, Hkv, d, P, n = c["R"], c["Hq"], c["Hkv"], c["d"], c["P"], s["max_q"]
    G, T = Hq // Hkv, s["q"].shape[0]
    # the cached rows of each request, padded to the longest: [R, Hkv, L, d], in the rotated basis
    table = s["table"].clamp(min=0).long()
    L = table.shape[1] * P
    rows = lambda codes, norms: (unpacked(codes[table], s["centroids"]) * norms[table][..., None]).transpose(1, 2).reshape(R, Hkv, L, d)  # noqa: E731
    start, lens = s["cu_q"][:-1].long(), s["cu_q"].diff().long()
    i = torch.arange(n, device=DEV)
    row = (start[:, None] + i).clamp(max=T - 1)
    q = ((s["q"].float() * s["signs_k"]) @ s["H"])[row]                      # [R, n, Hq, d]
    q = q.view(R, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, d)
    logits = (q @ rows(s["kcodes"], s["knorms"]).transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(R, Hkv, n, G, L)
    # query i stands at kv_len - q_len + i and sees no later token, and at most `window` of them
    at = (s["kv_lens"].long() - lens)[:, None] + i
    j = torch.arange(L, device=DEV)
    seen = (j <= at[..., None]) & (j < s["kv_lens"][:, None, None])
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    logits.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = logits.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(R, Hkv, n * G, L) @ rows(s["vcodes"], s["vnorms"])
    o = torch.where(total > 0, o.view(R, Hkv, n, G, d) / total, 0.0)
    o = ((o @ s["H"]) * s["signs_v"]).permute(0, 2, 1, 3, 4).reshape(R * n, Hq, d)
    # back to the ragged rows
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(s["cu_q"][1:].contiguous(), t, right=True)
    return o[r * n + t - start[r]].to(TYPES[c["dtype"]])


# ------------------------------------------------- the definition in 64 bits

def fwht64(x):
    """Walsh-Hadamard transform over the last axis, over sqrt(d), by butterflies."""
    d, h = x.shape[-1], 1
    while h < d:
        y = x.reshape(*x.shape[:-1], d // (2 * h), 2, h)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(*x.shape[:-1], d)
        h *= 2
    return x / math.sqrt(d)


def levels64(d):
    """The stored (32-bit) centroids and thresholds, as 64-bit values."""
    c = np.concatenate([-np.array(LEVELS)[::-1], np.array(LEVELS)]) / math.sqrt(d)
    t = (0.5 * (c[1:] + c[:-1])).astype(np.float32).astype(np.float64)
    return torch.from_numpy(c.astype(np.float32).astype(np.float64)).to(DEV), torch.from_numpy(t).to(DEV)


def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(case, seed)
    d = c["d"]
    cent, thr = levels64(d)
    sk = torch.from_numpy(seeded_signs(SEED_K, d)).to(DEV)
    sv = torch.from_numpy(seeded_signs(SEED_V, d)).to(DEV)

    def values(codes, norms):
        b = codes.to(torch.int64)
        both = torch.empty((*codes.shape, 2), dtype=torch.float64, device=DEV)
        both[..., 0], both[..., 1] = cent[b % 16], cent[b // 16]
        return both.reshape(*codes.shape[:-1], d) * norms.double().unsqueeze(-1)

    if c["op"] == "dequant":
        x = torch.empty((c["T"], c["H"], d), dtype=torch.float64, device=DEV)
        for a in range(0, c["T"], 8192):
            sl = s["slots"][a:a + 8192]
            page = torch.div(sl, c["P"], rounding_mode="floor")
            x[a:a + 8192] = fwht64(values(s["codes"][page, :, sl - page * c["P"]], s["norms"][page, :, sl - page * c["P"]])) * sk
        return x
    if c["op"] == "append":
        Hq, Hkv, rot = c["Hq"], c["Hkv"], c["rot"]
        x = s["qkv"].double()
        theta = torch.empty((c["T"], rot // 2), dtype=torch.float64, device=DEV)
        for i in range(rot // 2):
            theta[:, i] = s["positions"][int(s["axis"][i])].double() * float(s["inv_freq"][i])
        turn = torch.polar(torch.ones_like(theta), theta)[:, None]
        y = x[:, :Hq + Hkv].clone()
        if c["pairing"] == "half":
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag

        def stored(rows, signs):
            n = torch.linalg.vector_norm(rows, dim=-1, keepdim=True)
            u = fwht64(rows * signs) / n
            i = torch.zeros(u.shape, dtype=torch.int64, device=DEV)
            for j in range(15):
                i += u > thr[j]
            return fwht64(cent[i] * n) * signs

        return {"q": y[:, :Hq], "k": stored(y[:, Hq:], sk), "v": stored(x[:, Hq + Hkv:], sv)}
    qs, kv = attend_lengths(c)
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros((sum(qs), c["Hq"], d), dtype=torch.float64, device=DEV)
    t0 = 0
    for r in range(c["R"]):
        n, m = qs[r], kv[r]
        pages = s["table"][r, :pages_of(m, c["P"])].long()
        qr = fwht64(s["q"][t0:t0 + n].double() * sk)
        for h in range(c["Hkv"] if m else 0):
            K = values(s["kcodes"][pages, h].reshape(-1, d // 2)[:m], s["knorms"][pages, h].reshape(-1)[:m])
            V = values(s["vcodes"][pages, h].reshape(-1, d // 2)[:m], s["vnorms"][pages, h].reshape(-1)[:m])
            j = torch.arange(m, device=DEV)[None]
            for a in range(0, n, 512):
                e = min(n, a + 512)
                p = (m - n + torch.arange(a, e, device=DEV))[:, None]
                seen = (j <= p) & ((j > p - c["window"]) if c["window"] else (j >= 0))
                some = seen.any(1)
                for hq in range(h * G, (h + 1) * G):
                    z = (qr[a:e, hq] @ K.T) / math.sqrt(d)
                    z = torch.where(seen, z, -math.inf)[some]
                    if z.shape[0]:
                        o = torch.zeros((e - a, d), dtype=torch.float64, device=DEV)
                        o[some] = torch.softmax(z, 1) @ V
                        out[t0 + a:t0 + e, hq] = fwht64(o) * sv
        t0 += n
    return out

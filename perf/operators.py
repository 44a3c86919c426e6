"""What is measured of the language-model serving operators: the calls, their inputs and their plain forms.

Five operators make up one serving step of a causal model over a paged 4-bit
cache: ``cache_plan`` (block tables, slot maps), ``rope`` (rotary positions),
``kv4_append`` / ``kv4_read`` (the cache's rows), ``kv4_attn`` (attention over
the cache) and ``window_attn`` (attention with a sliding window and first
tokens that stay visible, for prefill and for single tokens over 16-bit K, V).

``run`` computes them in elementary torch operations where ``own`` is false
and through the package's public calls where it is true.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One decode step of 48 requests over 16-bit caches of 4352 places: the LM workload's heads and window.
        dict(name="window_decode_batch", op="window", B=48, Hq=32, Hkv=8, Nq=1, Nk=4352, d=128, dtype="bf16",
             window=4096, sinks=128, ragged=True),
        # Prefill of a padded batch of prompts of odd lengths.
        dict(name="window_prefill_padded", op="window", B=3, Hq=32, Hkv=8, Nq=2777, Nk=2777, d=128, dtype="bf16",
             window=1024, sinks=4, ragged=True),
        # Prefill of the LM workload: 131,072 tokens, window 4096, 128 anchors.
        dict(name="window_prefill_131k", op="window", B=1, Hq=32, Hkv=8, Nq=131072, Nk=131072, d=128, dtype="bf16",
             window=4096, sinks=128, ragged=False),
        # A small fp32 model (tests, calibration against 16 bits): other head width, no tensor-core kernel.
        dict(name="window_fp32", op="window", B=2, Hq=8, Hkv=8, Nq=1000, Nk=1000, d=64, dtype="fp32",
             window=256, sinks=1, ragged=False),
        # Decode of one request with a chat's history.
        dict(name="kv4_attn_one", op="kv4_attn", B=1, Hq=32, Hkv=8, d=128, page=16, min_len=5003, max_len=5003,
             q_max=1, window=0, sinks=0),
        # Decode of a mixed batch, lengths from one token to the LM workload's 131,072.
        dict(name="kv4_attn_mixed", op="kv4_attn", B=16, Hq=32, Hkv=8, d=128, page=64, min_len=1, max_len=131072,
             q_max=1, window=0, sinks=0),
        # One new token of each of 64 requests into the cache.
        dict(name="kv4_append_decode", op="kv4_append", T=64, Hkv=8, d=128, page=16, pages=4096, run=1),
        # A prefill's keys and values into the cache.
        dict(name="kv4_append_prefill", op="kv4_append", T=16411, Hkv=8, d=128, page=64, pages=512, run=16411),
        # The new tokens of 64 requests at far positions, interleaved pairs over half of the head.
        dict(name="rope_decode", op="rope", T=64, Hq=32, Hkv=8, d=128, rot=64, layout="interleaved", scaling="none",
             dtype="bf16", max_pos=131072, inverse=False),
        # A prefill's queries and keys, the whole head, scaled to four times the trained length.
        dict(name="rope_prefill", op="rope", T=16411, Hq=32, Hkv=8, d=128, rot=128, layout="half", scaling="yarn",
             dtype="bf16", max_pos=131072, inverse=False),
        # A decode step's tables: 256 requests, one token each, a few that end.
        dict(name="plan_decode", op="plan", B=256, page=16, max_blocks=1024, max_new=1, max_old=16000, release=0.03),
        # A prefill step's tables: chunks of up to 4096 tokens of 48 requests.
        dict(name="plan_prefill", op="plan", B=48, page=64, max_blocks=2048, max_new=4096, max_old=120000,
             release=0.1),
    ]


def _log_int(rng, lo, hi):
    """An integer between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (24, 24), (8, 8), (16, 2), (8, 1), (4, 2), (12, 4)]


def draw(rng):
    op = rng.choice(["window", "window", "kv4_attn", "kv4_attn", "kv4_append", "rope", "plan"])
    Hq, Hkv = rng.choice(HEADS)
    if op == "window":
        kind = rng.choice(["decode", "prefill", "prefill", "fp32"])
        window = rng.choice([0, _log_int(rng, 1, 8192), _log_int(rng, 16, 4096)])
        sinks = rng.choice([0, 1, 4, rng.randrange(0, 300)])
        if kind == "decode":
            return dict(op=op, B=_log_int(rng, 1, 64), Hq=Hq, Hkv=Hkv, Nq=rng.choice([1, 1, 2, 3]),
                        Nk=_log_int(rng, 3, 8192), d=rng.choice([64, 128, 128]), dtype="bf16", window=window,
                        sinks=sinks, ragged=rng.choice([True, False]))
        if kind == "prefill":
            n = _log_int(rng, 16, 6000)
            return dict(op=op, B=rng.choice([1, 2, 3]), Hq=Hq, Hkv=Hkv, Nq=n,
                        Nk=n + rng.choice([0, 0, _log_int(rng, 1, 2000)]), d=128, dtype="bf16", window=window,
                        sinks=sinks, ragged=rng.choice([True, False]))
        n = _log_int(rng, 1, 1500)
        return dict(op=op, B=rng.choice([1, 2]), Hq=Hq, Hkv=Hkv, Nq=n, Nk=n, d=rng.choice([16, 64, 128]),
                    dtype="fp32", window=window, sinks=sinks, ragged=rng.choice([True, False]))
    if op == "kv4_attn":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 131072 // B if B > 1 else 131072)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                    min_len=rng.choice([1, max(1, hi // 2), hi]), max_len=hi, q_max=rng.choice([1, 1, 2, 4]),
                    window=rng.choice([0, 0, _log_int(rng, 16, 8192)]), sinks=rng.choice([0, 4, 128]))
    if op == "kv4_append":
        T = _log_int(rng, 1, 16000)
        page = rng.choice([16, 32, 64, 128])
        return dict(op=op, T=T, Hkv=Hkv, d=rng.choice([64, 128]), page=page, pages=-(-T // page) + rng.randrange(1, 60),
                    run=rng.choice([1, 7, T]))
    if op == "rope":
        d = rng.choice([64, 128, 256])
        return dict(op=op, T=_log_int(rng, 1, 12000), Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d // 2, d // 4]),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), max_pos=_log_int(rng, 100, 1000000),
                    inverse=rng.choice([False, False, True]))
    page = rng.choice([16, 32, 64, 128])
    return dict(op=op, B=_log_int(rng, 1, 1024), page=page, max_blocks=-(-20000 // page) + 8,
                max_new=_log_int(rng, 1, 200), max_old=_log_int(rng, 1, 19800), release=rng.choice([0.0, 0.1, 0.5]))


def _lens(case):
    """(query lengths, key lengths) of the sequences, from the case alone: a user's program knows them."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    B = case["B"]
    if case["op"] == "window":
        if not case["ragged"]:
            return [case["Nq"]] * B, [case["Nk"]] * B
        nk = [case["Nk"]] + [r.randint(max(1, case["Nk"] // 8), case["Nk"]) for _ in range(B - 1)]
        nq = [min(case["Nq"], n) for n in nk]
        return nq, nk
    if case["op"] == "kv4_attn":
        nk = [case["max_len"]] + [_log_int(r, case["min_len"], case["max_len"]) for _ in range(B - 1)]
        return [min(n, r.randint(1, case["q_max"])) for n in nk], nk
    # plan: new tokens (-1 releases the request), tokens already cached
    old = [r.randint(0, case["max_old"]) for _ in range(B)]
    new = [-1 if r.random() < case["release"] else r.randint(min(1, case["max_new"]), case["max_new"])
           for _ in range(B)]
    return new, old


def _visible(p, n, window, sinks):
    """Keys that a query at position p of n sees."""
    hi = min(p, n - 1)
    if hi < 0:
        return 0
    if window == 0 or p + 1 <= window:
        return hi + 1
    lo = p - window + 1
    return max(0, hi - lo + 1) + min(sinks, lo)


def _pairs(case):
    """(visible pairs, keys that some query of the sequence sees), summed over the sequences."""
    nq, nk = _lens(case)
    pairs = keys = 0
    for a, b in zip(nq, nk):
        w, s = case["window"], case["sinks"]
        if a * 1.0 * len(nq) < 20000:
            pairs += sum(_visible(b - a + i, b, w, s) for i in range(a))
        else:
            i = torch.arange(a, dtype=torch.float64) + (b - a)
            lo = (i - w + 1).clamp_min(0) if w else torch.zeros_like(i)
            pairs += int((i + 1 - lo + lo.clamp_max(s)).sum())
        lo = max(0, b - a - w + 1) if w else 0
        keys += b - lo + min(s, lo)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "window":
        es = 2 if case["dtype"] == "bf16" else 4
        pairs, keys = _pairs(case)
        rows = sum(_lens(case)[0]) * case["Hq"]
        return {"bytes": 2 * keys * case["Hkv"] * case["d"] * es + rows * (2 * case["d"] * es + 4),
                "flops": 4.0 * pairs * case["Hq"] * case["d"]}
    if op == "kv4_attn":
        pairs, keys = _pairs(case)
        rows = sum(_lens(case)[0]) * case["Hq"]
        per = 2 * (case["d"] // 2 + case["d"] // 16)   # codes and scales of K and V
        return {"bytes": keys * case["Hkv"] * per + rows * (4 * case["d"] + 4),
                "flops": 4.0 * pairs * case["Hq"] * case["d"]}
    if op == "kv4_append":
        n = case["T"] * case["Hkv"] * case["d"]
        return {"bytes": 2 * n * (2 + 2 * 0.5625 + 2) + 8 * case["T"], "flops": 8.0 * n}
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * case["T"], "flops": 3.0 * n}
    new, old = _lens(case)
    tokens = sum(max(0, n) for n in new)
    pages = sum(-(-(o + max(0, n)) // case["page"]) - -(-o // case["page"]) if n >= 0 else -(-o // case["page"])
                for n, o in zip(new, old))
    return {"bytes": 8 * tokens + 8 * pages + 16 * case["B"], "flops": 4 * tokens}


# ---------------------------------------------------------------------------
# The cache's pages: uint8 [pages][Hkv][page / 16][576 G], G = d / 32
# ---------------------------------------------------------------------------
# A subtile holds 16 tokens of one head: K codes (256 G bytes), V codes (256 G), K scales (32 G), V scales (32 G).
# A byte holds two neighbouring channels of one token, the lower channel in the low nibble, each as code + 8.
#   K codes   [token][q4][g][j / 2]               channel 32 g + 8 q4 + j
#   V codes   [p][c8][t4][g][hi][i / 2]           channel 32 g + 4 c8 + i, token 8 p + 2 t4 + hi
#   K scales  [token][g], V scales [p][t4][g][hi] bf16

def _pack(kc, vc, ks, vs):
    """codes + 8 [..., 16, d] and scales [..., 16, G] of 16 tokens each to [..., 576 G] bytes."""
    lead, d = kc.shape[:-2], kc.shape[-1]
    G = d // 32
    kb = kc[..., 0::2] | (kc[..., 1::2] << 4)                       # [.., 16, d/2]
    vb = vc[..., 0::2] | (vc[..., 1::2] << 4)
    n = len(lead)
    at = lambda *o: list(range(n)) + [n + x for x in o]             # noqa: E731
    kb = kb.reshape(*lead, 16, G, 4, 4).permute(at(0, 2, 1, 3)).reshape(*lead, 256 * G)
    vb = vb.reshape(*lead, 2, 4, 2, G, 8, 2).permute(at(0, 4, 1, 3, 2, 5)).reshape(*lead, 256 * G)
    ks = ks.contiguous().view(torch.uint8).reshape(*lead, 32 * G)
    vs = vs.reshape(*lead, 2, 4, 2, G).permute(at(0, 1, 3, 2)).contiguous().view(torch.uint8).reshape(*lead, 32 * G)
    return torch.cat([kb, vb, ks, vs], dim=-1)


def _unpack(sub, dtype):
    """[..., 576 G] bytes to K and V values [..., 16, d] in `dtype`."""
    lead, n = sub.shape[:-1], sub.dim() - 1
    G = sub.shape[-1] // 576
    at = lambda *o: list(range(n)) + [n + x for x in o]             # noqa: E731
    kb = sub[..., :256 * G].reshape(*lead, 16, 4, G, 4).permute(at(0, 2, 1, 3))
    vb = sub[..., 256 * G:512 * G].reshape(*lead, 2, 8, 4, G, 2, 2).permute(at(0, 2, 4, 3, 1, 5))
    ks = sub[..., 512 * G:544 * G].contiguous().view(BF16).reshape(*lead, 16, G)
    vs = sub[..., 544 * G:].contiguous().view(BF16).reshape(*lead, 2, 4, G, 2).permute(at(0, 1, 3, 2))
    got = []
    for b, s in ((kb, ks), (vb, vs)):
        x = torch.stack([b & 15, b >> 4], dim=-1).reshape(*lead, 16, G, 32).to(dtype) - 8
        got.append((x * s.reshape(*lead, 16, G, 1).to(dtype)).reshape(*lead, 16, 32 * G))
    return got


def _quantise(x):
    """bf16 [..., d] to codes + 8 (uint8) and bf16 scales [..., d / 32]."""
    g = x.float().reshape(*x.shape[:-1], -1, 32)
    s = (g.abs().amax(-1) / 7).to(BF16)
    sf = s.float().unsqueeze(-1)
    c = torch.where(sf > 0, torch.round(g / sf), torch.zeros_like(g))
    return (c.reshape(x.shape) + 8).to(torch.uint8), s


def _row_bytes(G, dev):
    """Byte offsets of a token's rows in its subtile: K and V codes [16, 16 G], K and V scales [16, 2 G]."""
    t, m = torch.arange(16, device=dev)[:, None], torch.arange(16 * G, device=dev)[None]   # m: channel pair
    g, q4, jb = m // 16, m % 16 // 4, m % 4
    k = t * 16 * G + q4 * 4 * G + g * 4 + jb
    c8, ib = m % 16 // 2, m % 2
    p, t4, hi = t // 8, t % 8 // 2, t % 2
    v = 256 * G + p * 128 * G + (c8 * 4 + t4) * 4 * G + g * 4 + hi * 2 + ib
    m = torch.arange(2 * G, device=dev)[None]
    return k, v, 512 * G + t * 2 * G + m, 544 * G + p * 16 * G + t4 * 4 * G + (m // 2) * 4 + hi * 2 + m % 2


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _lowrank(g, heads, basis, n, d, dtype=BF16):
    """[heads, n, d]: rank-16 structure shared by the heads' queries and keys, and noise, as the LM workload draws them."""
    z = torch.randn(heads, n, 16, device=DEV, generator=g)
    x = torch.randn(heads, n, d, device=DEV, generator=g)
    return x.baddbmm_(z, basis).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)     # noqa: E731
    s = {"case": case}
    if op == "window":
        dt = BF16 if case["dtype"] == "bf16" else torch.float32
        B, Hq, Hkv, Nq, Nk, d = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
        basis = torch.randn(Hkv, 16, d, device=DEV, generator=g) / 4
        bq = basis.repeat_interleave(Hq // Hkv, 0)
        s["q"] = torch.stack([_lowrank(g, Hq, bq, Nq, d, dt) for _ in range(B)])
        s["k"] = torch.stack([_lowrank(g, Hkv, basis, Nk, d, dt) for _ in range(B)])
        s["v"] = torch.randn(B, Hkv, Nk, d, device=DEV, generator=g).to(dt)
        nq, nk = _lens(case)
        s["q_len"], s["kv_len"] = (i32(nq), i32(nk)) if case["ragged"] else (None, None)
        s["out"] = torch.zeros(B, Hq, Nq, d, dtype=dt, device=DEV)
        s["lse"] = torch.zeros(B, Hq, Nq, dtype=torch.float32, device=DEV)
    elif op == "kv4_attn":
        B, Hq, Hkv, d, page = (case[k] for k in ("B", "Hq", "Hkv", "d", "page"))
        nq, nk = _lens(case)
        blocks = [-(-n // page) for n in nk]
        pages = sum(blocks) + 3
        basis = torch.randn(Hkv, 16, d, device=DEV, generator=g) / 4
        cache = torch.empty(pages, Hkv, page // 16, 18 * d, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 28) // (page * Hkv * d))
        for a in range(0, pages, step):
            n = min(step, pages - a)
            cut = lambda x: x.reshape(Hkv, n, page // 16, 16, -1).transpose(0, 1)     # noqa: E731
            kc, ks = _quantise(_lowrank(g, Hkv, basis, n * page, d))
            vc, vs = _quantise(torch.randn(Hkv, n * page, d, device=DEV, generator=g).to(BF16))
            cache[a:a + n] = _pack(cut(kc), cut(vc), cut(ks), cut(vs))
        s["cache"] = cache
        order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
        table = torch.full((B, max(blocks) + 1), -1, dtype=torch.int32, device=DEV)
        used = 0
        for b, n in enumerate(blocks):
            table[b, :n] = order[used:used + n]
            used += n
        s["table"], s["kv_len"] = table, i32(nk)
        T = sum(nq)
        s["cu_q"] = i32([sum(nq[:b]) for b in range(B + 1)])
        bq = basis.repeat_interleave(Hq // Hkv, 0)
        s["q"] = _lowrank(g, Hq, bq, T, d).transpose(0, 1).contiguous()
        s["out"] = torch.empty(T, Hq, d, dtype=BF16, device=DEV)
        s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=DEV)
    elif op == "kv4_append":
        T, H, d, page, pages = (case[k] for k in ("T", "Hkv", "d", "page", "pages"))
        basis = torch.randn(H, 16, d, device=DEV, generator=g) / 4
        s["k"] = _lowrank(g, H, basis, T, d).transpose(0, 1).contiguous()
        s["v"] = torch.randn(T, H, d, device=DEV, generator=g).to(BF16)
        # Each request's new tokens lie one behind the other in its pages; the pages lie anywhere.
        if case["run"] == 1:
            slots = torch.randperm(pages * page, device=DEV, generator=g)[:T]
        else:
            order = torch.randperm(pages, device=DEV, generator=g)
            at = torch.arange(T, device=DEV)
            slots = order[at // page] * page + at % page
        s["slots"] = slots.to(torch.int32)
        s["cache"] = torch.zeros(pages, H, page // 16, 18 * d, dtype=torch.uint8, device=DEV)
        s["k_out"] = torch.empty(T, H, d, dtype=BF16, device=DEV)
        s["v_out"] = torch.empty(T, H, d, dtype=BF16, device=DEV)
    elif op == "rope":
        dt = BF16 if case["dtype"] == "bf16" else torch.float32
        T, Hq, Hkv, d = (case[k] for k in ("T", "Hq", "Hkv", "d"))
        s["q"] = torch.randn(T, Hq, d, device=DEV, generator=g).to(dt)
        s["k"] = torch.randn(T, Hkv, d, device=DEV, generator=g).to(dt)
        s["pos"] = torch.randint(0, case["max_pos"], (T,), device=DEV, generator=g).to(torch.int32)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    else:
        B, page, mb = case["B"], case["page"], case["max_blocks"]
        new, old = _lens(case)
        held = [-(-n // page) for n in old]
        need = sum(-(-(o + max(0, n)) // page) for n, o in zip(new, old))
        num = need + 64
        order = torch.randperm(num, device=DEV, generator=g).to(torch.int32)
        h = i32(held)
        cols = torch.arange(mb, device=DEV)[None]
        first = torch.cumsum(h, 0) - h
        index = (first[:, None] + cols).clamp_max(num - 1)
        s["table"] = torch.where(cols < h[:, None], order[index], torch.full_like(order[index], -1))
        n_held = sum(held)
        free = torch.full((num,), -1, dtype=torch.int32, device=DEV)
        free[:num - n_held] = order[n_held:]
        s["free"], s["free_count"] = free, i32([num - n_held])
        s["old"], s["new"] = i32(old), i32(new)
        tokens = sum(max(0, n) for n in new) + 13        # a buffer with a few places to spare
        s["num_pages"] = num
        s["new_len"], s["cu_q"] = i32([0] * B), i32([0] * (B + 1))
        s["slots"], s["positions"] = (torch.empty(tokens, dtype=torch.int32, device=DEV) for _ in range(2))
        s["free_count_out"] = i32([0])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

ROPE = dict(base=10000.0, factor=4.0, original_len=32768, beta_fast=32.0, beta_slow=1.0)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from long_context_mean_b200 import sa
        if op == "window":
            if "ws" not in s:
                s["ws"] = sa.workspace(sa.window_attn_workspace(s["q"], s["k"], s["v"]), DEV)
            sa.window_attn(s["q"], s["k"], s["v"], s["out"], s["lse"], window=c["window"], sinks=c["sinks"],
                           q_len=s["q_len"], kv_len=s["kv_len"], ws=s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "kv4_attn":
            if "kv4" not in s:
                s["kv4"] = sa.KV4Cache(s["cache"], c["page"], c["d"])
                s["ws"] = sa.workspace(sa.kv4_attn_workspace(s["kv4"], c["Hq"]), DEV)
            sa.kv4_attn(s["q"], s["kv4"], s["table"], s["kv_len"], s["out"], s["lse"], cu_q=s["cu_q"],
                        window=c["window"], sinks=c["sinks"], ws=s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "kv4_append":
            if "kv4" not in s:
                s["kv4"] = sa.KV4Cache(s["cache"], c["page"], c["d"])
            sa.kv4_append(s["k"], s["v"], s["slots"], s["kv4"])
            sa.kv4_read(s["kv4"], s["slots"], s["k_out"], s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if op == "rope":
            if "rope" not in s:
                s["rope"] = sa.Rope(c["rot"], layout=c["layout"], scaling=c["scaling"], device=DEV, **ROPE)
            sa.rope(s["rope"], s["pos"], s["q"], s["q_out"], s["k"], s["k_out"], inverse=c["inverse"])
            return {"q": s["q_out"], "k": s["k_out"]}
        sa.cache_plan(s["old"], s["new"], s["table"], s["free"], s["free_count"], c["page"], s["new_len"], s["cu_q"],
                      s["slots"], s["positions"], s["free_count_out"])
        return {"table": s["table"], "free": s["free"], "free_count": s["free_count_out"], "new_len": s["new_len"],
                "cu_q": s["cu_q"], "slots": s["slots"], "positions": s["positions"]}
    if op == "window":
        return _plain_window(s, c)
    if op == "kv4_attn":
        return _plain_kv4_attn(s, c)
    if op == "kv4_append":
        return _plain_append(s, c)
    if op == "rope":
        return _plain_rope(s, c)
    return _plain_plan(s, c)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _softmax_v(S, V):
    """softmax over the last axis (a row of -inf gives zeros) times V, and the log of the sum."""
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = torch.exp(S.sub_(m))
    l = P.sum(-1, keepdim=True)
    O = torch.matmul(P, V) / torch.where(l > 0, l, torch.ones_like(l))
    return O, (m + torch.log(l)).squeeze(-1)


def _mask(p, j, n, window, sinks):
    """Which keys j of n the queries at positions p see."""
    see = (j <= p) & (j < n)
    return see & ((p - j < window) | (j < sinks)) if window else see


def _plain_window(s, c):
    B, Hq, Hkv, Nq, Nk, d = (c[k] for k in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
    w, sinks, G = c["window"], c["sinks"], Hq // Hkv
    dev = s["q"].device
    nq = s["q_len"].long() if s["q_len"] is not None else torch.full((B,), Nq, device=dev)
    nk = s["kv_len"].long() if s["kv_len"] is not None else torch.full((B,), Nk, device=dev)
    q = s["q"].float().reshape(B, Hkv, G, Nq, d)
    k, v = s["k"].float(), s["v"].float()
    out, lse = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    banded = s["q_len"] is None and w and w + sinks + 1024 < Nk
    step = Nq if not banded and B * Hq * Nq * Nk <= (1 << 30) else 1024
    for i0 in range(0, Nq, step):
        i1 = min(Nq, i0 + step)
        i = torch.arange(i0, i1, device=dev)
        j = torch.arange(Nk, device=dev)
        if banded:
            lo = max(0, Nk - Nq + i0 - w + 1)
            j = torch.cat([j[:min(sinks, lo)], j[lo:Nk - Nq + i1]])
        kj, vj = (k, v) if not banded else (k[:, :, j], v[:, :, j])
        p = (nk - nq)[:, None] + i
        see = _mask(p[:, :, None], j, nk[:, None, None], w, sinks)[:, None, None]
        S = torch.matmul(q[:, :, :, i0:i1].reshape(B, Hkv, -1, d), kj.transpose(-1, -2)) / math.sqrt(d)
        S = S.reshape(B, Hkv, G, i1 - i0, -1).masked_fill_(~see, -math.inf)
        O, L = _softmax_v(S.reshape(B, Hkv, -1, S.shape[-1]), vj)
        live = (i < nq[:, None])[:, None]                            # rows behind a sequence stay as they were
        out[:, :, i0:i1] = torch.where(live[..., None], O.reshape(B, Hq, -1, d), 0.0).to(out.dtype)
        lse[:, :, i0:i1] = torch.where(live, L.reshape(B, Hq, -1), 0.0)
    return {"out": out, "lse": lse}


def _plain_kv4_attn(s, c):
    B, Hq, Hkv, d, page = (c[k] for k in ("B", "Hq", "Hkv", "d", "page"))
    dev = s["q"].device
    L, G = c["max_len"], Hq // Hkv
    blocks = -(-L // page)
    nk, cu = s["kv_len"].long(), s["cu_q"].long()
    nq = cu[1:] - cu[:-1]
    sub = s["cache"][s["table"][:, :blocks].long().clamp_min(0)]     # [B, blocks, Hkv, page / 16, bytes]
    sub = sub.transpose(1, 2).reshape(B, Hkv, blocks * page // 16, -1)
    k, v = (x.reshape(B, Hkv, blocks * page, d) for x in _unpack(sub, torch.float32))
    # Pages behind a sequence's end hold other requests' rows: they are masked.
    Q = min(c["q_max"], L)
    i = torch.arange(Q, device=dev)
    row = (cu[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"].float()[row].reshape(B, Q, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, d)
    S = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    p = (nk - nq)[:, None] + i
    see = _mask(p[:, :, None], torch.arange(blocks * page, device=dev), nk[:, None, None], c["window"], c["sinks"])
    S = S.reshape(B, Hkv, G, Q, -1).masked_fill_(~see[:, None, None], -math.inf).reshape(B, Hkv, G * Q, -1)
    O, lse = _softmax_v(S, v)
    live = i < nq[:, None]
    O = O.reshape(B, Hkv, G, Q, d).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, d)
    lse = lse.reshape(B, Hkv, G, Q).permute(0, 3, 1, 2).reshape(B, Q, Hq)
    return {"out": O[live].to(BF16), "lse": lse[live].contiguous()}


def _plain_append(s, c):
    H, d, page = c["Hkv"], c["d"], c["page"]
    G, slots, cache = d // 32, s["slots"].long(), s["cache"]
    h = torch.arange(H, device=slots.device)[None]
    sub = ((slots // page)[:, None] * H + h) * (page // 16) + (slots % page // 16)[:, None]
    ats = [(sub * 576 * G)[..., None] + o[slots % 16][:, None] for o in _row_bytes(G, slots.device)]
    (kc, ks), (vc, vs) = _quantise(s["k"]), _quantise(s["v"])
    flat = cache.reshape(-1)
    for at, x in zip(ats, (kc[..., 0::2] | (kc[..., 1::2] << 4), vc[..., 0::2] | (vc[..., 1::2] << 4),
                           ks.view(torch.uint8), vs.view(torch.uint8))):
        flat[at] = x
    got = []
    for codes, scales in ((ats[0], ats[2]), (ats[1], ats[3])):
        b, sc = flat[codes], flat[scales].view(BF16).float()
        x = torch.stack([b & 15, b >> 4], -1).reshape(*b.shape[:2], G, 32).float() - 8
        got.append((x * sc[..., None]).reshape(*b.shape[:2], d).to(BF16))
    return {"k": got[0], "v": got[1]}


def _frequencies(c):
    """Angle per position of each pair in 64 bits, and the factor on the rotated channels."""
    rot, base, f = c["rot"], ROPE["base"], ROPE["factor"]
    e = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    if c["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    w = base ** -e
    if c["scaling"] == "linear":
        return w / f, 1.0
    if c["scaling"] != "yarn":
        return w, 1.0
    # Pairs that turn often over the trained length keep their angle, slow ones are stretched, between lies a ramp.
    n = ROPE["original_len"]
    pair = lambda turns: rot * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
    lo = max(0, math.floor(pair(ROPE["beta_fast"])))
    hi = min(rot - 1, math.ceil(pair(ROPE["beta_slow"])))
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return w * (1 - ramp) + w / f * ramp, 0.1 * math.log(f) + 1


def _plain_rope(s, c):
    w, mag = _frequencies(c)
    a = s["pos"].double()[:, None] * w.to(s["pos"].device)
    cos, sin = (torch.cos(a) * mag).float()[:, None], (torch.sin(a) * mag).float()[:, None]
    if c["inverse"]:
        sin = -sin
    rot, got = c["rot"], {}
    for name in ("q", "k"):
        x = s[name].float()
        if c["layout"] == "half":
            x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        else:
            x1, x2 = x[..., :rot:2], x[..., 1:rot:2]
        y = [x1 * cos - x2 * sin, x2 * cos + x1 * sin]
        y = torch.cat(y, -1) if c["layout"] == "half" else torch.stack(y, -1).flatten(-2)
        got[name] = torch.cat([y, x[..., rot:]], -1).to(s[name].dtype)
    return got


def _plain_plan(s, c):
    page, dev = c["page"], s["old"].device
    old, new = s["old"].long(), s["new"].long()
    ends = new < 0
    add = new.clamp_min(0)
    held = (old + page - 1) // page
    grown = torch.where(ends, torch.zeros_like(old), (old + add + page - 1) // page - held)
    gone = torch.where(ends, held, torch.zeros_like(old))
    table, free = s["table"], s["free"]
    count = s["free_count"].long()
    cols = torch.arange(table.shape[1], device=dev)[None]
    # Pages of requests that end go on the stack, in the order of the requests and their blocks.
    released = table[(cols < gone[:, None])]
    free[count + torch.arange(released.numel(), device=dev)] = released
    top = count + released.numel()
    # New blocks take pages off the top, in the order of the requests and their blocks.
    fresh = (cols >= held[:, None]) & (cols < (held + grown)[:, None])
    taken = torch.arange(int(fresh.sum()), device=dev)
    table[fresh] = free[top - 1 - taken]
    cu = torch.zeros(c["B"] + 1, dtype=torch.int64, device=dev)
    cu[1:] = add.cumsum(0)
    b = torch.repeat_interleave(torch.arange(c["B"], device=dev), add)
    p = old[b] + torch.arange(b.numel(), device=dev) - cu[b]
    slots, positions = torch.full_like(s["slots"], -1), torch.zeros_like(s["positions"])
    slots[:b.numel()] = table[b, p // page] * page + (p % page).int()
    positions[:b.numel()] = p.int()
    return {"table": table, "free": free, "free_count": (top - taken.numel()).int(),
            "new_len": torch.where(ends, 0, old + add).int(), "cu_q": cu.int(), "slots": slots,
            "positions": positions}


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(q, k, v, first, window, sinks):
    """Attention of queries [H, n, d] at positions first.. over keys [H, m, d], row block by row block."""
    n, m, d = q.shape[1], k.shape[1], q.shape[2]
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=q.dtype, device=q.device)
    step = 512
    for a in range(0, n, step):
        b = min(n, a + step)
        last = min(m, first + b)
        if last <= 0:
            continue
        lo = max(0, first + a - window + 1) if window else 0
        keys = torch.arange(last, device=q.device)
        keys = torch.cat([keys[:min(lo, sinks)], keys[lo:]])
        dots = torch.einsum("hnd,hmd->hnm", q[:, a:b], k[:, keys]) * d ** -0.5
        back = (first + torch.arange(a, b, device=q.device))[:, None] - keys[None]
        hidden = back < 0
        if window:
            hidden = hidden | ((back >= window) & (keys[None] >= sinks))
        dots.masked_fill_(hidden, -math.inf)
        lse[:, a:b] = torch.logsumexp(dots, -1)
        weight = torch.exp(dots - lse[:, a:b, None].clamp_min(-1e300))
        out[:, a:b] = torch.einsum("hnm,hmd->hnd", weight, v[:, keys])
    return out, lse


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "window":
        nq, nk = _lens(case)
        G = case["Hq"] // case["Hkv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            for h in range(case["Hkv"]):
                k, v = (s[x][b, h, :nk[b]].double()[None].expand(G, -1, -1) for x in "kv")
                o, l = _exact_rows(s["q"][b, h * G:(h + 1) * G, :nq[b]].double(), k, v, nk[b] - nq[b],
                                   case["window"], case["sinks"])
                out[b, h * G:(h + 1) * G, :nq[b]], lse[b, h * G:(h + 1) * G, :nq[b]] = o, l
        return {"out": out, "lse": lse}
    if op == "kv4_attn":
        nq, nk = _lens(case)
        G, page = case["Hq"] // case["Hkv"], case["page"]
        outs, lses, at = [], [], 0
        for b in range(case["B"]):
            pages = s["table"][b, :-(-nk[b] // page)].long()
            k, v = (x.transpose(0, 1).reshape(case["Hkv"], -1, case["d"])[:, :nk[b]].repeat_interleave(G, 0)
                    for x in (y.reshape(pages.numel(), case["Hkv"], page, -1) for y in _unpack(s["cache"][pages], torch.float64)))
            o, l = _exact_rows(s["q"][at:at + nq[b]].double().transpose(0, 1), k, v, nk[b] - nq[b], case["window"],
                               case["sinks"])
            outs.append(o.transpose(0, 1))
            lses.append(l.transpose(0, 1))
            at += nq[b]
        return {"out": torch.cat(outs), "lse": torch.cat(lses).contiguous()}
    if op == "kv4_append":
        got = {}
        for name in "kv":
            x = s[name].double().unflatten(-1, (-1, 32))
            top = x.abs().max(-1, keepdim=True).values / 7
            unit = torch.exp2(torch.floor(torch.log2(top)) - 7)          # bf16 keeps 8 bits
            scale = torch.round(top / unit) * unit
            got[name] = (torch.round(x / scale) * scale).nan_to_num(0.0).flatten(-2)
        return got
    w, mag = _frequencies(case)
    turn = torch.polar(torch.full((1,), mag, dtype=torch.float64, device=DEV),
                       s["pos"].double()[:, None] * w.to(DEV) * (-1 if case["inverse"] else 1))[:, None]
    rot, got = case["rot"], {}
    for name in ("q", "k"):
        x = s[name].double()
        r = x[..., :rot]
        r = r.unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else r.unflatten(-1, (-1, 2))
        r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn)
        r = (r.transpose(-1, -2) if case["layout"] == "half" else r).flatten(-2)
        got[name] = torch.cat([r, x[..., rot:]], -1)
    return got

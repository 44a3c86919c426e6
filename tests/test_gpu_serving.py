"""The serving operators on the GPU against the plain 64-bit forms: window
attention, the 4-bit cache's rows, attention over it, rotary positions, the
cache plan, and a run of steps of all of them together.

Tolerances.  u = 2^-8 is half a bf16 step relative to the value.  A kernel's
score is off by at most e = (d + 8) 2^-24 sum |q_c k_c| scale (fp32 products and
sums, the scaling, the difference to the maximum; the power of two adds
2^-22), so a weight is off by 2 e + 2^-21 relative (numerator and normaliser);
bf16 weights (and for the 4-bit cache bf16 weight times scale) add u each, the
output's rounding u |o|, and sums of n terms n 2^-24.  The cache's K enters as
(code + 8) with 8 sum q taken off in the accumulator: every term and partial
sum of a 32-channel group is then at most sum |q_c| (|code_c| + 8) times its scale,
so e counts |k_c| + 8 s_c in the place of |k_c|, with 3 x 32 products, 32 terms of the
sum of q, the offset, the scale and the 4 groups: below (d + 8) roundings of 2^-24 for
d = 128 and below 140 for either d.
O's partial sums round (or are cut) by 2^-23 of sum w |v| at most with each product of 16
tokens and each joining of parts, n / 16 + 16 of them.
"""

import math

import numpy as np
import pytest

from oracle import serving as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def sa():
    from long_context_mean_b200 import sa
    return sa


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_rows(out, lse, want, d, n, dtype, roundings):
    """One head's rows against attention()'s result; roundings: bf16 roundings of a weight."""
    o, l, absv, size = want
    assert np.isfinite(out).all()
    e = (d + 8) * 2.0 ** -24 * size[:, None]
    rel = 2 * e + 2.0 ** -21 + n * 2.0 ** -23 + roundings * 2.0 ** -8 * (1 + 2.0 ** -7)
    last = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    off = (rel + (n / 16 + 16) * 2.0 ** -23) * absv
    assert (np.abs(out - o) <= last * (np.abs(o) + off) + off + 1e-38).all(), np.abs(out - o).max()
    none = np.isinf(l)
    assert np.array_equal(np.isneginf(lse), none) and (out[none] == 0).all()
    ok = ~none
    lse, l = np.where(ok, lse, 0), np.where(ok, l, 0)
    # bf16 weights enter the output only: the normaliser sums them unrounded
    assert (np.abs(lse - l)[ok] <= (2 * e[:, 0] + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(l))[ok]).all()


# ---------------------------------------------------------------------------
# Window attention
# ---------------------------------------------------------------------------

# B, Hq, Hkv, Nq, Nk, d, dtype, window, sinks, q_len, kv_len
WINDOW = [
    (2, 4, 2, 1, 77, 128, "bf16", 0, 0, None, None),
    (3, 8, 2, 1, 300, 128, "bf16", 64, 5, None, [300, 1, 0]),
    (1, 32, 8, 1, 1000, 128, "bf16", 256, 128, None, None),
    (2, 4, 4, 1, 65, 64, "bf16", 1, 0, None, [64, 17]),
    (2, 16, 2, 3, 90, 128, "bf16", 33, 2, [3, 2], [90, 2]),
    (1, 8, 1, 2, 50, 64, "bf16", 7, 40, None, None),
    (2, 12, 4, 5, 200, 128, "bf16", 100, 30, [5, 0], [200, 150]),
    (1, 2, 1, 130, 130, 128, "bf16", 0, 0, None, None),
    (2, 4, 2, 300, 300, 128, "bf16", 64, 4, [300, 131], [300, 131]),
    (1, 4, 2, 129, 400, 128, "bf16", 100, 70, None, None),
    (2, 2, 2, 257, 190, 128, "bf16", 50, 3, [257, 256], [190, 0]),     # more rows than keys: rows that see nothing
    (1, 2, 1, 513, 700, 128, "bf16", 1, 0, None, None),
    (2, 4, 2, 200, 260, 128, "bf16", 128, 129, [17, 200], [260, 201]),
    (1, 3, 3, 640, 640, 128, "bf16", 320, 64, None, None),
    (1, 4, 1, 150, 150, 64, "bf16", 40, 3, [149], [150]),
    (1, 2, 1, 70, 90, 16, "bf16", 20, 3, None, None),
    (1, 2, 2, 40, 40, 256, "bf16", 11, 2, None, None),
    (1, 2, 1, 66, 66, 104, "bf16", 0, 0, None, None),
    (2, 4, 2, 1, 1, 64, "fp32", 0, 0, None, None),
    (2, 4, 2, 100, 100, 64, "fp32", 30, 2, [100, 37], [90, 37]),
    (1, 4, 4, 65, 200, 128, "fp32", 64, 1, None, None),
    (1, 2, 1, 70, 33, 16, "fp32", 9, 0, None, None),
    (2, 2, 2, 128, 128, 256, "fp32", 0, 7, None, [128, 0]),
    (1, 2, 1, 90, 90, 20, "fp32", 64, 64, None, None),
]


def window_inputs(torch, c, seed=0):
    B, Hq, Hkv, Nq, Nk, d, dtype, window, sinks, ql, kl = c
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = (torch.randn(B, Hq, Nq, d, device="cuda", generator=g) * 1.5).to(dt)
    k = torch.randn(B, Hkv, Nk, d, device="cuda", generator=g).to(dt)
    v = torch.randn(B, Hkv, Nk, d, device="cuda", generator=g).to(dt)
    return q, k, v, ql or [Nq] * B, kl or [Nk] * B


def paths(c):
    """The kernels that a case can be sent to: the library's own choice, the decode, prefill and CUDA-core ones."""
    return [0, 8, 16, 1] if c[6] == "bf16" and c[5] in (64, 128) else [0]


@pytest.mark.parametrize("c,flags", [(c, f) for c in WINDOW for f in paths(c)],
                         ids=lambda x: str(x) if isinstance(x, int) else "-".join(map(str, x[:9])))
@pytest.mark.parametrize("poison", [False, True])
def test_window_attn(torch, sa, c, flags, poison):
    B, Hq, Hkv, Nq, Nk, d, dtype, window, sinks, ql, kl = c
    q, k, v, nq, nk = window_inputs(torch, c)
    if poison:   # whatever no row sees may be anything, and rows behind a sequence too
        for b in range(B):
            seen = S.visible(nq[b], nk[b], window, sinks).any(0)
            hidden = torch.ones(Nk, dtype=torch.bool)
            hidden[:nk[b]] = torch.from_numpy(~seen)
            k[b, :, hidden], v[b, :, hidden] = math.nan, math.inf
            q[b, :, nq[b]:] = math.nan
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    status = i32(torch, [0])
    ws = sa.workspace(sa.window_attn_workspace(q, k, v), "cuda")
    ws.fill_(255)
    sa.window_attn(q, k, v, out, lse, window=window, sinks=sinks, q_len=ql and i32(torch, ql),
                   kv_len=kl and i32(torch, kl), status=status, ws=ws, flags=flags)
    assert sa.read_status(status) == 0
    o, l, qn, kn, vn = (f64(t) for t in (out, lse, q, k, v))
    for b in range(B):
        for h in range(Hq):
            want = S.attention(qn[b, h, :nq[b]], kn[b, h * Hkv // Hq, :nk[b]], vn[b, h * Hkv // Hq, :nk[b]], window, sinks)
            check_rows(o[b, h, :nq[b]], l[b, h, :nq[b]], want, d, nk[b], dtype,
                       1 if dtype == "bf16" and d in (64, 128) and flags != 1 else 0)
        assert (o[b, :, nq[b]:] == 7).all() and (l[b, :, nq[b]:] == 7).all()
    again = torch.full_like(out, 7.0)
    sa.window_attn(q, k, v, again, window=window, sinks=sinks, q_len=ql and i32(torch, ql), kv_len=kl and i32(torch, kl),
                   flags=flags)
    assert torch.equal(again, out)


@pytest.mark.parametrize("c,flags", [(WINDOW[1], 8), (WINDOW[8], 16), (WINDOW[8], 8), (WINDOW[19], 0)], ids=str)
def test_window_attn_bad_lengths_stay_inside(torch, sa, c, flags):
    q, k, v, nq, nk = window_inputs(torch, c)
    B = q.shape[0]
    status = i32(torch, [0])
    out = torch.empty_like(q)
    sa.window_attn(q, k, v, out, window=9, kv_len=i32(torch, [1 << 30] + [-5] * (B - 1)), status=status,
                   flags=flags)
    assert sa.read_status(status) == sa.SA_ERR_INVALID_ARG
    status.zero_()
    sa.window_attn(q, k, v, out, window=9, q_len=i32(torch, [-1] + [1 << 30] * (B - 1)), status=status,
                   flags=flags)
    assert sa.read_status(status) == sa.SA_ERR_INVALID_ARG


@pytest.mark.parametrize("flags", [8, 16, 1])
def test_window_attn_scale_and_large_scores(torch, sa, flags):
    c = (1, 2, 1, 140, 140, 128, "bf16", 90, 2, None, None)
    q, k, v, _, _ = window_inputs(torch, c)
    q *= 8
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    sa.window_attn(q, k, v, out, lse, window=90, sinks=2, scale=0.3, flags=flags)
    o, l, qn, kn, vn = (f64(t) for t in (out, lse, q, k, v))
    for h in range(2):
        check_rows(o[0, h], l[0, h], S.attention(qn[0, h], kn[0, 0], vn[0, 0], 90, 2, 0.3), 128, 140, "bf16", 1)


@pytest.mark.parametrize("c,flags", [(WINDOW[0], 8), (WINDOW[7], 8), (WINDOW[7], 16), (WINDOW[20], 0)], ids=str)
def test_window_attn_nan_in_a_visible_key_shows(torch, sa, c, flags):
    q, k, v, _, _ = window_inputs(torch, c)
    v[0, 0, 3, 5] = math.nan
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    sa.window_attn(q, k, v, out, lse, flags=flags)
    assert torch.isnan(out[0, 0, -1, 5]) and not torch.isnan(out[0, 0, -1, 6])
    k[0, 0, 2] = math.nan
    sa.window_attn(q, k, v, out, lse, flags=flags)
    assert torch.isnan(out[0, 0, -1]).all() and torch.isnan(lse[0, 0, -1])
    if q.shape[0] > 1:
        assert torch.isfinite(out[1]).all()


@pytest.mark.parametrize("c,flags", [(WINDOW[2], 8), (WINDOW[8], 16), (WINDOW[19], 0)], ids=["decode", "prefill", "fp32"])
def test_window_attn_other_stream_and_graph(torch, sa, c, flags):
    B, Hq, Hkv, Nq, Nk, d, dtype, window, sinks, ql, kl = c
    q, k, v, _, _ = window_inputs(torch, c)
    want = torch.empty_like(q)
    sa.window_attn(q, k, v, want, window=window, sinks=sinks, flags=flags)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(q)
    ws = sa.workspace(sa.window_attn_workspace(q, k, v), "cuda")
    sa.window_attn(q, k, v, got, window=window, sinks=sinks, ws=ws, stream=side, flags=flags)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.window_attn(q, k, v, got, window=window, sinks=sinks, ws=ws, flags=flags)
    got.zero_()
    graph.replay()
    assert torch.equal(got, want)
    q2, k2, v2, _, _ = window_inputs(torch, c, 5)
    for a, b in ((q, q2), (k, k2), (v, v2)):
        a.copy_(b)
    graph.replay()
    sa.window_attn(q2, k2, v2, want, window=window, sinks=sinks, flags=flags)
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# The cache's rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("H,d,page,T", [(1, 64, 16, 1), (3, 128, 16, 37), (2, 64, 128, 130), (8, 128, 64, 200)])
def test_kv4_append_is_the_plain_form(torch, sa, H, d, page, T):
    g = torch.Generator(device="cuda").manual_seed(T)
    pages = T // page + 3
    # rows of a packed projection (strided), and some that matter: zeros, one large channel, subnormals, inf, NaN
    packed = torch.randn(T, 3 * H, d, device="cuda", generator=g).to(torch.bfloat16)
    k, v = packed[:, H:2 * H], packed[:, 2 * H:]
    k[0, 0, :32] = 0
    v[0, 0, 32:64] = 0
    v[0, 0, 40] = 3e38
    if T > 5:
        k[1, 0, 0], v[2, 0, 33], k[3, 0] = math.inf, math.nan, 1e-39
        k[4, 0, :32], v[4, 0, 5] = 9.2e-41, -math.inf
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:T].to(torch.int32)
    if T > 5:
        slots[5] = -1
    cache = sa.KV4Cache.allocate(pages, H, page, d)
    cache.pages.fill_(0x5A)
    status = i32(torch, [0])
    sa.kv4_append(k, v, slots, cache, status=status)
    want = np.full(cache.pages.shape, 0x5A, np.uint8)
    kn, vn, sl = f64(k), f64(v), slots.cpu().numpy()
    with np.errstate(invalid="ignore"):
        (kc, ks), (vc, vs) = S.quantise(kn), S.quantise(vn)
    for t in range(T):
        for h in range(H):
            if sl[t] >= 0:
                S.store(want, sl[t], h, kc[t, h], ks[t, h], vc[t, h], vs[t, h])
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    ko, vo = (torch.full((T, H, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sa.kv4_read(cache, slots, ko, vo, status=status)
    assert sa.read_status(status) == 0
    for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
        x = S.round_bf16(np.nan_to_num(S.values(c, s), nan=0)) + np.where(np.isnan(S.values(c, s)), np.nan, 0)
        x[sl < 0] = 9
        assert np.array_equal(f64(got), x, equal_nan=True)


def test_kv4_rows_bad_slots(torch, sa):
    cache = sa.KV4Cache.allocate(2, 2, 16, 64)
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (32, -2, 1 << 30):
        status = i32(torch, [0])
        cache.pages.zero_()
        sa.kv4_append(k, k, i32(torch, [3, bad, 4]), cache, status=status)
        assert sa.read_status(status) == sa.SA_ERR_INVALID_ARG
        o = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        sa.kv4_read(cache, i32(torch, [3, bad, 4]), o, torch.zeros_like(o))
        assert (o[0] == 1).all() and (o[1] == 0).all() and (o[2] == 1).all()


# ---------------------------------------------------------------------------
# Attention over the cache
# ---------------------------------------------------------------------------

# Hq, Hkv, d, page, kv_len, q_len, window, sinks
KV4 = [
    (4, 2, 128, 16, [1], [1], 0, 0),
    (8, 2, 128, 16, [5, 0, 33, 200], [1, 1, 1, 1], 0, 0),
    (32, 8, 128, 64, [700], [1], 0, 0),
    (4, 4, 64, 32, [31, 32, 33], [1, 1, 1], 0, 0),
    (16, 2, 128, 128, [129, 400], [3, 2], 50, 3),
    (8, 1, 64, 16, [300, 17], [4, 17], 64, 20),
    (24, 24, 128, 16, [100, 3, 250], [1, 0, 2], 16, 0),
    (12, 4, 128, 32, [512, 90], [1, 5], 1, 40),
    (4, 2, 128, 16, [10, 20], [12, 3], 0, 0),           # more rows than keys
    (32, 8, 128, 16, [3000, 1, 64], [1, 1, 1], 1000, 4),
]


def paged(torch, sa, c, seed=0):
    """The operator's inputs, and each sequence's K and V values [n, Hkv, d] in 64 bits."""
    Hq, Hkv, d, page, nk, nq, window, sinks = c
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [-(-n // page) for n in nk]
    total = sum(blocks) + 2
    cache = sa.KV4Cache.allocate(total, Hkv, page, d)
    cache.pages.fill_(255)      # scales of NaN wherever nothing is written
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(nk), max(blocks) + 2), -7, dtype=torch.int32)
    vals, used = [], 0
    for b, n in enumerate(nk):
        table[b, :blocks[b]] = torch.tensor(order[used:used + blocks[b]], dtype=torch.int32)
        k, v = (torch.randn(n, Hkv, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
        slots = torch.tensor([order[used + i // page] * page + i % page for i in range(n)], dtype=torch.int32, device="cuda")
        sa.kv4_append(k, v, slots, cache)
        vals.append([S.values(*S.quantise(f64(x))) for x in (k, v)] + [8 * np.repeat(S.quantise(f64(k))[1], 32, -1)])
        used += blocks[b]
    q = (torch.randn(sum(nq) + 2, Hq, d, device="cuda", generator=g) * 1.5).to(torch.bfloat16)
    cu = i32(torch, [sum(nq[:i]) for i in range(len(nq) + 1)])
    return q, cache, table, i32(torch, nk), cu, vals


@pytest.mark.parametrize("c", KV4, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_kv4_attn(torch, sa, c):
    Hq, Hkv, d, page, nk, nq, window, sinks = c
    q, cache, table, kv_len, cu, vals = paged(torch, sa, c)
    for b in range(len(nk)):    # blocks without a key that some row sees may have been given away
        seen = S.visible(nq[b], nk[b], window, sinks).any(0)
        for i in range(-(-nk[b] // page)):
            if not seen[i * page:(i + 1) * page].any():
                table[b, i] = -7
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    status = i32(torch, [0])
    ws = sa.workspace(sa.kv4_attn_workspace(cache, Hq), "cuda")
    ws.fill_(255)
    sa.kv4_attn(q, cache, table.cuda(), kv_len, out, lse, cu_q=cu, window=window, sinks=sinks, status=status, ws=ws)
    assert sa.read_status(status) == 0
    o, l, qn, at = f64(out), f64(lse), f64(q), 0
    for b, (n, k) in enumerate(zip(nq, nk)):
        for h in range(Hq):
            kh, vh, extra = (x[:, h * Hkv // Hq] for x in vals[b])
            want = S.attention(qn[at:at + n, h], kh, vh, window, sinks, extra=extra)
            check_rows(o[at:at + n, h], l[at:at + n, h], want, 132, k, "bf16", 2)
        at += n
    assert (o[at:] == 7).all() and (l[at:] == 7).all()
    again = torch.empty_like(out)
    packed = torch.zeros(q.shape[0], 2 * Hq, d, dtype=q.dtype, device="cuda")    # strided queries, another workspace
    packed[:, :Hq] = q
    sa.kv4_attn(packed[:, :Hq], cache, table.cuda(), kv_len, again, cu_q=cu, window=window, sinks=sinks)
    assert torch.equal(again[:at], out[:at])


def test_kv4_attn_bad_tables_and_lengths_stay_inside(torch, sa):
    c = KV4[1]
    q, cache, table, kv_len, cu, _ = paged(torch, sa, c)
    table = table.cuda()
    out = torch.empty_like(q)

    def run(**kw):
        status = i32(torch, [0])
        a = dict(table=table, kv_len=kv_len, cu_q=cu)
        a.update(kw)
        sa.kv4_attn(q, cache, a["table"], a["kv_len"], out, cu_q=a["cu_q"], status=status)
        return sa.read_status(status)
    assert run() == 0
    assert run(table=torch.full_like(table, 1 << 30)) == sa.SA_ERR_INVALID_ARG
    assert run(table=torch.full_like(table, -1)) == sa.SA_ERR_INVALID_ARG
    assert run(kv_len=i32(torch, [1 << 30, -3, 1, 1])) == sa.SA_ERR_INVALID_ARG
    assert run(cu_q=i32(torch, [0, 1, 1 << 30, 2, 3])) == sa.SA_ERR_INVALID_ARG
    assert run(cu_q=i32(torch, [-4, 3, 1, 2, 4])) == sa.SA_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

ROPE = [
    (1, 4, 2, 128, 128, "half", "bf16", {}), (33, 4, 4, 128, 64, "interleaved", "bf16", {}),
    (2500, 2, 1, 128, 128, "half", "bf16", dict(scaling="yarn", factor=4.0, original_len=32768)),
    (2400, 3, 0, 64, 32, "interleaved", "fp32", dict(scaling="ntk", factor=4.0)),
    (17, 1, 1, 256, 64, "half", "fp32", dict(scaling="linear", factor=3.0)),
    (9, 2, 2, 80, 40, "half", "bf16", {}), (7, 2, 1, 66, 6, "interleaved", "bf16", {}), (5, 3, 2, 35, 2, "half", "fp32", {}),
    (11, 2, 1, 72, 72, "half", "bf16", {}),
]


def rope_check(got, x, pos, r, kw, layout, dtype, inverse):
    w, mag = S.rope_frequencies(r.rot_dim, **kw)
    want, size = S.rope(f64(x), pos, w, mag, layout, inverse)
    # angle 2^-24, sine and cosine 2^-23, magnitude 2^-24, two products and a sum 3 x 2^-24, all at most |x1| + |x2|
    # times 7 2^-24 < 2^-21; the last rounding
    tol = 2.0 ** -21 * size + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * (np.abs(want) + 2.0 ** -21 * size)
    assert (np.abs(f64(got) - want) <= tol).all(), (np.abs(f64(got) - want) - tol).max()
    rot = r.rot_dim
    assert np.array_equal(f64(got)[..., rot:], f64(x)[..., rot:])


@pytest.mark.parametrize("c", ROPE, ids=lambda c: "-".join(map(str, c[:7])))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(torch, sa, c, inverse):
    T, Hq, Hk, d, rot, layout, dtype, kw = c
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(T)
    packed = torch.randn(T, Hq + 2 * Hk, d, device="cuda", generator=g).to(dt)
    q, k = packed[:, :Hq], packed[:, Hq:Hq + Hk] if Hk else None
    pos = torch.randint(0, 1000000, (T,), device="cuda", generator=g).to(torch.int32)
    pos[0] = 2 ** 31 - 1 if T > 1 else 0
    r = sa.Rope(rot, layout=layout, **kw)
    qo, ko = torch.full((T, Hq, d), 7, dtype=dt, device="cuda"), torch.full((T, Hk, d), 7, dtype=dt, device="cuda") if Hk else None
    sa.rope(r, pos, q, qo, k, ko, inverse=inverse)
    p = pos.cpu().numpy()
    # a position of 2^31 times the rounded frequency of the 64-bit form is itself off by 2^31 2^-53 = 2^-22 rad
    p0, far = p.copy(), slice(1, None) if T > 1 else slice(None)
    rope_check(qo[far], q[far], p0[far], r, kw, layout, dtype, inverse)
    if Hk:
        rope_check(ko[far], k[far], p0[far], r, kw, layout, dtype, inverse)
    assert torch.isfinite(qo).all()
    # in place, within the packed rows; the values behind the keys stay
    rest = packed[:, Hq + Hk:].clone()
    sa.rope(r, pos, q, q, k, k, inverse=inverse)
    assert torch.equal(q, qo) and (not Hk or torch.equal(k, ko)) and torch.equal(packed[:, Hq + Hk:], rest)


def test_rope_batches_and_heads_first(torch, sa):
    B, N, H, d = 3, 21, 4, 64
    x = torch.randn(B, H, N, d, device="cuda")
    q = x.transpose(1, 2)                                  # BNSD memory as [B, N, H, d]
    pos = torch.randint(0, 5000, (B, N), device="cuda").to(torch.int32)
    r = sa.Rope(64, layout="half")
    out = torch.empty_like(x).transpose(1, 2)
    for p in (pos, pos[1]):
        sa.rope(r, p, q, out)
        rope_check(out, q, p.cpu().numpy(), r, {}, "half", "fp32", False)
    with pytest.raises(sa.SAError):                        # rows that overlap
        sa.rope(r, pos[0], x[0].transpose(0, 1), x[0, :1].expand(H, N, d).transpose(0, 1))


def test_rope_inverse_is_the_gradient(torch, sa):
    """<g, R x> = <R' g, x>, and the slope of <g, R x> along a direction by differences."""
    r = sa.Rope(48, layout="interleaved", scaling="yarn", factor=4.0, original_len=64)
    T, H, d = 13, 2, 64
    x, g, e = (torch.randn(T, H, d, device="cuda") for _ in range(3))
    pos = torch.arange(T, device="cuda").to(torch.int32) * 777
    y, gx, hi, lo = (torch.empty_like(x) for _ in range(4))
    sa.rope(r, pos, x, y)
    sa.rope(r, pos, g, gx, inverse=True)
    n = x.numel()
    # each side is a sum of n products of numbers with relative error below 2^-20
    bound = 2.0 ** -19 * float((g.double().abs() * (y.double().abs() + 1)).sum()) + n * 2.0 ** -24
    assert abs(float((g.double() * y.double()).sum() - (gx.double() * x.double()).sum())) <= bound
    sa.rope(r, pos, x + e, hi)                             # linear in x: a difference of any step
    sa.rope(r, pos, x - e, lo)
    slope = float((g.double() * (hi.double() - lo.double())).sum()) / 2
    size = float((g.double().abs() * (hi.double().abs() + lo.double().abs() + 1)).sum())
    assert abs(slope - float((gx.double() * e.double()).sum())) <= 2.0 ** -19 * size


# ---------------------------------------------------------------------------
# The cache plan
# ---------------------------------------------------------------------------

class Book:
    """A cache's books on the device, and one step of them."""

    def __init__(self, torch, sa, B, max_blocks, num, page, max_tokens):
        self.t, self.sa, self.page, self.tokens = torch, sa, page, max_tokens
        z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")   # noqa: E731
        self.table = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.free = torch.arange(num, device="cuda").flip(0).to(torch.int32)
        self.count, self.count_out, self.kv_len, self.new_len = i32(torch, [num]), z(1), z(B), z(B)
        self.cu, self.slots, self.pos, self.status = z(B + 1), z(max_tokens), z(max_tokens), z(1)

    def step(self, q_len):
        self.status.zero_()
        self.sa.cache_plan(self.kv_len, i32(self.t, q_len), self.table, self.free, self.count, self.page, self.new_len,
                           self.cu, self.slots, self.pos, self.count_out, status=self.status)
        return self.sa.read_status(self.status)

    def turn(self):
        self.kv_len, self.new_len = self.new_len, self.kv_len
        self.count, self.count_out = self.count_out, self.count


@pytest.mark.parametrize("B,page,max_new", [(1, 16, 3), (7, 16, 40), (64, 32, 1), (300, 64, 70), (1100, 128, 9), (5, 16, 5000)])
def test_cache_plan_steps(torch, sa, B, page, max_new):
    rng = np.random.default_rng(B)
    mb = -(-max_new // page) * 4 + 2
    num = B * mb // 2 + mb
    k = Book(torch, sa, B, mb, num, page, B * max_new + 3)
    lens, table, free = [0] * B, k.table.tolist(), k.free.tolist()
    done = 0
    for step in range(12):
        new = [-1 if rng.random() < 0.25 else int(rng.integers(0, max_new + 1)) for _ in range(B)]
        before = k.table.clone(), k.free.clone()
        code = k.step(new)
        try:
            if any(a > 0 and o + a > mb * page for a, o in zip(new, lens)):
                raise MemoryError
            r = S.plan(lens, new, table, free, page, k.tokens)
        except MemoryError:
            assert code == sa.SA_ERR_CAPACITY
            assert torch.equal(k.table, before[0]) and torch.equal(k.free, before[1])
            assert k.new_len.tolist() == lens and int(k.count_out) == len(free) and int(k.cu.abs().sum()) == 0
            assert (k.slots == -1).all() and (k.pos == 0).all()
            new = [-1 if i % 2 else 0 for i in range(B)]
            assert k.step(new) == 0
            r = S.plan(lens, new, table, free, page, k.tokens)
        assert k.status.item() == 0
        assert k.table.tolist() == r["table"] and k.free[:len(r["free"])].tolist() == r["free"]
        assert int(k.count_out) == len(r["free"]) and k.new_len.tolist() == r["new_len"] and k.cu.tolist() == r["cu_q"]
        assert k.slots.tolist() == r["slots"] and k.pos.tolist() == r["positions"]
        # the stack above its top keeps what the step took from it
        assert k.free[len(r["free"]):len(r["peak"])].tolist() == r["peak"][len(r["free"]):]
        lens, table, free = r["new_len"], r["table"], r["free"]
        k.turn()
        done += 1
    assert done == 12


def test_cache_plan_refuses_bad_lengths(torch, sa):
    k = Book(torch, sa, 4, 6, 20, 16, 50)
    assert k.step([3, -2, 0, 1]) == sa.SA_ERR_INVALID_ARG and k.cu.tolist() == [0] * 5
    assert k.step([3, 97, 0, 1]) == sa.SA_ERR_CAPACITY          # 6 blocks of 16
    assert k.step([20, 20, 10, 1]) == sa.SA_ERR_CAPACITY        # 50 token places
    k.kv_len[2] = -1
    assert k.step([1, 1, 1, 1]) == sa.SA_ERR_INVALID_ARG
    k.kv_len[2] = 0
    k.count[0] = 21
    assert k.step([1, 1, 1, 1]) == sa.SA_ERR_INVALID_ARG
    k.count[0] = 20
    k.free.fill_(1 << 20)                                       # pages that do not exist
    assert k.step([1, 1, 1, 1]) == sa.SA_ERR_INVALID_ARG and (k.slots == -1).all()


# ---------------------------------------------------------------------------
# The steps of a served model, together
# ---------------------------------------------------------------------------

def test_steps_together(torch, sa):
    """Prompts of several lengths, then tokens one by one, one request that ends and its place taken by another:
    plan, rope, append and attend, every step against the same from the 64-bit forms on the rows' values."""
    Hq, Hkv, d, page, B, window, sinks = 8, 2, 128, 16, 3, 40, 4
    rng = np.random.default_rng(0)
    g = torch.Generator(device="cuda").manual_seed(0)
    k = Book(torch, sa, B, 8, 20, page, 140)
    cache = sa.KV4Cache.allocate(20, Hkv, page, d)
    cache.pages.fill_(255)
    rope = sa.Rope(64, layout="half")
    ws = sa.workspace(sa.kv4_attn_workspace(cache, Hq), "cuda")
    past = [[np.zeros((0, Hkv, d))] * 3 for _ in range(B)]
    q_in, k_in = (torch.zeros(140, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
    v_in, out = torch.zeros_like(k_in), torch.zeros_like(q_in)
    lse = torch.zeros(140, Hq, device="cuda")
    for new in ([50, 7, 33], [1, 1, 1], [1, -1, 2], [1, 60, 1], [1, 1, 1], [0, 1, 1]):
        for t in (q_in, k_in, v_in):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        assert k.step(new) == 0
        qr, kr = torch.empty_like(q_in), torch.empty_like(k_in)
        sa.rope(rope, k.pos, q_in, qr, k_in, kr)
        sa.kv4_append(kr, v_in, k.slots, cache, status=k.status)
        sa.kv4_attn(qr, cache, k.table, k.new_len, out, lse, cu_q=k.cu, window=window, sinks=sinks, ws=ws, status=k.status)
        assert sa.read_status(k.status) == 0
        at, o, l, qn = 0, f64(out), f64(lse), f64(qr)
        for b, n in enumerate(new):
            if n < 0:
                past[b] = [x[:0] for x in past[b]]
                continue
            rows = slice(at, at + n)
            for i, x in enumerate((kr, v_in)):
                past[b][i] = np.concatenate([past[b][i], S.values(*S.quantise(f64(x[rows])))])
            past[b][2] = np.concatenate([past[b][2], 8 * np.repeat(S.quantise(f64(kr[rows]))[1], 32, -1)])
            for h in range(Hq):
                kh, vh, extra = (x[:, h * Hkv // Hq] for x in past[b])
                want = S.attention(qn[rows, h], kh, vh, window, sinks, extra=extra)
                check_rows(o[rows, h], l[rows, h], want, 132, len(past[b][0]), "bf16", 2)
            at += n
        k.turn()


def test_a_captured_step_runs_on_new_inputs(torch, sa):
    """One decode step (plan, rope, append, attend) as a graph gives what the calls give."""
    Hq, Hkv, d, page, B = 8, 2, 128, 16, 5
    lens = [3, 100, 31, 64, 0]

    def build():
        k = Book(torch, sa, B, 9, 40, page, B)
        big = Book(torch, sa, B, 9, 40, page, 200)
        assert big.step(lens) == 0
        k.table, k.free, k.count = big.table, big.free, big.count_out
        k.kv_len.copy_(i32(torch, lens))
        g = torch.Generator(device="cuda").manual_seed(3)
        cache = sa.KV4Cache.allocate(40, Hkv, page, d)
        x = torch.randn(200, Hkv, d, device="cuda", generator=g).to(torch.bfloat16)
        sa.kv4_append(x, x, big.slots, cache)
        q = torch.randn(B, Hq, d, device="cuda", generator=g).to(torch.bfloat16)
        kv = torch.randn(B, Hkv, d, device="cuda", generator=g).to(torch.bfloat16)
        return k, cache, q, kv, torch.zeros_like(q)
    rope = sa.Rope(128)
    ones = i32(torch, [1] * B)

    def step(k, cache, q, kv, out, ws):
        sa.cache_plan(k.kv_len, ones, k.table, k.free, k.count, page, k.new_len, k.cu, k.slots, k.pos, k.count_out)
        sa.rope(rope, k.pos, q, q, kv, kv)
        sa.kv4_append(kv, kv, k.slots, cache)
        sa.kv4_attn(q, cache, k.table, k.new_len, out, cu_q=k.cu, ws=ws)
        k.kv_len.copy_(k.new_len)
        k.count.copy_(k.count_out)
    a, b = build(), build()
    wa, wb = (sa.workspace(sa.kv4_attn_workspace(a[1], Hq), "cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*b, wb)
    for i in range(20):      # over page borders
        for s in (a, b):
            g = torch.Generator(device="cuda").manual_seed(i)
            s[2].copy_(torch.randn(s[2].shape, device="cuda", generator=g))
            s[3].copy_(torch.randn(s[3].shape, device="cuda", generator=g))
        step(*a, wa)
        graph.replay()
        assert torch.equal(a[4], b[4]) and torch.equal(a[1].pages, b[1].pages) and torch.equal(a[0].table, b[0].table)
        assert a[0].kv_len.tolist() == b[0].kv_len.tolist() == [n + i + 1 for n in lens]


# ---------------------------------------------------------------------------
# Few sinks before a far window
# ---------------------------------------------------------------------------

FEW_SINKS = [
    (1, 4, 2, 300, 600, 128, "bf16", 100, 1, None, None),
    (2, 4, 2, 260, 700, 64, "bf16", 64, 32, [260, 131], [700, 400]),
    (1, 3, 3, 400, 500, 128, "bf16", 150, 31, None, None),
    (1, 2, 1, 257, 520, 128, "bf16", 90, 33, None, None),
    (1, 2, 2, 513, 900, 64, "bf16", 200, 4, None, None),
    (1, 2, 1, 128, 355, 128, "bf16", 100, 7, None, None),     # the window starts on the second tile's border
    (1, 2, 1, 128, 354, 128, "bf16", 100, 7, None, None),     # and one key before it
    (2, 2, 2, 300, 300, 128, "bf16", 20, 16, [300, 5], [300, 290]),
]


@pytest.mark.parametrize("c", FEW_SINKS, ids=lambda c: "-".join(map(str, c[:9])))
@pytest.mark.parametrize("poison", [False, True])
def test_window_attn_few_sinks(torch, sa, c, poison):
    test_window_attn(torch, sa, c, 16, poison)


def test_window_attn_few_sinks_of_any_score(torch, sa):
    """Sinks far above and far below the window's scores, and at minus infinity."""
    q, k, v, _, _ = window_inputs(torch, (1, 2, 1, 200, 500, 64, "bf16", 70, 3, None, None))
    q.abs_()
    for size in (30.0, -30.0, -math.inf):
        k[:, :, :3] = size
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        sa.window_attn(q, k, v, out, lse, window=70, sinks=3, flags=16)
        o, l, qn, vn = (f64(t) for t in (out, lse, q, v))
        kn = f64(k) if size != -math.inf else np.where(np.isinf(f64(k)), -1e30, f64(k))
        for h in range(2):
            check_rows(o[0, h], l[0, h], S.attention(qn[0, h], kn[0, 0], vn[0, 0], 70, 3), 64, 500, "bf16", 1)


# ---------------------------------------------------------------------------
# Many units, and offsets past 32 bits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,d,window", [(16, 4, 128, 300), (11, 11, 64, 0)])
def test_window_attn_prefill_of_many_units(torch, sa, Hq, Hkv, d, window):
    """More units than SMs, so that blocks take a second one, in a padded batch."""
    c = (2, Hq, Hkv, 1700, 1900, d, "bf16", window, 5, [1700, 1333], [1900, 1334])
    q, k, v, nq, nk = window_inputs(torch, c)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    sa.window_attn(q, k, v, out, lse, window=window, sinks=5, q_len=i32(torch, nq), kv_len=i32(torch, nk), flags=16)
    o, l, qn, kn, vn = (f64(t) for t in (out, lse, q, k, v))
    for b in range(2):
        for h in (0, 1, Hq - 1):
            kh = h * Hkv // Hq
            want = S.attention(qn[b, h, :nq[b]], kn[b, kh, :nk[b]], vn[b, kh, :nk[b]], window, 5)
            check_rows(o[b, h, :nq[b]], l[b, h, :nq[b]], want, d, nk[b], "bf16", 1)
        assert (o[b, :, nq[b]:] == 7).all() and (l[b, :, nq[b]:] == 7).all()
    other = torch.empty_like(q)
    sa.window_attn(q, k, v, other, window=window, sinks=5, q_len=i32(torch, nq), kv_len=i32(torch, nk), flags=8)
    for b in range(2):
        # two kernels, each within 2 (2^-8 (1 + 2^-7) sum w |v| + 2^-8 |o|) of the truth, |v| < 6
        assert (out[b, :, :nq[b]].float() - other[b, :, :nq[b]].float()).abs().max() <= 4 * 2.0 ** -8 * 6


def test_offsets_past_32_bits(torch, sa):
    """K and V of more than 2^31 elements, and a cache of more than 2^32 bytes: the last heads and pages."""
    B, Hkv, Nk, d = 1, 8, 2 ** 21 + 100, 128
    k, v = (torch.zeros(B, Hkv, Nk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(0)
    tail = 700
    k[:, :, -tail:].copy_(torch.randn(B, Hkv, tail, d, device="cuda", generator=g))
    v[:, :, -tail:].copy_(torch.randn(B, Hkv, tail, d, device="cuda", generator=g))
    for Nq, flags in ((1, 8), (130, 16), (20, 1)):
        q = torch.randn(B, 2 * Hkv, Nq, d, device="cuda", generator=g).to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        sa.window_attn(q, k, v, out, lse, window=500, sinks=0, flags=flags)
        for h in (0, 2 * Hkv - 1):
            want = S.attention(f64(q[0, h]), f64(k[0, h // 2, -tail:]), f64(v[0, h // 2, -tail:]), 500, 0)
            check_rows(f64(out[0, h]), f64(lse[0, h]), want, d, tail, "bf16", 1)
    del k, v
    cache = sa.KV4Cache.allocate(30000, 8, 128, 128)
    assert cache.pages.numel() > 2 ** 32
    x = [torch.randn(200, 8, 128, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    slots = torch.cat([torch.arange(128) + 29999 * 128, torch.arange(72) + 29123 * 128]).to(torch.int32).cuda()
    sa.kv4_append(*x, slots, cache)
    back = [torch.empty_like(t) for t in x]
    sa.kv4_read(cache, slots, *back)
    vals = [S.values(*S.quantise(f64(t))) for t in x]
    for t, want in zip(back, vals):
        assert np.array_equal(f64(t), S.round_bf16(want))
    q = torch.randn(1, 8, 128, device="cuda", generator=g).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    sa.kv4_attn(q, cache, i32(torch, [[29999, 29123]]), i32(torch, [200]), out, lse, cu_q=i32(torch, [0, 1]))
    extra = 8 * np.repeat(S.quantise(f64(x[0]))[1], 32, -1)
    for h in range(8):
        want = S.attention(f64(q[:, h]), vals[0][:, h], vals[1][:, h], 0, 0, extra=extra[:, h])
        check_rows(f64(out[:, h]), f64(lse[:, h]), want, 132, 200, "bf16", 2)


def test_two_streams_with_workspaces_of_their_own(torch, sa):
    """Calls that overlap on the GPU do not share anything but their inputs."""
    c = (4, 8, 2, 1, 3001, 128, "bf16", 0, 0, None, None)
    q, k, v, _, _ = window_inputs(torch, c)
    want = torch.empty_like(q)
    sa.window_attn(q, k, v, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[torch.zeros_like(q) for _ in range(20)] for _ in streams]
    for i in range(20):
        for s, st in enumerate(streams):
            sa.window_attn(q, k, v, outs[s][i], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for s in outs for o in s)


# ---------------------------------------------------------------------------
# Refusals of the binding, and the ends of the queries' range
# ---------------------------------------------------------------------------

def test_the_binding_refuses(torch, sa):
    z = lambda *n, dt=torch.bfloat16, dev="cuda": torch.zeros(*n, dtype=dt, device=dev)   # noqa: E731
    q, k = z(2, 4, 3, 64), z(2, 2, 9, 64)
    i2 = i32(torch, [3, 3])

    def window(q=q, k=k, v=k, out=None, **kw):
        sa.window_attn(q, k, v, torch.zeros_like(q) if out is None else out, **kw)
    window()
    for kw, what in ((dict(k=k.float()), "k must be a"), (dict(k=k.cpu(), v=k.cpu()), "same CUDA device"), (dict(v=z(2, 2, 8, 64)), "shape"),
                     (dict(out=z(2, 4, 3, 128)), "out must have shape"), (dict(q=q.transpose(1, 2)), "contiguous|shape"),
                     (dict(q_len=i2.long()), "q_len"), (dict(q_len=i2[:1]), "q_len"), (dict(kv_len=i2.cpu()), "kv_len"),
                     (dict(lse=z(2, 4, 3)), "lse"), (dict(ws=z(512, dt=torch.uint8, dev="cpu")), "ws"),
                     (dict(q=q.half(), k=k.half(), v=k.half(), out=q.half()), "unsupported dtype")):
        with pytest.raises(ValueError, match=what):
            window(**kw)
    with pytest.raises(sa.SAError, match="WORKSPACE"):
        window(ws=z(256, dt=torch.uint8))
    with pytest.raises(sa.SAError, match="overlap"):
        window(out=q)
    with pytest.raises(sa.SAError, match="UNSUPPORTED"):
        sa.window_attn(*(z(1, 1, 2, 20) for _ in range(4)))       # 40 bytes a row
    cache = sa.KV4Cache.allocate(2, 2, 16, 64)
    row, slots = z(5, 2, 64), i32(torch, range(5))
    for args, what in (((row[:4], row, slots), "v must have shape"), ((row, row, slots[:4]), "slots"),
                       ((row.float(), row, slots), "k must be a"), ((z(5, 64, 2).transpose(1, 2), row, slots), "channels"),
                       ((row.cpu(), row, slots), "same CUDA device")):
        with pytest.raises(ValueError, match=what):
            sa.kv4_append(*args, cache)
    with pytest.raises(ValueError, match="k must"):
        sa.kv4_read(cache, slots, row[:, :1], row)
    with pytest.raises(sa.SAError, match="8-byte|strides"):
        sa.kv4_append(z(5, 2, 65)[..., 1:], row, slots, cache)
    with pytest.raises(ValueError, match="cu_q"):
        sa.kv4_attn(z(1, 2, 64), cache, i32(torch, [[0]]), i32(torch, [4]), z(1, 2, 64), cu_q=i32(torch, [0]))
    r = sa.Rope(64)
    for args, what in (((i32(torch, range(4)), row, row), "pos"), ((i32(torch, range(5)), row, row[:, :1]), "q_out"),
                       ((i32(torch, range(5)), row, row, row), "k and k_out")):
        with pytest.raises(ValueError, match=what):
            sa.rope(r, *args)
    with pytest.raises(sa.SAError, match="rot_dim"):
        sa.rope(sa.Rope(128), i32(torch, range(5)), row, torch.zeros_like(row))
    b = Book(torch, sa, 3, 4, 5, 16, 9)
    b.cu = b.cu[:3]
    with pytest.raises(ValueError, match="cu_q"):
        b.step([1, 1, 1])


@pytest.mark.parametrize("size,scale", [(0.0, 0.0), (0.0, 1e-30), (1e-36, 0.0), (1e30, 1e-30)])
def test_kv4_attn_queries_of_any_size(torch, sa, size, scale):
    """Zero, tiny and huge queries: the power of two that fp16 takes them at follows their size."""
    c = (8, 2, 128, 16, [100, 40], [1, 2], 30, 2)
    q, cache, table, kv_len, cu, vals = paged(torch, sa, c)
    q = (q.float() * size).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    sa.kv4_attn(q, cache, table.cuda(), kv_len, out, lse, cu_q=cu, window=30, sinks=2, scale=scale)
    o, l, qn, at = f64(out), f64(lse), f64(q), 0
    for b, (n, k) in enumerate(zip(c[5], c[4])):
        for h in range(8):
            kh, vh, extra = (x[:, h // 4] for x in vals[b])
            want = S.attention(qn[at:at + n, h], kh, vh, 30, 2, scale, extra=extra)
            check_rows(o[at:at + n, h], l[at:at + n, h], want, 132, k, "bf16", 2)
        at += n


# ---------------------------------------------------------------------------
# Workspaces that a call allocates, beside work queued on another stream
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("op", ["decode", "prefill", "kv4"])
def test_a_calls_own_workspace_is_not_shared_with_queued_work(torch, sa, op):
    """The current stream holds a long queue that still fills and reads a freed temporary of the workspace's
    size, while the call runs on a side stream without `ws`: both keep their results."""
    if op == "kv4":
        c = (32, 8, 128, 64, [3000], [1], 0, 0)
        q, cache, table, kv_len, cu, _ = paged(torch, sa, c)
        q, table = q[:1], table.cuda()
        n = sa.kv4_attn_workspace(cache, 32)

        def call(out, **kw):
            sa.kv4_attn(q, cache, table, kv_len, out, cu_q=cu, **kw)
    else:
        Nq, Nk, flags = (1, 3000, 8) if op == "decode" else (700, 900, 16)
        q, k, v, _, _ = window_inputs(torch, (2, 32, 8, Nq, Nk, 128, "bf16", 300, 5, None, None))
        n = sa.window_attn_workspace(q, k, v)

        def call(out, **kw):
            sa.window_attn(q, k, v, out, window=300, sinks=5, flags=flags, **kw)
    want, out = torch.empty_like(q), torch.empty_like(q)
    call(want)
    side, kept = torch.cuda.Stream(), torch.empty(n, dtype=torch.uint8, device="cuda")
    x = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for i in range(20):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        temp = torch.empty(n, dtype=torch.uint8, device="cuda")
        for _ in range(10):
            x = torch.clamp(x @ x, -1, 1)
            temp.fill_(i)
        kept.copy_(temp)
        del temp
        call(out, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and (kept == i).all()


# ---------------------------------------------------------------------------
# Waits that run out
# ---------------------------------------------------------------------------

def test_kv4_attn_timeout_path_reports_and_recovers(torch, sa):
    """A block whose copies are never reported whole: its wait runs out (after 10 ms here), it stops, and the status
    says so.  One sequence over 20,000 keys is 8 units of 8 + 313 tiles, 6 a block: block 1 begins the first kv head's
    unit, whose rows then stay as they were; block 2 is inside it, and its rows become NaN.  All others are untouched
    by it, and later calls run as before."""
    import ctypes
    c = (32, 8, 128, 64, [20000], [1], 0, 0)
    q, cache, table, kv_len, cu, _ = paged(torch, sa, c)
    q, table = q[:1], table.cuda()
    want, want_lse = torch.empty_like(q), torch.empty(1, 32, device="cuda")
    sa.kv4_attn(q, cache, table, kv_len, want, want_lse, cu_q=cu)
    ws = sa.workspace(sa.kv4_attn_workspace(cache, 32), "cuda")
    lib = sa.load()
    fn = lib.sa_kv4_attn_stalled
    fn.restype, fn.argtypes = ctypes.c_int32, [ctypes.c_int32] + lib.sa_kv4_attn.argtypes
    status = i32(torch, [0])
    for block in (1, 2, 2, 1):
        out, lse = torch.full_like(q, 7.0), torch.full((1, 32), 7.0, device="cuda")
        status.zero_()
        p = lambda t: ctypes.c_void_p(t.data_ptr())   # noqa: E731
        code = fn(block, p(q), 1, 32, ctypes.byref((ctypes.c_int64 * 2)(32 * 128, 128)), p(cu), 1, p(cache.pages),
                  ctypes.byref(cache.desc), p(table), table.shape[1], p(kv_len), 0, 0, 0.0, p(out), p(lse), p(status),
                  p(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert code == sa.SA_OK and sa.read_status(status) == sa.SA_ERR_TIMEOUT
        assert torch.equal(out[:, 4:], want[:, 4:]) and torch.equal(lse[:, 4:], want_lse[:, 4:])
        if block == 1:
            assert (out[:, :4] == 7).all() and (lse[:, :4] == 7).all()
        else:
            assert torch.isnan(out[:, :4]).all() and torch.isnan(lse[:, :4]).all()
        status.zero_()
        sa.kv4_attn(q, cache, table, kv_len, out, lse, cu_q=cu, ws=ws, status=status)
        assert sa.read_status(status) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


# ---------------------------------------------------------------------------
# Rotary positions at the ends of their range
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot,kw", [(64, {}), (128, dict(base=500000.0, scaling="yarn", factor=40.0, original_len=4096)),
                                    (32, dict(scaling="ntk", factor=4.0)), (2, dict(scaling="linear", factor=3.0))])
def test_rope_far_and_negative_positions(torch, sa, rot, kw, layout):
    """Against angles from 60 decimal digits, reduced exactly: within rope_check's 2^-21 of |x1| + |x2| everywhere
    (an angle is off by 2^-25 at most)."""
    p = [2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 2 ** 31 - 12345, -1, -77, 0, 5, -1000003, 2 ** 30 + 7, -2 ** 29 - 1, 2 ** 24 + 1]
    r = sa.Rope(rot, layout=layout, **kw)
    x = torch.randn(len(p), 3, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rot))
    y, back = torch.empty_like(x), torch.empty_like(x)
    pos = i32(torch, p)
    mag = S.rope_frequencies(rot, **kw)[1]
    angles = S.far_angles(p, S.rope_turns(rot, **kw))
    for inverse, got in ((False, y), (True, back)):
        sa.rope(r, pos, x, got, inverse=inverse)
        for t in range(len(p)):
            want, size = S.rope(f64(x[t:t + 1]), [1], angles[t], mag, layout, inverse)
            tol = 2.0 ** -21 * size + 2.0 ** -24 * (np.abs(want) + 2.0 ** -21 * size)
            assert (np.abs(f64(got[t:t + 1]) - want) <= tol).all(), p[t]


# ---------------------------------------------------------------------------
# The cache plan's refusals on the device
# ---------------------------------------------------------------------------

def test_cache_plan_says_the_same_of_a_step_with_two_faults(torch, sa):
    """A request with a bad length and one without room, in either order and far apart: always the bad length."""
    B = 600
    for bad, full in ((0, B - 1), (B - 1, 0), (3, 4), (4, 3)):
        new = [1] * B
        new[bad], new[full] = -2, 1000
        for _ in range(5):
            k = Book(torch, sa, B, 6, B, 16, B)
            assert k.step(new) == sa.SA_ERR_INVALID_ARG
            assert k.new_len.tolist() == [0] * B and int(k.count_out) == B and (k.slots == -1).all()


@pytest.mark.parametrize("where", ["free", "released", "deep in a released row", "filled up"])
@pytest.mark.parametrize("page_id", [-1, 40, 1 << 30])
@pytest.mark.parametrize("tokens", [200, 40000])     # 8 and 40 blocks of threads
def test_cache_plan_with_a_page_outside_the_cache_changes_nothing(torch, sa, where, page_id, tokens):
    k = Book(torch, sa, 5, 12, 40, 16, tokens)
    assert k.step([33, 130, 16, 5, 0]) == 0
    k.turn()
    spare = k.table.clone()
    k.table[0, 3], k.table[3, 1], k.free[30] = 1 << 20, -5, 1 << 20    # entries that the step does not come to
    new = [1, -1, 20, 2, 3]
    if where == "free":         # 9 pages come back, 3 are taken: the stack's own are not; so nobody ends
        new[1] = 0
        k.free[int(k.count) - 2] = page_id
    elif where == "released":
        k.table[1, 0] = page_id
    elif where == "deep in a released row":
        k.table[1, 7] = page_id
    else:
        k.table[3, 0] = page_id
    before = [t.clone() for t in (k.table, k.free, k.kv_len, k.count)]
    for t in (k.new_len, k.cu, k.slots, k.pos, k.count_out):
        t.fill_(77)
    assert k.step(new) == sa.SA_ERR_INVALID_ARG
    for t, want in zip((k.table, k.free, k.new_len, k.count_out), before):
        assert torch.equal(t, want)
    assert (k.cu == 0).all() and (k.slots == -1).all() and (k.pos == 0).all()
    # with the page put right the same step goes through, whatever stands in the entries that it does not come to
    keep = (0, 3), (3, 1)
    lens, free = k.kv_len.tolist(), k.free[:int(k.count)].tolist()
    if where == "free":
        k.free[int(k.count) - 2] = free[-2] = 40 - 1 - (int(k.count) - 2)
    else:
        k.table.copy_(spare)
        for b, i in keep:
            k.table[b, i] = before[0][b, i]
    rows = k.table.tolist()
    assert k.step(new) == 0
    r = S.plan(lens, new, rows, free, 16, k.tokens)
    assert k.table.tolist() == r["table"] and k.free[:len(r["free"])].tolist() == r["free"]
    assert k.slots.tolist() == r["slots"] and k.new_len.tolist() == r["new_len"]


# ---------------------------------------------------------------------------
# The kernels' forms for large calls
# ---------------------------------------------------------------------------

LARGE_SIMT = [     # 592 tiles of 16 rows and more: two warps a tile
    (2, 8, 4, 600, 640, 64, "fp32", 100, 3, [600, 417], [640, 417]),
    (1, 16, 4, 595, 595, 128, "fp32", 0, 0, None, None),
    (3, 8, 8, 400, 400, 16, "fp32", 33, 9, [400, 1, 0], [390, 400, 77]),
    (1, 16, 2, 600, 633, 256, "fp32", 64, 1, None, None),
    (2, 8, 2, 600, 600, 96, "bf16", 70, 2, [600, 599], [600, 600]),
]


@pytest.mark.parametrize("c", LARGE_SIMT, ids=lambda c: "-".join(map(str, c[:9])))
@pytest.mark.parametrize("poison", [False, True])
def test_window_attn_many_rows_on_the_cuda_cores(torch, sa, c, poison):
    test_window_attn(torch, sa, c, 0, poison)


@pytest.mark.parametrize("c", [(1, 4, 1, 1, 20000, 128, "bf16", 0, 0, None, None),
                               (4, 8, 2, 1, 3001, 128, "bf16", 0, 0, None, [3001, 1, 2999, 0]),
                               (1, 8, 1, 4, 9000, 64, "bf16", 0, 0, None, None),
                               (1, 16, 1, 3, 12000, 128, "bf16", 9000, 500, None, None)],
                         ids=lambda c: "-".join(map(str, c[:9])))
def test_window_attn_few_rows_over_many_keys(torch, sa, c):
    """Units of more parts than one round of the join takes."""
    test_window_attn(torch, sa, c, 8, False)


@pytest.mark.parametrize("c", [(4, 1, 128, 64, [20000], [1], 0, 0), (4, 1, 64, 16, [20011], [1], 0, 0),
                               (4, 1, 128, 64, [20000], [4], 0, 0), (8, 2, 64, 128, [21003], [2], 15000, 300),
                               (8, 2, 128, 64, [1, 30000, 1, 2], [1, 1, 1, 1], 0, 0),
                               (8, 2, 64, 32, [30000, 3, 1, 900], [1, 3, 1, 5], 0, 0)],
                         ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_kv4_attn_many_keys(torch, sa, c):
    test_kv4_attn(torch, sa, c)


@pytest.mark.parametrize("H,d,T", [(8, 128, 700), (8, 128, 1001), (8, 128, 2000), (5, 128, 2000), (5, 64, 2000), (8, 64, 1999)])
def test_kv4_rows_of_a_prompt(torch, sa, H, d, T):
    """Warps that walk 2, 3 and 4 blocks of heads, with and without a tail; runs of tokens, single ones and left out ones."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    page = 32
    pages = T // page + 5
    k, v = (torch.randn(T, H, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    k[3, H - 1, :32], v[T - 1, H - 1, 5] = 0, math.nan
    slots = torch.arange(T, device="cuda", dtype=torch.int32) + 5        # a run from an odd place
    some = torch.randperm(T, device="cuda", generator=g)[:T // 3]
    slots[some] = slots[some[torch.randperm(len(some), device="cuda", generator=g)]]
    slots[some[:4]] = -1
    cache = sa.KV4Cache.allocate(pages, H, page, d)
    cache.pages.fill_(0x5A)
    status = i32(torch, [0])
    sa.kv4_append(k, v, slots, cache, status=status)
    want = np.full(cache.pages.shape, 0x5A, np.uint8)
    sl = slots.cpu().numpy()
    (kc, ks), (vc, vs) = S.quantise(f64(k)), S.quantise(f64(v))
    for t in range(T):
        for h in range(H):
            if sl[t] >= 0:
                S.store(want, sl[t], h, kc[t, h], ks[t, h], vc[t, h], vs[t, h])
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    ko, vo = (torch.full((T, H, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sa.kv4_read(cache, slots, ko, vo, status=status)
    assert sa.read_status(status) == 0
    for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
        x = S.values(c, s)
        x = S.round_bf16(np.nan_to_num(x, nan=0)) + np.where(np.isnan(x), np.nan, 0)
        x[sl < 0] = 9
        assert np.array_equal(f64(got), x, equal_nan=True)


@pytest.mark.parametrize("B,page,max_new", [(5000, 16, 5), (18000, 32, 2)])
def test_cache_plan_of_many_requests(torch, sa, B, page, max_new):
    test_cache_plan_steps(torch, sa, B, page, max_new)


@pytest.mark.parametrize("c", [(2400, 2, 1, 66, 6, "interleaved", "bf16", {}), (2401, 3, 2, 35, 2, "half", "fp32", {}),
                               (2403, 1, 1, 72, 72, "half", "bf16", {})], ids=lambda c: "-".join(map(str, c[:7])))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_of_many_tokens_without_aligned_vectors(torch, sa, c, inverse):
    test_rope(torch, sa, c, inverse)


@pytest.mark.parametrize("op", ["window", "kv4"])
def test_a_captured_call_on_a_forked_stream_has_a_workspace_of_its_own(torch, sa, op):
    """In a captured graph, calls without `ws` run on a forked stream beside work of the capturing one, which
    allocates and frees blocks of the workspace's size in between; every replay gives what the calls give."""
    if op == "kv4":
        q, cache, table, kv_len, cu, _ = paged(torch, sa, (32, 8, 128, 64, [3000], [1], 0, 0))
        q, table = q[:1], table.cuda()
        n = sa.kv4_attn_workspace(cache, 32)

        def call(out, **kw):
            sa.kv4_attn(q, cache, table, kv_len, out, cu_q=cu, **kw)
    else:
        q, k, v, _, _ = window_inputs(torch, (2, 32, 8, 1, 3000, 128, "bf16", 0, 0, None, None))
        n = sa.window_attn_workspace(q, k, v)

        def call(out, **kw):
            sa.window_attn(q, k, v, out, flags=8, **kw)
    want, outs = torch.empty_like(q), [torch.empty_like(q) for _ in range(4)]
    call(want)
    kept = torch.empty(4, n, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for i, out in enumerate(outs):
            call(out, stream=side)
            temp = torch.full((n,), i, dtype=torch.uint8, device="cuda")
            temp += 10
            kept[i].copy_(temp)
            del temp
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(10):
        kept.zero_()
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)
        assert all((kept[i] == 10 + i).all() for i in range(4))

"""The serving operators without a GPU: argument refusals of the C ABI and of
the binding, the rotary frequencies, and the plain forms themselves."""

import ctypes
import math
import os
from fractions import Fraction

import numpy as np
import pytest

from long_context_mean_b200 import sa
from oracle import serving as S

BAD, UNSUP, WS = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED, sa.SA_ERR_WORKSPACE
NULL = ctypes.c_void_p(None)


def at(mib):
    """A made-up 256-byte aligned device address; nothing is read from it."""
    return ctypes.c_void_p(0x100000000 + (mib << 20))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sa.LIB_PATH):
        from long_context_mean_b200 import build
        build.build()
    return sa.load()


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

def window_code(lib, shape=(2, 4, 2, 5, 70, 128, sa.SA_BF16), window=8, sinks=1, scale=0.0, ws_bytes=None, flags=0, **kw):
    s = sa.WindowShape(*shape, 0)
    p = dict(q=at(0), k=at(64), v=at(128), out=at(192), lse=at(256), ws=at(320))
    p.update(kw)
    n = lib.sa_window_attn_workspace(ctypes.byref(s)) if ws_bytes is None else ws_bytes
    return lib.sa_window_attn(p["q"], p["k"], p["v"], ctypes.byref(s), window, sinks, NULL, NULL, scale, p["out"],
                              p["lse"], NULL, p["ws"], n, flags, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(shape=(0, 4, 2, 5, 70, 128, 0)), BAD), (dict(shape=(2, 4, 3, 5, 70, 128, 0)), BAD),
    (dict(shape=(2, 4, 2, 5, 70, 128, 7)), BAD), (dict(shape=(2, 4, 2, 5, 70, 36, 0)), UNSUP),
    (dict(shape=(2, 4, 2, 5, 70, 264, 1)), UNSUP), (dict(shape=(1, 64, 2, 1 << 26, 70, 128, 0)), UNSUP),
    (dict(shape=(1, 4, 2, 1 << 40, 70, 128, 0)), UNSUP),
    (dict(window=-1), BAD), (dict(sinks=-1), BAD), (dict(window=1 << 33), UNSUP), (dict(scale=-1.0), BAD),
    (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(q=NULL), BAD), (dict(out=NULL), BAD),
    (dict(q=ctypes.c_void_p(0x100000008)), BAD), (dict(out=at(0)), BAD), (dict(out=at(64)), BAD),
    (dict(lse=at(192)), BAD), (dict(ws=NULL), WS), (dict(ws_bytes=100), WS),
    (dict(ws=ctypes.c_void_p(0x100000080)), WS), (dict(flags=2), BAD),
    (dict(flags=sa.SA_FLAG_FORCE_PREFILL, shape=(2, 4, 2, 5, 70, 128, 1)), UNSUP)])
def test_window_attn_refusals(lib, kw, code):
    assert window_code(lib, **kw) == code


def kv4(pages=8, H=2, page=16, d=128):
    return sa.KV4Desc(pages, H, page, d)


@pytest.mark.parametrize("desc,size", [(kv4(), 8 * 2 * 18 * 128), (kv4(3, 5, 128, 64), 3 * 5 * 8 * 18 * 64),
                                       (kv4(0), 0), (kv4(H=0), 0), (kv4(page=48), 0), (kv4(page=8), 0),
                                       (kv4(d=96), 0), (kv4(pages=1 << 28), 0)])
def test_kv4_bytes(lib, desc, size):
    assert lib.sa_kv4_bytes(ctypes.byref(desc)) == size
    assert (lib.sa_kv4_attn_workspace(ctypes.byref(desc), desc.Hkv) > 0) == (size > 0)


def test_kv4_row_refusals(lib):
    I2 = ctypes.c_int64 * 2

    def append(k=at(0), v=at(64), T=9, ks=(256, 128), vs=(256, 128), slots=at(128), desc=kv4(), cache=at(192)):
        return lib.sa_kv4_append(k, v, T, ctypes.byref(I2(*ks)), ctypes.byref(I2(*vs)), slots, ctypes.byref(desc), cache,
                                 NULL, NULL)

    def read(k=at(0), v=at(64), T=9, slots=at(128), desc=kv4(), cache=at(192)):
        return lib.sa_kv4_read(cache, ctypes.byref(desc), slots, T, k, v, NULL, NULL)
    for kw, code in ((dict(k=NULL), BAD), (dict(T=-1), BAD), (dict(ks=(258, 128)), BAD), (dict(vs=(-256, 128)), BAD),
                     (dict(k=ctypes.c_void_p(0x100000004)), BAD), (dict(cache=at(0)), BAD),
                     (dict(desc=kv4(page=20)), UNSUP), (dict(slots=NULL), BAD), (dict(T=0, slots=NULL), 0)):
        assert append(**kw) == code, kw
    for kw, code in ((dict(k=NULL), BAD), (dict(T=-1), BAD), (dict(v=at(0)), BAD), (dict(cache=at(64)), BAD),
                     (dict(k=ctypes.c_void_p(0x100000008)), BAD), (dict(T=0), 0)):
        assert read(**kw) == code, kw


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(T=1 << 29, Hq=8), UNSUP), (dict(Hq=3), BAD), (dict(Hq=0), BAD), (dict(mb=0), BAD), (dict(mb=1 << 40), UNSUP),
    (dict(q=NULL), BAD), (dict(cu=NULL), BAD), (dict(table=NULL), BAD), (dict(kv_len=NULL), BAD),
    (dict(qs=(516, 128)), BAD), (dict(q=ctypes.c_void_p(0x100000008)), BAD), (dict(out=at(0)), BAD),
    (dict(out=at(64)), BAD), (dict(lse=at(128)), BAD), (dict(ws=NULL), WS), (dict(n=64), WS),
    (dict(window=-3), BAD), (dict(scale=math.nan), BAD), (dict(desc=kv4(d=80)), UNSUP),
    (dict(T=0, q=NULL), 0), (dict(B=0), 0)])
def test_kv4_attn_refusals(lib, kw, code):
    a = dict(q=at(0), T=6, Hq=4, qs=(512, 128), cu=at(32), B=2, cache=at(64), desc=kv4(), table=at(96), mb=4,
             kv_len=at(100), window=0, sinks=0, scale=0.0, out=at(128), lse=at(160), ws=at(192), n=None)
    a.update(kw)
    n = lib.sa_kv4_attn_workspace(ctypes.byref(kv4()), 4) if a["n"] is None else a["n"]
    got = lib.sa_kv4_attn(a["q"], a["T"], a["Hq"], ctypes.byref((ctypes.c_int64 * 2)(*a["qs"])), a["cu"], a["B"],
                          a["cache"], ctypes.byref(a["desc"]), a["table"], a["mb"], a["kv_len"], a["window"], a["sinks"],
                          a["scale"], a["out"], a["lse"], NULL, a["ws"], n, NULL)
    assert got == code


@pytest.mark.parametrize("kw,code", [
    (dict(rot=3), BAD), (dict(rot=0), BAD), (dict(rot=130), BAD), (dict(layout=2), BAD), (dict(dtype=5), BAD),
    (dict(inverse=2), BAD), (dict(mag=math.inf), BAD), (dict(B=-1), BAD), (dict(d=2048), UNSUP),
    (dict(q=NULL), BAD), (dict(pos=NULL), BAD), (dict(k_out=NULL), BAD), (dict(q_out=at(64)), BAD),
    (dict(q_out=ctypes.c_void_p(0x100000040)), BAD), (dict(qo=(0, 64, 128)), BAD),        # rows overlap
    (dict(q_out=at(0), qo=(0, 1024, 128)), BAD),                                          # in place, other strides
    (dict(qs=(0, -512, 128)), BAD), (dict(N=0, q=NULL), 0)])
def test_rope_refusals(lib, kw, code):
    a = dict(B=1, N=7, Hq=4, Hk=2, d=128, rot=64, layout=0, dtype=sa.SA_BF16, inverse=0, mag=1.0, q=at(0), q_out=at(32),
             k=at(64), k_out=at(96), pos=at(128), qs=(0, 512, 128), qo=(0, 512, 128), ks=(0, 256, 128), ko=(0, 256, 128))
    a.update(kw)
    I3 = ctypes.c_int64 * 3
    desc = sa.RopeDesc(a["B"], a["N"], a["Hq"], a["Hk"], a["d"], I3(*a["qs"]), I3(*a["qo"]), I3(*a["ks"]), I3(*a["ko"]), 0,
                       a["rot"], a["layout"], a["dtype"], a["inverse"], a["mag"], 0)
    assert lib.sa_rope(a["q"], a["q_out"], a["k"], a["k_out"], a["pos"], at(160), ctypes.byref(desc), NULL) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), BAD), (dict(mb=0), BAD), (dict(pages=0), BAD), (dict(tokens=-1), BAD), (dict(page=24), UNSUP),
    (dict(B=20000), UNSUP), (dict(pages=1 << 30), UNSUP), (dict(kv=NULL), BAD), (dict(slots=NULL), BAD),
    (dict(new=at(0)), BAD), (dict(fout=at(4)), BAD), (dict(pos=at(6)), BAD), (dict(cu=at(7)), BAD)])
def test_cache_plan_refusals(lib, kw, code):
    a = dict(kv=at(0), ql=at(1), B=5, mb=9, pages=40, tokens=30, page=16, table=at(2), free=at(3), fin=at(4), fout=at(5),
             new=at(6), cu=at(9), slots=at(7), pos=at(10))
    a.update(kw)
    desc = sa.PlanDesc(a["B"], a["mb"], a["pages"], a["tokens"], a["page"], 0)
    assert lib.sa_cache_plan(a["kv"], a["ql"], ctypes.byref(desc), a["table"], a["free"], a["fin"], a["fout"], a["new"],
                             a["cu"], a["slots"], a["pos"], NULL, NULL) == code


def test_the_binding_refuses_what_is_not_on_a_gpu_or_of_another_type(lib):
    import torch
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        sa.window_attn(q, q, q, torch.zeros_like(q))
    with pytest.raises(ValueError, match="uint8"):
        sa.KV4Cache(torch.zeros(2, 2, 1, 18 * 64), 16, 64)
    with pytest.raises(ValueError, match="layout"):
        sa.Rope(64, layout="other", device="cpu")
    with pytest.raises(ValueError, match="scaling"):
        sa.Rope(64, scaling="other", device="cpu")


# ---------------------------------------------------------------------------
# Rotary frequencies
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rot,kw", [(128, {}), (2, dict(scaling="ntk", factor=8.0)), (64, dict(scaling="linear", factor=3.0)),
                                    (96, dict(scaling="ntk", factor=4.0)),
                                    (128, dict(scaling="yarn", factor=4.0, original_len=32768)),
                                    (64, dict(base=500000.0, scaling="yarn", factor=40.0, original_len=4096))])
def test_frequencies_are_the_formula(lib, rot, kw):
    r = sa.Rope(rot, device="cpu", **kw)
    w, mag = S.rope_frequencies(rot, **kw)
    got = np.array([Fraction(int(np.uint64(x)), 1 << 64) for x in r.host_freqs.numpy().view(np.uint64)])
    # a few roundings of 64-bit floats (pow and log are good to an ulp or two), and half a unit of 2^-64 turns
    for f, x in zip(got, w):
        assert abs(float(f) * 2 * math.pi - x) <= 32 * 2.0 ** -53 * x + 2 * math.pi * 2.0 ** -65
    assert r.magnitude == np.float32(mag)


@pytest.mark.parametrize("kw", [dict(base=1.0), dict(base=math.inf), dict(scaling="linear", factor=0.5),
                                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_len=9, beta_slow=0.0),
                                dict(scaling="ntk", factor=math.nan)])
def test_bad_frequencies_are_refused(lib, kw):
    with pytest.raises(sa.SAError):
        sa.Rope(64, device="cpu", **kw)


@pytest.mark.parametrize("rot", [0, 3, -2, 2000])
def test_bad_rot_dim_is_refused(lib, rot):
    with pytest.raises(sa.SAError):
        sa.Rope(rot, device="cpu")


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n_q,n_k,window,sinks", [(1, 9, 4, 1), (5, 5, 0, 0), (7, 4, 2, 0), (6, 11, 3, 20), (3, 0, 5, 1)])
def test_plain_attention_is_the_definition(n_q, n_k, window, sinks):
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((n_q, 4)), rng.standard_normal((n_k, 4)), rng.standard_normal((n_k, 4))
    out, lse, *_ = S.attention(q, k, v, window, sinks)
    for i in range(n_q):
        p = n_k - n_q + i
        keys = [j for j in range(n_k) if j <= p and (window == 0 or p - j < window or j < sinks)]
        e = [math.exp(float(q[i] @ k[j]) / 2) for j in keys]
        want = sum((x * v[j] for x, j in zip(e, keys)), np.zeros(4)) / (sum(e) or 1)
        assert np.allclose(out[i], want, rtol=1e-12, atol=1e-12)
        assert lse[i] == -math.inf if not keys else abs(lse[i] - math.log(sum(e))) < 1e-12


def test_plain_rounding_and_codes():
    import torch
    x = np.random.default_rng(2).standard_normal(4000) * np.exp(np.random.default_rng(3).uniform(-95, 80, 4000))
    assert np.array_equal(S.round_bf16(x), torch.from_numpy(x).to(torch.bfloat16).double().numpy())
    c, s = S.quantise(S.round_bf16(x).reshape(-1, 160))
    assert np.abs(c).max() == 7 and (np.abs(c.reshape(-1, 5, 32)).max(-1) == 7).all()
    big = np.abs(x.reshape(-1, 5, 32)).max(-1, keepdims=True)
    assert (np.abs(S.values(c, s).reshape(-1, 5, 32) - x.reshape(-1, 5, 32)) <= big / 7 * (0.5 + 7 * 2 ** -8)).all()


def test_plain_plan_keeps_every_page_once():
    rng = np.random.default_rng(4)
    page, B, mb, num = 16, 12, 20, 90
    lens, table, free = [0] * B, [[-1] * mb for _ in range(B)], list(range(num))
    for _ in range(40):
        new = [-1 if rng.random() < 0.2 else int(rng.integers(0, 40)) for _ in range(B)]
        try:
            r = S.plan(lens, new, table, free, page, 600)
        except MemoryError:
            new = [-1] * B
            r = S.plan(lens, new, table, free, page, 600)
        lens, table, free = r["new_len"], r["table"], r["free"]
        held = [t for row, n in zip(table, lens) for t in row[:-(-n // page)]]
        assert sorted(held + free) == list(range(num))
        live = [s for s in r["slots"] if s >= 0]
        assert len(set(live)) == len(live)


# ---------------------------------------------------------------------------
# Workspaces of a call
# ---------------------------------------------------------------------------

def test_a_calls_own_workspace_comes_from_the_stream_that_it_runs_on(monkeypatch):
    """A block of the current stream's pool may still be in use by work queued there while `stream` writes it."""
    import contextlib
    from types import SimpleNamespace

    import torch
    current = ["current"]

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(sa, "workspace", lambda n, device: SimpleNamespace(n=n, pool=current[-1]))
    t = SimpleNamespace(is_cuda=True, device="cuda:0")
    ws = sa._call_workspace(512, t, "q", "side")
    assert (ws.n, ws.pool, current) == (512, "side", ["current"])
    assert sa._call_workspace(512, t, "q", None).pool == "current"


# ---------------------------------------------------------------------------
# Rotary frequencies at far positions
# ---------------------------------------------------------------------------

FREQUENCIES = [(128, {}), (256, dict(base=500000.0)), (2, dict(scaling="ntk", factor=8.0)), (96, dict(scaling="ntk", factor=4.0)),
               (64, dict(scaling="linear", factor=3.0)), (128, dict(scaling="yarn", factor=4.0, original_len=32768)),
               (64, dict(base=1000000.0, scaling="yarn", factor=40.0, original_len=4096))]


@pytest.mark.parametrize("rot,kw", FREQUENCIES)
def test_frequencies_to_a_few_units(lib, rot, kw):
    """Against 60 decimal digits, in units u = 2^-64 turns.  Relative to w, in roundings of 2^-64 of a 64-bit
    mantissa: the exponent |ln w|, the power 2, two pi and its division 2; a linear factor 1; ntk's base ln f r / (r - 2) + 3;
    yarn's ramp and blend 6; and half a unit at the end."""
    r = sa.Rope(rot, device="cpu", **kw)
    f = kw.get("factor", 1.0)
    for got, t in zip(r.host_freqs.numpy().view(np.uint64), S.rope_turns(rot, **kw)):
        w = float(t) * 2 * math.pi
        bound = 0.5 + float(t) * (abs(math.log(w)) + 14 + 2 * math.log(f))
        assert abs(int(got) - t * 2 ** 64) <= bound < 4
    # an angle at 2^31 positions is then off by less than 1e-8 rad; 53 bits of mantissa leave 50 units and more
    assert 2 ** 31 * 4 * 2.0 ** -64 * 2 * math.pi < 1e-8


def test_far_angles_are_those_of_small_positions():
    w, _ = S.rope_frequencies(64)
    pos = np.array([0, 1, 17, -17, 4000])
    got, want = S.far_angles(pos, S.rope_turns(64)), pos[:, None] * w
    assert np.abs(np.exp(1j * got) - np.exp(1j * want)).max() < 4000 * 2.0 ** -50


# ---------------------------------------------------------------------------
# A scale below 32 bits' range
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("scale", [1e-50, -1e-50, 5e-324])
def test_a_scale_that_32_bits_round_to_zero_is_not_the_default(lib, scale):
    """0 means 1 / sqrt(d); a scale that is not 0 never does."""
    import torch
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="scale"):
        sa.window_attn(q, q, q, torch.zeros_like(q), scale=scale, ws=ws)
    cache = sa.KV4Cache.allocate(2, 2, 16, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="scale"):
        sa.kv4_attn(q[0], cache, i[None], i[:1], torch.zeros_like(q[0]), cu_q=i, scale=scale, ws=ws)
    for good in (0.0, -0.0, 2e-45, 0.5):      # these come as far as the tensors' device
        with pytest.raises(ValueError, match="CUDA device"):
            sa.window_attn(q, q, q, torch.zeros_like(q), scale=good, ws=ws)

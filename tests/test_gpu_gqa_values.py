"""What values can do to the grouped-query attention calls: NaN and infinities
in keys, queries and values, one key that outweighs thousands, magnitudes at
the ends of the types, FP8 scales far apart; and calls from two host threads.

Bounds are those of gqa_util; where a value is not finite it has to be the
same one, sign and all."""

import threading

import numpy as np
import pytest
import torch

from gqa_util import ACT, Paged, check_out, f64
from oracle import gqa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_gated_b200 import build
    build.build()
    import long_context_sparse_gated_b200 as m
    return m


def _params(lib, act="bf16", kv="act", **kw):
    return lib.make_gqa_params(act_fmt=lib.ACT_BF16 if act == "bf16" else lib.ACT_F16,
                               kv_fmt=lib.KV_ACT if kv == "act" else lib.KV_FP8, **kw)


def _randn(shape, act, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(ACT[act])


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(lens):
    return _i32([0] + list(np.cumsum(lens)))


def _same(got, want, mag, zmag, act, what=""):
    """check_out, and infinities and NaN exactly as wanted."""
    got = f64(got)
    odd = ~np.isfinite(want)
    np.testing.assert_array_equal(got[odd], want[odd], err_msg=what)
    check_out(got[~odd], want[~odd], mag[~odd], zmag, act, what)


def _prompt(lib, q, k, v, nq, nk, act, scale, window=0, sink=None):
    """gqa_prompt_attn of CPU rows; the output on the CPU."""
    H, d = q.shape[1:]
    p = _params(lib, act, B=len(nq), n_heads=H, n_kv_heads=k.shape[1], d=d, window=window, softmax_scale=scale)
    out, err = torch.full(q.shape, 9.0, device="cuda").to(q.dtype), torch.zeros(4, dtype=torch.int32, device="cuda")
    lib.gqa_prompt_attn(p, q.cuda(), k.cuda(), v.cuda(), _starts(nq), _starts(nk), out,
                        sink=None if sink is None else sink.cuda(), err=err)
    assert int(err[0]) == 0
    return out.cpu()


def _decode(lib, q, cache, table, lens, T, act, kv, G, page, scale, window=0, sink=None):
    H, d = q.shape[1:]
    p = _params(lib, act, kv, B=len(lens), n_heads=H, n_kv_heads=G, d=d, page=page, window=window, softmax_scale=scale)
    n_max = max(lens)
    ws = torch.full((max(16, lib.gqa_decode_attn_workspace_bytes(p, T, n_max)),), 255, dtype=torch.uint8, device="cuda")
    out, err = torch.full(q.shape, 9.0, device="cuda").to(q.dtype), torch.zeros(4, dtype=torch.int32, device="cuda")
    lib.gqa_decode_attn(p, q.cuda(), cache, table, _i32(lens), T, n_max, out, ws, sink=None if sink is None else sink.cuda(), err=err)
    assert int(err[0]) == 0
    return out.cpu()


# ---- NaN in keys and queries ---------------------------------------------------

@pytest.mark.parametrize("act,d", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
def test_prompt_nan_in_a_key_at_every_column(lib, act, d):
    """The last four queries of 300 keys see two tiles of 128 whole and a part
    of a third; a NaN in any one key makes every row that sees it NaN, and the
    heads of the other KV head stay exact."""
    cols = list(range(256)) + [256, 270, 298]
    n, m, H, G = 4, 300, 2, 2
    B = len(cols)
    q, k, v = _randn((n * B, H, d), act, 1), _randn((m * B, G, d), act, 2), _randn((m * B, G, d), act, 3)
    bad = k.clone()
    for b, c in enumerate(cols):
        bad[b * m + c, 0, (7 * c) % d] = float("nan")
    out = _prompt(lib, q, bad, v, [n] * B, [m] * B, act, d ** -0.5)
    for b, c in enumerate(cols):
        t = np.arange(m - n, m)
        want, mag, zmag = gqa.attend(f64(q[b * n:(b + 1) * n]), f64(k[b * m:(b + 1) * m]), f64(v[b * m:(b + 1) * m]), t, d ** -0.5)
        want[t >= c, 0] = np.nan
        _same(out[b * n:(b + 1) * n], want, mag, zmag, act, f"key {c}")


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_prompt_infinite_logit_is_not_hidden(lib, act):
    """A logit of +infinity makes its rows NaN, wherever the key lies."""
    n, m, d = 2, 300, 64
    cols = list(range(0, 298, 3))
    B = len(cols)
    q, k, v = _randn((n * B, 1, d), act, 1), _randn((m * B, 1, d), act, 2), _randn((m * B, 1, d), act, 3)
    q[:, 0, 5] = 1.0
    for b, c in enumerate(cols):
        k[b * m + c, 0, 5] = float("inf")
    assert _prompt(lib, q, k, v, [n] * B, [m] * B, act, d ** -0.5).isnan().all()


@pytest.mark.parametrize("act,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("window", [0, 70])
def test_prompt_nan_in_keys_and_queries_reach_only_who_sees_them(lib, act, d, window):
    nq, H, G = [300, 290], 4, 2
    q, k, v = _randn((590, H, d), act, 1), _randn((590, G, d), act, 2), _randn((590, G, d), act, 3)
    bad_q, bad_k = q.clone(), k.clone()
    bad_q[150, 3, 0] = bad_q[0, 0, 1] = float("nan")
    bad_k[40, 0, 3] = bad_k[299, 1, 5] = bad_k[300 + 130, 1, 0] = float("nan")
    out = _prompt(lib, bad_q, bad_k, v, nq, nq, act, d ** -0.5, window)
    at = 0
    for n in nq:
        t = np.arange(n)
        want, mag, zmag = gqa.attend(f64(q[at:at + n]), f64(k[at:at + n]), f64(v[at:at + n]), t, d ** -0.5, window)
        want[np.isnan(f64(bad_q[at:at + n])).any(-1)] = np.nan
        for j, g in np.argwhere(np.isnan(f64(bad_k[at:at + n])).any(-1)):
            rows = (t >= j) & ((t < j + window) if window else True)
            want[rows, g * (H // G):(g + 1) * (H // G)] = np.nan
        _same(out[at:at + n], want, mag, zmag, act, f"sequence at {at}")
        at += n


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "act"), ("bf16", "fp8")])
@pytest.mark.parametrize("T,H", [(1, 4), (3, 8), (5, 8)])
def test_decode_nan_in_keys_and_queries_reach_only_who_sees_them(lib, act, kv, T, H):
    G, d, page, window = 2, 128, 16, 40
    lens = [50, 700, 67]
    ks, vs = ([_randn((n, G, d), act, s + b) for b, n in enumerate(lens)] for s in (1, 50))
    q = _randn((len(lens) * T, H, d), act, 3)
    clean = Paged(ks, vs, page, kv, act)
    bad = [x.clone() for x in ks]
    bad[0][-1, 0, 5] = bad[1][-1, 1, 7] = bad[1][3, 0, 0] = bad[2][30, 1, 9] = float("nan")
    c, bad_q = Paged(bad, vs, page, kv, act), q.clone()
    bad_q[T - 1, H - 1, 4] = float("nan")
    for w in (0, window):
        out = _decode(lib, bad_q, c.handle(), c.table, lens, T, act, kv, G, page, d ** -0.5, w)
        for b, n in enumerate(lens):
            t = np.arange(n - T, n)
            want, mag, zmag = gqa.attend(f64(q[b * T:(b + 1) * T]), *clean.rows(b, n), t, d ** -0.5, w)
            want[np.isnan(f64(bad_q[b * T:(b + 1) * T])).any(-1)] = np.nan
            for j, g in np.argwhere(np.isnan(f64(bad[b])).any(-1)):
                rows = (t >= j) & ((t < j + w) if w else True)
                want[rows, g * (H // G):(g + 1) * (H // G)] = np.nan
            _same(out[b * T:(b + 1) * T], want, mag, zmag, act, f"length {n}, window {w}")


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("n", [40, 3000])
def test_decode_infinite_logit_is_not_hidden(lib, act, n):
    d, page = 128, 32
    q = _randn((2, 4, d), act, 1)
    q[:, :, 5] = 1.0
    for at in (0, 17, n - 2):
        k, v = _randn((n, 1, d), act, 2), _randn((n, 1, d), act, 3)
        k[at, 0, 5] = float("inf")
        c = Paged([k], [v], page, "act", act)
        assert _decode(lib, q, c.handle(), c.table, [n], 2, act, "act", 1, page, d ** -0.5).isnan().all()


# ---- values that are not finite ------------------------------------------------

@pytest.mark.parametrize("act,d", [("bf16", 128), ("f16", 64), ("f16", 128)])
@pytest.mark.parametrize("window", [0, 100, 300])
def test_prompt_infinities_in_values(lib, act, d, window):
    """Infinities arrive with their signs (two of opposite signs as NaN), on
    both sides of tile borders, and only at rows that see them."""
    nq, H, G = [700, 290, 64], 4, 2
    q, k, v = _randn((1054, H, d), act, 1), _randn((1054, G, d), act, 2), _randn((1054, G, d), act, 3)
    inf = float("inf")
    for row, g, dim, x in ((0, 0, 1, inf), (127, 1, 2, -inf), (128, 1, 2, inf), (255, 0, 63, -inf), (256, 0, 0, float("nan")),
                           (511, 1, 9, inf), (640, 0, 33, -inf), (699, 1, 4, inf), (700, 0, 5, -inf), (989, 1, 6, inf), (990, 1, 7, inf)):
        v[row, g, dim] = x
    out = _prompt(lib, q, k, v, nq, nq, act, d ** -0.5, window)
    at = 0
    for n in nq:
        want, mag, zmag = gqa.attend(f64(q[at:at + n]), f64(k[at:at + n]), f64(v[at:at + n]), np.arange(n), d ** -0.5, window)
        _same(out[at:at + n], want, mag, zmag, act, f"sequence at {at}")
        at += n


def test_prompt_infinities_in_values_more_keys_and_an_odd_group(lib):
    """Positions that do not begin at a tile, units of neighbouring position
    tiles in one CTA (a group of one and of three heads)."""
    inf = float("inf")
    for H, G, act, d in ((2, 2, "bf16", 128), (3, 1, "f16", 64)):
        for window in (0, 200):
            nq, nk = [400, 9], [577, 333]
            q, k, v = _randn((409, H, d), act, 1), _randn((910, G, d), act, 2), _randn((910, G, d), act, 3)
            for row, dim, x in ((3, 1, inf), (176, 2, -inf), (177, 3, inf), (305, 4, -inf), (383, 5, inf), (384, 6, float("nan")),
                                (576, 7, -inf), (577, 8, inf), (900, 9, inf), (909, 10, -inf)):
                v[row, :, dim] = x
            out = _prompt(lib, q, k, v, nq, nk, act, d ** -0.5, window)
            aq = ak = 0
            for n, m in zip(nq, nk):
                want, mag, zmag = gqa.attend(f64(q[aq:aq + n]), f64(k[ak:ak + m]), f64(v[ak:ak + m]), np.arange(m - n, m), d ** -0.5, window)
                _same(out[aq:aq + n], want, mag, zmag, act, f"{n} of {m}, window {window}")
                aq, ak = aq + n, ak + m


@pytest.mark.parametrize("act,d", [("bf16", 128), ("f16", 64)])
def test_prompt_one_query_behind_a_value_that_is_not_finite(lib, act, d):
    """A single query with a window, odd values before it, inside it and in
    both places, after a few keys and after many."""
    H, G, inf = 4, 2, float("inf")
    nk = [2, 5, 12, 16, 17, 40, 130, 300]
    B = len(nk)
    at = np.cumsum([0] + nk)
    sink = torch.tensor([0.5, -1.0, 2.0, 0.0])
    for window, back in ((1, [1]), (3, [1, 4]), (4, [3])):
        q, k, v = _randn((B, H, d), act, 1), _randn((sum(nk), G, d), act, 2), _randn((sum(nk), G, d), act, 3)
        for b, m in enumerate(nk):
            for x, j in enumerate(back):
                if j < m:
                    v[at[b] + m - 1 - j, x % G, 5 + x] = (inf, -inf, float("nan"))[b % 3]
        out = _prompt(lib, q, k, v, [1] * B, nk, act, d ** -0.5, window, sink)
        for b, m in enumerate(nk):
            s = slice(at[b], at[b] + m)
            want, mag, zmag = gqa.attend(f64(q[b:b + 1]), f64(k[s]), f64(v[s]), [m - 1], d ** -0.5, window, f64(sink))
            _same(out[b:b + 1], want, mag, zmag, act, f"{m} keys, window {window}")


@pytest.mark.parametrize("T,H,G", [(1, 4, 2), (3, 4, 2), (5, 8, 2)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_decode_infinities_in_values(lib, act, T, H, G):
    d, page, inf = 64, 16, float("inf")
    lens = [50, 700, 67]
    ks, vs = ([_randn((n, G, d), act, s + b) for b, n in enumerate(lens)] for s in (1, 50))
    vs[0][-1, 0, 5], vs[0][-2, 0, 6], vs[1][-1, 1, 7], vs[1][3, 0, 8] = inf, -inf, -inf, inf
    vs[2][-1, 0, 9], vs[2][20, 0, 9], vs[2][-1, 1, 9] = inf, -inf, inf
    c = Paged(ks, vs, page, "act", act)
    q = _randn((len(lens) * T, H, d), act, 3)
    for window in (0, 40):
        out = _decode(lib, q, c.handle(), c.table, lens, T, act, "act", G, page, d ** -0.5, window)
        for b, n in enumerate(lens):
            want, mag, zmag = gqa.attend(f64(q[b * T:(b + 1) * T]), *c.rows(b, n), np.arange(n - T, n), d ** -0.5, window)
            _same(out[b * T:(b + 1) * T], want, mag, zmag, act, f"length {n}, window {window}")


@pytest.mark.parametrize("where", ["first key", "every 97th key", "last key", "every key"])
@pytest.mark.parametrize("window", [0, 1000])
def test_prompt_values_that_are_not_finite_take_a_bounded_time(lib, where, window):
    """A long prompt with NaN among its values: right at every row, and within
    some 40 times the time without (a warp computes 32 rows again by 16 blocks of
    16 x 16 for a tile of 128 keys, each a few thousand clocks, as a tile takes
    otherwise; row by row and key by key it would be 800 times)."""
    n, H, G, d = 6000, 8, 1, 128
    q, k, v = _randn((n, H, d), "bf16", 1).cuda(), _randn((n, G, d), "bf16", 2).cuda(), _randn((n, G, d), "bf16", 3).cuda()
    bad = v.clone()
    rows = {"first key": [0], "every 97th key": range(0, n, 97), "last key": [n - 1], "every key": range(n)}[where]
    for j in rows:
        bad[j, 0, j % d] = float("nan")
    p = _params(lib, B=1, n_heads=H, n_kv_heads=G, d=d, window=window, softmax_scale=d ** -0.5)
    cu = _i32([0, n])
    us = {}
    for name, x in (("clean", v), ("odd", bad)):
        out, times = torch.empty_like(q), []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            lib.gqa_prompt_attn(p, q, k, x, cu, cu, out)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        us[name] = min(times[1:])
    t = np.unique(np.concatenate([np.arange(0, 200), np.arange(n - 140, n), np.arange(1000, 1010), np.arange(0, n, 331)]))
    want, mag, zmag = gqa.attend(f64(q[t.tolist()]), f64(k), f64(bad), t, d ** -0.5, window)
    _same(out[t.tolist()], want, mag, zmag, "bf16", where)
    assert us["odd"] < 40 * us["clean"] + 200, us


@pytest.mark.parametrize("d", [64, 128])
def test_decode_fp8_row_with_an_infinity(lib, d):
    """A value row that holds an infinity has it as its scale: whoever sees
    the row is NaN, whoever does not is exact."""
    lens, G, H, T, page = [40, 300], 1, 2, 3, 16
    ks, vs = ([_randn((n, G, d), "bf16", s + b) for b, n in enumerate(lens)] for s in (1, 50))
    c = Paged(ks, vs, page, "fp8", "bf16")
    q = _randn((2 * T, H, d), "bf16", 3)
    rows = [c.rows(b, n) for b, n in enumerate(lens)]
    for b, j in ((0, 38), (1, 200)):
        at = c.table[b, j // page].long(), 0, j % page
        codes = torch.zeros(d, device="cuda")
        codes[3] = float("nan")
        c.v[at] = codes.to(torch.float8_e4m3fn)
        c.v_scale[at] = float("inf")
    out = _decode(lib, q, c.handle(), c.table, lens, T, "bf16", "fp8", G, page, d ** -0.5)
    for b, (n, j) in enumerate(zip(lens, (38, 200))):
        t = np.arange(n - T, n)
        want, mag, zmag = gqa.attend(f64(q[b * T:(b + 1) * T]), *rows[b], t, d ** -0.5)
        want[t >= j] = np.nan
        _same(out[b * T:(b + 1) * T], want, mag, zmag, "bf16", f"length {n}")


# ---- weights and magnitudes far apart ------------------------------------------

def _sink_like(n, d, act, nats, at, seed):
    """Keys of which one outweighs the others by e^nats, with a value of zero,
    among values of one sign."""
    k, v = _randn((n, 1, d), act, seed, 0.02), (_randn((n, 1, d), act, seed + 1).float().abs() + 0.5).to(ACT[act])
    k[at] = nats / d ** 0.5
    v[at] = 0
    return k, v


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("nats", [8, 12, 14, 16])
@pytest.mark.parametrize("at", [0, 1030])
def test_prompt_one_key_outweighs_thousands(lib, act, nats, at):
    """What the others hold comes out with the accuracy of its own sum: their
    weights, 2^-23 of the largest, keep the activation type's precision."""
    for n, m, d in ((2100, 2100, 64), (5, 16384, 128)):
        q = torch.ones(n, 2, d).to(ACT[act])
        k, v = _sink_like(m, d, act, nats, at, 5)
        out = _prompt(lib, q, k, v, [n], [m], act, d ** -0.5)
        t = np.arange(m - n, m)
        want, mag, zmag = gqa.attend(f64(q), f64(k), f64(v), t, d ** -0.5)
        _same(out, want, mag, zmag, act, f"{n} queries, {m} keys")


@pytest.mark.parametrize("act,kv", [("f16", "act"), ("bf16", "act"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("nats", [8, 12, 14, 16])
@pytest.mark.parametrize("T,H", [(1, 2), (2, 8), (5, 8)])
def test_decode_one_key_outweighs_thousands(lib, act, kv, nats, T, H):
    d, page = 128, 64
    for m, at in ((300, 2), (2100, 1030), (9000, 0)):
        k, v = _sink_like(m, d, act, nats, at, 5)
        if kv == "fp8":
            v[at, 0, 0] = 1.0  # a scale like the others', codes of zero
        q = torch.ones(T, H, d).to(ACT[act])
        c = Paged([k], [v], page, kv, act)
        out = _decode(lib, q, c.handle(), c.table, [m], T, act, kv, 1, page, d ** -0.5)
        want, mag, zmag = gqa.attend(f64(q), *c.rows(0, m), np.arange(m - T, m), d ** -0.5)
        _same(out, want, mag, zmag, act, f"{m} keys")


@pytest.mark.parametrize("act,d", [("bf16", 64), ("bf16", 128), ("f16", 64), ("f16", 128)])
def test_values_at_the_end_of_the_type(lib, act, d):
    """Averages of the type's largest values are such values, not infinities."""
    n, H, G, page = 700, 4, 2, 32
    top = torch.finfo(ACT[act]).max
    q, k = _randn((n, H, d), act, 1), _randn((n, G, d), act, 2)
    v = (_randn((n, G, d), act, 3).float().abs().clamp(0.25, 1.0) * (0.98 * top)).to(ACT[act])
    v[:, 0] = 0.75 * top
    out = _prompt(lib, q, k, v, [n], [n], act, d ** -0.5)
    want, mag, zmag = gqa.attend(f64(q), f64(k), f64(v), np.arange(n), d ** -0.5)
    _same(out, want, mag, zmag, act, "prompt")
    c = Paged([k], [v], page, "act", act)
    for T in (1, 9):
        out = _decode(lib, q[-T:], c.handle(), c.table, [n], T, act, "act", G, page, d ** -0.5)
        _same(out, want[-T:], mag[-T:], zmag, act, "decode")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** -118, 2.0 ** -100, 2.0 ** 100])
def test_values_far_from_one(lib, d, size):
    """BF16 values of 2^-118 and 2^100 on average weigh as those of 1 do.  (fp32
    sums lose 2^-149 a product at most; with weights of 2^-18 on average that is
    2^-131 of the result, 2^-13 of values of 2^-118.)"""
    n, H, G, page = 700, 4, 2, 32
    q, k = _randn((n, H, d), "bf16", 1), _randn((n, G, d), "bf16", 2)
    v = (_randn((n, G, d), "bf16", 3).float() * size).bfloat16()
    want, mag, zmag = gqa.attend(f64(q), f64(k), f64(v), np.arange(n), d ** -0.5)
    _same(_prompt(lib, q, k, v, [n], [n], "bf16", d ** -0.5), want, mag, zmag, "bf16", "prompt")
    c = Paged([k], [v], page, "act", "bf16")
    for T in (1, 9):
        out = _decode(lib, q[-T:], c.handle(), c.table, [n], T, "bf16", "act", G, page, d ** -0.5)
        _same(out, want[-T:], mag[-T:], zmag, "bf16", "decode")


@pytest.mark.parametrize("act,size", [("f16", 6e4), ("bf16", 3e3), ("bf16", 1e9), ("bf16", 5e17)])
def test_equal_logits_of_any_size(lib, act, size):
    """Logits of up to 10^37, all equal: the average of the values."""
    n, H, d = 300, 2, 128
    q, k = torch.full((n, H, d), size).to(ACT[act]), torch.full((n, H, d), size).to(ACT[act])
    q[:, 1] *= -1
    v = _randn((n, H, d), act, 3)
    want = np.cumsum(f64(v), 0) / np.arange(1, n + 1)[:, None, None]
    mag = np.cumsum(np.abs(f64(v)), 0) / np.arange(1, n + 1)[:, None, None]
    _same(_prompt(lib, q, k, v, [n], [n], act, 1.0), want, mag, 0.0, act, "prompt")
    c = Paged([k], [v], 16, "act", act)
    _same(_decode(lib, q[-3:], c.handle(), c.table, [n], 3, act, "act", H, 16, 1.0), want[-3:], mag[-3:], 0.0, act, "decode")


@pytest.mark.parametrize("act,kv", [("f16", "act"), ("bf16", "act"), ("bf16", "fp8"), ("f16", "fp8")])
def test_decode_equal_logits_around_fp32s_last_bit(lib, act, kv):
    """Logits of 10^6 to 10^10, where fp32's step goes from a fraction to more
    than all that a weight's range holds: still the average.  (With an FP8 cache
    the value's log-scale shares the logit's rounding, as any error of a logit.)"""
    n, H, d = 150, 2, 128
    v = [_randn((n, H, d), act, 3)]
    for size in (128.0, 256.0, 512.0, 736.0, 1040.0, 1472.0, 2080.0, 4160.0, 8320.0):
        q, k = torch.full((3, H, d), size).to(ACT[act]), torch.full((n, H, d), size).to(ACT[act])
        q[:, 1] *= -1
        c = Paged([k], v, 16, kv, act)
        x = c.rows(0, n)[1]
        want, mag = (np.stack([y[:m].mean(0) for m in (n - 2, n - 1, n)]) for y in (x, np.abs(x)))
        _same(_decode(lib, q, c.handle(), c.table, [n], 3, act, kv, H, 16, 1.0), want, mag,
              0.0 if kv == "act" else 128 * size * size, act, f"{kv} {size}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("far", [0, 20, 45])
def test_decode_fp8_scales_far_apart(lib, d, far):
    """Value rows up to 2^90 apart in size: small ones still count in the
    denominator."""
    n, H, G, page = 400, 4, 2, 16
    ks, vs = [_randn((n, G, d), "bf16", 1)], [_randn((n, G, d), "bf16", 2)]
    c = Paged(ks, vs, page, "fp8", "bf16")
    big = torch.rand(c.v_scale.shape, generator=torch.Generator().manual_seed(4)).cuda() < 0.3
    c.v_scale.mul_(torch.where(big, 2.0 ** (far + 2), 2.0 ** (2 - far)))
    q = _randn((3, H, d), "bf16", 3)
    sink = torch.tensor([0.0, 2.0, -3.0, 1.0])
    for s in (None, sink):
        out = _decode(lib, q, c.handle(), c.table, [n], 3, "bf16", "fp8", G, page, d ** -0.5, sink=s)
        want, mag, zmag = gqa.attend(f64(q), *c.rows(0, n), np.arange(n - 3, n), d ** -0.5, 0, None if s is None else f64(s))
        _same(out, want, mag, zmag, "bf16")


# ---- batches and host threads --------------------------------------------------

def test_prompt_bits_do_not_depend_on_the_batch(lib):
    lens, H, G, d = [700, 40, 256, 1, 129], 6, 2, 128
    n = sum(lens)
    q, k, v = _randn((n, H, d), "bf16", 1), _randn((n, G, d), "bf16", 2), _randn((n, G, d), "bf16", 3)
    whole, at = _prompt(lib, q, k, v, lens, lens, "bf16", d ** -0.5), 0
    for m in lens:
        s = slice(at, at + m)
        assert torch.equal(_prompt(lib, q[s], k[s], v[s], [m], [m], "bf16", d ** -0.5), whole[s])
        at += m


def test_two_host_threads(lib):
    """Two threads with a stream, a cache and a workspace each, of different
    forms, give what they give alone."""
    def layer(i):
        act, kv, d, page, H, G, n = (("bf16", "act", 128, 32, 8, 2, 900), ("f16", "fp8", 64, 16, 6, 1, 700))[i]
        c = Paged([_randn((n, G, d), act, 1 + i)], [_randn((n, G, d), act, 3 + i)], page, kv, act, extra_cols=3)
        c.table[0, -(-n // page):] = c.k.shape[0] - 1
        p = _params(lib, act, kv, B=1, n_heads=H, n_kv_heads=G, d=d, r=d, page=page, softmax_scale=d ** -0.5, rope_theta=(1e4, 5e5)[i])
        q, new = _randn((3, H, d), act, 5 + i).cuda(), _randn((3, G, d), act, 7 + i).cuda()
        ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 3, n + 3)), dtype=torch.uint8, device="cuda")
        cu, pos0, lens = _i32([0, 3]), _i32([n]), _i32([n + 3])

        def step():
            qo, ko, out, po = torch.empty_like(q), torch.empty_like(new), torch.empty_like(q), torch.empty_like(q)
            lib.gqa_cache_append(p, q, new, new, cu, pos0, c.handle(), c.table, q_out=qo, k_out=ko)
            lib.gqa_decode_attn(p, qo, c.handle(), c.table, lens, 3, n + 3, out, ws)
            lib.gqa_prompt_attn(p, qo, ko, new, cu, cu, po)
            return qo, ko, out, po
        return step

    layers = [layer(0), layer(1)]
    alone = [f() for f in layers]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    got = layers[i]()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                    wrong.append(f"thread {i}: other bits")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong

"""gqa_cache_append, gqa_decode_attn and gqa_prompt_attn against the fp64
oracle: types, head layouts, lengths from zero to several tiles, pages that
end inside a tile, windows, sinks, masked garbage, strides, streams and
graphs, and a run of the three together."""

import numpy as np
import pytest
import torch

from gqa_util import ACT, Paged, check_fp8, check_out, check_turned, f64
from gqa_util import quantise as _quantise
from oracle import gqa

pytestmark = pytest.mark.gpu
THETA = 1e4


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
                               kv_fmt=lib.KV_ACT if kv == "act" else lib.KV_FP8, rope_theta=THETA, **kw)


def _randn(shape, act, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(ACT[act])


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(lens):
    return _i32([0] + list(np.cumsum(lens)))


def _err():
    return torch.zeros(4, dtype=torch.int32, device="cuda")


# ---- append --------------------------------------------------------------------

def _append(lib, act, kv, lens, pos0, heads, G, d, r, page, tail=0, seed=0, spoil=None, fused=False):
    """Appends random rows to a poisoned cache and checks every cache byte,
    q_out and k_out."""
    n = sum(lens) + tail
    H = heads
    qkv = _randn((n, H + 2 * G, d), act, seed, 2.0).cuda()
    if len(lens) > 1 and sum(lens) > 2:
        qkv[1, H] = 0  # a key row of zeros (FP8: scale 1)
    q, k, v = qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.transpose(0, 1).contiguous().transpose(0, 1)
    cols = max(-(-(p + m) // page) for p, m in zip(pos0, lens)) if lens else 1
    cols = max(cols, 1)
    rng = np.random.RandomState(seed)
    reached = [(b, c) for b, (p, m) in enumerate(zip(pos0, lens)) if m for c in range(p // page, (p + m - 1) // page + 1)]
    n_pages = len(reached) + 2
    table = np.full((len(lens), cols), -1, np.int32)
    for i, at in enumerate(rng.permutation(n_pages)[:len(reached)]):
        table[reached[i]] = at
    if spoil is not None:
        table[reached[spoil]] = n_pages
    shape = (n_pages, G, page, d)
    dt = ACT[act] if kv == "act" else torch.float8_e4m3fn
    poison = torch.full(shape, 3.0).to(dt)
    kc, vc = poison.cuda(), poison.clone().cuda()
    ks = vs = None
    if kv != "act":
        ks, vs = torch.full(shape[:3], 7.0, device="cuda"), torch.full(shape[:3], 7.0, device="cuda")
    qo, ko = torch.full((n, H, d), 5.0, device="cuda").to(ACT[act]), torch.full((n, G, d), 5.0, device="cuda").to(ACT[act])
    err = _err()
    p = _params(lib, act, kv, B=len(lens), n_heads=H, n_kv_heads=G, d=d, r=r, page=page)
    lib.gqa_cache_append(p, q, k, v, _starts(lens), _i32(pos0), lib.make_gqa_cache(kc, vc, ks, vs),
                         torch.from_numpy(table).cuda(), q_out=qo, k_out=ko, err=err)
    torch.cuda.synchronize()
    m = sum(lens)
    pos = np.concatenate([np.arange(a, a + c) for a, c in zip(pos0, lens)] + [np.zeros(0, int)]).astype(np.int64)
    seq = np.concatenate([np.full(c, b) for b, c in enumerate(lens)] + [np.zeros(0, int)]).astype(np.int64)
    wq, wk, wv = gqa.rotate(f64(q[:m]), pos, r, THETA), gqa.rotate(f64(k[:m]), pos, r, THETA), f64(v[:m])
    check_turned(qo[:m], wq, q[:m], act, "q_out")
    check_turned(ko[:m], wk, k[:m], act, "k_out")
    assert (qo[m:] == 5).all() and (ko[m:] == 5).all(), "rows behind the last sequence"
    at, slot = table[seq, pos // page], pos % page
    ok = at < n_pages
    assert int(err[0]) == (0 if ok.all() else lib.DEV_ERR_INDEX)
    mask = np.zeros(shape[:3], bool)
    for name, cache, scale, want, x in (("k", kc, ks, wk, k), ("v", vc, vs, wv, v)):
        idx = (torch.from_numpy(at[ok]).long(), slice(None), torch.from_numpy(slot[ok]).long())
        got = cache.cpu()[idx]
        if kv == "act":
            if name == "v":
                assert torch.equal(got, v[:m].cpu()[torch.from_numpy(ok)])
            elif m:
                check_turned(got, want[ok], x[:m], act, name)
        else:
            check_fp8(got, scale.cpu()[idx], want[ok], name)
        mask[at[ok], :, slot[ok]] = True
        left = torch.from_numpy(~mask)
        assert (cache.cpu().float()[left] == 3).all(), f"{name}: slots of no token"
        if scale is not None:
            assert (scale.cpu()[left] == 7).all()


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "act"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("H,G,d,r,page", [(8, 2, 128, 128, 64), (5, 1, 64, 32, 16), (6, 3, 128, 64, 256), (4, 4, 64, 64, 32), (3, 1, 128, 0, 128)])
def test_append(lib, act, kv, H, G, d, r, page):
    _append(lib, act, kv, [1, 0, 37, 2, 130], [0, 5, 13, 131071, 1000], H, G, d, r, page)


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "fp8"), ("bf16", "fp8"), ("f16", "act")])
@pytest.mark.parametrize("H,G,d,r", [(32, 8, 128, 64), (28, 7, 128, 128), (16, 4, 64, 64), (9, 1, 64, 32), (128, 64, 128, 128)])
def test_append_many_tokens(lib, act, kv, H, G, d, r):
    """Enough tokens for several a CTA, in two and in three pieces a thread."""
    _append(lib, act, kv, [1100, 1, 0, 398], [7, 0, 3, 50000], H, G, d, r, 64, tail=3, seed=8)


@pytest.mark.parametrize("kv", ["act", "fp8"])
def test_append_one_token_each(lib, kv):
    _append(lib, "bf16", kv, [1] * 33, [17 * i for i in range(33)], 32, 8, 128, 128, 16, seed=3)


@pytest.mark.parametrize("kv", ["act", "fp8"])
def test_append_rows_behind_the_last_sequence_fused_projection(lib, kv):
    _append(lib, "bf16", kv, [0, 9, 0, 4, 0], [3, 60, 1, 0, 9], 7, 1, 128, 64, 16, tail=6, seed=4, fused=True)
    _append(lib, "f16", kv, [0], [0], 4, 2, 64, 64, 16, tail=3, seed=5)


def test_append_bad_page_is_skipped(lib):
    _append(lib, "bf16", "act", [40, 5], [10, 0], 4, 2, 128, 64, 16, spoil=1, seed=6)


def test_append_bad_positions(lib):
    p = _params(lib, B=3, n_heads=2, n_kv_heads=1, d=64, r=64, page=16)
    k = _randn((3, 1, 64), "bf16", 1).cuda()
    q = _randn((3, 2, 64), "bf16", 2).cuda()
    kc = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    err = _err()
    ko = torch.zeros_like(k)
    lib.gqa_cache_append(p, None, k, k, _i32([0, 1, 2, 3]), _i32([-1, 32, 31]), lib.make_gqa_cache(kc, vc),
                         _i32([[0, 1], [2, 3], [3, 2]]), k_out=ko, err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == lib.DEV_ERR_RANGE
    assert torch.equal(vc[2, 0, 15], k[2, 0]) and int((vc != 0).any(-1).sum()) == 1
    check_turned(ko, gqa.rotate(f64(k), [-1, 32, 31], 64, THETA), k, "bf16")


def test_append_in_place_and_without_outputs(lib):
    p = _params(lib, B=1, n_heads=4, n_kv_heads=2, d=128, r=128, page=16)
    q, k, v = _randn((21, 4, 128), "bf16", 1).cuda(), _randn((21, 2, 128), "bf16", 2).cuda(), _randn((21, 2, 128), "bf16", 3).cuda()
    caches = [torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    table, cu, pos0 = _i32([[1, 0]]), _i32([0, 21]), _i32([4])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    lib.gqa_cache_append(p, q, k, v, cu, pos0, lib.make_gqa_cache(*caches[:2]), table, q_out=qo, k_out=ko)
    k2 = k.clone()
    lib.gqa_cache_append(p, q, k2, v, cu, pos0, lib.make_gqa_cache(*caches[2:]), table, q_out=q, k_out=k2)
    lib.gqa_cache_append(p, None, k, v, cu, pos0, lib.make_gqa_cache(*caches[2:]), table)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k2, ko)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_append_far_positions(lib):
    """Angles stay exact to fp32 at positions near 2^27."""
    far = (1 << 27) - 5
    p = _params(lib, "f16", B=1, n_heads=1, n_kv_heads=1, d=64, r=64, page=256)
    k = _randn((4, 1, 64), "f16", 9).cuda()
    ko = torch.empty_like(k)
    cache = torch.zeros(1, 1, 256, 64, dtype=torch.float16, device="cuda")
    lib.gqa_cache_append(p, None, k, k, _i32([0, 4]), _i32([far]), lib.make_gqa_cache(cache, cache.clone()),
                         torch.zeros(1, 1 << 19, dtype=torch.int32, device="cuda"), k_out=ko)
    check_turned(ko, gqa.rotate(f64(k), np.arange(far, far + 4), 64, THETA), k, "f16")


# ---- decode --------------------------------------------------------------------

LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 517]


def _decode(lib, lens, act="bf16", kv="act", H=8, G=2, d=128, page=16, T=1, window=0, sink=False, gain=1.0, seed=0,
            n_max=None, bad=(), v_odd=None):
    ks = [_randn((n, G, d), act, seed + 10 + b) for b, n in enumerate(lens)]
    vs = [_randn((n, G, d), act, seed + 500 + b) for b, n in enumerate(lens)]
    if v_odd is not None:
        v_odd(vs)
    c = Paged(ks, vs, page, kv, act, seed=seed)
    live = [None] * len(lens)
    for b, col in bad:
        c.table[b, col] = c.k.shape[0] if col % 2 else -1
        live[b] = np.ones(lens[b], bool) if live[b] is None else live[b]
        live[b][col * page:(col + 1) * page] = False
    q = _randn((len(lens) * T, H, d), act, seed + 1, gain).cuda()
    sk = (torch.randn(H, generator=torch.Generator().manual_seed(seed + 2)) * 2).cuda() if sink else None
    p = _params(lib, act, kv, B=len(lens), n_heads=H, n_kv_heads=G, d=d, page=page, window=window, softmax_scale=d ** -0.5)
    n_max = max(lens) if n_max is None else n_max
    out = torch.full_like(q, 9.0)
    ws = torch.full((max(16, lib.gqa_decode_attn_workspace_bytes(p, T, n_max)),), 255, dtype=torch.uint8, device="cuda")
    err = _err()
    lib.gqa_decode_attn(p, q, c.handle(), c.table, _i32(lens), T, n_max, out, ws, sink=sk, err=err)
    torch.cuda.synchronize()
    seen_bad = any(max(0, lens[b] - T - window + 1 if window else 0) < (col + 1) * page for b, col in bad)
    assert int(err[0]) == (lib.DEV_ERR_INDEX if seen_bad else 0)
    for b, n in enumerate(lens):
        if bad:
            k, v = (np.asarray(f64(x[b])) for x in (ks, vs))
        else:
            k, v = c.rows(b, n)
        want, mag, zmag = gqa.attend(f64(q[b * T:(b + 1) * T]), k, v, np.arange(n - T, n), d ** -0.5, window,
                                     None if sk is None else f64(sk), live[b])
        check_out(out[b * T:(b + 1) * T], want, mag, zmag, act, f"length {n}")
    return out


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "act"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("H,G,d", [(8, 2, 128), (8, 1, 64), (5, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_decode_lengths(lib, act, kv, H, G, d, page):
    _decode(lib, LENS, act, kv, H, G, d, page)


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("window", [1, 16, 100])
@pytest.mark.parametrize("T,sink", [(1, True), (3, False), (9, True)])
def test_decode_window_tokens_sink(lib, page, window, T, sink):
    for act, kv in (("bf16", "act"), ("f16", "fp8")):
        _decode(lib, LENS, act, kv, 8, 4, 128, page, T, window, sink, seed=window)


@pytest.mark.parametrize("kv", ["act", "fp8"])
@pytest.mark.parametrize("H,G,T", [(16, 1, 1), (32, 2, 2), (128, 1, 1), (24, 1, 1), (128, 2, 64), (1, 1, 64)])
def test_decode_many_rows_share_a_kv_head(lib, kv, H, G, T):
    _decode(lib, [0, 1, 40, 64, 333], "bf16", kv, H, G, 128, 32, T, 0, True, seed=H)
    _decode(lib, [70, 333], "f16", kv, H, G, 64, 32, T, 50, False, seed=H)


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "fp8")])
@pytest.mark.parametrize("lens", [[1023, 1024, 1025], [4096, 100, 5000], [20000]])
def test_decode_splits(lib, act, kv, lens):
    _decode(lib, lens, act, kv, 8, 2, 128, 64, seed=5, sink=True)
    _decode(lib, lens, act, kv, 4, 4, 64, 16, T=2, seed=6, gain=4.0)
    _decode(lib, lens, act, kv, 4, 2, 128, 32, window=777, seed=7, n_max=max(lens) + 30)


def test_decode_bad_pages_are_skipped(lib):
    _decode(lib, [200, 64, 40, 16], "bf16", "act", 8, 2, 128, 16, bad=[(0, 0), (0, 5), (0, 12), (3, 0)])
    _decode(lib, [200, 700], "bf16", "act", 8, 2, 64, 64, T=2, bad=[(0, 3), (1, 0), (1, 1), (1, 10)])
    _decode(lib, [700], "bf16", "act", 8, 2, 64, 128, bad=[(0, 1)], window=300)


def test_decode_length_past_its_bounds(lib):
    """lens over n_max is cut there; negative lengths count as none."""
    ks = [_randn((100, 2, 64), "bf16", b) for b in range(2)]
    c = Paged(ks, ks, 16, "act", "bf16")
    p = _params(lib, B=2, n_heads=4, n_kv_heads=2, d=64, page=16, softmax_scale=0.125)
    q = _randn((2, 4, 64), "bf16", 7).cuda()
    ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 1, 80)), dtype=torch.uint8, device="cuda")
    out, err = torch.empty_like(q), _err()
    lib.gqa_decode_attn(p, q, c.handle(), c.table, _i32([100, -5]), 1, 80, out, ws, err=err)
    assert int(err[0]) == lib.DEV_ERR_RANGE
    k, v = c.rows(0, 80)
    want, mag, zmag = gqa.attend(f64(q[:1]), k, v, [79], 0.125)
    check_out(out[:1], want, mag, zmag, "bf16")
    assert (out[1] == 0).all()


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "act"), ("bf16", "fp8")])
def test_decode_odd_values_reach_only_who_sees_them(lib, act, kv):
    """NaN and infinities in values of the last tokens and before a window:
    queries that do not see them stay exact."""
    def odd(vs):
        vs[0][-1, 0, 5] = float("nan")   # seen by the last of the three queries alone
        vs[1][-1, 1, 7] = float("nan")
        vs[1][0] = float("nan")          # before the window of all
        if kv == "act":
            vs[2][-2, 0, 9] = float("inf")
            vs[2][-2, 1, 9] = float("-inf")
    _decode(lib, [50, 200, 67], act, kv, 4, 2, 64, 16, T=3, window=40, v_odd=odd)


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "act"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("T,H,G,window", [(1, 17, 1, 0), (3, 11, 1, 500), (4, 40, 8, 0), (8, 32, 8, 33), (33, 2, 2, 0)])
def test_decode_rows_of_one_item_and_a_few_more(lib, act, kv, T, H, G, window):
    """17, 20, 32 and 33 query rows a KV head: an item with columns to spare,
    a full one, one row in a second item."""
    for d in (64, 128):
        _decode(lib, [0, 1, 16, 40, 300, 1100], act, kv, H, G, d, 32, T, window, T != 3, seed=T + d)


@pytest.mark.parametrize("act,kv", [("bf16", "act"), ("f16", "act"), ("bf16", "fp8")])
@pytest.mark.parametrize("T,H,G", [(4, 16, 2), (8, 8, 2), (5, 4, 1)])
def test_decode_odd_values_among_many_rows(lib, act, kv, T, H, G):
    """As above, with 20 to 32 rows an item."""
    def odd(vs):
        vs[0][-1, 0, 5] = float("nan")
        vs[1][-1, G - 1, 7] = float("nan")
        vs[1][0] = float("nan")
        vs[2][-2, 0, 9] = float("nan")
    for d in (64, 128):
        _decode(lib, [50, 700, 67], act, kv, H, G, d, 16, T, window=40, v_odd=odd, seed=3)
    if kv == "act":  # (the helper compares bad pages with rows that were not quantised)
        _decode(lib, [200, 700], act, kv, H, G, 128, 64, T, bad=[(0, 3), (1, 0), (1, 1), (1, 10)])


@pytest.mark.parametrize("act,kv,d", [("bf16", "act", 128), ("f16", "fp8", 64)])
@pytest.mark.parametrize("T,H,G", [(1, 12, 4), (3, 12, 2)])
def test_decode_joins_of_few_and_many_splits(lib, act, kv, d, T, H, G):
    """Twelve splits are joined by a warp, thirteen by a CTA; a batch that
    holds both, and one whose bound allows only few, give the same bits."""
    lens = [12288, 300, 12289, 0, 256, 257, 13500]
    whole = _decode(lib, lens, act, kv, H, G, d, 128, T, seed=11, sink=True)
    few = [0, 300, 0, 0, 256, 257, 0]
    ks = [_randn((n, G, d), act, 40 + b) for b, n in enumerate(lens)]
    vs = [_randn((n, G, d), act, 540 + b) for b, n in enumerate(lens)]
    c = Paged(ks, vs, 128, kv, act)
    q = _randn((len(lens) * T, H, d), act, 1).cuda()
    p = _params(lib, act, kv, B=len(lens), n_heads=H, n_kv_heads=G, d=d, page=128, softmax_scale=d ** -0.5)
    outs = []
    for lengths, n_max in ((lens, max(lens)), (few, 300), (few, 12288), (few, max(lens))):
        ws = torch.full((lib.gqa_decode_attn_workspace_bytes(p, T, n_max),), 255, dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, 9.0)
        lib.gqa_decode_attn(p, q, c.handle(), c.table, _i32(lengths), T, n_max, out, ws)
        outs.append(out.view(len(lens), T, H, d))
    for b, n in enumerate(few):
        if n:
            for x in outs[1:]:
                assert torch.equal(x[b], outs[0][b]), n
    for x in outs[1:]:
        assert not x[[0, 2, 3, 6]].any()
    assert whole.isfinite().all()


@pytest.mark.parametrize("kv", ["act", "fp8"])
def test_decode_large_and_small_magnitudes(lib, kv):
    """Logits in the hundreds (one key takes all), keys and values of any
    size that the activation type holds."""
    _decode(lib, [300, 77], "bf16", kv, 4, 2, 128, 16, gain=100.0)
    for scale in (2.0 ** -40, 2.0 ** 30):
        k = _randn((90, 2, 64), "bf16", 1) * 1.0
        v = (_randn((90, 2, 64), "bf16", 2).float() * scale).bfloat16()
        v[7] *= 2.0 ** -20  # rows of one tile far apart in size
        c = Paged([k], [v], 16, kv, "bf16")
        p = _params(lib, "bf16", kv, B=1, n_heads=4, n_kv_heads=2, d=64, page=16, softmax_scale=0.125)
        q = (_randn((1, 4, 64), "bf16", 3).float() * torch.tensor([1e-30, 1.0, 3.0, 1e-3])[None, :, None]).bfloat16().cuda()
        out = torch.empty_like(q)
        ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 1, 90)), dtype=torch.uint8, device="cuda")
        lib.gqa_decode_attn(p, q, c.handle(), c.table, _i32([90]), 1, 90, out, ws)
        kk, vv = c.rows(0, 90)
        want, mag, zmag = gqa.attend(f64(q), kk, vv, [89], 0.125)
        check_out(out, want, mag, zmag, "bf16", f"values of {scale}")


def test_decode_strided_rows(lib):
    """Queries inside a fused projection, outputs head-major."""
    n, G, d = 150, 2, 128
    ks, vs = [_randn((n, G, d), "bf16", 1)], [_randn((n, G, d), "bf16", 2)]
    c = Paged(ks, vs, 32, "act", "bf16")
    p = _params(lib, B=1, n_heads=4, n_kv_heads=G, d=d, page=32, softmax_scale=0.1)
    big = _randn((2, 9, d), "bf16", 3).cuda()
    outs = torch.full((4, 2, 2 * d), 9.0, dtype=torch.bfloat16, device="cuda")
    out = outs[:, :, :d].transpose(0, 1)
    ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 2, n)), dtype=torch.uint8, device="cuda")
    lib.gqa_decode_attn(p, big[:, 3:7], c.handle(), c.table, _i32([n]), 2, n, out, ws)
    want, mag, zmag = gqa.attend(f64(big[:, 3:7]), *c.rows(0, n), [n - 2, n - 1], 0.1)
    check_out(out, want, mag, zmag, "bf16")
    assert (outs[:, :, d:] == 9).all()


def test_decode_offsets_past_32_bits(lib):
    """Pages more than 2^32 elements (and bytes) into the cache."""
    d, page, G = 128, 256, 8
    n_pages = (1 << 32) // (d * page * G) + 40
    k = torch.zeros(n_pages, G, page, d, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    s = torch.ones(n_pages, G, page, device="cuda")
    kk, vv = _randn((300, G, d), "f16", 1).to(torch.float8_e4m3fn), _randn((300, G, d), "f16", 2).to(torch.float8_e4m3fn)
    ids = [n_pages - 1, n_pages - 9]
    for c, i in enumerate(ids):
        m = min(300 - 256 * c, 256)
        k[i, :, :m], v[i, :, :m] = kk[256 * c:256 * c + m].transpose(0, 1).cuda(), vv[256 * c:256 * c + m].transpose(0, 1).cuda()
    p = _params(lib, "f16", "fp8", B=1, n_heads=16, n_kv_heads=G, d=d, page=page, softmax_scale=0.1)
    q = _randn((1, 16, d), "f16", 3).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 1, 300)), dtype=torch.uint8, device="cuda")
    lib.gqa_decode_attn(p, q, lib.make_gqa_cache(k, v, s, s), _i32([ids]), _i32([300]), 1, 300, out, ws)
    want, mag, zmag = gqa.attend(f64(q), f64(kk.float()), f64(vv.float()), [299], 0.1)
    check_out(out, want, mag, zmag, "f16")
    # and a token stored there
    new = _randn((1, G, d), "f16", 4).cuda()
    p = _params(lib, "f16", "fp8", B=1, n_heads=16, n_kv_heads=G, d=d, r=64, page=page)
    lib.gqa_cache_append(p, None, new, new, _i32([0, 1]), _i32([300]), lib.make_gqa_cache(k, v, s, s.clone()), _i32([ids]))
    check_fp8(v[ids[1], :, 44].cpu(), torch.from_numpy(gqa.row_scale(f64(new[0]))), f64(new[0]))
    del k, v, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kv", ["act", "fp8"])
def test_decode_bits_do_not_depend_on_the_batch(lib, kv):
    lens = [3000, 1, 0, 517, 1024, 9000, 64]
    G, d = 2, 128
    ks, vs = ([_randn((n, G, d), "bf16", s + b) for b, n in enumerate(lens)] for s in (1, 50))
    c = Paged(ks, vs, 32, kv, "bf16")
    q = _randn((len(lens), 8, d), "bf16", 3).cuda()

    def run(rows, n_max):
        p = _params(lib, "bf16", kv, B=len(rows), n_heads=8, n_kv_heads=G, d=d, page=32, softmax_scale=0.1)
        ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 1, n_max)), dtype=torch.uint8, device="cuda")
        out = torch.empty(len(rows), 8, d, dtype=torch.bfloat16, device="cuda")
        lib.gqa_decode_attn(p, q[rows].contiguous(), c.handle(), c.table[rows].contiguous(), _i32([lens[b] for b in rows]),
                            1, n_max, out, ws)
        return out

    full = run(list(range(len(lens))), 9000)
    assert torch.equal(full, run(list(range(len(lens))), 9000))
    for b in range(len(lens)):
        assert torch.equal(run([b], max(1, lens[b])), full[b:b + 1]), f"sequence {b}"


# ---- prompt --------------------------------------------------------------------

def _prompt(lib, nq, nk=None, act="bf16", H=4, G=2, d=128, window=0, sink=False, gain=1.0, seed=0, tail=0, layout="plain",
            v_odd=None):
    nk = nq if nk is None else nk
    q = _randn((sum(nq) + tail, H, d), act, seed + 1, gain)
    k, v = _randn((sum(nk) + tail, G, d), act, seed + 2), _randn((sum(nk) + tail, G, d), act, seed + 3)
    # rows of nobody hold NaN
    q[sum(nq):], k[sum(nk):], v[sum(nk):] = float("nan"), float("nan"), float("nan")
    if v_odd is not None:
        v_odd(v)
    if layout == "fused" and nq == nk:
        x = torch.cat([q, k, v], 1).cuda()
        q, k, v = x[:, :H], x[:, H:H + G], x[:, H + G:]
    elif layout == "heads":
        q, k, v = (x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in (q, k, v))
    else:
        q, k, v = q.cuda(), k.cuda(), v.cuda()
    sk = (torch.randn(H, generator=torch.Generator().manual_seed(seed + 4)) * 2).cuda() if sink else None
    p = _params(lib, act, B=len(nq), n_heads=H, n_kv_heads=G, d=d, window=window, softmax_scale=d ** -0.5)
    if layout == "heads":
        out = torch.full((H, len(q), d), 9.0, device="cuda").to(ACT[act]).transpose(0, 1)
    else:
        out = torch.full((len(q), H, d), 9.0, device="cuda").to(ACT[act])
    err = _err()
    lib.gqa_prompt_attn(p, q, k, v, _starts(nq), _starts(nk), out, sink=sk, err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    aq = ak = 0
    for b, (n, m) in enumerate(zip(nq, nk)):
        want, mag, zmag = gqa.attend(f64(q[aq:aq + n]), f64(k[ak:ak + m]), f64(v[ak:ak + m]), np.arange(m - n, m), d ** -0.5,
                                     window, None if sk is None else f64(sk))
        check_out(out[aq:aq + n], want, mag, zmag, act, f"sequence {b}: {n} queries, {m} keys")
        aq, ak = aq + n, ak + m
    assert (out[aq:] == 9).all(), "rows behind the last sequence"
    return out


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("H,G,d", [(4, 2, 128), (4, 1, 64), (3, 3, 128), (5, 1, 64)])
def test_prompt_lengths(lib, act, H, G, d):
    _prompt(lib, [1, 0, 2, 31, 64, 127, 128, 129, 255, 256, 257, 300], None, act, H, G, d, tail=5)


@pytest.mark.parametrize("n", [1, 100, 511, 513, 900])
@pytest.mark.parametrize("layout", ["plain", "fused", "heads"])
def test_prompt_single(lib, n, layout):
    _prompt(lib, [n], layout=layout, seed=n)
    _prompt(lib, [n], layout=layout, act="f16", d=64, H=2, G=2, seed=n)


@pytest.mark.parametrize("window", [1, 5, 64, 128, 129, 400])
@pytest.mark.parametrize("sink", [False, True])
def test_prompt_window_sink(lib, window, sink):
    _prompt(lib, [300, 77, 0, 513], window=window, sink=sink, seed=window)
    _prompt(lib, [300, 77, 0, 513], act="f16", d=64, window=window, sink=sink, seed=window, layout="fused")


@pytest.mark.parametrize("window", [0, 150])
def test_prompt_more_or_fewer_keys_than_queries(lib, window):
    _prompt(lib, [5, 130, 1, 256], [700, 131, 1000, 300], window=window, seed=1)
    _prompt(lib, [200, 7, 300, 40], [100, 0, 299, 1], window=window, sink=True, seed=2)  # queries before the first key: zeros
    _prompt(lib, [200, 7], [3, 6], act="f16", d=64, window=window, seed=3)
    _prompt(lib, [20], [0], seed=4)


def test_prompt_large_logits(lib):
    _prompt(lib, [400, 130], gain=60.0)
    _prompt(lib, [400, 130], act="f16", d=64, gain=200.0)


@pytest.mark.parametrize("act,d", [("bf16", 128), ("f16", 64)])
def test_prompt_odd_values_reach_only_who_sees_them(lib, act, d):
    """NaN and infinities in values: earlier queries, other sequences and
    queries whose window has passed stay exact."""
    def odd(v):
        v[40, 0, 3] = float("nan")
        v[299, 1, 5] = float("inf")     # the last key of the first sequence
        v[300, 0, 7] = float("nan")     # the first key of the second
        v[520, 1, 9] = float("-inf")
    _prompt(lib, [300, 290], act=act, d=d, v_odd=odd)
    _prompt(lib, [300, 290], act=act, d=d, v_odd=odd, window=100, sink=True)


def test_prompt_sequence_outside_the_rows(lib):
    p = _params(lib, B=3, n_heads=2, n_kv_heads=1, d=64, softmax_scale=0.125)
    q, k = _randn((30, 2, 64), "bf16", 1).cuda(), _randn((30, 1, 64), "bf16", 2).cuda()
    out, err = torch.full_like(q, 9.0), _err()
    lib.gqa_prompt_attn(p, q, k, k, _i32([0, 10, 20, 30]), _i32([0, 10, 20, 31]), out, err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == lib.DEV_ERR_RANGE
    for a in (0, 10):
        want, mag, zmag = gqa.attend(f64(q[a:a + 10]), f64(k[a:a + 10]), f64(k[a:a + 10]), np.arange(10), 0.125)
        check_out(out[a:a + 10], want, mag, zmag, "bf16")
    assert (out[20:] == 9).all()


def test_prompt_run_to_run_and_batch(lib):
    a = _prompt(lib, [700, 40, 256], seed=8)
    b = _prompt(lib, [700, 40, 256], seed=8)
    assert torch.equal(a, b)


# ---- streams, graphs, together -------------------------------------------------

def test_streams_and_graphs(lib):
    """All three calls captured into a graph and replayed on new inputs, while
    the same calls run on another stream with a workspace of their own."""
    n, G, H, d, page = 600, 2, 8, 128, 32
    dev = []
    for i in range(2):
        c = Paged([_randn((n, G, d), "bf16", 1)], [_randn((n, G, d), "bf16", 2)], page, "act", "bf16", extra_cols=3)
        c.table[0, -(-n // page):] = c.k.shape[0] - 1
        c.k.nan_to_num_()
        c.v.nan_to_num_()
        pd = _params(lib, B=1, n_heads=H, n_kv_heads=G, d=d, r=64, page=page, softmax_scale=0.1)
        dev.append(dict(c=c, p=pd, q=_randn((3, H, d), "bf16", 3).cuda(), kv=_randn((3, G, d), "bf16", 4).cuda(),
                        qo=torch.zeros(3, H, d, dtype=torch.bfloat16, device="cuda"), out=torch.zeros(3, H, d, dtype=torch.bfloat16, device="cuda"),
                        po=torch.zeros(3, H, d, dtype=torch.bfloat16, device="cuda"), cu=_i32([0, 3]), pos0=_i32([n]), lens=_i32([n + 3]),
                        ws=torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(pd, 3, 640)), dtype=torch.uint8, device="cuda")))

    def step(s):
        lib.gqa_cache_append(s["p"], s["q"], s["kv"], s["kv"], s["cu"], s["pos0"], s["c"].handle(), s["c"].table, q_out=s["qo"])
        lib.gqa_decode_attn(s["p"], s["qo"], s["c"].handle(), s["c"].table, s["lens"], 3, 640, s["out"], s["ws"])
        lib.gqa_prompt_attn(s["p"], s["q"], s["kv"], s["kv"], s["cu"], s["cu"], s["po"])

    step(dev[0])
    torch.cuda.synchronize()
    first = dev[0]["out"].clone(), dev[0]["po"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(dev[0])
    dev[0]["out"].zero_()
    dev[0]["po"].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        graph.replay()
        with torch.cuda.stream(side):
            step(dev[1])
    torch.cuda.synchronize()
    for s in dev:
        assert torch.equal(s["out"], first[0]) and torch.equal(s["po"], first[1])
    dev[0]["q"].neg_()
    dev[1]["q"].neg_()
    torch.cuda.synchronize()
    graph.replay()
    with torch.cuda.stream(side):
        step(dev[1])
    torch.cuda.synchronize()
    assert not torch.equal(dev[0]["out"], first[0])
    assert torch.equal(dev[0]["out"], dev[1]["out"]) and torch.equal(dev[0]["po"], dev[1]["po"])


@pytest.mark.parametrize("act,kv,d,page,window,sink", [("bf16", "act", 128, 16, 0, False), ("f16", "act", 64, 64, 60, True),
                                                        ("bf16", "fp8", 128, 32, 0, True)])
def test_a_layer_from_prompt_to_tokens(lib, act, kv, d, page, window, sink):
    """Prompts go through append and prompt attention, then tokens one and two
    at a time through append and decode attention; every output equals causal
    attention over the whole sequence."""
    prompts, steps, H, G = [70, 1, 131], [1, 1, 2, 1, 2, 2], 6, 2
    B, extra = len(prompts), sum(steps)
    total = [n + extra for n in prompts]
    X = [{x: _randn((n, h, d), act, 10 * b + i) for i, (x, h) in enumerate((("q", H), ("k", G), ("v", G)))} for b, n in enumerate(total)]
    cols = -(-max(total) // page)
    table = torch.from_numpy(np.random.RandomState(1).permutation(B * cols).reshape(B, cols).astype(np.int32)).cuda()
    shape = (B * cols, G, page, d)
    dt = ACT[act] if kv == "act" else torch.float8_e4m3fn
    kc, vc = torch.full(shape, float("nan")).to(dt).cuda(), torch.full(shape, float("nan")).to(dt).cuda()
    sc = [None if kv == "act" else torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2)]
    cache = lib.make_gqa_cache(kc, vc, *sc)
    sk = torch.randn(H, generator=torch.Generator().manual_seed(3)).cuda() if sink else None
    p = _params(lib, act, kv, B=B, n_heads=H, n_kv_heads=G, d=d, r=d // 2, page=page, window=window, softmax_scale=d ** -0.5)
    ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 2, max(total))), dtype=torch.uint8, device="cuda")
    err = _err()

    def packed(x, at, n):
        return torch.cat([X[b][x][a:a + m] for b, (a, m) in enumerate(zip(at, n))]).cuda()

    # prompts
    q, k, v = (packed(x, [0] * B, prompts) for x in "qkv")
    cu = _starts(prompts)
    lib.gqa_cache_append(p, q, k, v, cu, _i32([0] * B), cache, table, q_out=q, k_out=k, err=err)
    out = torch.empty_like(q)
    lib.gqa_prompt_attn(p, q, k, v, cu, cu, out, sink=sk, err=err)
    outs = [[o] for o in out.split(prompts)]
    turned, kept = [[t] for t in q.split(prompts)], k.split(prompts)
    lens = list(prompts)
    for T in steps:
        q, k, v = (packed(x, lens, [T] * B) for x in "qkv")
        lib.gqa_cache_append(p, q, k, v, _starts([T] * B), _i32(lens), cache, table, q_out=q, err=err)
        lens = [n + T for n in lens]
        out = torch.empty_like(q)
        lib.gqa_decode_attn(p, q, cache, table, _i32(lens), T, max(lens), out, ws, sink=sk, err=err)
        for b in range(B):
            outs[b].append(out[b * T:(b + 1) * T])
            turned[b].append(q[b * T:(b + 1) * T])
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    for b, n in enumerate(total):
        pos = np.arange(n)
        tq = torch.cat(turned[b])
        check_turned(tq, gqa.rotate(f64(X[b]["q"]), pos, d // 2, THETA), X[b]["q"], act, "queries")
        check_turned(kept[b], gqa.rotate(f64(X[b]["k"][:prompts[b]]), pos[:prompts[b]], d // 2, THETA), X[b]["k"], act, "keys")
        # attention over the rows as the calls read them: the packed turned
        # keys in the prompt, the cache's rows afterwards
        got, m = torch.cat(outs[b]), prompts[b]
        pages = table[b].long().cpu()
        rows = []
        for x, s in ((kc, sc[0]), (vc, sc[1])):
            y = x.cpu()[pages].double()
            if s is not None:
                y = y * s.cpu()[pages].double()[..., None]
            rows.append(y.transpose(1, 2).reshape(-1, G, d)[:n].numpy())
        want, mag, zmag = gqa.attend(f64(tq[:m]), f64(kept[b]), f64(X[b]["v"][:m]), pos[:m], d ** -0.5, window, None if sk is None else f64(sk))
        check_out(got[:m], want, mag, zmag, act, f"prompt {b}")
        want, mag, zmag = gqa.attend(f64(tq[m:]), rows[0], rows[1], pos[m:], d ** -0.5, window, None if sk is None else f64(sk))
        check_out(got[m:], want, mag, zmag, act, f"tokens {b}")


@pytest.mark.parametrize("kv", ["act", "fp8"])
def test_decode_many_passes_over_a_large_cache(lib, kv):
    """300 passes over a cache larger than L2, whose tiles arrive out of
    order: every pass gives the same bits, and those of a plain softmax."""
    B, n, H, G, d, page = 4, 40000, 16, 8, 128, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    cols = -(-n // page)
    k, v = (torch.randn((B * cols, G, page, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.randperm(B * cols, generator=g, device="cuda").int().view(B, cols)
    ks = vs = None
    kf, vf = k.float(), v.float()
    if kv == "fp8":
        (k, ks), (v, vs) = ([x for x in _quantise(y)] for y in (kf, vf))
        kf, vf = k.float() * ks[..., None], v.float() * vs[..., None]
    q = torch.randn((B, H, d), generator=g, device="cuda").bfloat16()
    p = _params(lib, "bf16", kv, B=B, n_heads=H, n_kv_heads=G, d=d, page=page, softmax_scale=0.1)
    lens = [n, n - 1, n - 777, n // 2]
    ws = torch.empty(lib.gqa_decode_attn_workspace_bytes(p, 1, n), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    err, lens_t, wrong = _err(), _i32(lens), torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        lib.gqa_decode_attn(p, q, lib.make_gqa_cache(k, v, ks, vs), table, lens_t, 1, n, outs[min(i, 1)], ws, err=err)
        if i:
            wrong += (outs[0] != outs[1]).sum()
    assert int(err[0]) == 0 and int(wrong) == 0
    for b in range(B):
        kk, vv = (x[table[b].long()].transpose(1, 2).reshape(-1, G, d)[:lens[b]].transpose(0, 1) for x in (kf, vf))
        z = torch.einsum("ghd,gmd->ghm", q[b].float().view(G, H // G, d), kk) * 0.1
        want = torch.softmax(z, -1) @ vv
        # weights of tens of thousands of keys, each off by 2^-8 at most
        assert (outs[0][b].float().view(G, H // G, d) - want).abs().max() < 2.0 ** -8 * (want.abs().max() + vv.abs().mean())


# ---- the ends of the ranges ----------------------------------------------------

def test_decode_more_than_64k_keys(lib):
    """Sequences on both sides of the length where splits grow again, one of
    them with a window."""
    lens, G, H, d, page = [66000, 65536, 65537, 3], 1, 4, 64, 256
    g = torch.Generator(device="cuda").manual_seed(5)
    cols = -(-max(lens) // page)
    k, v = (torch.randn((4 * cols, G, page, d), generator=g, device="cuda").half() for _ in range(2))
    table = torch.randperm(4 * cols, generator=g, device="cuda").int().view(4, cols)
    q = torch.randn((4, H, d), generator=g, device="cuda").half()
    for window in (0, 65600):
        p = _params(lib, "f16", B=4, n_heads=H, n_kv_heads=G, d=d, page=page, softmax_scale=0.2, window=window)
        ws = torch.empty(lib.gqa_decode_attn_workspace_bytes(p, 1, 66000), dtype=torch.uint8, device="cuda")
        out, err = torch.empty_like(q), _err()
        lib.gqa_decode_attn(p, q, lib.make_gqa_cache(k, v), table, _i32(lens), 1, 66000, out, ws, err=err)
        assert int(err[0]) == 0
        for b, n in enumerate(lens):
            kk, vv = (x[table[b].long()].transpose(1, 2).reshape(-1, G, d)[:n] for x in (k, v))
            want, mag, zmag = gqa.attend(f64(q[b:b + 1]), f64(kk), f64(vv), [n - 1], 0.2, window)
            check_out(out[b:b + 1], want, mag, zmag, "f16", f"{n} keys, window {window}")


def test_a_thousand_sequences(lib):
    """B at its limit, lengths of 0 to 40, through all three calls."""
    B, H, G, d, page = 1024, 4, 2, 64, 16
    rng = np.random.RandomState(3)
    lens = rng.randint(0, 41, B)
    lens[[0, 500, 1023]] = [0, 40, 1]
    n = int(lens.sum())
    p = _params(lib, B=B, n_heads=H, n_kv_heads=G, d=d, r=d, page=page, softmax_scale=0.2)
    q, k, v = _randn((n, H, d), "bf16", 1).cuda(), _randn((n, G, d), "bf16", 2).cuda(), _randn((n, G, d), "bf16", 3).cuda()
    cols = 3
    table = torch.from_numpy(rng.permutation(B * cols).reshape(B, cols).astype(np.int32)).cuda()
    kc, vc = (torch.zeros(B * cols, G, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu, err, ko, qo = _starts(lens), _err(), torch.empty_like(k), torch.empty_like(q)
    lib.gqa_cache_append(p, q, k, v, cu, _i32([0] * B), lib.make_gqa_cache(kc, vc), table, q_out=qo, k_out=ko, err=err)
    out = torch.empty_like(q)
    lib.gqa_prompt_attn(p, qo, ko, v, cu, cu, out, err=err)
    # each sequence's last query again, from the cache
    last = torch.from_numpy(np.maximum(np.cumsum(lens) - 1, 0)).cuda()
    dq = qo[last].contiguous()
    do = torch.empty_like(dq)
    ws = torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 1, 40)), dtype=torch.uint8, device="cuda")
    lib.gqa_decode_attn(p, dq, lib.make_gqa_cache(kc, vc), table, _i32(list(lens)), 1, 40, do, ws, err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    starts = np.concatenate([[0], np.cumsum(lens)])
    check_turned(ko, gqa.rotate(f64(k), np.concatenate([np.arange(m) for m in lens]), d, THETA), k, "bf16")
    for b, m in enumerate(lens):
        a = starts[b]
        want, mag, zmag = gqa.attend(f64(qo[a:a + m]), f64(ko[a:a + m]), f64(v[a:a + m]), np.arange(m), 0.2)
        check_out(out[a:a + m], want, mag, zmag, "bf16", f"prompt {b}")
        if m:
            check_out(do[b:b + 1], want[-1:], mag[-1:], zmag, "bf16", f"token {b}")
        else:
            assert (do[b] == 0).all()


def test_nothing_to_do(lib):
    """No tokens, no keys, an empty batch of lengths: outputs are zeros or left
    alone."""
    p = _params(lib, B=2, n_heads=4, n_kv_heads=2, d=64, r=64, page=16, softmax_scale=0.1)
    kc = torch.full((2, 2, 16, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    empty, kv = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    zero, table = _i32([0, 0, 0]), _i32([[0], [1]])
    lib.gqa_cache_append(p, empty, kv, kv, zero, _i32([0, 0]), lib.make_gqa_cache(kc, kc.clone()), table, q_out=empty, k_out=kv)
    lib.gqa_prompt_attn(p, empty, kv, kv, zero, zero, empty)
    q = _randn((2, 4, 64), "bf16", 1).cuda()
    out = torch.full_like(q, 9.0)
    lib.gqa_prompt_attn(p, q, kv, kv, _i32([0, 1, 2]), zero, out)
    assert (out == 0).all() and (kc == 3).all()
    out.fill_(9.0)
    lib.gqa_decode_attn(p, q, lib.make_gqa_cache(kc, kc.clone()), table, _i32([0, 0]), 1, 0, out,
                        sink=torch.zeros(4, device="cuda"))
    assert (out == 0).all()


def test_windows_wider_than_any_sequence(lib):
    for window in ((1 << 30) - 1, 1 << 30, (1 << 31) - 1):
        _prompt(lib, [200, 5], window=window)
        _decode(lib, [200, 5, 0], "bf16", "act", 4, 2, 64, 16, T=3, window=window)


def test_prompt_bad_sequences_between_good_ones(lib):
    p = _params(lib, B=5, n_heads=2, n_kv_heads=1, d=64, softmax_scale=0.125)
    q, k = _randn((60, 2, 64), "bf16", 1).cuda(), _randn((60, 1, 64), "bf16", 2).cuda()
    out, err = torch.full_like(q, 9.0), _err()
    # the third runs backwards, the fourth has keys from before the first
    lib.gqa_prompt_attn(p, q, k, k, _i32([0, 10, 25, 20, 40, 60]), _i32([0, 10, 25, -3, 40, 60]), out, err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == lib.DEV_ERR_RANGE
    for a, b in ((0, 10), (10, 25), (40, 60)):
        want, mag, zmag = gqa.attend(f64(q[a:b]), f64(k[a:b]), f64(k[a:b]), np.arange(b - a), 0.125)
        check_out(out[a:b], want, mag, zmag, "bf16")
    assert (out[25:40] == 9).all()


def test_append_rows_near_zero_and_not_finite(lib):
    """FP8 rows whose scale would be below fp32's smallest step are zeros; a
    NaN or an infinity shows in the row's scale and reaches who sees the row."""
    p = _params(lib, "bf16", "fp8", B=1, n_heads=2, n_kv_heads=1, d=64, r=0, page=16, softmax_scale=0.1)
    k = _randn((5, 1, 64), "bf16", 1).cuda()
    v = _randn((5, 1, 64), "bf16", 2).cuda()
    v[1] = 0
    v[1, 0, 3] = 2.0 ** -133
    v[3, 0, 7], v[4, 0, 9] = float("nan"), float("inf")
    kc, vc = (torch.zeros(1, 1, 16, 64, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(1, 1, 16, device="cuda") for _ in range(2))
    cache = lib.make_gqa_cache(kc, vc, ks, vs)
    lib.gqa_cache_append(p, None, k, v, _i32([0, 5]), _i32([0]), cache, _i32([[0]]))
    s = vs[0, 0, :5].cpu()
    assert torch.isfinite(s[:3]).all() and (s[:3] > 0).all() and torch.isnan(s[3]) and torch.isinf(s[4])
    back = vc[0, 0, :3].float().cpu() * s[:3, None]
    assert torch.isfinite(back).all() and back[1].abs().max() <= 2.0 ** -132
    q = _randn((3, 2, 64), "bf16", 3).cuda()
    out = torch.empty_like(q)
    lib.gqa_decode_attn(p, q, cache, _i32([[0]]), _i32([4]), 3, 16, out,
                        torch.empty(max(16, lib.gqa_decode_attn_workspace_bytes(p, 3, 16)), dtype=torch.uint8, device="cuda"))
    assert torch.isfinite(out[:2].float()).all() and torch.isnan(out[2].float()).all()

"""Host-side refusals of the grouped-query attention calls (no GPU needed,
nothing is launched).  The C calls run in a subprocess that sees no device."""

import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CALLS = r"""
import ctypes, sys
sys.path.insert(0, ROOT)
import long_context_sparse_gated_b200 as m
from long_context_sparse_gated_b200 import GqaRows, GqaCache
L = m.lib()
A = 0x10000  # a fake, 16-byte aligned address; every case below fails validation first
OK = dict(B=2, n_heads=8, n_kv_heads=2, d=128, r=64, page=64)
Q, KV, NONE = GqaRows(A, 1024, 128), GqaRows(A, 256, 128), GqaRows(None, 0, 0)
CACHE = GqaCache(A, A, None, None, 10)
def P(**kw):
    return ctypes.byref(m.make_gqa_params(**{**OK, **kw}))
def append(p=None, q=Q, k=KV, v=KV, n=4, cu=A, pos0=A, cache=CACHE, table=A, cols=8, qo=Q, ko=KV, **kw):
    return L.gqa_cache_append(P(**kw) if p is None else p, q, k, v, n, cu, pos0, cache, table, cols, qo, ko, None, None)
def decode(q=Q, cache=CACHE, table=A, cols=8, lens=A, T=1, n_max=100, sink=None, out=Q, ws=A, ws_bytes=0, **kw):
    return L.gqa_decode_attn(P(**kw), q, cache, table, cols, lens, T, n_max, sink, out, ws, ws_bytes, None, None)
def prompt(q=Q, k=KV, v=KV, n_q=4, n_k=4, cu_q=A, cu_k=A, sink=None, out=Q, **kw):
    return L.gqa_prompt_attn(P(**kw), q, k, v, n_q, n_k, cu_q, cu_k, sink, out, None, None)
r = []
def want(code, got, what):
    if got != code: r.append((what, got, code))
want(-1, L.gqa_cache_append(None, Q, KV, KV, 4, A, A, CACHE, A, 8, Q, KV, None, None), "no params")
for call in (append, decode, prompt):
    n = call.__name__
    want(-1, call(B=0), n + " B"); want(-2, call(B=2049), n + " B large")
    want(-1, call(n_kv_heads=3), n + " groups"); want(-2, call(n_heads=256), n + " heads")
    want(-2, call(d=96), n + " d"); want(-2, call(d=512), n + " d large"); want(-1, call(window=-1), n + " window")
    want(-2, call(act_fmt=m.ACT_F32), n + " act"); want(-1, call(softmax_scale=float("nan")), n + " scale")
    want(-1, call(softmax_scale=0.0), n + " scale 0"); want(-1, call(softmax_scale=float("inf")), n + " scale inf")
    want(-1, call(q=GqaRows(A, 64, 128)), n + " row stride"); want(-1, call(q=GqaRows(A, 1024, 0)), n + " broadcast heads")
    want(-1, call(q=GqaRows(A, -1024, 128)), n + " negative stride")
    want(-3, call(q=GqaRows(A + 2, 1024, 128)), n + " q address"); want(-3, call(q=GqaRows(A, 1028, 128)), n + " q stride")
    want(-2, call(q=GqaRows(A, 1 << 40, 128)), n + " q stride large")
for call in (append, decode):
    n = call.__name__
    want(-2, call(page=48), n + " page"); want(-2, call(page=8), n + " small page"); want(-2, call(kv_fmt=m.KV_FP8_BF16), n + " kv")
    want(-1, call(cache=GqaCache(None, A, None, None, 10)), n + " no k"); want(-1, call(kv_fmt=m.KV_FP8), n + " no scales")
    want(-1, call(cache=GqaCache(A, A, None, None, 0)), n + " no pages"); want(-1, call(table=None), n + " no table")
    want(-2, call(cache=GqaCache(A, A, None, None, 1 << 31)), n + " page ids"); want(-2, call(cols=1 << 30), n + " positions")
    want(-3, call(cache=GqaCache(A + 8, A, None, None, 10)), n + " cache address"); want(-3, call(table=A + 4), n + " table address")
    want(-3, call(kv_fmt=m.KV_FP8, cache=GqaCache(A, A, A + 4, A, 10)), n + " scale address")
want(-2, append(r=12), "r"); want(-2, append(r=136), "r over d"); want(-1, append(rope_theta=0.0), "theta")
want(-1, append(q=NONE), "q_out alone"); want(-1, append(qo=NONE), "q alone"); want(-1, append(k=NONE), "no k")
want(-1, append(cu=None), "no cu"); want(-1, append(pos0=None), "no pos0"); want(-1, append(n=-1), "n")
want(-2, append(n=1 << 31), "n large"); want(-3, append(cu=A + 4), "cu address"); want(0, append(n=0), "nothing")
want(-1, decode(lens=None), "no lens"); want(-1, decode(T=0), "T"); want(-2, decode(T=65), "T large")
want(-1, decode(n_max=-1), "n_max"); want(-1, decode(n_max=513), "n_max past the table"); want(-1, decode(out=NONE), "no out")
want(-3, decode(sink=A + 4), "sink address"); want(-3, decode(lens=A + 4), "lens address")
big = m.make_gqa_params(**OK)
need = L.gqa_decode_attn_workspace_bytes(ctypes.byref(big), 1, 100000)
if need:
    want(-4, decode(n_max=100000, cols=2000, ws_bytes=need - 1), "small ws")
    want(-4, decode(n_max=100000, cols=2000, ws=None, ws_bytes=need), "no ws")
want(-1, prompt(cu_q=None), "no cu_q"); want(-1, prompt(cu_k=None), "no cu_k"); want(-1, prompt(n_q=-1), "n_q")
want(-1, prompt(k=NONE), "no k"); want(-1, prompt(out=NONE), "no out"); want(-3, prompt(sink=A + 4), "sink address")
want(-2, prompt(n_k=1 << 31), "n_k large"); want(0, prompt(n_q=0), "nothing")
print(repr(r))
"""


def test_refusals():
    from long_context_sparse_gated_b200 import build
    build.build()
    out = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + _CALLS], capture_output=True, text=True,
                         env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), timeout=300)
    assert out.returncode == 0, out.stderr
    assert eval(out.stdout.strip().splitlines()[-1]) == []


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import long_context_sparse_gated_b200 as lib
    p = lib.make_gqa_params(B=1, n_heads=4, n_kv_heads=2, d=64)
    x, kv = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(TypeError):
        lib.gqa_prompt_attn(p, x, kv, kv, cu, cu, torch.empty_like(x))
    with pytest.raises(ValueError):
        lib.gqa_prompt_attn(p, x, kv, kv[:2], cu, cu, torch.empty_like(x))
    with pytest.raises(ValueError):
        lib.gqa_cache_append(p, x[:2], kv, kv, cu, cu, None, cu[None])
    with pytest.raises(ValueError):
        lib.gqa_decode_attn(p, x, None, cu[None], cu, 1, 3, torch.empty_like(x))
    with pytest.raises(ValueError):
        lib.make_gqa_cache(kv, kv[:1])


class _Cuda(torch.Tensor):
    """A host tensor that says it is on the current device, for the binding's
    checks (every call below fails one of them before a pointer is used)."""

    is_cuda = True

    def get_device(self):
        return 0


def _fake(x):
    return x.as_subclass(_Cuda)


def test_binding_refuses_wrong_types_and_caches(monkeypatch):
    import long_context_sparse_gated_b200 as lib
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class Unreached:
        def __getattr__(self, name):
            return lambda *a: pytest.fail("a refused call reached the library")

    monkeypatch.setattr(lib, "lib", lambda *a: Unreached())
    p = lib.make_gqa_params(B=1, n_heads=4, n_kv_heads=2, d=64, page=16)
    q, kv = _fake(torch.zeros(1, 4, 64).bfloat16()), _fake(torch.zeros(1, 2, 64).bfloat16())
    pages = _fake(torch.zeros(3, 2, 16, 64).bfloat16())
    codes, scale = _fake(torch.zeros(3, 2, 16, 64, dtype=torch.uint8)), _fake(torch.zeros(3, 2, 16))
    table, one, cu = (_fake(torch.zeros(s, dtype=torch.int32)) for s in ((1, 4), (1,), (2,)))
    cache = lib.make_gqa_cache(pages, pages)
    decode = lambda c=cache, t=table, n=one, x=q, o=q, **kw: lib.gqa_decode_attn(p, x, c, t, n, 1, 9, o, **kw)
    for call, what in ((lambda: decode(lib.make_gqa_cache(pages[:, :1], pages[:, :1])), ValueError),   # KV heads
                       (lambda: decode(lib.make_gqa_cache(codes, codes, scale, scale)), ValueError),     # FP8 for 16 bits
                       (lambda: decode(lib.make_gqa_cache(pages[:, :, :8], pages[:, :, :8])), (TypeError, ValueError)),
                       (lambda: decode(t=table.long()), TypeError), (lambda: decode(n=one.float()), TypeError),
                       (lambda: decode(t=_fake(torch.zeros(2, 4, dtype=torch.int32))), ValueError),
                       (lambda: decode(n=cu), ValueError), (lambda: decode(x=q.half()), TypeError),
                       (lambda: decode(sink=_fake(torch.zeros(3))), ValueError),
                       (lambda: decode(sink=_fake(torch.zeros(4, dtype=torch.float64))), ValueError),
                       (lambda: decode(o=_fake(torch.zeros(1, 4, 128).bfloat16())[:, :, ::2]), ValueError),
                       (lambda: lib.gqa_cache_append(p, None, kv, kv, one, one, cache, table), ValueError),
                       (lambda: lib.gqa_cache_append(p, None, kv, kv, cu, cu, cache, table), ValueError),
                       (lambda: lib.gqa_prompt_attn(p, q, kv, kv, cu, one, q), ValueError),
                       (lambda: lib.make_gqa_cache(codes, codes), ValueError),
                       (lambda: lib.make_gqa_cache(pages, pages, scale, scale), ValueError),
                       (lambda: lib.make_gqa_cache(codes, codes, scale, scale[:2]), ValueError)):
        with pytest.raises(what):
            call()
    # another device than the current one
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="device"):
        decode()


def test_binding_refuses_caches_and_workspaces_of_another_type_or_device(monkeypatch):
    import long_context_sparse_gated_b200 as lib
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class Elsewhere(_Cuda):
        def get_device(self):
            return 1

    class Unreached:
        def __getattr__(self, name):
            return lambda *a: pytest.fail("a refused call reached the library")

    monkeypatch.setattr(lib, "lib", lambda *a: Unreached())
    p = lib.make_gqa_params(B=1, n_heads=4, n_kv_heads=2, d=64, page=16)
    q, kv = _fake(torch.zeros(1, 4, 64).bfloat16()), _fake(torch.zeros(1, 2, 64).bfloat16())
    pages = torch.zeros(3, 2, 16, 64).bfloat16()
    codes, scale = _fake(torch.zeros(3, 2, 16, 64, dtype=torch.uint8)), _fake(torch.zeros(3, 2, 16))
    table, one, cu = (_fake(torch.zeros(s, dtype=torch.int32)) for s in ((1, 4), (1,), (2,)))
    cache = lib.make_gqa_cache(_fake(pages), _fake(pages))
    half = lib.make_gqa_cache(_fake(pages.half()), _fake(pages.half()))
    there = lib.make_gqa_cache(pages.as_subclass(Elsewhere), pages.as_subclass(Elsewhere))
    far = torch.zeros(64, dtype=torch.int32).as_subclass(Elsewhere)
    decode = lambda c, **kw: lib.gqa_decode_attn(p, q, c, table, one, 1, 9, q, **kw)
    append = lambda c, **kw: lib.gqa_cache_append(p, None, kv, kv, cu, one, c, table, **kw)
    for call, what in ((lambda: decode(half), TypeError), (lambda: append(half), TypeError),
                       (lambda: decode(there), ValueError), (lambda: append(there), ValueError),
                       (lambda: decode(cache, ws=far), ValueError), (lambda: decode(cache, err=far), ValueError),
                       (lambda: append(cache, err=far), ValueError),
                       (lambda: lib.gqa_prompt_attn(p, q, kv, kv, cu, cu, _fake(torch.zeros(1, 4, 64).bfloat16()), err=far), ValueError),
                       (lambda: lib.make_gqa_cache(codes, codes, scale.int(), scale.int()), ValueError),
                       (lambda: lib.make_gqa_cache(codes.view(torch.float8_e5m2), codes.view(torch.float8_e5m2), scale, scale), ValueError)):
        with pytest.raises(what):
            call()


def test_prompt_in_place_is_refused():
    code = """
import ctypes, sys
sys.path.insert(0, ROOT)
import long_context_sparse_gated_b200 as m
A, B, C = 0x10000, 0x20000, 0x30000
rows = lambda at: m.GqaRows(at, 512, 128)
p = ctypes.byref(m.make_gqa_params(B=1, n_heads=4, n_kv_heads=4, d=128))
for out in (A, B, C):
    st = m.lib().gqa_prompt_attn(p, rows(A), rows(B), rows(C), 4, 4, A, A, None, rows(out), None, None)
    assert st == -1, (hex(out), st)
""".replace("ROOT", repr(ROOT))
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": ""}
    done = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr

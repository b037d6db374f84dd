"""Host-side bounds of the grouped-query attention calls (no GPU needed,
nothing is launched)."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_sparse_gated_b200 import build
    build.build()


def _run(code):
    """The last line that `code` prints, in a process that sees no device."""
    head = f"ROOT = {ROOT!r}\nimport ctypes, sys\nsys.path.insert(0, ROOT)\nimport long_context_sparse_gated_b200 as m\nL = m.lib()\n"
    done = subprocess.run([sys.executable, "-c", head + code], capture_output=True, text=True, timeout=300,
                          env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert done.returncode == 0, done.stderr
    return eval(done.stdout.strip().splitlines()[-1])


def _splits(length, T, window, n_max):
    """Splits that the device gives a sequence: its seen keys in blocks of 32,
    8 to 64 blocks a split."""
    length = max(0, min(length, n_max))
    lo = max(0, length - T - window + 1) if 0 < window < 1 << 30 else 0
    n = -(-length // 32) - lo // 32 if length > lo else 0
    c = 64 if n > 2048 else next((c for c in (8, 16) if c * 12 >= n), 32)
    return max(1, -(-n // c))


CASES = [(T, window, n_max) for T in (1, 64) for window in (0, 1, 500, 70000, (1 << 30) - 1, 1 << 30, (1 << 31) - 1)
         for n_max in (0, 1, 300, 3000, 6150, 66000, (1 << 30) - 1)]


def test_decode_workspace_holds_every_split():
    B, H, d = 3, 4, 64
    got = _run(f"print([L.gqa_decode_attn_workspace_bytes(ctypes.byref(m.make_gqa_params(B={B}, n_heads={H}, n_kv_heads=2, d={d}, "
               f"window=w)), T, n) for T, w, n in {CASES}])")
    for (T, window, n_max), size in zip(CASES, got):
        lengths = {n_max, n_max // 2, min(n_max, window), min(n_max, window + T), min(n_max, window + T + 31), 2049 * 32, 2048 * 32,
                   96 * 32, 192 * 32, 97 * 32, 193 * 32, 256, 257}
        most = max(_splits(n, T, window, n_max) for n in lengths if n <= n_max)
        assert size >= (0 if most == 1 else B * most * T * H * (d + 2) * 4), (T, window, n_max)


def test_decode_refuses_lengths_of_2_to_the_30():
    """Sums of positions and windows are 32-bit on the device, and a window of
    2^30 counts as none there; pages may repeat in a table, so such lengths
    need no such memory."""
    code = """
A = 0x10000
rows, cache = m.GqaRows(A, 1024, 128), m.GqaCache(A, A, None, None, 10)
def decode(n_max, window):
    p = ctypes.byref(m.make_gqa_params(B=2, n_heads=8, n_kv_heads=2, d=128, page=256, window=window))
    need = L.gqa_decode_attn_workspace_bytes(p, 1, n_max)
    # (with one byte too few, so that nothing is launched whatever the answer)
    return L.gqa_decode_attn(p, rows, cache, A, (1 << 23) - 1, A, 1, n_max, None, rows, A, max(0, need - 1), None, None), need > 0
print([decode(n, w) for n in ((1 << 30) - 1, 1 << 30, (1 << 30) + (1 << 20), (1 << 31) - 257) for w in (0, 1 << 30)])
"""
    assert _run(code) == [(-4, True)] * 2 + [(-2, False)] * 6


def test_strides_of_a_single_row_or_head_do_not_count():
    """A view of one row or one head may have any stride there (rows of a
    tensor whose width is no multiple of 8, a broadcast dim)."""
    import torch

    import long_context_sparse_gated_b200 as lib

    class OnDevice(torch.Tensor):
        def get_device(self):
            return 0

    def rows(x, n, heads):
        r = lib._rows(x.as_subclass(OnDevice), torch.bfloat16, 0, n, heads, 64)
        return r.row_stride, r.head_stride

    x = torch.zeros(5, 4 * 64 + 3, dtype=torch.bfloat16)
    assert rows(x[:1, :256].view(1, 4, 64), 1, 4) == (64, 64)
    y = torch.zeros(6, 3, 64, dtype=torch.bfloat16)
    assert rows(y.as_strided((6, 1, 64), (192, 1, 1)), 6, 1) == (192, 64)
    assert rows(y.as_strided((1, 3, 64), (0, 64, 1)), 1, 3) == (64, 64)
    assert rows(y, 6, 3) == (192, 64) and rows(y.transpose(0, 1), 3, 6) == (64, 192)

"""Inputs and bounds shared by the grouped-query attention tests.

Bounds, element by element (eps / 2 is half a step of the activation type,
relative: 2^-8 for BF16, 2^-11 for FP16):

* attention outputs: the result is rounded once (eps/2 |o|), and each
  probability may be rounded to 16 bits before it weighs its value (eps/2
  sum p|v|).  Logits are fp32 sums of at most 128 exact products; any order
  of summation in tensor-core blocks of 16 stays within 16 roundings of at
  most 2^-23 of the sum of magnitudes, as does the scale's; an error dz of a
  logit changes p by dz and the denominator by as much, and the exponential
  and the long fp32 sums add a few 2^-22.  With an FP8 cache the value times
  its scale is another fp32 rounding.
* turned rows: rounded once, after fp32 products of cosines that are within
  2^-22 (angles are reduced in fp64).
* FP8 rows: a scale within 2^-21; a value within half a step of its code
  (2^-4 relative, 2^-10 of the scale below 2^-6 of it), plus the fp32 error
  of the value.
"""

import numpy as np
import torch

from oracle import gqa

ACT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def f64(x):
    return x.detach().double().cpu().numpy()


def check_out(got, want, mag, zmag, act, what=""):
    got = f64(got) if torch.is_tensor(got) else got
    same = ~np.isfinite(want)
    np.testing.assert_array_equal(np.isnan(got[same]), np.isnan(want[same]), err_msg=what)
    dz = 2 * 16 * 2.0 ** -23 * zmag
    tol = HALF_STEP[act] * (np.abs(want) + mag) + (2 * dz + 2.0 ** -19) * mag
    if act == "f16":
        tol = tol + 2.0 ** -24  # the smallest FP16 step
    bad = ~(np.abs(got - want) <= tol) & ~same
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]}, allowed {tol[bad][0]}")


def check_turned(got, want, x, act, what=""):
    tol = HALF_STEP[act] * np.abs(want) + 2.0 ** -20 * np.abs(f64(x)).max(initial=0)
    if act == "f16":
        tol = tol + 2.0 ** -24
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), f"{what}: {f64(got)[bad][0]} for {want[bad][0]}"


def check_fp8(codes, scale, want, what=""):
    """Rows of codes [..., d] and scales [...] for values `want`."""
    s = gqa.row_scale(want)
    scale = f64(scale)
    np.testing.assert_allclose(scale, s, rtol=2.0 ** -21, err_msg=what)
    amax = np.abs(want).max(-1, keepdims=True)
    got = f64(codes.float()) * scale[..., None]
    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s[..., None]) + 2.0 ** -20 * amax
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {got[bad][0]} for {want[bad][0]}"


def quantise(x):
    """Rows of a float tensor as E4M3 codes and fp32 scales."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


class Paged:
    """A paged cache holding the given keys and values, with NaN everywhere
    else (slots behind a sequence, pages of nobody)."""

    def __init__(self, ks, vs, page, kv, act, extra_cols=1, seed=0, device="cuda"):
        self.page, self.kv, self.act, self.device = page, kv, act, device
        lens = [len(x) for x in ks]
        G, d = ks[0].shape[1:]
        used = [-(-n // page) for n in lens]
        n_pages = sum(used) + 2
        cols = max(used) + extra_cols
        order = np.random.RandomState(seed).permutation(n_pages)
        # what no sequence reaches: page ids that are no pages
        table = np.full((len(lens), cols), 0x7fffffff, np.int32)
        table[:, 1::2] = -1
        shape = (n_pages, G, page, d)
        k = torch.full(shape, float("nan"))
        v = torch.full(shape, float("nan"))
        at = 0
        for b, n in enumerate(lens):
            for c in range(used[b]):
                table[b, c] = order[at]
                rows = slice(c * page, min(n, (c + 1) * page))
                m = rows.stop - rows.start
                k[order[at], :, :m] = torch.as_tensor(ks[b][rows]).transpose(0, 1).float()
                v[order[at], :, :m] = torch.as_tensor(vs[b][rows]).transpose(0, 1).float()
                at += 1
        self.table = torch.from_numpy(table).to(device)
        self.k_scale = self.v_scale = None
        if kv == "act":
            self.k, self.v = k.to(ACT[act]).to(device), v.to(ACT[act]).to(device)
        else:
            (self.k, self.k_scale), (self.v, self.v_scale) = ([y.to(device) for y in quantise(x)] for x in (k, v))

    def handle(self):
        import long_context_sparse_gated_b200 as lib
        return lib.make_gqa_cache(self.k, self.v, self.k_scale, self.v_scale)

    def rows(self, b, n):
        """Sequence b's keys and values as the cache holds them, [n, G, d]."""
        out = []
        for x, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            pages = self.table[b, :-(-n // self.page)].long().cpu()
            y = x.cpu()[pages].double()
            if s is not None:
                y = y * s.cpu()[pages].double()[..., None]
            out.append(y.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n].numpy())
        return out

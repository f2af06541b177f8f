"""Helpers of the paged-cache and attention tests: caches with known
contents, the 64-bit reference, and the error bounds.

Bounds, in the oracle's a = sum_j p_j |v_j| / sum_j p_j and e = scale * max_j
sum_d |q_d k_jd| (u = torch.finfo(type).eps / 2, half a step):

* a score is a sum of up to 128 products in at most 16 fp32 steps, each off by
  up to 2^-23 of the sum of absolute values, and its operands carry at least 22
  bits: it is off by at most 2^-18 e.  exp2 adds 2^-21.  An error x of every
  exponent moves o by at most 2 x a (numerator and denominator).
* the products with the values are summed in fp32: n keys in at most n/16 + 32
  steps, 2^-23 a each.
* a probability rounded to type t for that product is off by u_t of itself; one
  below fp16's normal range by up to 2^-25 of the row's largest, hence n 2^-25
  max|v|.  (bf16 and tf32 have fp32's range.)
* the result is rounded once: u |o|, and 2^-25 below fp16's normal range.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle as o

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8,
             "tf32": 2.0 ** -11}      # fp32's range, fp16's significand


def bound(ref, a, e, n, vmax, out_dtype, p_dtype):
    """Largest |o - ref| allowed, for n keys whose values are up to vmax."""
    err = a * (2 * (2.0 ** -18 * e[..., None] + 2.0 ** -21) + (n / 16 + 32) * 2.0 ** -23)
    if p_dtype != torch.float32:
        err = err + a * HALF_STEP[p_dtype]
    if p_dtype == torch.float16:
        err = err + n * 2.0 ** -25 * vmax
    err = err + HALF_STEP[out_dtype] * (np.abs(ref) + err)
    return err + (2.0 ** -25 if out_dtype == torch.float16 else 1e-37)


def check(got, ref, tol, what=""):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    err = np.abs(got - ref)
    worst = np.max(err / tol) if err.size else 0.0
    assert np.all(err <= tol), f"{what}: max err/bound {worst:.3g}, max err {err.max():.3g}"


class Cache:
    """A paged cache filled by the oracle's quantiser, its pages handed out
    in no order; free pages and the ends of last pages hold codes under NaN
    and infinite scales, unused table entries -1."""

    def __init__(self, lens, heads, page, dim, seed=0, spare=2, extra_cols=1, key_gain=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.page, self.dim = list(lens), heads, page, dim
        used = [-(-n // page) for n in lens]
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages)
        cols = max(used + [0]) + extra_cols
        self.table = np.full((len(lens), cols), -1, np.int32)
        shape = (self.n_pages, heads, page)
        codes = rng.integers(-127, 128, (2,) + shape + (dim,)).astype(np.int8)
        scales = np.where(rng.random((2,) + shape + (dim // 32,)) < 0.5, np.nan, np.inf).astype(np.float16)
        self.rows = []                                  # (k, v) fp32 rows as written
        at = 0
        for b, n in enumerate(lens):
            self.table[b, : used[b]] = order[at: at + used[b]]
            at += used[b]
            x = rng.standard_normal((2, n, heads, dim)).astype(np.float32)
            x[0, :, :, : max(1, dim // 32)] *= 4 * key_gain      # key channels that stand out
            self.rows.append((x[0], x[1]))
            if n == 0:
                continue
            pos = np.arange(n)
            pg, off = self.table[b, pos // page], pos % page
            for w in range(2):
                qq, dd = o.quantize_q8_0(x[w].reshape(n * heads, dim))
                codes[w][pg, :, off] = qq.reshape(n, heads, dim)
                scales[w][pg, :, off] = dd.view(np.float16).reshape(n, heads, dim // 32)
        self.codes, self.scales = codes, scales

    def device(self):
        t = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in
             (self.codes[0], self.scales[0], self.codes[1], self.scales[1])]
        return tuple(t)

    def values(self, b):
        """The dequantised (k, v) of sequence b, fp64 [n, heads, dim]."""
        pos = np.arange(self.lens[b])
        pg, off = self.table[b, pos // self.page], pos % self.page
        out = []
        for w in range(2):
            c = self.codes[w][pg, :, off].astype(np.float64)
            s = self.scales[w][pg, :, off].astype(np.float64)
            out.append(c * np.repeat(s, 32, axis=-1))
        return out

    def dev_table(self):
        return torch.from_numpy(self.table).cuda()

    def dev_lens(self):
        return torch.tensor(self.lens, dtype=torch.int32).cuda()


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()

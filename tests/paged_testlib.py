"""Shared helpers of the paged-cache tests: small caches with hostile unused
memory, the calls through the binding, and tolerances from the arithmetic."""

from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

from kv_cache_sparsity_b200 import hylra as H

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def pool_tensor(pages, heads, page, d, dtype, layout, device="cuda"):
    """A [pages, heads, page, d] tensor in one of three memory layouts, filled with NaN."""
    if layout == "hnd":
        t = torch.empty(pages, heads, page, d, dtype=dtype, device=device)
    elif layout == "nhd":
        t = torch.empty(pages, page, heads, d, dtype=dtype, device=device).transpose(1, 2)
    else:  # "slice": every second half of rows twice as long, in a pool of K and V pages
        t = torch.empty(pages, 2, heads, page, 2 * d, dtype=dtype, device=device)[:, 1, :, :, d:]
    return t.fill_(math.nan)


@dataclasses.dataclass
class Cache:
    page: int
    hq: int
    hkv: int
    d: int
    dtype: str
    lens: tuple
    keys: torch.Tensor
    vals: torch.Tensor
    table: torch.Tensor
    seqlens: torch.Tensor
    q: torch.Tensor
    shape: H.PagedShape
    ws: torch.Tensor
    scale: float

    def status(self):
        torch.cuda.synchronize()
        return H.read_status(self.ws, clear=True)

    def result(self):
        B = len(self.lens)
        return (torch.full((B, self.hq, self.d), math.nan, device="cuda"),
                torch.full((B, self.hq), math.nan, device="cuda"))

    def decode(self, **kw):
        out, lse = self.result()
        H.paged_decode(self.shape, self.q, self.keys, self.vals, self.table, self.seqlens, out,
                       self.ws, lse=lse, **kw)
        return out, lse

    def decode_topk(self, idx, **kw):
        out, lse = self.result()
        H.paged_decode_topk(self.shape, self.q, self.keys, self.vals, self.table, self.seqlens,
                            idx, out, self.ws, lse=lse, **kw)
        return out, lse


def workspace(shape):
    ws = torch.empty(H.paged_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    H.workspace_init(ws)
    return ws


def make_cache(lens, page=16, hq=8, hkv=2, d=128, dtype="bf16", layout="hnd", seed=0, scale=0.0,
               spare=3, cols=None, sharp=1.0):
    """Random keys and values in randomly placed pages.  Rows past a sequence's
    end, unused pages and unused table entries hold NaN and ids out of range."""
    g = torch.Generator().manual_seed(seed)
    t = DTYPES[dtype]
    have = [-(-n // page) for n in lens]
    pool = sum(have) + spare
    cols = cols or max(1, max(have))
    order = torch.randperm(pool, generator=g)
    table = torch.full((len(lens), cols), 2**30, dtype=torch.int32)
    keys = pool_tensor(pool, hkv, page, d, t, layout)
    vals = pool_tensor(pool, hkv, page, d, t, layout)
    at = 0
    for b, n in enumerate(lens):
        pages = order[at:at + have[b]]
        at += have[b]
        table[b, : have[b]] = pages.to(torch.int32)
        for i, p in enumerate(pages.tolist()):
            rows = min(page, n - i * page)
            keys[p, :, :rows] = torch.randn(hkv, rows, d, generator=g).to(t).cuda()
            vals[p, :, :rows] = torch.randn(hkv, rows, d, generator=g).to(t).cuda()
    q = (sharp * torch.randn(len(lens), hq, d, generator=g)).to(t).cuda()
    shape = H.make_paged_shape(len(lens), hq, hkv, page, pool, cols,
                               dtype=H.BF16 if dtype == "bf16" else H.FP16, head_dim=d, pool=keys,
                               scale=scale)
    return Cache(page, hq, hkv, d, dtype, tuple(lens), keys, vals, table.cuda(),
                 torch.tensor(lens, dtype=torch.int32, device="cuda"), q, shape, workspace(shape),
                 scale or 1.0 / math.sqrt(d))


def attention_tolerance(c: Cache):
    """(largest error of an output element, of an lse) that the arithmetic allows.

    A logit is a sum of d exact products in fp32.  Each addition of the matrix
    unit may be off by one unit of the running sum (2^-23: it need not round to
    nearest), so a logit is off by at most d * 2^-23 * S, S = the largest
    scale * sum |q_i k_i|.  Subtracting the maximum and multiplying by the scale
    in one fused step adds 2^-24 of a number below 2 S * log2(e), and the scale
    itself is rounded to fp32: 3 S * 2^-24 more.  A weight exp(x) is then off
    by that much, by 2^-22 (exponential) and by its split into 16-bit terms:
    at most (eps/2)^3 = 2^-24 (three bf16 terms) or (eps/2)^2 = 2^-22 (two fp16
    terms).  out = sum p v / sum p doubles the weights' part; the sums have at
    most n additions of 2^-23 each, but run in tiles: at most 8 * 16 in the
    matrix unit, then one a tile of one CTA, 8 for its four warps, and one a CTA that
    holds part of the head: the tiles of 64 tokens or more that one CTA adds up
    and the CTAs are together below n / 128 + 256.  The result is stored in
    fp32 (2^-24), all times the largest |v|.  lse: the same once, plus the
    logarithm's 2^-22 of a number below S + log n.
    """
    ok = [n for n in c.lens if n > 0]
    if not ok:
        return 0.0, 0.0
    fin = lambda t: torch.nan_to_num(t.float(), nan=0.0).abs()  # noqa: E731
    k, v = fin(c.keys).amax((0, 2)), float(fin(c.vals).max())
    r = c.hq // c.hkv
    S = float((c.q.float().abs().view(-1, c.hkv, r, c.d) * k[None, :, None]).sum(-1).max()) * c.scale
    logit = c.d * 2.0**-23 * S + 3 * S * 2.0**-24 + 2 * 2.0**-24 * S * 1.4427
    weight = logit + 2.0**-22 + 2.0**-22
    adds = 128 + max(ok) / 128 + 8 + 256
    out = v * (2 * weight + 2 * adds * 2.0**-23 + 2.0**-24)
    return out, weight + adds * 2.0**-23 + (S + math.log(max(ok)) + 20) * 2.0**-22


def check_attention(c: Cache, got, want, what=""):
    (out, lse), (o_ref, l_ref) = got, want
    tol_o, tol_l = attention_tolerance(c)
    o, l = f64(out), f64(lse)
    assert np.array_equal(np.isneginf(l), np.isneginf(l_ref)), what
    assert np.isfinite(o).all(), what
    live = np.isfinite(l_ref)
    assert np.all(o[~live] == 0), what
    err_o = float(np.abs(o - o_ref).max(initial=0.0))
    err_l = float(np.abs(l[live] - l_ref[live]).max(initial=0.0))
    assert err_o <= tol_o and err_l <= tol_l, (what, err_o, tol_o, err_l, tol_l)
    return err_o, err_l


# Inputs whose outputs show the weights themselves: keys and queries along the first dimension
# (a raw logit is one exact product), values that are unit vectors (token t: dimension t mod d).

FACTORS = (1.0, -1.0, 2.0, 0.5)  # the query of each of four heads


def ladder(n, seed=0):
    """The keys' first elements: multiples of 2^-5 below 8, exact in every type; the first is 0 and
    the second the largest, so that every head's range of logits is the same for all n >= 2."""
    c = np.random.default_rng(seed).integers(0, 256, n) / 32
    c[:2] = (0, 255 / 32)
    return c


def ladder_weights(c, scale):
    """[heads, n]: the weights relative to the largest, in 64 bits."""
    a = scale * np.outer(FACTORS, c)
    return np.exp(a - a.max(1, keepdims=True))


def ladder_result(c, w, scale, d):
    """(out [heads, d], lse [heads]) of these weights."""
    z = w.sum(1)
    out = np.stack([np.bincount(np.arange(len(c)) % d, x, d) for x in w]) / z[:, None]
    return out, scale * np.outer(FACTORS, c).max(1) + np.log(z)


def ladder_tolerance(n, d, dtype, scale, heads=1):
    """(relative, absolute) largest error of an output element, and the largest of an lse.

    A logit less the largest is exact; the scale in base 2 and its product are rounded (2^-24 each), so
    that exp2's argument is off by X * 2^-23, X its largest size, and a weight by that times ln 2 and
    by 2^-22 (the exponential).  It goes into the product with V as 16-bit terms: three of bf16 leave
    2^-24 of it, two of fp16 2^-22 of it or 2^-37 of the largest.  A unit of at most 128 tokens adds to the
    denominator at most four weights in a lane, then three times over lanes and four over warps (12 of
    2^-24), and to an output at most two weights of a token's dimension, in the matrix unit (2 of 2^-23),
    the terms (2 of 2^-24) and the running sum (2^-24).  Dividing is two roundings.
    More than one unit of 64 tokens or more: a weight is rescaled by the maxima of the units after it in its
    CTA and then by those of the CTAs, in the join twice.  The arguments of these exponentials add up to X at
    most; each costs 2^-22 and two roundings; and a sum of one CTA or one of CTAs is rounded per unit.
    out is a quotient of two such sums.
    """
    x = scale * 1.4426950408889634 * max(abs(f) for f in FACTORS) * 255 / 32
    split = 2.0**-24 if dtype == "bf16" else 2.0**-22
    weight = math.log(2) * x * 2.0**-23 + 2.0**-22
    adds = 12 * 2.0**-24
    unit = 64 if d == 128 else 128
    if n > unit:
        units = -(-n // unit)
        # two CTAs to an SM or more on 148 SMs
        rescales = -(-units * heads // 296) + 2
        weight += math.log(2) * x * 2.0**-23 + rescales * (2.0**-22 + 2.0**-23)
        adds += (units + 16) * 2.0**-24
    out = 2 * (weight + adds) + split + 2 * 2.0**-23 + 5 * 2.0**-24
    # an lse: its denominator's error, the logarithm's 2^-22 and the roundings of a sum below this
    size = x * math.log(2) + math.log(n) + 9
    return out, (2.0**-37 if dtype == "fp16" else 0.0), weight + adds + size * (2.0**-22 + 4 * 2.0**-24)


def ladder_check(got, want, tol):
    """Whether out and lse are within the tolerance everywhere."""
    (out, lse), (o, l), (rel, low, abs_l) = got, want, tol
    return bool(np.all(np.abs(out - o) <= rel * o + low) and np.all(np.abs(lse - l) <= abs_l))

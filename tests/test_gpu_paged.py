"""Paged-cache calls on the GPU against the 64-bit oracle: every page size,
head dimension, type and pool layout; lengths around the page and tile edges;
empty rows; hostile unused memory; refused requests and bad indices; the calls
in a row, on other streams and in CUDA graphs."""

import math

import numpy as np
import pytest
import torch

from kv_cache_sparsity_b200 import build as hbuild
from kv_cache_sparsity_b200 import hylra as H
from oracle import paged_oracle as O

import paged_testlib as T

pytestmark = pytest.mark.gpu

EDGES = (0, 1, 15, 16, 17, 127, 128, 129, 255, 1000)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hbuild.build()
    H.load()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------- tables


class Requests:
    """Inputs of paged_tables with random pages, and the oracle's answer."""

    def __init__(self, cached, new, page=16, free=None, cols=None, pad=0, seed=0, slots=None):
        rng = np.random.default_rng(seed)
        have = [O.pages_of(max(0, c), page) for c in cached]
        # the pool and the free list cover every request that a table row could hold
        need = [O.pages_of(max(0, c) + min(max(0, w), H.MAX_SEQLEN // 2), page)
                for c, w in zip(cached, new)]
        self.page, self.cached, self.new = page, cached, new
        self.cols = cols or max(1, max(need))
        pool = sum(have) + sum(need) + 8
        order = rng.permutation(pool)
        self.num_pages = pool
        self.table = np.full((len(cached), self.cols), -5, dtype=np.int64)
        at = 0
        for b, n in enumerate(have):
            n = min(n, self.cols)
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free_pages = order[at:]
        self.free = len(self.free_pages) if free is None else free
        self.slots = sum(max(0, w) for w in new) + pad if slots is None else slots
        self.shape = H.make_paged_shape(len(cached), 8, 2, page, pool, self.cols)
        self.ws = T.workspace(self.shape)

    def run(self, alias=False):
        B = len(self.cached)
        cached, free = i32(self.cached), i32([self.free])
        table = i32(self.table.tolist())
        lens = cached if alias else torch.full((B,), -9, dtype=torch.int32, device="cuda")
        left = free if alias else i32([-9])
        cu = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
        slots = torch.full((self.slots,), -9, dtype=torch.int32, device="cuda")
        H.paged_tables(self.shape, cached, i32(self.new), i32(self.free_pages.tolist()), free,
                       table, lens, cu, slots, left, self.ws)
        torch.cuda.synchronize()
        return tuple(x.cpu().numpy() for x in (table, slots, lens, cu, left))

    def check(self, alias=False):
        want = O.tables(self.cached, self.new, self.free_pages, self.free, self.table, self.page,
                        self.num_pages, self.slots)
        got = self.run(alias)
        for name, a, b in zip(("table", "slots", "seqlens", "cu", "left"), got, want):
            assert np.array_equal(a, np.asarray(b).reshape(a.shape)), name
        bits = (H.STATUS_BAD_SEQLEN * want[5] | H.STATUS_NO_PAGES * want[6]
                | H.STATUS_BAD_INDEX * want[7])
        assert H.read_status(self.ws) == bits
        return got


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("alias", [False, True])
def test_tables_edges(page, alias):
    cached = [0, 0, 1, page - 1, page, page + 1, 5 * page, 0, 3 * page - 1, 7]
    new = [0, 1, 1, 1, 1, page, 2 * page + 3, 10 * page, 1, 0]
    Requests(cached, new, page, pad=13, seed=page).check(alias)


@pytest.mark.parametrize("batch,hi,new_hi", [(1, 1, 1), (1, 100000, 5000), (7, 300, 40),
                                             (255, 900, 3), (256, 900, 3), (257, 100, 1),
                                             (1024, 4000, 1), (1023, 50, 100), (64, 2000, 4000)])
def test_tables_random(batch, hi, new_hi):
    rng = np.random.default_rng(batch)
    cached = rng.integers(0, hi + 1, batch).tolist()
    new = rng.integers(0, new_hi + 1, batch).tolist()
    Requests(cached, new, 16, pad=3, seed=batch).check()
    # again with too few pages, down to none
    for free in (0, 1, batch // 2):
        Requests(cached, new, 16, free=free, seed=batch).check(alias=True)


def test_tables_refuses_requests_in_order():
    # 2 free pages: the first takes one, the second needs two, the third none, the fourth one
    r = Requests([16, 15, 3, 32], [1, 18, 4, 1], 16, free=2)
    table, slots, lens, cu, left = r.check()
    assert lens.tolist() == [17, 15, 7, 32] and left.tolist() == [1]
    assert cu.tolist() == [0, 1, 19, 23, 24] and (slots[1:19] == -1).all()


def test_tables_bad_lengths():
    # negative lengths, a row that is too short, too few slots
    Requests([5, -1, 10, 40, 8], [3, 4, -2, 200, 2], 16, cols=4, pad=5).check()
    Requests([5, 6, 7, 8], [3, 30, 4, 2], 16, slots=20).check()
    Requests([0, 0], [2**31 - 1, 2**31 - 1], 128, cols=4, slots=64).check()


def test_tables_bad_pages():
    r = Requests([5, 40, 16], [20, 3, 40], 16, seed=3)
    r.table[1, 2] = r.num_pages  # the partial page of request 1
    r.free_pages[r.free - 2] = -7
    r.check()
    for free in (-1, 10**6):
        Requests([5, 40], [20, 3], 16, free=free).check()


def test_tables_needs_no_free_list_or_slots():
    Requests([5, 40], [3, 0], 16, free=0, seed=1).check()
    Requests([5, 40], [0, 0], 16, seed=1, slots=0).check()


# ------------------------------------------------------------------- append


def append_case(held, new, page, hkv=2, d=128, dtype="bf16", layout="hnd", fused=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = T.DTYPES[dtype]
    total = [a + b for a, b in zip(held, new)]
    have = [O.pages_of(n, page) for n in total]
    pool = sum(have) + 2
    order = torch.randperm(pool, generator=g).tolist()
    keys, vals = (T.pool_tensor(pool, hkv, page, d, t, layout) for _ in range(2))
    slots, at = [], 0
    for n, w, m in zip(held, new, have):
        pages = order[at:at + m]
        at += m
        for pos in range(n):
            keys[pages[pos // page], :, pos % page] = torch.randn(hkv, d, generator=g).to(t).cuda()
        slots += [pages[pos // page] * page + pos % page for pos in range(n, n + w)]
    heads = 3 * hkv if fused else hkv
    rows = torch.randn(2, len(slots), heads, d, generator=g).to(t).cuda()
    k_new, v_new = rows[0][:, :hkv], rows[1][:, heads - hkv:]
    means = torch.full((pool, hkv, d), math.nan, dtype=t, device="cuda")
    shape = H.make_paged_shape(max(1, len(held)), hkv, hkv, page, pool, 8,
                               dtype=H.BF16 if dtype == "bf16" else H.FP16, head_dim=d, pool=keys)
    return shape, keys, vals, means, k_new, v_new, slots


def check_append(case, page, slots=None):
    shape, keys, vals, means, k_new, v_new, own = case
    slots = own if slots is None else slots
    k, v, m = T.f64(keys), T.f64(vals), T.f64(means)
    O.append(k, v, m, T.f64(k_new), T.f64(v_new), slots, page)
    ws = T.workspace(shape)
    H.paged_append(shape, k_new, v_new, i32(slots), keys, vals, means, ws)
    torch.cuda.synchronize()
    assert np.array_equal(T.f64(keys), k, equal_nan=True)
    assert np.array_equal(T.f64(vals), v, equal_nan=True)
    got = T.f64(means)
    assert np.array_equal(np.isnan(got), np.isnan(m))
    # a sum of `page` values in fp32 (2^-24 an addition), one division, one rounding to 16 bits
    live = ~np.isnan(m)
    size = np.nanmax(np.abs(k), initial=0.0)
    tol = np.abs(m[live]) * torch.finfo(means.dtype).eps / 2 + size * (page + 1) * 2.0**-24
    # fp16 rounds values below 2^-14 to multiples of 2^-24
    tol = tol + (2.0**-25 if means.dtype == torch.float16 else 0.0)
    assert np.all(np.abs(got[live] - m[live]) <= tol)
    return H.read_status(ws)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,dtype,layout", [(128, "bf16", "hnd"), (64, "fp16", "nhd"),
                                            (128, "fp16", "slice"), (64, "bf16", "slice")])
def test_append(page, d, dtype, layout):
    held = [0, 1, page - 1, page, 3, 2 * page - 2, 0]
    new = [1, 1, 1, page, 2 * page, 5, 3 * page + 1]
    case = append_case(held, new, page, d=d, dtype=dtype, layout=layout, fused=page == 32, seed=page)
    assert check_append(case, page) == 0


@pytest.mark.parametrize("tokens,hkv", [(1, 1), (3, 8), (700, 1), (1500, 8)])
def test_append_lengths(tokens, hkv):
    assert check_append(append_case([5], [tokens], 64, hkv=hkv, seed=tokens), 64) == 0
    # one token each
    held = [i % 64 for i in range(tokens)]
    if tokens <= 700:
        assert check_append(append_case(held, [1] * tokens, 64, hkv=hkv, seed=tokens), 64) == 0


@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 64), (3, 128), (11, 128), (40, 64)])
def test_append_heads(hkv, d):
    """Fewer and more columns than a CTA takes, and K and V meeting inside one."""
    case = append_case([3, 0, 31], [40, 70, 1], 32, hkv=hkv, d=d, dtype="fp16", seed=hkv)
    assert check_append(case, 32) == 0


def test_append_skips_slots():
    case = append_case([0, 3], [40, 20], 16)
    slots = list(case[6])
    slots[3] = slots[50] = -1
    slots[31] = -1  # the page's last row is not written: no mean
    assert check_append(case, 16, slots) == 0
    case = append_case([0], [20], 16)
    slots = list(case[6])
    slots[2], slots[5] = -2, case[1].shape[0] * 16
    assert check_append(case, 16, slots) == H.STATUS_BAD_INDEX


def with_left_out(case, gaps):
    """The case with gaps[i] tokens that are left out before its token i, which take no slot."""
    shape, keys, vals, means, k_new, v_new, slots = case
    at = np.concatenate([[-1] * gaps.get(i, 0) + [i] for i in range(len(slots) + 1)])[:-1]
    rows = torch.from_numpy(np.maximum(at, 0)).cuda()
    out = torch.from_numpy(at < 0).cuda()[:, None, None]
    nan = torch.full_like(k_new[:1], math.nan)
    return (shape, keys, vals, means, torch.where(out, nan, k_new[rows]),
            torch.where(out, nan, v_new[rows]), [slots[i] if i >= 0 else -1 for i in at])


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("gap", [1, 2, 50, 256, 1000])
def test_append_left_out_tokens_inside_a_page(page, gap):
    """Tokens left out between two of a page's: its mean takes the rows before them from this call."""
    held, new = [0, 5, page - 2, 3, 0, page // 2], [page, page, 2, 3 * page + 7, 2 * page, 2]
    case = append_case(held, new, page, d=64, dtype="fp16", layout="nhd", seed=gap)
    first = np.cumsum([0] + new)
    places = [5, page - 1, page + 3, 2 * page + 1, first[3] + page, first[3] + page + 4, first[5] + 1]
    case = with_left_out(case, {int(i): gap for i in places})
    assert check_append(case, page) == 0


@pytest.mark.parametrize("tokens,page,hkv", [(500, 16, 2), (3000, 64, 1), (40000, 128, 1),
                                             (40000, 16, 3)])
def test_append_left_out_tokens_anywhere(tokens, page, hkv):
    """Tiles of every size, gaps inside them, at their edges and over several."""
    rng = np.random.default_rng(tokens + page)
    lens = [tokens // 3, 1, tokens // 3, tokens - 1 - 2 * (tokens // 3)]
    case = append_case([3, page - 1, 0, 1], lens, page, hkv=hkv, d=64, seed=tokens)
    places = rng.choice(tokens + 1, tokens // 6, replace=False)
    gaps = {int(i): int(g) for i, g in zip(places, rng.choice([1, 1, 2, 3, 70], len(places)))}
    assert check_append(with_left_out(case, gaps), page) == 0


@pytest.mark.parametrize("skew", [0, 1, 2, 3])
@pytest.mark.parametrize("gap", [30, 1021, 5000])
def test_append_slot_maps_at_any_address(skew, gap):
    """A slot map that begins inside a 16-byte group, searched back to its first token."""
    shape, keys, vals, means, k_new, v_new, slots = with_left_out(
        append_case([2, 16, 0, 7], [1, 3, 16, 9], 16, d=64, seed=skew), {0: 5, 1: 2, 10: gap, 21: gap + 1})
    k, v, m = T.f64(keys), T.f64(vals), T.f64(means)
    O.append(k, v, m, T.f64(k_new), T.f64(v_new), slots, 16)
    at = i32([999] * skew + slots + [999])[skew:-1]  # neighbours that are slots of the pool
    H.paged_append(shape, k_new, v_new, at, keys, vals, means, T.workspace(shape))
    assert np.array_equal(T.f64(keys), k, equal_nan=True)
    got, live = T.f64(means), ~np.isnan(m)
    assert np.array_equal(np.isnan(got), ~live)
    # as in check_append
    tol = np.abs(m) * 2.0**-8 + np.nanmax(np.abs(k)) * 17 * 2.0**-24
    assert np.all(np.abs(got - m)[live] <= tol[live])


def test_append_bad_slots_inside_a_page():
    """A slot outside the pool leaves its token out, as -1 does, and says so."""
    case = with_left_out(append_case([0, 2], [40, 30], 16, seed=1), {7: 1, 20: 3, 50: 2})
    slots = [s if s >= 0 else (-7, 2**30)[i % 2] for i, s in enumerate(case[6])]
    assert check_append(case, 16, slots) == H.STATUS_BAD_INDEX


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_largest_and_smallest_keys(page, dtype):
    """Means of keys whose sum no fp32 number holds, beside others and alone, and of very small ones."""
    case = append_case([0, 5], [2 * page, page], page, d=64, dtype=dtype, seed=page)
    k_new, big = case[4], torch.finfo(T.DTYPES[dtype]).max
    k_new[:page] = big
    k_new[2 * page::3] = -big
    assert check_append(case, page) == 0
    case = append_case([0, 0], [2 * page, page], page, d=64, dtype=dtype, seed=page)
    case[4].mul_(2.0 ** (-120 if dtype == "bf16" else -14))
    shape, keys, vals, means, k_new, v_new, slots = case
    k, v, m = T.f64(keys), T.f64(vals), T.f64(means)
    O.append(k, v, m, T.f64(k_new), T.f64(v_new), slots, page)
    H.paged_append(shape, k_new, v_new, i32(slots), keys, vals, means, T.workspace(shape))
    # as in check_append, and half a step of the type's subnormal numbers: means of small keys fall
    # below its smallest normal one (bf16 2^-126, in steps of 2^-133; fp16 2^-14, of 2^-24)
    tol = np.abs(m) * torch.finfo(means.dtype).eps / 2 + np.nanmax(np.abs(k)) * (page + 1) * 2.0**-24
    tol = tol + (2.0**-134 if dtype == "bf16" else 2.0**-25)
    live = ~np.isnan(m)
    assert np.all(np.abs(T.f64(means) - m)[live] <= tol[live])


def test_append_without_means_and_without_tokens():
    shape, keys, vals, means, k_new, v_new, slots = append_case([0], [33], 16)
    ws = T.workspace(shape)
    H.paged_append(shape, k_new, v_new, i32(slots), keys, vals, None, ws)
    before = keys.clone()
    H.paged_append(shape, k_new[:0], v_new[:0], i32([]), keys, vals, means, ws)
    assert torch.equal(before.nan_to_num(), keys.nan_to_num())
    assert torch.isnan(means).all() and H.read_status(ws) == 0


# ------------------------------------------------------------------- decode


def oracle_decode(c, lists=None):
    return O.decode(T.f64(c.q), np.nan_to_num(T.f64(c.keys)), np.nan_to_num(T.f64(c.vals)),
                    c.table.cpu().numpy(), c.lens, c.page, c.scale, lists)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,layout", [("bf16", "hnd"), ("fp16", "nhd"), ("bf16", "slice")])
def test_decode_edges(page, d, dtype, layout):
    c = T.make_cache(EDGES, page, 8, 2, d, dtype, layout, seed=page + d)
    T.check_attention(c, c.decode(), oracle_decode(c))
    assert c.status() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (9, 3), (4, 1), (5, 1), (12, 2), (7, 1),
                                    (16, 2), (40, 8)])
def test_decode_groups(hq, hkv):
    c = T.make_cache((300, 0, 77), 32, hq, hkv, 128, "bf16", seed=hq)
    T.check_attention(c, c.decode(), oracle_decode(c))
    c = T.make_cache((300, 0, 77), 32, hq, hkv, 64, "fp16", seed=hq)
    T.check_attention(c, c.decode(), oracle_decode(c))
    assert c.status() == 0


@pytest.mark.parametrize("lens,hq,hkv,d,dtype", [
    ((40000,), 4, 1, 128, "bf16"),         # every CTA holds a part of one head
    ((40000,), 8, 1, 64, "fp16"),
    ((20000, 3), 3, 3, 128, "fp16"),
    ((9000, 1, 0, 5000), 16, 8, 128, "bf16"),
    ((2000,) * 40, 8, 4, 64, "bf16"),      # most heads whole in one CTA
])
def test_decode_split_and_join(lens, hq, hkv, d, dtype):
    c = T.make_cache(lens, 128 if d == 128 else 64, hq, hkv, d, dtype, seed=len(lens))
    first = c.decode()
    T.check_attention(c, first, oracle_decode(c))
    again = c.decode()  # no order of arrival changes a bit
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert c.status() == 0


def test_decode_many_short_sequences():
    lens = tuple(int(x) for x in np.random.default_rng(1).integers(0, 300, 1024))
    c = T.make_cache(lens, 16, 4, 2, 64, "bf16", seed=1)
    T.check_attention(c, c.decode(), oracle_decode(c))
    assert c.status() == 0


@pytest.mark.parametrize("batch,d,dtype", [(400, 64, "bf16"), (500, 128, "fp16"),
                                           (900, 128, "bf16"), (1000, 64, "fp16"),
                                           (1024, 128, "bf16")])
def test_decode_batch_sizes(batch, d, dtype):
    """Batches whose lengths leave room for fewer CTAs per SM, or for fewer stages."""
    lens = tuple(int(x) for x in np.random.default_rng(batch).integers(0, 100, batch))
    c = T.make_cache(lens, 16, 2, 1, d, dtype, seed=batch)
    T.check_attention(c, c.decode(), oracle_decode(c))
    lists = np.random.default_rng(0).integers(0, 3, (batch, 1, 3))
    lists = np.where(lists < np.array([O.pages_of(n, 16) for n in lens])[:, None, None], lists, -1)
    T.check_attention(c, c.decode_topk(i32(lists.tolist())), oracle_decode(c, lists))
    assert c.status() == 0


@pytest.mark.parametrize("page", [16, 128])
def test_decode_single_page_pool_and_single_head(page):
    """Dimensions of one element, whose strides mean nothing."""
    c = T.make_cache((page - 3,), page, 4, 1, 128, "bf16", seed=page, spare=0)
    c.keys = c.keys.as_strided(c.keys.shape, (1, 3, 128, 1))
    c.vals = c.vals.as_strided(c.vals.shape, (7, 5, 128, 1))
    c.shape = H.make_paged_shape(1, 4, 1, page, 1, 1, pool=c.keys)
    T.check_attention(c, c.decode(), oracle_decode(c))
    assert c.status() == 0


def test_decode_sharp_and_scaled():
    # large logits: the running maximum moves often, and most weights vanish
    for scale in (0.0, 1.0, 0.01):
        c = T.make_cache((3000, 500), 64, 8, 2, 128, "bf16", seed=9, scale=scale, sharp=3.0)
        T.check_attention(c, c.decode(), oracle_decode(c), scale)
    # one key per head far above the rest, late in the sequence
    c = T.make_cache((2000,), 128, 4, 1, 128, "fp16", seed=10)
    p = int(c.table[0, 14])
    c.keys[p, 0, 5] = 4 * c.q[0, 1]
    T.check_attention(c, c.decode(), oracle_decode(c))

@pytest.mark.parametrize("dtype,d,size", [("fp16", 64, 60000.0), ("fp16", 128, 60000.0),
                                          ("bf16", 128, 1e15), ("bf16", 64, -3e9)])
@pytest.mark.parametrize("n", [70, 9000])
def test_decode_very_large_logits(dtype, d, size, n):
    """Logits of up to 2^100: the largest keys' weights are 1, the others 0.

    Queries and keys lie along the first dimension, so that a raw logit is one exact product and
    equal keys give equal logits.  The other keys are half as long or zero: their logits are 2^27 or
    more below, weights of 0 in 64 bits too.  out: a sum of values below 6, with 2^-23 of the sum of
    their magnitudes for an addition: 128 of them in a tile, one for each of at most n / 64 tiles and
    256 CTAs, and a division.  lse: the scale, its product with the logit, the sum with the logarithm
    and the change of its base round once each, and the base's constant is rounded: 5 * 2^-24."""
    c = T.make_cache((n, 33), 64, 4, 1, d, dtype, seed=n)
    c.keys.zero_()
    c.q.zero_()
    c.q[:, :, 0] = size
    for b, length in enumerate(c.lens):
        for i in range(length):
            c.keys[int(c.table[b, i // 64]), 0, i % 64, 0] = (1, 0.5, 0)[i % 3] * size
    want, l_ref = oracle_decode(c)
    every = torch.arange(c.shape.max_pages, dtype=torch.int32, device="cuda").expand(2, 1, -1)
    for out, lse in (c.decode(), c.decode_topk(every.contiguous())):
        assert np.abs(T.f64(out) - want).max() <= 6 * (128 + n / 64 + 256 + 2) * 2.0**-23
        assert np.all(np.abs(T.f64(lse) - l_ref) <= 5 * 2.0**-24 * np.abs(l_ref))
    assert c.status() == 0


def test_decode_non_finite_inputs_stay_in_their_rows():
    c = T.make_cache((700, 300), 32, 4, 2, 128, "bf16", seed=2)
    want = oracle_decode(c)
    c.q[0, 1] = math.nan                         # one query head
    c.keys[int(c.table[1, 3]), 1, 4] = math.inf  # one key of KV head 1 of sequence 1
    out, lse = (T.f64(x) for x in c.decode())
    bad = np.zeros((2, 4), dtype=bool)
    bad[0, 1] = bad[1, 2] = bad[1, 3] = True
    assert np.isnan(out[bad]).all()
    tol_o, tol_l = T.attention_tolerance(T.make_cache((700, 300), 32, 4, 2, 128, "bf16", seed=2))
    assert np.abs(out - want[0])[~bad].max() <= tol_o
    assert np.abs(lse - want[1])[~bad].max() <= tol_l


def test_decode_lowest_values_and_infinities_in_masked_rows():
    for fill in (math.inf, -math.inf, torch.finfo(torch.bfloat16).min, 3e38):
        c = T.make_cache((130, 17), 16, 4, 2, 128, "bf16", seed=4)
        for t in (c.keys, c.vals):
            t.copy_(torch.where(torch.isnan(t), torch.full_like(t, fill), t))
        ref = T.make_cache((130, 17), 16, 4, 2, 128, "bf16", seed=4)
        T.check_attention(ref, c.decode(), oracle_decode(ref), fill)


def test_decode_bad_pages_and_lengths():
    c = T.make_cache((100, 60, 200, 5), 16, 4, 2, 64, "bf16", seed=5)
    c.table[0, 2] = -1
    c.table[2, 12] = c.keys.shape[0]
    T.check_attention(c, c.decode(), oracle_decode(c))
    assert c.status() == H.STATUS_BAD_INDEX
    c = T.make_cache((100, 60, 200, 5), 16, 4, 2, 64, "bf16", seed=5)
    lens = list(c.lens)
    c.seqlens[1], c.seqlens[2] = -3, c.table.shape[1] * 16 + 1
    lens[1] = lens[2] = 0
    c.lens = tuple(lens)
    T.check_attention(c, c.decode(), oracle_decode(c))
    assert c.status() == H.STATUS_BAD_SEQLEN


@pytest.mark.parametrize("n", [2, 50, 64, 700, 9000, 40000])
@pytest.mark.parametrize("d,dtype,page", [(128, "bf16", 64), (128, "fp16", 128), (64, "bf16", 128),
                                          (64, "fp16", 64), (128, "bf16", 16), (64, "fp16", 16)])
def test_decode_shows_every_weight(n, d, dtype, page):
    """Outputs that are sums of at most n / d weights, within a few units in the last place of fp32:
    weights in fewer 16-bit terms, or a token lost, would show."""
    c = T.make_cache((n, 3), page, len(T.FACTORS), 1, d, dtype, seed=n)
    ladders = [T.ladder(k, seed=k) for k in c.lens]
    c.q.zero_()
    c.q[:, :, 0] = torch.tensor(T.FACTORS, device="cuda")
    for b, x in enumerate(ladders):
        pos = torch.arange(len(x), device="cuda")
        at = (c.table[b, pos // page].long(), torch.zeros_like(pos), pos % page)
        rows = torch.zeros(len(x), d, device="cuda", dtype=c.keys.dtype)
        rows[:, 0] = torch.from_numpy(x).cuda().to(rows.dtype)
        c.keys[at] = rows
        c.vals[at] = torch.eye(d, device="cuda", dtype=c.vals.dtype)[pos % d]
    results = [c.decode()]
    if c.shape.max_pages <= H.MAX_TOPK:
        lists = torch.arange(c.shape.max_pages, dtype=torch.int32, device="cuda")
        results.append(c.decode_topk(lists.expand(2, 1, -1).contiguous()))
    for out, lse in results:
        for b, x in enumerate(ladders):
            want = T.ladder_result(x, T.ladder_weights(x, c.scale), c.scale, d)
            tol = T.ladder_tolerance(len(x), d, dtype, c.scale, heads=2)
            assert T.ladder_check((T.f64(out[b]), T.f64(lse[b])), want, tol)
    assert c.status() == 0


def test_decode_without_lse_and_with_shared_pages():
    c = T.make_cache((200, 190), 32, 4, 2, 128, "bf16", seed=6)
    c.table[1, :4] = c.table[0, :4]  # a common prefix of 128 tokens
    out, lse = c.decode()
    T.check_attention(c, (out, lse), oracle_decode(c))
    plain = torch.empty_like(out)
    H.paged_decode(c.shape, c.q, c.keys, c.vals, c.table, c.seqlens, plain, c.ws)
    assert torch.equal(out, plain)


def test_decode_joins_parts_by_lse():
    """lse joins outputs over disjoint parts of a sequence."""
    c = T.make_cache((400,), 16, 4, 2, 128, "fp16", seed=7)
    whole, lse = c.decode()
    n = 16 * 11
    front = T.Cache(**{**c.__dict__, "lens": (n,), "seqlens": i32([n])})
    back_table = torch.cat([c.table[:, 11:], c.table[:, :11]], 1).contiguous()
    back = T.Cache(**{**c.__dict__, "lens": (400 - n,), "seqlens": i32([400 - n]),
                      "table": back_table})
    (o1, l1), (o2, l2) = front.decode(), back.decode()
    w = torch.softmax(torch.stack([l1, l2]).double(), 0)
    joined = w[0, ..., None] * o1.double() + w[1, ..., None] * o2.double()
    T.check_attention(c, (joined, torch.logaddexp(l1.double(), l2.double())),
                      (T.f64(whole), T.f64(lse)))


def test_decode_in_a_pool_past_32_bits():
    """Element and byte offsets past 2^31 and 2^32."""
    page, hkv, d = 128, 8, 128
    pool = (1 << 32) // (page * hkv * d) + 9
    keys, vals = (torch.empty(pool, hkv, page, d, dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
    c = T.make_cache((1000, 129), page, 16, hkv, d, "bf16", seed=8)
    table = c.table.clone()
    far = torch.arange(pool - 1, pool - 1 - c.keys.shape[0], -1, device="cuda")
    keys[far], vals[far] = c.keys, c.vals
    live = c.table < c.keys.shape[0]
    table[live] = far[c.table[live].long()].to(torch.int32)
    shape = H.make_paged_shape(2, 16, hkv, page, pool, table.shape[1], pool=keys)
    out, lse = c.result()
    H.paged_decode(shape, c.q, keys, vals, table, c.seqlens, out, c.ws, lse=lse)
    T.check_attention(c, (out, lse), oracle_decode(c))
    # rows appended there, and the means of its pages
    means = torch.zeros(pool, hkv, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(2, page, hkv, d, device="cuda").bfloat16()
    slots = (pool - 1) * page + torch.arange(page, dtype=torch.int32, device="cuda")
    H.paged_append(shape, rows[0], rows[1], slots, keys, vals, means, c.ws)
    assert torch.equal(keys[pool - 1], rows[0].transpose(0, 1))
    assert torch.equal(vals[pool - 1], rows[1].transpose(0, 1))
    assert float(means[: pool - 1].abs().sum()) == 0 and float(means[pool - 1].abs().sum()) > 0
    assert c.status() == 0


# -------------------------------------------------------------- decode_topk


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,dtype,layout", [(128, "bf16", "nhd"), (64, "fp16", "hnd")])
@pytest.mark.parametrize("k", [1, 3, 9, 40])
def test_decode_topk(page, d, dtype, layout, k):
    c = T.make_cache(EDGES, page, 6, 2, d, dtype, layout, seed=page + k)
    rng = np.random.default_rng(k)
    lists = np.full((len(EDGES), 2, k), -1)
    for b, n in enumerate(EDGES):
        for h in range(2):
            p = rng.permutation(O.pages_of(n, page))[:k]
            lists[b, h, : len(p)] = p
    idx = i32(lists.tolist())
    T.check_attention(c, c.decode_topk(idx), oracle_decode(c, lists))
    assert c.status() == 0


def test_decode_topk_skips_and_repeats():
    c = T.make_cache((500, 100, 64, 0), 16, 4, 2, 128, "bf16", seed=11)
    lists = np.full((4, 2, 12), -1)
    lists[0, 0] = [5, -1, 5, 31, 0, -1, 30, 2, 7, 9, 11, 13]  # page 5 twice, the last page
    lists[0, 1] = -1                                          # nothing
    lists[1, 0, :3] = [6, 0, 6]
    lists[1, 1, :2] = [-1, 4]
    lists[2, :, 4:] = 3  # entries past the sequence's four pages are not read
    lists[2, 0, :4] = [0, 1, 2, 3]
    idx = i32(lists.tolist())
    T.check_attention(c, c.decode_topk(idx), oracle_decode(c, lists))
    assert c.status() == 0
    lists[0, 0, 4], lists[1, 1, 0] = 32, -2
    T.check_attention(c, c.decode_topk(i32(lists.tolist())), oracle_decode(c, lists))
    assert c.status() == H.STATUS_BAD_INDEX


def test_decode_topk_of_every_page_is_decode():
    c = T.make_cache((3000, 700), 32, 8, 2, 128, "fp16", seed=12)
    idx = torch.arange(94, dtype=torch.int32, device="cuda").expand(2, 2, 94).contiguous()
    a, b = c.decode(), c.decode_topk(idx)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    long = torch.arange(1024, dtype=torch.int32, device="cuda").expand(2, 2, 1024).contiguous()
    b = c.decode_topk(long)
    assert torch.equal(a[0], b[0]) and c.status() == 0


# ------------------------------------------------------------------- select


def make_means(c, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(c.keys.shape[0], c.hkv, c.d, generator=g).to(c.keys.dtype).cuda()


def run_select(c, means, k, sink, recent):
    idx = torch.full((len(c.lens), c.hkv, k), -9, dtype=torch.int32, device="cuda")
    H.paged_select(c.shape, c.q, means, c.table, c.seqlens, idx, c.ws, sink=sink, recent=recent)
    torch.cuda.synchronize()
    return idx.cpu().numpy()


def oracle_select(c, means, k, sink, recent):
    return O.select(T.f64(c.q), T.f64(means), c.table.cpu().numpy(), c.lens, c.page, c.scale, k,
                    sink, recent)[0]


@pytest.mark.parametrize("page,d,dtype", [(16, 128, "bf16"), (32, 64, "fp16"), (64, 128, "fp16"),
                                          (128, 64, "bf16")])
@pytest.mark.parametrize("k,sink,recent", [(1, 0, 1), (4, 1, 1), (5, 2, 3), (33, 0, 2), (2, 3, 4),
                                           (200, 1, 2)])
def test_select(page, d, dtype, k, sink, recent):
    c = T.make_cache(EDGES + (3000,), page, 6, 2, d, dtype, seed=k)
    means = make_means(c, k)
    assert np.array_equal(run_select(c, means, k, sink, recent),
                          oracle_select(c, means, k, sink, recent))
    assert c.status() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (8, 1), (15, 3), (7, 7)])
def test_select_groups(hq, hkv):
    c = T.make_cache((5000, 130), 32, hq, hkv, 128, "bf16", seed=hq)
    means = make_means(c, hq)
    assert np.array_equal(run_select(c, means, 20, 1, 1), oracle_select(c, means, 20, 1, 1))
    assert c.status() == 0


@pytest.mark.parametrize("k", [7, 64, 257, 1000, 1024])
def test_select_long(k):
    """A table as long as the limit allows, from one cluster per head."""
    c = T.make_cache((40000, 100), 16, 8, 1, 64, "bf16", seed=k, cols=16384)
    means = make_means(c, k)
    assert np.array_equal(run_select(c, means, k, 4, 8), oracle_select(c, means, k, 4, 8))
    assert c.status() == 0


@pytest.mark.parametrize("hq,hkv,d,k", [(8, 1, 64, 1024), (4, 2, 128, 40)])
def test_select_largest_table(hq, hkv, d, k):
    """Every column of the longest table holds a page."""
    c = T.make_cache((H.MAX_SEQLEN - 3, 50), 16, hq, hkv, d, "bf16", seed=k)
    means = make_means(c, k)
    assert np.array_equal(run_select(c, means, k, 2, 3), oracle_select(c, means, k, 2, 3))
    assert c.status() == 0


def test_select_many_heads():
    lens = tuple(int(x) for x in np.random.default_rng(3).integers(0, 2000, 150))
    c = T.make_cache(lens, 32, 8, 4, 64, "fp16", seed=3)
    means = make_means(c, 3)
    assert np.array_equal(run_select(c, means, 12, 1, 2), oracle_select(c, means, 12, 1, 2))


def test_select_ties_take_the_lower_page():
    c = T.make_cache((16 * 600,), 16, 4, 2, 64, "bf16", seed=13)
    means = torch.ones(c.keys.shape[0], 2, 64, dtype=torch.bfloat16, device="cuda")
    assert np.array_equal(run_select(c, means, 300, 0, 1)[0, 0], [599] + list(range(299)))
    # two values: the better pages first, each kind in order
    better = list(range(3, 600, 7))
    rows = torch.tensor([int(c.table[0, j]) for j in better], device="cuda")
    means[rows] = 2 * torch.sign(c.q[0].float().view(2, 2, 64).sum(1)).bfloat16()
    got = run_select(c, means, 128, 0, 1)
    assert np.array_equal(got, oracle_select(c, means, 128, 0, 1))
    assert c.status() == 0


@pytest.mark.parametrize("n", [513, 1500, 2049, 3000, 5000])
@pytest.mark.parametrize("k", [3, 300, 1024])
def test_select_many_equal_and_far_scores(n, k):
    """More equal scores than one sort takes, and wanted pages far below the best."""
    c = T.make_cache((16 * (n + 1),), 16, 2, 1, 64, "bf16", seed=n)
    rows = torch.tensor([int(x) for x in c.table[0, : n + 1]], device="cuda")
    means = torch.ones(c.keys.shape[0], 1, 64, dtype=torch.bfloat16, device="cuda")
    assert np.array_equal(run_select(c, means, k, 0, 1)[0, 0],
                          ([n] + list(range(min(k - 1, n))) + [-1] * k)[:k])
    # the same with a few better and a few much better pages
    sign = torch.sign(c.q[0].float().sum(0)).bfloat16()
    means[rows[5:n:97]] = sign * 1.5
    means[rows[7:n:301]] = sign * 4
    assert np.array_equal(run_select(c, means, k, 0, 1), oracle_select(c, means, k, 0, 1))
    # scores over hundreds of binades
    far = torch.linspace(-40, 40, n + 1, device="cuda")[torch.randperm(n + 1, device="cuda")]
    means[rows] = (far[:, None, None] * sign).bfloat16()
    assert np.array_equal(run_select(c, means, k, 0, 1), oracle_select(c, means, k, 0, 1))
    assert c.status() == 0


def test_select_vanishing_scores():
    """Scores that underflow to zero tie, and still come in order."""
    c = T.make_cache((16 * 300,), 16, 2, 1, 64, "bf16", seed=14, sharp=30.0)
    means = (30 * make_means(c, 14).float()).bfloat16()
    assert np.array_equal(run_select(c, means, 200, 1, 1), oracle_select(c, means, 200, 1, 1))
    assert c.status() == 0


def test_select_bad_input():
    c = T.make_cache((16 * 40, 100), 16, 4, 2, 64, "bf16", seed=15)
    means = make_means(c)
    # means of pages that are always taken are not read
    for j in (0, 39):
        means[int(c.table[0, j])] = math.nan
    assert np.array_equal(run_select(c, means, 8, 1, 1), oracle_select(c, means, 8, 1, 1))
    assert c.status() == 0
    means[int(c.table[0, 7]), 1] = math.nan  # every score of this head is lost: pages in order
    got = run_select(c, means, 8, 1, 1)
    assert got[0, 1].tolist() == [0, 39, 1, 2, 3, 4, 5, 6]
    assert np.array_equal(got[0, 0], oracle_select(c, make_means(c), 8, 1, 1)[0, 0])
    assert c.status() == H.STATUS_NONFINITE
    c = T.make_cache((16 * 40, 100), 16, 4, 2, 64, "bf16", seed=15)
    means = make_means(c)
    best = int(oracle_select(c, means, 8, 1, 1)[0, 0, 2])
    c.table[0, best] = -1
    got = run_select(c, means, 38, 1, 1)
    assert best not in got[0, 0].tolist()
    assert c.status() == H.STATUS_BAD_INDEX


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(4, 2, 64, "bf16"), (8, 1, 128, "fp16")])
def test_select_bad_entries_beside_a_page_without_a_mean(fill, hq, hkv, d, dtype):
    """A table entry outside the pool scores 0 and changes no other score, whatever the means of
    pages that no sequence holds are."""
    n = 700
    c = T.make_cache((16 * n, 100), 16, hq, hkv, d, dtype, seed=15)
    means = make_means(c)
    held = torch.cat([c.table[0], c.table[1, :7]]).long()
    if (held == 0).any():  # page 0 is no sequence's: another takes its place
        spare = sorted(set(range(c.keys.shape[0])) - set(held.tolist()))[0]
        means[spare] = means[0]
        c.table[c.table == 0] = spare
    means[0] = fill
    bad = {7: -1, 8: 2**30, 300: c.keys.shape[0], 650: -(2**31)}
    # the others rank as in a sequence without these pages
    keep = [j for j in range(n) if j not in bad]
    want = O.select(T.f64(c.q)[:1], T.f64(means), c.table.cpu().numpy()[:1, keep], (16 * len(keep),),
                    16, c.scale, len(keep), 1, 1)[0][0]
    for j, page in bad.items():
        c.table[0, j] = page
    got = run_select(c, means, n, 1, 1)[0]
    assert np.array_equal(got[:, : len(keep)], np.array(keep)[want])
    assert np.array_equal(got[:, len(keep):], [sorted(bad)] * hkv)
    assert c.status() == H.STATUS_BAD_INDEX


# ------------------------------------------------------------------ together


class Loop:
    """A serving loop over a paged pool, with the plain record of every sequence beside it."""

    def __init__(self, batch, page, hq, hkv, d, dtype="bf16", pool=400, k=6, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.t, self.page, self.hq, self.hkv, self.d, self.k = T.DTYPES[dtype], page, hq, hkv, d, k
        self.keys = T.pool_tensor(pool, hkv, page, d, self.t, "nhd")
        self.vals = T.pool_tensor(pool, hkv, page, d, self.t, "nhd")
        self.means = torch.full((pool, hkv, d), math.nan, dtype=self.t, device="cuda")
        cols = 40
        self.shape = H.make_paged_shape(batch, hq, hkv, page, pool, cols,
                                        dtype=H.BF16 if dtype == "bf16" else H.FP16, head_dim=d,
                                        pool=self.keys)
        self.ws = T.workspace(self.shape)
        self.table = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pool, generator=self.g).to(torch.int32).cuda()
        self.count, self.lens = i32([pool]), i32([0] * batch)
        self.cu = i32([0] * (batch + 1))
        self.new = i32([0] * batch)
        self.record = [[np.zeros((0, hkv, d)), np.zeros((0, hkv, d))] for _ in range(batch)]
        self.out = torch.empty(batch, hq, d, device="cuda")
        self.sparse = torch.empty_like(self.out)
        self.lse = torch.empty(batch, hq, device="cuda")
        self.idx = torch.empty(batch, hkv, k, dtype=torch.int32, device="cuda")
        self.q = torch.empty(batch, hq, d, dtype=self.t, device="cuda")

    def buffers(self, tokens):
        self.slots = i32([0] * tokens)
        self.rows = torch.empty(2, tokens, self.hkv, self.d, dtype=self.t, device="cuda")

    def fill(self, new):
        """New lengths, rows and queries of one step, in place."""
        self.new.copy_(i32(new))
        n = sum(new)
        rows = torch.randn(2, n, self.hkv, self.d, generator=self.g).to(self.t)
        self.rows[:, :n].copy_(rows)
        at = 0
        for b, w in enumerate(new):
            for i in range(2):
                self.record[b][i] = np.concatenate([self.record[b][i], T.f64(rows[i, at:at + w])])
            at += w
        self.q.copy_(torch.randn(self.q.shape, generator=self.g).to(self.t))

    def step(self):
        H.paged_tables(self.shape, self.lens, self.new, self.free, self.count, self.table,
                       self.lens, self.cu, self.slots, self.count, self.ws)
        H.paged_append(self.shape, self.rows[0], self.rows[1], self.slots, self.keys, self.vals,
                       self.means, self.ws)
        H.paged_decode(self.shape, self.q, self.keys, self.vals, self.table, self.lens, self.out,
                       self.ws, lse=self.lse)
        H.paged_select(self.shape, self.q, self.means, self.table, self.lens, self.idx, self.ws,
                       sink=1, recent=2)
        H.paged_decode_topk(self.shape, self.q, self.keys, self.vals, self.table, self.lens,
                            self.idx, self.sparse, self.ws)

    def check(self):
        torch.cuda.synchronize()
        assert H.read_status(self.ws) == 0
        lens = [len(r[0]) for r in self.record]
        assert self.lens.tolist() == lens
        q, scale, r = T.f64(self.q), 1 / math.sqrt(self.d), self.hq // self.hkv
        idx, out, sparse = self.idx.cpu().numpy(), T.f64(self.out), T.f64(self.sparse)
        lse, means, table = T.f64(self.lse), T.f64(self.means), self.table.cpu().numpy()
        # N(0, 1) inputs: |logit| sum below 8 sqrt(d), |v| below 6 (see attention_tolerance)
        S = 8 * math.sqrt(self.d)
        tol = 6 * 2 * (self.d * 2.0**-23 * S + 6 * S * 2.0**-24 + 2.0**-21 + 400 * 2.0**-23)
        want_idx = O.select(q, np.nan_to_num(means), table, lens, self.page, scale, self.k, 1, 2)[0]
        assert np.array_equal(idx, want_idx)
        for b, (k, v) in enumerate(self.record):
            for h in range(self.hkv):
                at = slice(h * r, h * r + r)
                o, l = O.attention(q[b, at], k[:, h], v[:, h], scale)
                assert np.abs(out[b, at] - o).max() <= tol
                assert np.array_equal(np.isneginf(lse[b, at]), np.isneginf(l))
                pos = [j * self.page + i for j in idx[b, h] if j >= 0 for i in range(self.page)]
                pos = [x for x in pos if x < len(k)]
                o, _ = O.attention(q[b, at], k[pos, h], v[pos, h], scale)
                assert np.abs(sparse[b, at] - o).max() <= tol


@pytest.mark.parametrize("page,d,dtype", [(16, 64, "bf16"), (32, 128, "fp16")])
def test_serving_loop(page, d, dtype):
    s = Loop(5, page, 8, 2, d, dtype)
    for new in ([70, 0, 1, 200, 33], [1, 90, 1, 1, 1], [1, 1, 14, 0, 1], [1] * 5, [0] * 5):
        s.buffers(sum(new) + 3)
        s.fill(new)
        s.step()
        s.check()


def test_serving_loop_in_a_graph_and_on_another_stream():
    s = Loop(4, 16, 8, 2, 128)
    s.buffers(8)
    s.fill([2, 1, 0, 3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    side.synchronize()
    s.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for i in range(40):
        s.fill([1, i % 2, 2, i % 3])
        graph.replay()
        if i % 13 == 0:
            s.check()
    s.check()


def test_calls_of_two_streams_with_their_own_workspaces():
    a = T.make_cache((9000,), 64, 8, 2, 128, "bf16", seed=20)
    b = T.make_cache((5000, 200), 16, 8, 2, 64, "fp16", seed=21)
    want = a.decode(), b.decode()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        for c, st in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(st):
                got.append(c.decode())
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_calls_in_a_row_without_waiting_for_any():
    """Each call starts beside the end of the one before it, of every other kind."""
    a = T.make_cache((9000, 40), 64, 8, 2, 128, "bf16", seed=30)
    b = T.make_cache((700,) * 30, 16, 8, 2, 64, "fp16", seed=31)
    r = Requests(list(range(60)), [1] * 60, 16, seed=5)
    means = make_means(a), make_means(b)
    dense = torch.randn(2, 1, 2, 640, 128, device="cuda").bfloat16()
    dshape = H.make_shape(1, 8, 2, 3, 640, kv_capacity=640)
    dws = torch.empty(H.workspace_bytes(dshape), dtype=torch.uint8, device="cuda")
    H.workspace_init(dws)

    def everything():
        got = []
        for c, m in ((a, means[0]), (b, means[1])):
            idx = torch.empty(len(c.lens), c.hkv, 5, dtype=torch.int32, device="cuda")
            got += [*c.decode(), idx]
            H.paged_select(c.shape, c.q, m, c.table, c.seqlens, idx, c.ws)
            got += c.decode_topk(idx)
            out = torch.empty(1, 8, 128, device="cuda")
            tk = torch.empty(1, 2, 3, dtype=torch.int32, device="cuda")
            H.decode_full(dshape, a.q[:1].contiguous(), dense[0], dense[1], i32([640]), out, tk,
                          dws)
            got += [out, tk, *c.decode()]
        return got

    want = everything()
    r.check()
    torch.cuda.synchronize()
    rounds = [everything() for _ in range(25)]
    torch.cuda.synchronize()
    for got in rounds:
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert a.status() == 0 and b.status() == 0


def test_one_workspace_serves_every_shape():
    a = T.make_cache((9000,), 64, 8, 2, 128, "bf16", seed=22)
    b = T.make_cache((500, 200) * 30, 16, 8, 2, 64, "fp16", seed=23)
    want = a.decode(), b.decode()
    b.ws = a.ws
    for _ in range(3):
        for c, w in ((a, want[0]), (b, want[1])):
            o, l = c.decode()
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


@pytest.mark.parametrize("batch,hkv,slack", [(40, 8, 0), (3, 2, 0), (40, 8, 5 << 20), (200, 4, 300)])
def test_one_workspace_serves_dense_and_paged_calls(batch, hkv, slack):
    """The dense fp32 calls keep state in their workspace; the paged calls leave it as it is."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    n = 700
    q = torch.randn(batch, 4 * hkv, 128, generator=g, device="cuda")
    kv = torch.randn(2, batch, hkv, n, 128, generator=g, device="cuda")
    lens = i32([n - b % 5 * 100 for b in range(batch)])
    shape = H.make_shape(batch, 4 * hkv, hkv, 3, n, dtype=H.FP32, kv_capacity=n)
    c = T.make_cache((9000, 3, 0, 2000), 64, 8, 2, 128, "bf16", seed=25)
    r = Requests([5, 0, 40], [3, 100, 2000], 16, seed=6)
    nbytes = max(H.workspace_bytes(shape), H.paged_workspace_bytes(c.shape)) + slack
    own = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    both = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def dense(ws):
        out = torch.full((batch, 4 * hkv, 128), math.nan, device="cuda")
        topk = torch.full((batch, hkv, 3), -9, dtype=torch.int32, device="cuda")
        H.decode_full(shape, q, kv[0], kv[1], lens, out, topk, ws)
        return out, topk

    H.workspace_init(own)
    H.workspace_init(both)
    want, paged = dense(own), c.decode()
    c.ws = r.ws = both
    for _ in range(3):
        got = c.decode()
        assert torch.equal(got[0], paged[0]) and torch.equal(got[1], paged[1])
        r.check()
        for x, y in zip(dense(both), want):
            assert torch.equal(x, y)
    assert c.status() == 0


def test_wait_limit_ends_decode_with_a_status():
    """A wait that gives up: the call ends, says so, and leaves the workspace usable."""
    c = T.make_cache((9000, 100), 64, 8, 2, 128, "bf16", seed=24)
    want = c.decode()
    assert c.status() == 0
    H.set_wait_limit(1)
    try:
        c.decode()
        assert c.status() & H.STATUS_TIMEOUT
    finally:
        H.set_wait_limit(0)
    o, l = c.decode()
    assert torch.equal(o, want[0]) and torch.equal(l, want[1]) and c.status() == 0

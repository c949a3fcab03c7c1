"""Paged-cache calls without a GPU: refusals before any launch, the binding's
checks, and pins of the 64-bit oracle."""

import copy
import ctypes
import math
import pickle

import numpy as np
import pytest
import torch

from kv_cache_sparsity_b200 import build as hbuild
from kv_cache_sparsity_b200 import hylra as H
from oracle import paged_oracle as O

import paged_testlib as T

INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return H.load()


def _shape(**kw):
    strides = {k: kw.pop(k) for k in ("page_stride", "head_stride", "token_stride") if k in kw}
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, page_size=16, num_pages=10, max_pages=5)
    base.update(kw)
    s = H.make_paged_shape(**base)
    for k, v in strides.items():
        setattr(s, k, v)
    return s


# a non-null, aligned address for arguments that a refused call never touches
PTR = 1 << 20


def _calls(lib, shape, **kw):
    """Return codes of every entry point for this shape, with the given arguments changed.

    The workspace is too small for any call: one whose arguments all pass ends there, the last check
    before a launch, and no launch with these addresses happens on a machine with a GPU."""
    a = dict(q=PTR, K=PTR, V=PTR, table=PTR, lens=PTR, out=PTR, lse=None, ws=PTR, nbytes=1,
             k=4, idx=PTR, means=PTR, sink=1, recent=1, new_stride=256, tokens=3, slots=PTR,
             free_cap=5, slot_cap=5)
    a.update(kw)
    s = ctypes.byref(shape) if shape is not None else None
    yield "tables", lib.hylra_paged_tables(s, a["lens"], a["lens"], a["slots"], a["free_cap"],
                                           a["lens"], a["table"], a["lens"], a["lens"], a["slots"],
                                           a["slot_cap"], a["lens"], a["ws"], a["nbytes"], None)
    yield "append", lib.hylra_paged_append(s, a["K"], a["V"], a["new_stride"], a["slots"],
                                           a["tokens"], a["K"], a["V"], a["means"], a["ws"],
                                           a["nbytes"], None)
    yield "decode", lib.hylra_paged_decode(s, a["q"], a["K"], a["V"], a["table"], a["lens"],
                                           a["out"], a["lse"], a["ws"], a["nbytes"], None)
    yield "select", lib.hylra_paged_select(s, a["q"], a["means"], a["table"], a["lens"], a["k"],
                                           a["sink"], a["recent"], a["idx"], a["ws"], a["nbytes"],
                                           None)
    yield "topk", lib.hylra_paged_decode_topk(s, a["q"], a["K"], a["V"], a["table"], a["lens"],
                                              a["idx"], a["k"], a["out"], a["lse"], a["ws"],
                                              a["nbytes"], None)


ALL = {"tables", "append", "decode", "select", "topk"}
POOL = {"append", "decode", "topk"}


@pytest.mark.parametrize("kw,code,who", [
    (dict(batch=0), INVALID, ALL), (dict(batch=1025), UNSUPPORTED, ALL),
    (dict(num_q_heads=0), INVALID, ALL), (dict(num_q_heads=7), INVALID, ALL),
    (dict(num_kv_heads=0, num_q_heads=1), INVALID, ALL),
    (dict(num_q_heads=18), UNSUPPORTED, ALL),
    (dict(head_dim=96), UNSUPPORTED, ALL), (dict(head_dim=256), UNSUPPORTED, ALL),
    (dict(page_size=8), UNSUPPORTED, ALL), (dict(page_size=48), UNSUPPORTED, ALL),
    (dict(page_size=256), UNSUPPORTED, ALL), (dict(page_size=0), UNSUPPORTED, ALL),
    (dict(dtype=H.FP32), UNSUPPORTED, ALL), (dict(dtype=5), INVALID, ALL),
    (dict(num_pages=0), INVALID, ALL), (dict(max_pages=0), INVALID, ALL),
    (dict(num_pages=1 << 27), UNSUPPORTED, ALL), (dict(max_pages=16385), UNSUPPORTED, ALL),
    (dict(scale=-1.0), INVALID, ALL), (dict(scale=math.nan), INVALID, ALL),
    (dict(scale=math.inf), INVALID, ALL),
    (dict(num_q_heads=1 << 20, num_kv_heads=1 << 20), UNSUPPORTED, ALL),
    (dict(page_stride=4096 - 8), INVALID, POOL), (dict(token_stride=120), INVALID, POOL),
    (dict(token_stride=132), INVALID, POOL), (dict(head_stride=0), INVALID, POOL),
    (dict(page_stride=-4096), INVALID, POOL), (dict(page_stride=1 << 39), UNSUPPORTED, POOL),
    (dict(page_stride=0), INVALID, POOL), (dict(num_pages=1 << 20, page_stride=1 << 30),
                                           UNSUPPORTED, POOL),
])
def test_shapes_refused(lib, kw, code, who):
    s = _shape(**kw)
    for name, rc in _calls(lib, s):
        if name in who:
            assert rc == code, name
    if who is ALL:
        n = ctypes.c_size_t(7)
        assert lib.hylra_paged_workspace_bytes(ctypes.byref(s), ctypes.byref(n)) == code
        assert n.value == 7


@pytest.mark.parametrize("kw,code,who", [
    (dict(q=0), INVALID, {"decode", "select", "topk"}), (dict(q=PTR + 8), INVALID, {"decode"}),
    (dict(K=None), INVALID, POOL), (dict(V=PTR + 2), INVALID, POOL),
    (dict(table=None), INVALID, {"tables", "decode", "select", "topk"}),
    (dict(lens=PTR + 1), INVALID, {"tables", "decode", "select", "topk"}),
    (dict(out=None), INVALID, {"decode", "topk"}), (dict(lse=PTR + 2), INVALID, {"decode"}),
    (dict(k=0), INVALID, {"select", "topk"}), (dict(k=1025), UNSUPPORTED, {"select", "topk"}),
    (dict(idx=None), INVALID, {"select", "topk"}), (dict(sink=-1), INVALID, {"select"}),
    (dict(recent=0), INVALID, {"select"}), (dict(means=None), INVALID, {"select"}),
    (dict(means=PTR + 4), INVALID, {"append", "select"}),
    (dict(new_stride=248), INVALID, {"append"}), (dict(new_stride=260), INVALID, {"append"}),
    (dict(new_stride=1 << 31), UNSUPPORTED, {"append"}), (dict(tokens=-1), INVALID, {"append"}),
    (dict(slots=None), INVALID, {"append", "tables"}),
    (dict(free_cap=-1), INVALID, {"tables"}), (dict(slot_cap=-1), INVALID, {"tables"}),
])
def test_arguments_refused(lib, kw, code, who):
    for name, rc in _calls(lib, _shape(), **kw):
        if name in who:
            assert rc == code, name


def test_scale_past_fp32_refused(lib):
    """A scale whose product with log2(e) no fp32 number holds; the selection works in 64 bits."""
    big = dict(_calls(lib, _shape(scale=2.0**127)))
    ok = dict(_calls(lib, _shape(scale=2.0**126)))
    for name in ("decode", "topk"):
        assert big[name] == UNSUPPORTED and ok[name] != UNSUPPORTED
    assert big["select"] != UNSUPPORTED


def test_null_shape(lib):
    assert all(rc == INVALID for _, rc in _calls(lib, None))
    assert lib.hylra_paged_workspace_bytes(None, None) == INVALID


# what a call with good arguments ends with: the device query or, past it, the workspace check
PASSED = {-3, -4}


def test_calls_of_these_tests_end_before_a_launch(lib):
    assert {rc for _, rc in _calls(lib, _shape())} <= PASSED
    assert dict(_calls(lib, _shape(), tokens=0))["append"] in PASSED


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 1, 3)])
def test_layouts_accepted(lib, order):
    """Any order of the dimensions passes the pool check (the next refusal is the workspace's)."""
    shape = (10, 2, 16, 128)
    t = torch.empty([shape[i] for i in order], dtype=torch.bfloat16)
    t = t.permute([order.index(i) for i in range(4)])
    s = _shape(pool=t)
    codes = dict(_calls(lib, s, ws=None))
    # without a device the call ends at the device query, past the checks of the shape
    assert all(codes[n] != UNSUPPORTED for n in POOL)


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 1, 3), (1, 0, 2, 3),
                                   (1, 2, 0, 3), (2, 1, 0, 3)])
def test_layouts_pass_the_pool_check(lib, order):
    """Every order of the dimensions, padded rows and slices, down to the workspace check; the same
    with one stride eight elements less than its rows and their padding allow is refused."""
    extents = (10, 2, 16, 128)
    for row in (128, 136, 256):
        t = torch.empty([extents[i] for i in order[:3]] + [row], dtype=torch.bfloat16)[..., :128]
        t = t.permute([order.index(i) for i in range(4)])
        codes = dict(_calls(lib, _shape(pool=t)))
        assert {codes[n] for n in POOL} <= PASSED
        for at, name in enumerate(("page_stride", "head_stride", "token_stride")):
            # what stands before the next element of the dimension ends in one row's padding
            codes = dict(_calls(lib, _shape(pool=t, **{name: t.stride(at) - (row - 128) - 8})))
            assert {codes[n] for n in POOL} == {INVALID}
            codes = dict(_calls(lib, _shape(pool=t, **{name: t.stride(at) - (row - 128)})))
            assert {codes[n] for n in POOL} <= PASSED


def test_binding_checks_tensors(lib):
    s = _shape()
    pool = torch.zeros(10, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _shape(pool=pool[..., :64])
    with pytest.raises(ValueError):
        _shape(pool=torch.zeros(10, 2, 128, 16, dtype=torch.bfloat16).transpose(2, 3))
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, 5, dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    out = torch.zeros(2, 8, 128)
    ws = torch.zeros(1 << 22, dtype=torch.uint8)
    good = [s, q, pool, pool, i, n, out, ws]
    bad = {1: [q.float(), q[:1], q.transpose(0, 1).contiguous().transpose(0, 1)],
           2: [pool.half(), pool[:5], torch.zeros(10, 16, 2, 128, dtype=torch.bfloat16).transpose(1, 2)],
           4: [i.long(), i[:, :4]], 5: [n.long(), n[:1]], 6: [out.bfloat16(), out[:, :4]],
           7: [ws]}  # nothing may live on the CPU
    for at, values in bad.items():
        for v in values:
            args = list(good)
            args[at] = v
            with pytest.raises(ValueError):
                H.paged_decode(*args)


class _FakeCuda:
    """A tensor's description without its memory: what the binding looks at."""

    def __init__(self, t, dev=0):
        self.t, self.dev = t, dev
        self.dtype, self.shape, self.nbytes = t.dtype, t.shape, t.nbytes
        self.device = f"cuda:{dev}"

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def calls(monkeypatch):
    """The paged calls reach a recorder in the library's place: (name, shape's fields, stream)."""
    made = []

    def entry(name):
        def call(shape, *args):
            made.append((name, bytes(shape._obj), args[-1]))
            return 0
        call.__name__ = name
        return call

    class Recorder:
        def __getattr__(self, name):
            return entry(name)

    monkeypatch.setattr(H, "_lib", Recorder())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    return made


def _decode_args(shape):
    s, t = shape, torch.bfloat16
    pool = torch.empty(s.num_pages, s.num_kv_heads, s.page_size, s.head_dim, dtype=t)
    return [shape] + [_FakeCuda(x) for x in (
        torch.empty(s.batch, s.num_q_heads, s.head_dim, dtype=t), pool, pool,
        torch.empty(s.batch, s.max_pages, dtype=torch.int32), torch.empty(s.batch, dtype=torch.int32),
        torch.empty(s.batch, s.num_q_heads, s.head_dim), torch.empty(4096, dtype=torch.uint8))]


def test_shapes_changed_and_copied_between_calls(calls):
    """The library gets the fields that the tensors were checked against."""
    a = _shape()
    H.paged_decode(*_decode_args(a))
    for copied in (copy.copy(a), copy.deepcopy(a), pickle.loads(pickle.dumps(a))):
        before = _decode_args(copied)
        a.batch += 1  # the copy keeps its own fields
        H.paged_decode(*before)
        assert calls[-1][1] == bytes(copied) and copied.batch == 2
        with pytest.raises(ValueError):
            H.paged_decode(a, *before[1:])
        H.paged_decode(*_decode_args(a))
        assert calls[-1][1] == bytes(a)
        a.batch = 2


def test_workspace_calls_run_on_the_workspaces_device(calls, monkeypatch):
    """A workspace of another device than the current one is zeroed and read on the stream that the
    paged calls with it use."""
    current = [0]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.before

    class Stream:
        cuda_stream = property(lambda self: 100 + current[0])

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    made = []
    lib = H._lib
    for name in ("hylra_workspace_init", "hylra_read_status"):
        monkeypatch.setattr(type(lib), name, staticmethod(
            lambda *args, name=name: made.append((name, current[0], args[-1])) or 0), raising=False)
    for dev in (0, 1):
        args = _decode_args(_shape())
        for t in args[1:]:
            t.dev = dev
        H.workspace_init(args[-1])
        H.paged_decode(*args)
        H.read_status(args[-1])
        assert calls[-1][2] == 100 + dev
        assert made[-2:] == [("hylra_workspace_init", dev, 100 + dev),
                             ("hylra_read_status", dev, 100 + dev)]
        assert current[0] == 0


@pytest.mark.parametrize("dtype,code", [(H.FP32, UNSUPPORTED), (7, INVALID)])
def test_type_of_a_shape_refused_by_name(calls, dtype, code):
    """A type that the paged calls lack is what is refused, not a tensor that has it."""
    args = _decode_args(_shape())
    args[0].dtype = dtype
    for t in args[1:4]:
        t.dtype = torch.float32
    with pytest.raises(H.HylraError) as e:
        H.paged_decode(*args)
    assert e.value.code == code and not calls


# ------------------------------------------- what the precision tests can see

LADDERS = [(n, d, t) for d in (64, 128) for t in ("bf16", "fp16") for n in (2, 50, 64, 700, 9000, 40000)]


def _in_terms(w, dtype, terms):
    """Weights as the sum of this many 16-bit terms, as the kernel splits them."""
    t, up = (torch.bfloat16, 1.0) if dtype == "bf16" else (torch.float16, 4096.0)
    left = torch.from_numpy(w).float() * up
    total = torch.zeros(w.shape, dtype=torch.float64)
    for _ in range(terms):
        part = left.to(t).float()
        left = left - part
        total += part.double()
    return (total / up).numpy()


@pytest.mark.parametrize("n,d,dtype", LADDERS)
def test_precision_tolerance_tells_terms_and_tokens(n, d, dtype):
    """Weights in the kernel's terms pass; one term, a term less at the sizes of one unit, and a lost
    token fail.  (Over tens of thousands of tokens the roundings of single fp16 terms average out.)"""
    scale = 1 / math.sqrt(d)
    c = T.ladder(n, seed=n)
    w = T.ladder_weights(c, scale)
    want = T.ladder_result(c, w, scale, d)
    tol = T.ladder_tolerance(n, d, dtype, scale)

    def passes(out_weights, z_weights):
        out, _ = T.ladder_result(c, out_weights, scale, d)
        _, lse = T.ladder_result(c, z_weights, scale, d)
        out = out * (out_weights.sum(1) / z_weights.sum(1))[:, None]
        return T.ladder_check((out, lse), want, tol)

    full = 3 if dtype == "bf16" else 2
    assert passes(_in_terms(w, dtype, full), w)
    if 2 < n <= 9000:  # of two weights one is 1
        assert not passes(_in_terms(w, dtype, 1), w)
    if n in (50, 64) and dtype == "bf16":
        assert not passes(_in_terms(w, dtype, 2), w)
    for lost in sorted({1, n // 2, n - 1}):
        some = w.copy()
        some[:, lost] = 0
        assert not passes(some, some)


# ------------------------------------------------------------ oracle pins


def test_oracle_attention_is_softmax():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 8, generator=g, dtype=torch.float64) for n in (3, 11, 11))
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None])[0]
    out, lse = O.attention(q.numpy(), k.numpy(), v.numpy(), 1 / math.sqrt(8))
    assert np.allclose(out, want.numpy(), rtol=1e-13, atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(q @ k.T / math.sqrt(8), -1).numpy(), rtol=1e-13)
    out, lse = O.attention(q.numpy(), k.numpy()[:0], v.numpy()[:0], 1.0)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_oracle_decode_gathers_pages_in_order():
    rng = np.random.default_rng(0)
    k, v = rng.normal(size=(2, 7, 4))
    pool_k, pool_v = np.full((2, 5, 1, 3, 4), np.nan)
    table = np.array([[4, 1, 2, 99]])
    for j in range(3):
        rows = min(3, 7 - 3 * j)
        pool_k[table[0, j], 0, :rows] = k[3 * j:3 * j + rows]
        pool_v[table[0, j], 0, :rows] = v[3 * j:3 * j + rows]
    q = rng.normal(size=(1, 2, 4))
    out, lse = O.decode(q, pool_k, pool_v, table, [7], 3, 0.5)
    o, l = O.attention(q[0], k, v, 0.5)
    assert np.allclose(out[0], o) and np.allclose(lse[0], l)
    out, _ = O.decode(q, pool_k, pool_v, table, [7], 3, 0.5, np.array([[[2, 0]]]))
    rows = [6, 0, 1, 2]
    assert np.allclose(out[0], O.attention(q[0], k[rows], v[rows], 0.5)[0])


def test_oracle_select_by_hand():
    # one head, means 1-d in effect: logits 0, 1, 2, 3 on pages 0..3 of a five-page sequence
    means = np.zeros((5, 1, 2))
    means[:, 0, 0] = [0, 1, 2, 3, np.nan]
    q = np.array([[[1.0, 0.0]]])
    idx, scores = O.select(q, means, np.array([[0, 1, 2, 3, 4]]), [17], 4, 1.0, 4, 1, 1)
    assert idx[0, 0].tolist() == [0, 4, 3, 2]
    c0, s = scores[0, 0]
    assert c0 == 1 and np.allclose(s, np.exp([1, 2, 3]) / np.exp([1, 2, 3]).sum())
    # equal means: the lower page first; fewer pages than asked for: -1
    idx, _ = O.select(q, np.ones((5, 1, 2)), np.array([[0, 1, 2, 3, 4]]), [20], 4, 1.0, 7, 0, 1)
    assert idx[0, 0].tolist() == [4, 0, 1, 2, 3, -1, -1]


def test_oracle_tables_by_hand():
    table = [[7, -1, -1], [8, 9, -1]]
    got = O.tables([3, 8], [3, 1], [0, 1, 2], 3, table, 4, 10, 6)
    assert got[0].tolist() == [[7, 2, -1], [8, 9, 1]]
    assert got[1].tolist() == [31, 8, 9, 4, -1, -1]
    assert got[2].tolist() == [6, 9] and got[3].tolist() == [0, 3, 4] and got[4] == 1
    assert got[5:] == (False, False, False)


def test_oracle_append_by_hand():
    k, v, m = np.zeros((2, 1, 2, 1)), np.zeros((2, 1, 2, 1)), np.zeros((2, 1, 1))
    new = np.array([[[2.0]], [[4.0]], [[6.0]]])
    O.append(k, v, m, new, -new, [2, 3, -1], 2)
    assert k[1, 0, :, 0].tolist() == [2, 4] and v[1, 0, :, 0].tolist() == [-2, -4]
    assert m[:, 0, 0].tolist() == [0, 3]

"""Host-side validation of the calls on the paged key-value cache, without a GPU: bad arguments are
refused before any launch, empty problems return OK."""
import ctypes as C

import numpy as np
import pytest

from kv_common import E4M3, TableModel, quantize_rows

import binarized_transformer_b200 as bt

P = 0x10000           # 16-byte aligned, never dereferenced
Q = 0x10008           # not aligned
F = C.c_void_p


@pytest.fixture(scope="module")
def lib():
    from binarized_transformer_b200 import build as b
    b.build()
    return bt.load_library()


def cache(**kw):
    a = dict(k=P, v=P, ks=None, vs=None, n=10, ps=16, H=2, D=64, stride=None, ss=0, type=0)
    a.update(kw)
    if a["stride"] is None:
        a["stride"] = a["H"] * a["ps"] * a["D"]
    return bt.KvCacheC(a["k"], a["v"], a["ks"], a["vs"], a["n"], a["ps"], a["H"], a["D"], a["stride"], a["ss"], a["type"])


def table(**kw):
    a = dict(pages=P, ld=4, mp=4, n=3, len=P, ref=P)
    a.update(kw)
    return bt.KvTableC(a["pages"], a["ld"], a["mp"], a["n"], a["len"], a["ref"])


BAD_CACHES = [
    (dict(type=2), bt.BWTA_ERR_INVALID_ARG), (dict(n=-1), bt.BWTA_ERR_INVALID_ARG),
    (dict(H=0), bt.BWTA_ERR_INVALID_ARG), (dict(D=60), bt.BWTA_ERR_UNSUPPORTED),
    (dict(D=136), bt.BWTA_ERR_UNSUPPORTED), (dict(D=0), bt.BWTA_ERR_INVALID_ARG),
    (dict(ps=24), bt.BWTA_ERR_UNSUPPORTED), (dict(ps=0), bt.BWTA_ERR_INVALID_ARG),
    (dict(ps=65552), bt.BWTA_ERR_UNSUPPORTED), (dict(n=1 << 31), bt.BWTA_ERR_UNSUPPORTED),
    (dict(stride=2047), bt.BWTA_ERR_INVALID_ARG), (dict(stride=2052), bt.BWTA_ERR_ALIGNMENT),
    (dict(stride=1 << 41), bt.BWTA_ERR_UNSUPPORTED),
    (dict(k=None), bt.BWTA_ERR_INVALID_ARG), (dict(v=Q), bt.BWTA_ERR_ALIGNMENT),
    (dict(type=1, ss=32), bt.BWTA_ERR_INVALID_ARG), (dict(type=1, ks=P, vs=P, ss=31), bt.BWTA_ERR_INVALID_ARG),
    (dict(type=1, ks=P, vs=Q, ss=32), bt.BWTA_ERR_ALIGNMENT), (dict(type=1, ks=P, vs=P, ss=34), bt.BWTA_ERR_ALIGNMENT),
]
BAD_TABLES = [
    (dict(n=-1), bt.BWTA_ERR_INVALID_ARG), (dict(ld=3), bt.BWTA_ERR_INVALID_ARG),
    (dict(mp=-1), bt.BWTA_ERR_INVALID_ARG), (dict(len=None), bt.BWTA_ERR_INVALID_ARG),
    (dict(pages=None), bt.BWTA_ERR_INVALID_ARG), (dict(n=1 << 31), bt.BWTA_ERR_UNSUPPORTED),
]


def append(lib, c=None, t=None, slots=None, n_seq=3, cu=None, total=3, k=P, ldk=128, v=P, ldv=128, kind=1):
    c, t = c or cache(), t or table()
    return lib.bwta_kv_append(C.byref(c), C.byref(t), slots, n_seq, cu, total, k, ldk, v, ldv, kind, None, None)


def decode(lib, c=None, t=None, slots=None, n_seq=3, q=P, ldq=256, heads=4, scale=0.125, window=0, sinks=0, out=P,
           ldo=256, ws=P, ws_bytes=1 << 40):
    c, t = c or cache(), t or table()
    return lib.bwta_attn_decode_paged(C.byref(c), C.byref(t), slots, n_seq, q, ldq, heads, scale, window, sinks, out,
                                      ldo, ws, ws_bytes, None, None)


def prompt(lib, c=None, t=None, slots=None, n_seq=3, cu=P, total=9, q=P, ldq=256, heads=4, scale=0.125, window=0,
           sinks=0, out=P, ldo=256):
    c, t = c or cache(), t or table()
    return lib.bwta_attn_prompt_paged(C.byref(c), C.byref(t), slots, n_seq, cu, total, q, ldq, heads, scale, window,
                                      sinks, out, ldo, None, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(lib, kw, code):
    c = cache(**kw)
    t = table()
    for f in (append, decode, prompt):
        assert f(lib, c=c) == code
    assert lib.bwta_kv_fork(C.byref(c), 1, C.byref(t), P, P, 1, P, 1 << 30, None, None) == code
    assert lib.bwta_kv_compact(C.byref(c), 1, C.byref(t), None, P, 1 << 40, None, None) == code
    assert lib.bwta_kv_copy_pages(C.byref(c), C.byref(c), 1, P, P, 1, P, 1 << 30, None, None) == code


@pytest.mark.parametrize("kw,code", BAD_TABLES)
def test_bad_tables(lib, kw, code):
    t, c = table(**kw), cache()
    for f in (append, decode, prompt):
        assert f(lib, t=t) == code
    assert lib.bwta_kv_reserve(C.byref(t), 10, 16, P, P, 1, None, None) == code
    assert lib.bwta_kv_free(C.byref(t), 10, 16, P, 1, None, None) == code
    assert lib.bwta_kv_fork(C.byref(c), 1, C.byref(t), P, P, 1, P, 1 << 30, None, None) == code
    assert lib.bwta_kv_compact(C.byref(c), 1, C.byref(t), None, P, 1 << 30, None, None) == code


@pytest.mark.parametrize("f", [append, decode, prompt])
def test_null_structs(lib, f):
    for name in ("bwta_kv_append", "bwta_attn_decode_paged", "bwta_attn_prompt_paged"):
        fn = getattr(lib, name)
        rest = [None if a in (C.c_void_p,) else 0 for a in fn.argtypes[2:]]
        assert fn(None, C.byref(table()), *rest) == bt.BWTA_ERR_INVALID_ARG
        assert fn(C.byref(cache()), None, *rest) == bt.BWTA_ERR_INVALID_ARG


def test_append_arguments(lib):
    I, A = bt.BWTA_ERR_INVALID_ARG, bt.BWTA_ERR_ALIGNMENT
    assert append(lib, n_seq=-1) == I and append(lib, total=2) == I and append(lib, n_seq=4, total=4) == I
    assert append(lib, kind=2) == I and append(lib, ldk=127) == I and append(lib, v=None) == I
    assert append(lib, k=Q) == A and append(lib, ldv=130) == A and append(lib, ldk=132, kind=0) == A
    assert append(lib, n_seq=0, total=0) == bt.BWTA_OK
    assert append(lib, n_seq=0, cu=P, total=5) == bt.BWTA_OK
    assert append(lib, slots=P, n_seq=0, total=0, k=None, v=None) == bt.BWTA_OK


@pytest.mark.parametrize("f", [decode, prompt])
def test_attention_arguments(lib, f):
    I, A, U = bt.BWTA_ERR_INVALID_ARG, bt.BWTA_ERR_ALIGNMENT, bt.BWTA_ERR_UNSUPPORTED
    assert f(lib, n_seq=-1) == I and f(lib, n_seq=4) == I and f(lib, heads=3) == I and f(lib, heads=0) == I
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert f(lib, scale=s) == I
    assert f(lib, window=-1) == I and f(lib, sinks=1) == I and f(lib, window=5, sinks=-1) == I
    assert f(lib, ldq=255) == I and f(lib, ldo=248) == I and f(lib, q=None) == I and f(lib, out=None) == I
    assert f(lib, q=Q) == A and f(lib, out=Q) == A and f(lib, ldq=260) == A and f(lib, ldo=260) == A
    assert f(lib, heads=65536, ldq=1 << 23, ldo=1 << 23) == U
    assert f(lib, t=table(mp=1 << 27, ld=1 << 27)) == U     # positions past 31 bits
    assert f(lib, n_seq=0, **(dict(total=0) if f is prompt else {})) == bt.BWTA_OK


def test_prompt_and_workspace_arguments(lib):
    I = bt.BWTA_ERR_INVALID_ARG
    assert prompt(lib, cu=None) == I and prompt(lib, total=-1) == I
    assert prompt(lib, c=cache(H=1), heads=129, ldq=1 << 14, ldo=1 << 14) == bt.BWTA_ERR_UNSUPPORTED
    want = lib.bwta_attn_decode_workspace(4, 2, 64)
    if want:
        assert decode(lib, ws_bytes=want - 1) == I and decode(lib, ws=None) == I
    assert decode(lib, ws=Q) == bt.BWTA_ERR_ALIGNMENT


def test_page_call_arguments(lib):
    I, A, U = bt.BWTA_ERR_INVALID_ARG, bt.BWTA_ERR_ALIGNMENT, bt.BWTA_ERR_UNSUPPORTED
    t, c = table(), cache()

    def reserve(num=10, ps=16, s=P, g=P, n=1, t=t):
        return lib.bwta_kv_reserve(C.byref(t), num, ps, s, g, n, None, None)
    assert reserve(num=-1) == I and reserve(ps=0) == I and reserve(ps=20) == U and reserve(num=(1 << 19) + 1) == U
    assert reserve(s=None) == I and reserve(g=None) == I and reserve(n=-1) == I and reserve(n=2049) == U
    assert reserve(t=table(ref=None)) == I and reserve(n=0) == bt.BWTA_OK

    def free(s=P, n=1, t=t):
        return lib.bwta_kv_free(C.byref(t), 10, 16, s, n, None, None)
    assert free(s=None) == I and free(n=-1) == I and free(n=1 << 31) == U and free(n=0) == bt.BWTA_OK

    def fork(c=c, layers=1, s=P, d=P, n=1, ws=P, b=1 << 30, t=t):
        return lib.bwta_kv_fork(c if isinstance(c, C.Array) else C.byref(c), layers, C.byref(t), s, d, n, ws, b, None, None)
    need = lib.bwta_kv_pages_workspace(10, 1)
    assert fork(layers=0) == I and fork(layers=129) == U and fork(s=None) == I and fork(d=None) == I
    assert fork(n=-1) == I and fork(n=2049) == U and fork(b=need - 1) == I and fork(ws=None) == I and fork(ws=Q) == A
    assert fork(t=table(ref=None)) == I and fork(n=0) == bt.BWTA_OK
    for kw in (dict(n=11), dict(ps=32), dict(H=1), dict(D=32), dict(stride=4096), dict(type=1, ks=P, vs=P, ss=32)):
        assert fork(c=(bt.KvCacheC * 2)(cache(), cache(**kw)), layers=2) == I
    assert fork(c=cache(n=(1 << 19) + 1), b=1 << 40) == U

    def compact(ws=P, b=1 << 30):
        return lib.bwta_kv_compact(C.byref(c), 1, C.byref(t), None, ws, b, None, None)
    assert compact(b=lib.bwta_kv_pages_workspace(10, 0) - 1) == I and compact(ws=Q) == A

    def copy(a, b, n=1, s=P, d=P, layers=1, ws=P, wb=1 << 30):
        a, b = ((bt.KvCacheC * len(x))(*x) for x in (a, b))
        return lib.bwta_kv_copy_pages(a, b, layers, s, d, n, ws, wb, None, None)
    R = 0x90000
    assert copy([cache()], [cache(k=R, v=R, D=32)]) == I and copy([cache()], [cache(k=R, v=R)], n=-1) == I
    assert copy([cache()], [cache(k=R, v=R)], s=None) == I
    assert copy([cache()], [cache(k=R, v=R)], n=(1 << 19) + 1, wb=1 << 40) == U
    # pools that share some of their memory are neither one nor two
    assert copy([cache(v=R)], [cache(v=R + 0x1000)]) == I
    assert copy([cache(v=R)], [cache(k=R, v=P)]) == I
    assert copy([cache(k=P, v=P), cache(k=R, v=R)], [cache(k=R, v=R), cache(k=P, v=P)], layers=2) == I
    # one pool, described in two ways
    assert copy([cache(v=R)], [cache(v=R, n=11)]) == I and copy([cache(v=R, n=11)], [cache(v=R)]) == I
    assert copy([cache(v=R)], [cache(v=R, stride=8192)]) == I
    assert copy([cache()], [cache(k=R, v=R, n=3)], n=0) == bt.BWTA_OK
    assert lib.bwta_kv_pages_workspace(-1, 0) == 0


# ------------------------------------------------------------------ the models that the GPU tests use
def test_e4m3_model_rounds_to_nearest_even():
    v = np.sort(E4M3[:127])
    assert v[0] == 0 and v[-1] == 448 and (np.diff(v) > 0).all()
    mid = (v[:-1] + v[1:]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9)])
    # a row whose largest value is 448 has the scale 1
    rows = np.stack([x, np.full_like(x, 448.0)], 1)
    codes, scale = quantize_rows(rows)
    assert (scale == 1).all()
    got = E4M3[codes[:, 0]]
    assert (np.abs(got - x) <= np.abs(v[None] - x[:, None]).min(1)).all()
    ties = codes[len(v):len(v) + len(mid), 0]
    assert (ties % 2 == 0).all()


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (65504.0, 8), (57344.0, 7), (57345.0, 8),
                                   (1e-9, -15), (0.0, 0), (448 * 2.0 ** -15, -15)])
def test_e4m3_scale_rule(top, e):
    codes, scale = quantize_rows(np.array([[top, 0.0]]))
    assert scale[0] == 2.0 ** e
    val = E4M3[codes[0, 0]] * scale[0]
    assert val == np.float16(val)                             # every stored value is an fp16 value


def test_table_model_keeps_its_books():
    r = np.random.default_rng(0)
    m = TableModel(8, 10, 30, 16)
    for _ in range(200):
        k = r.integers(0, 4)
        if k == 0:
            m.reserve(r.integers(0, 8, 3).tolist(), r.integers(0, 40, 3).tolist())
        elif k == 1:
            m.free(r.integers(0, 8, 2).tolist())
        elif k == 2:
            m.fork(r.integers(0, 8, 3).tolist(), r.integers(0, 8, 3).tolist())
        else:
            m.compact()
        count = [0] * 30
        for s in range(8):
            for i in range(m.need(m.len[s])):
                count[m.pages[s][i]] += 1
        assert count == m.ref


def _pools(lib, a, b, n=1):
    a, b = ((bt.KvCacheC * len(x))(*x) for x in (a, b))
    return lib.bwta_kv_copy_pages(a, b, len(a), P, P, n, P, 1 << 30, None, None)


def test_copies_between_pools_that_coincide_in_some_layers(lib):
    """One pool in every layer or none: a layer copied within itself would race with the list's other copies."""
    I = bt.BWTA_ERR_INVALID_ARG
    A, B, D, E = 0x20000, 0x30000, 0x40000, 0x50000
    one, two, other = cache(k=A, v=B), cache(k=D, v=E), cache(k=0x60000, v=0x70000)
    assert _pools(lib, [one, two], [one, other]) == I
    assert _pools(lib, [two, one], [other, one]) == I
    assert _pools(lib, [one, two], [cache(k=A, v=B, n=11), cache(k=0x60000, v=0x70000, n=11)]) == I

    def e4m3(k, v, ks, vs):
        return cache(type=1, k=k, v=v, ks=ks, vs=vs, ss=32)
    x = e4m3(A, B, 0x1000, 0x2000)
    assert _pools(lib, [x], [e4m3(D, E, 0x1000, 0x3000)]) == I      # scales shared, bytes not
    assert _pools(lib, [x], [e4m3(D, E, 0x3000, 0x2000)]) == I
    assert _pools(lib, [x], [e4m3(D, E, 0x2000, 0x1000)]) == I
    assert _pools(lib, [x], [e4m3(A, B, 0x1000, 0x3000)]) == I      # bytes shared, scales not
    y = e4m3(D, E, 0x3000, 0x4000)
    assert _pools(lib, [x, y], [e4m3(0x60000, 0x70000, 0x3000, 0x6000), e4m3(0x80000, 0x90000, 0x7000, 0x8000)]) == I


def test_copies_of_two_layers_into_one(lib):
    """A target that is listed for two sources would hold parts of each."""
    I = bt.BWTA_ERR_INVALID_ARG
    one, two = cache(k=0x20000, v=0x30000), cache(k=0x40000, v=0x50000)
    assert _pools(lib, [one, two], [cache(k=0x60000, v=0x70000)] * 2) == I
    assert _pools(lib, [one, two], [cache(k=0x60000, v=0x70000), cache(k=0x60000, v=0x80000)]) == I
    a, b = (cache(type=1, k=0x20000 * i, v=0x30000 * i, ks=0x100 * i, vs=0x200 * i, ss=32) for i in (1, 5))
    to = [cache(type=1, k=0x500000 * i, v=0x700000 * i, ks=0x1000, vs=0x2000 * i, ss=32) for i in (1, 3)]
    assert _pools(lib, [a, b], to) == I

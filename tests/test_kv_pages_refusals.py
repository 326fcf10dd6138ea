"""Refusals of the paged KV cache's entry points, at the C ABI and in the
binding (CPU only: every call here is refused before any HIP call, or has
nothing to do)."""
import ctypes

import pytest
import torch

import bit_linear_layer_amd as nv

FAKE = 1 << 20


def pages(**kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, n_pages=8, heads=2, dim=128, page=32)
    a.update(kw)
    a.setdefault("ldc", a["heads"] * a["page"] * a["dim"])
    a.setdefault("lds", a["heads"] * a["page"])
    return nv._KVPages(a["k"], a["v"], a["ks"], a["vs"], a["n_pages"], a["ldc"], a["lds"], a["heads"], a["dim"], a["page"])


PAGES = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
    (dict(dim=96), -2), (dict(dim=0), -2), (dict(page=8), -2), (dict(page=48), -2), (dict(page=8192), -2), (dict(page=-16), -2),
    (dict(heads=0), -2), (dict(heads=4097), -2), (dict(n_pages=0), -2),
    (dict(n_pages=1 << 31), -11), (dict(n_pages=1 << 26), -11),
    (dict(ldc=2 * 32 * 128 - 16), -4), (dict(ldc=2 * 32 * 128 + 8), -4), (dict(lds=48), -4), (dict(lds=72), -4),
    (dict(k=FAKE + 8), -5), (dict(vs=FAKE + 4), -5),
]
ROWS = [
    (dict(x=None), -1), (dict(slots=None), -1), (dict(dt=5), -3), (dict(rows=-1), -2), (dict(rows=1 << 28), -11),
    (dict(ld=255), -4), (dict(ld=257), -4), (dict(x=FAKE + 8), -5), (dict(slots=FAKE + 4), -5), (dict(rows=0), 0),
    (dict(rows=0, x=None, slots=None), 0),
]


def write(p, x=FAKE, ld=256, dt=0, rows=4, slots=FAKE):
    return nv.load().nvfp4_kv_pages_write(ctypes.byref(p), x, ld, FAKE, 256, dt, rows, slots, None)


def read(p, x=FAKE, ld=256, dt=0, rows=4, slots=FAKE):
    return nv.load().nvfp4_kv_pages_read(ctypes.byref(p), rows, slots, FAKE, 256, x, ld, dt, None)


@pytest.mark.parametrize("kw,status", PAGES)
def test_bad_caches(kw, status):
    p = pages(**kw)
    assert write(p) == status and read(p) == status and attention(p) == status


@pytest.mark.parametrize("kw,status", ROWS)
def test_bad_rows(kw, status):
    assert write(pages(), **kw) == status and read(pages(), **kw) == status


def batch(**kw):
    a = dict(batch=3, q_len=1, lens=FAKE, max_len=100, table=FAKE, cols=4, ldt=4, prefix=FAKE, prefix_len=500)
    a.update(kw)
    return nv._KVBatch(a["batch"], a["q_len"], a["lens"], a["max_len"], a["table"], a["cols"], a["ldt"], a["prefix"],
                       a["prefix_len"])


def need(p, b, q_heads=4, dt=0):
    return nv.load().nvfp4_kv_pages_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), q_heads, dt)


def attention(p=None, b=None, q=FAKE, ldq=512, dt=0, q_heads=4, scale=0.1, out=FAKE, ldo=512, ws=FAKE, less=0, wsb=None):
    p, b = p or pages(), b or batch()
    n = need(p, b, q_heads, dt) - less if wsb is None else wsb
    return nv.load().nvfp4_kv_pages_attention(ctypes.byref(p), ctypes.byref(b), q, ldq, dt, q_heads, scale, out, ldo, ws, n,
                                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), -2), (dict(q_len=0), -2), (dict(max_len=-1), -2), (dict(prefix_len=-1), -2),
    (dict(batch=1 << 31), -11), (dict(q_len=1 << 31), -11), (dict(max_len=1 << 31, cols=1 << 30), -11),
    (dict(prefix_len=1 << 31), -11), (dict(batch=1 << 20, q_len=1 << 10), -11), (dict(batch=1 << 24), -11),
    (dict(lens=None), -1), (dict(table=None), -1), (dict(prefix=None), -1),
    (dict(max_len=129), -2), (dict(cols=3), -2), (dict(ldt=3), -4),
    (dict(lens=FAKE + 2), -5), (dict(table=FAKE + 1), -5), (dict(prefix=FAKE + 2), -5),
    (dict(batch=0), 0),
])
def test_bad_batches(kw, status):
    b = batch(**kw)
    assert attention(b=b, wsb=1 << 40) == status
    if status == -11:
        assert need(pages(), b) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -8), (dict(less=1), -8), (dict(ws=FAKE + 8), -5),
    (dict(dt=3, wsb=1 << 40), -3), (dict(q_heads=3, wsb=1 << 40), -2), (dict(q_heads=0, wsb=1 << 40), -2),
    (dict(ldq=508), -4), (dict(ldo=516), -4), (dict(q=FAKE + 8), -5), (dict(out=FAKE + 4), -5),
    (dict(scale=0.0), -12), (dict(scale=-1.0), -12), (dict(scale=float("nan")), -12), (dict(scale=float("inf")), -12),
    (dict(scale=3e38), -12),
])
def test_bad_attention_arguments(kw, status):
    assert attention(**kw) == status


def test_null_structs():
    lib = nv.load()
    assert lib.nvfp4_kv_pages_write(None, FAKE, 256, FAKE, 256, 0, 4, FAKE, None) == -1
    assert lib.nvfp4_kv_pages_read(None, 4, FAKE, FAKE, 256, FAKE, 256, 0, None) == -1
    p = pages()
    assert lib.nvfp4_kv_pages_attention(ctypes.byref(p), None, FAKE, 512, 0, 4, 0.1, FAKE, 512, FAKE, 1 << 30, None) == -1
    assert lib.nvfp4_kv_pages_attention_workspace_bytes(None, None, 4, 0) == 0


def test_workspace_covers_every_shape():
    """Positive, a multiple of 4, and not smaller for a longer bound."""
    last = 0
    for n in (1, 64, 256, 257, 4096, 1 << 20):
        b = batch(max_len=n, prefix_len=0, cols=1 << 20)
        got = need(pages(), b)
        assert got > 0 and got % 4 == 0 and got >= last
        last = got
    assert nv.nvfp4_status_string(-12) not in ("", "unknown status")


def test_binding_refuses_host_tensors():
    t = lambda *shape, dtype=torch.uint8: torch.zeros(shape, dtype=dtype)  # noqa: E731
    c = nv.KVPages(t(4, 2 * 16 * 64), t(4, 2 * 16 * 64), t(4, 32), t(4, 32), 2, 64, 16)
    slots = t(3, dtype=torch.int64)
    x = t(3, 128, dtype=torch.bfloat16)
    for call in (lambda: nv.kv_pages_write(c, x, x, slots), lambda: nv.kv_pages_read(c, slots),
                 lambda: nv.kv_pages_attention(x, c)):
        with pytest.raises(nv.NVFP4Error):
            call()


@pytest.mark.parametrize("kw,q_heads,taken", [
    (dict(max_len=1 << 30, cols=1 << 28), 4, False), (dict(prefix_len=1 << 30), 4, False),
    (dict(max_len=(1 << 30) - 1, cols=1 << 28, prefix_len=(1 << 30) - 1), 4, True),
    (dict(q_len=1 << 28, batch=1), 4, False), (dict(q_len=(1 << 28) - 1, batch=1), 4, True),
    (dict(batch=1 << 23, q_len=1), 2, False), (dict(batch=(1 << 23) - 1, q_len=64), 2, True), (dict(batch=1 << 23, q_len=64), 2, False),
])
def test_largest_shapes(kw, q_heads, taken):
    """The plan of the largest shapes stays within its integers: the workspace
    is 0 where a shape is refused, and otherwise below the partial results of
    every row and of every share (2 passes of at most 2048 shares of 128 rows)."""
    b = batch(**kw)
    heads, dim = 2, 128
    got = need(pages(heads=heads, dim=dim), b, q_heads)
    rows = b.batch * b.q_len * q_heads
    if not taken:
        assert got == 0 and attention(pages(heads=heads, dim=dim), b, q_heads=q_heads, ldq=dim * q_heads, ldo=dim * q_heads, wsb=1 << 50) == -11
    else:
        tiles = 2 * (-(-rows // 16) + b.batch * heads)  # a ragged last tile in each
        assert 0 < got <= 4 * (dim + 4) * (2 * rows + 128 * tiles + 2 * 2048 * 128)


@pytest.mark.parametrize("shape,q_len", [((4, 128), 0), ((4, 128), -1), ((4, 128), 3), ((512,), 1), ((2, 2, 128), 1)])
def test_binding_refuses_rows_that_are_no_batch(shape, q_len):
    t = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    c = nv.KVPages(t(4, 2 * 16 * 64), t(4, 2 * 16 * 64), t(4, 32), t(4, 32), 2, 64, 16)
    with pytest.raises(nv.NVFP4Error):
        nv.kv_pages_attention(torch.zeros(shape, dtype=torch.bfloat16), c, q_len=q_len)
    if len(shape) != 2:
        with pytest.raises(nv.NVFP4Error):
            nv.kv_pages_attention_workspace(torch.zeros(shape, dtype=torch.bfloat16), c, 4)

"""Drive the paged KV cache's entry points in a sanitized host build: random
calls, each either refused with a status of the header or passed on to a
launcher.  Run in a process that preloads the sanitizer runtime.
Usage: python kv_pages_driver.py LIB"""
import ctypes
import random
import sys

P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
FAKE = 1 << 20  # never dereferenced by the host layer


class Pages(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("ks", P), ("vs", P), ("n_pages", I64), ("ld_codes", I64), ("ld_scales", I64),
                ("heads", I32), ("dim", I32), ("page", I32)]


class Batch(ctypes.Structure):
    _fields_ = [("batch", I64), ("q_len", I64), ("lens", P), ("max_len", I64), ("table", P), ("cols", I64), ("ldt", I64),
                ("prefix", P), ("prefix_len", I64)]


libc = ctypes.CDLL(None)
libc.malloc.restype, libc.malloc.argtypes = P, [SZ]
libc.free.argtypes = [P]


def block(struct):
    """The struct in a malloc'ed block of its own size, so that a read past its end is seen."""
    at = libc.malloc(ctypes.sizeof(struct))
    ctypes.memmove(at, ctypes.byref(struct), ctypes.sizeof(struct))
    return at


def main(path):
    lib = ctypes.CDLL(path)
    lib.nvfp4_kv_pages_write.argtypes = [P, P, I64, P, I64, I32, I64, P, P]
    lib.nvfp4_kv_pages_read.argtypes = [P, I64, P, P, I64, P, I64, I32, P]
    lib.nvfp4_kv_pages_attention_workspace_bytes.argtypes = [P, P, I32, I32]
    lib.nvfp4_kv_pages_attention_workspace_bytes.restype = SZ
    lib.nvfp4_kv_pages_attention.argtypes = [P, P, P, I64, I32, I32, ctypes.c_float, P, I64, P, SZ, P]
    rng = random.Random(1)
    big = [-(1 << 63), -1, 0, 1, (1 << 24) - 1, 1 << 24, 1 << 28, (1 << 30) - 1, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 63) - 1]
    seen, ok = set(), 0

    def odd(value, chance=0.04):
        return rng.choice(big) if rng.random() < chance else value

    def odd32(value):
        v = odd(value)
        return max(min(v, (1 << 31) - 1), -(1 << 31))

    def pointer():
        return None if rng.random() < 0.02 else FAKE + (rng.choice([2, 4, 8]) if rng.random() < 0.02 else 0)

    for _ in range(20000):
        heads, dim, page = rng.choice([1, 2, 8, 4096]), rng.choice([64, 128, 256]), rng.choice([16, 64, 4096])
        c = Pages(pointer(), pointer(), pointer(), pointer(), odd(rng.randint(1, 5000)), odd(heads * page * dim),
                  odd(heads * page), odd32(heads), odd32(dim), odd32(page))
        b = Batch(odd(rng.randint(0, 9)), odd(rng.randint(1, 5)), pointer(), odd(rng.randint(0, 4 * page)), pointer(),
                  odd(4), odd(rng.randint(4, 5)), pointer(), odd(rng.randint(0, 9999)))
        cp, bp = block(c), block(b)
        calls = lib.nvfp4_kv_stub_calls()
        esz = rng.choice([0, 0, 1, 1, 7]) if rng.random() < 0.1 else rng.randint(0, 1)
        width = heads * dim
        which = rng.randint(0, 2)
        if which == 0:
            st = lib.nvfp4_kv_pages_write(cp, pointer(), odd(width), pointer(), odd(width), esz, odd(rng.randint(0, 9)), pointer(), None)
        elif which == 1:
            st = lib.nvfp4_kv_pages_read(cp, odd(rng.randint(0, 9)), pointer(), pointer(), odd(width), pointer(), odd(width), esz, None)
        else:
            q_heads = odd32(heads * rng.randint(1, 9))
            need = lib.nvfp4_kv_pages_attention_workspace_bytes(cp, bp, q_heads, esz)
            ld = odd(max(0, min(q_heads, 1 << 20)) * dim)
            scale = rng.choice([0.1] * 20 + [0.0, -1.0, float("nan"), float("inf"), 3e38])
            st = lib.nvfp4_kv_pages_attention(cp, bp, pointer(), ld, esz, q_heads, scale, pointer(), ld, pointer(),
                                              max(0, need - (rng.random() < 0.02)), None)
            if need and st == 0 and lib.nvfp4_kv_stub_calls() > calls:
                assert lib.nvfp4_kv_stub_group() * c.heads == q_heads
        assert -12 <= st <= 0, st
        launched = lib.nvfp4_kv_stub_calls() - calls
        assert launched in ((0, 1) if st == 0 else (0,)), (st, launched)
        if launched:
            assert 1 << lib.nvfp4_kv_stub_page_shift() == c.page
            ok += 1
        seen.add(st)
        libc.free(cp)
        libc.free(bp)
    assert ok > 2000 and seen >= {0, -1, -2, -3, -4, -5, -8, -11, -12}, (ok, seen)
    print("sanitized paged KV driver ok", ok)


main(sys.argv[1])

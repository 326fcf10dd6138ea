"""Drive the entry points of layer_api.hip in a sanitized host build: random
calls, each either refused with a status of the header or passed on to a
launcher with the sizes asked for.  Run in a process that preloads the
sanitizer runtime.  Usage: python layer_driver.py LIB"""
import ctypes
import random
import sys

P, I64, I32, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
FAKE = 1 << 20  # never dereferenced by the host layer


def struct(*fields):
    return type("S", (ctypes.Structure,), {"_fields_": [(f"f{i}", t) for i, t in enumerate(fields)]})


FP8 = struct(P, P, I64, I64, I64, I64, I32)
HEADS = struct(P, I64, I64, P, I64, I64, P, I32)
ROPE = struct(P, I64, P, P, I32, I32, I32)
CONV = struct(P, I64, P, I64, P, P, I64, I64, I64, I32, I32, P, P, I64, I64, P, P)
GDN = struct(*[t for _ in range(5) for t in (P, I64)])

libc = ctypes.CDLL(None)
libc.malloc.restype, libc.malloc.argtypes = P, [SZ]
libc.free.argtypes = [P]


def main(path):
    lib = ctypes.CDLL(path)
    lib.nvfp4_fp8_quantize.argtypes = [P, I32, I64, P, I32, P]
    lib.nvfp4_fp8_gemm.argtypes = [P, P, P, I32, I64, P, SZ, P]
    lib.nvfp4_fp8_gemm_workspace_bytes.argtypes, lib.nvfp4_fp8_gemm_workspace_bytes.restype = [I64], SZ
    lib.nvfp4_fp8_linear_workspace_bytes.argtypes, lib.nvfp4_fp8_linear_workspace_bytes.restype = [I64, I64], SZ
    lib.nvfp4_fp8_linear.argtypes = [P, I32, I64, I64, P, P, I32, I64, P, SZ, P]
    lib.nvfp4_qk_norm_rope.argtypes = [P, P, I32, I64, I32, F, F, P, P]
    lib.nvfp4_causal_conv.argtypes = [P, I32, P]
    lib.nvfp4_gdn_step.argtypes = [P, I32, I64, I64, I32, I32, I32, P, I64, I64, P, P, P, I32, I64, P]
    lib.nvfp4_layer_stub_seen.restype = I64
    rng = random.Random(1)
    big = [-(1 << 63), -1, 0, 1, (1 << 20) - 1, 1 << 22, 1 << 24, (1 << 31) - 1, 1 << 31, 1 << 40, (1 << 63) - 1]
    blocks = []

    def odd(v, chance=0.02):
        return rng.choice(big) if rng.random() < chance else v

    def odd32(v):
        return max(min(odd(v), (1 << 31) - 1), -(1 << 31))

    def at():
        return None if rng.random() < 0.01 else FAKE + (rng.choice([1, 2, 4, 8]) if rng.random() < 0.01 else 0)

    def block(s):
        """The struct in a malloc'ed block of its own size, so that a read past its end is seen."""
        if rng.random() < 0.01:
            return None
        p = libc.malloc(ctypes.sizeof(s))
        ctypes.memmove(p, ctypes.byref(s), ctypes.sizeof(s))
        blocks.append(p)
        return p

    def up(v, a):
        return -(-v // a) * a

    seen, ok = set(), [0] * 6
    for _ in range(40000):
        calls, which, dt = lib.nvfp4_layer_stub_calls(), rng.randint(0, 5), odd32(rng.randint(0, 1))
        want = None
        if which <= 2:
            m, n, k = rng.randint(0, 300), rng.randint(1, 500), 16 * rng.randint(1, 300)
            m, n, k = odd(m), odd(n), odd(k)
            safe = max(0, min(k, 1 << 40))
            ld, lds = odd(up(safe, 16)), odd(-(-safe // 128))
            a, w = FP8(at(), at(), m, k, ld, lds, odd32(1)), FP8(at(), at(), n, odd(k, 0.005), ld, lds, odd32(128))
            if which == 0:
                q = a if rng.random() < 0.5 else w
                st = lib.nvfp4_fp8_quantize(at(), dt, odd(up(safe, 16)), block(q), rng.choice([0, 0, 1, 1, 2]), None)
            elif which == 1:
                st = lib.nvfp4_fp8_gemm(block(a), block(w), at(), dt, odd(max(0, min(n, 1 << 40))), at(),
                                        max(0, lib.nvfp4_fp8_gemm_workspace_bytes(m) - (rng.random() < 0.02)), None)
                want = (m, n, k)
            else:
                need = lib.nvfp4_fp8_linear_workspace_bytes(m, k)
                st = lib.nvfp4_fp8_linear(at(), dt, m, odd(up(safe, 16)), block(w), at(), odd32(rng.randint(0, 1)), odd(max(0, min(n, 1 << 40))),
                                          at(), max(0, need - (rng.random() < 0.02)), None)
        elif which == 3:
            d, t = odd32(rng.choice([64, 128, 256])), odd(rng.randint(0, 99))
            side = []
            for _ in range(2):
                h, gap = odd32(rng.randint(1, 9)), 8 * rng.randint(0, 3)
                wide = max(0, min(h, 99)) * (max(0, min(d, 256)) + gap)
                side.append(block(HEADS(at(), odd(wide), odd(max(0, min(d, 256)) + gap), at(), odd(wide), odd(max(0, min(d, 256)) + gap), at(), h)))
            r = ROPE(at(), odd(max(0, min(t, 99))), at(), at(), odd32(rng.randint(1, 4)), odd32(16 * rng.randint(1, 4)), rng.randint(0, 1))
            st = lib.nvfp4_qk_norm_rope(side[0], side[1], dt, t, d, rng.choice([1e-6] * 30 + [0.0, -1.0, float("nan")]), 1.0, block(r), None)
            want = (t,)
        elif which == 4:
            t, c, b, w = odd(rng.randint(0, 99)), odd(8 * rng.randint(1, 99)), odd(rng.randint(0, 9)), odd32(rng.randint(2, 4))
            ld = odd(max(0, min(c, 1 << 22)))
            s = CONV(at(), ld, None if rng.random() < 0.01 else 2 * FAKE, ld, at(), at(), t, c, b, w, 1, at(), at(), odd(rng.randint(9, 12)),
                     odd(8 * max(0, min(c, 1 << 22))), at(), at())
            st = lib.nvfp4_causal_conv(block(s), dt, None)
            want = (t, c, b, w)
        else:
            b, n, hk, r = odd(rng.randint(0, 9)), odd(rng.randint(1, 5)), odd32(rng.randint(1, 9)), rng.randint(1, 4)
            hv = max(min(hk * r, (1 << 31) - 1), -(1 << 31))
            kw, vw = max(0, min(hk, 1 << 20)) * 128, max(0, min(hv, 1 << 20)) * 128
            i = GDN(at(), odd(kw), at(), odd(kw), at(), odd(vw), at(), odd(vw), at(), odd(vw))
            st = lib.nvfp4_gdn_step(block(i), dt, b, n, hk, hv, 1, at(), odd(rng.randint(9, 12)), odd(vw * 128), at(), at(), at(),
                                    odd32(rng.randint(0, 1)), odd(vw), None)
            want = (b, n, hk, hv)
        assert -12 <= st <= 0, st
        launched = lib.nvfp4_layer_stub_calls() - calls
        assert launched <= (2 if which == 2 else 1) and (st == 0 or launched == 0), (which, st, launched)
        if launched:
            ok[which] += 1
            if want is not None:
                assert tuple(lib.nvfp4_layer_stub_seen(j) for j in range(len(want))) == want, (which, want)
        seen.add(st)
        while blocks:
            libc.free(blocks.pop())
    assert min(ok) > 1000 and seen >= {0, -1, -2, -3, -4, -5, -8, -9, -11, -12}, (ok, seen)
    print("sanitized layer driver ok", ok)


main(sys.argv[1])

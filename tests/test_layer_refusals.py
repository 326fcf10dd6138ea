"""Refusals of the 8-bit linear layers, the norm with rotation, the short
convolution and the gated delta rule's next tokens, at the C ABI and in the
binding (CPU only: every call here is refused before any HIP call, or has
nothing to do)."""
import pytest
import torch

import bit_linear_layer_amd as nv

FAKE = 1 << 20
BIG = 1 << 62


def pack(f, *values):
    """The struct's bytes, for what its integers hold; a NULL pointer is None."""
    return f(*[0 if v is None else v for v in values])


# ------------------------------------------------------------ 8-bit layers

def fp8(**kw):
    a = dict(codes=FAKE, scales=FAKE, rows=5, cols=272, ldc=272, lds=3, block=1)
    a.update(kw)
    return pack(nv._FP8, a["codes"], a["scales"], a["rows"], a["cols"], a["ldc"], a["lds"], a["block"])


def quantize(q=None, x=FAKE, dt=0, ld=272, flags=0):
    return nv.load().nvfp4_fp8_quantize(x, dt, ld, q or fp8(), flags, None)


def gemm(a=None, w=None, out=FAKE, dt=0, ld=130, ws=FAKE, wsb=1 << 30):
    return nv.load().nvfp4_fp8_gemm(a or fp8(), w or fp8(rows=130, block=128), out, dt, ld, ws, wsb, None)


def linear(w=None, x=FAKE, dt=0, rows=5, ld=272, out=FAKE, odt=0, ldo=130, ws=FAKE, wsb=1 << 30):
    return nv.load().nvfp4_fp8_linear(x, dt, rows, ld, w or fp8(rows=130, block=128), out, odt, ldo, ws, wsb, None)


MATRICES = [
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(rows=-1), -2), (dict(cols=0), -2), (dict(cols=264), -2),
    (dict(block=0), -2), (dict(block=64), -2), (dict(ldc=256), -4), (dict(ldc=280), -4), (dict(lds=2), -4),
    (dict(codes=FAKE + 8), -5), (dict(scales=FAKE + 2), -5), (dict(rows=1 << 31), -11), (dict(rows=BIG), -11),
    (dict(cols=1 << 22, ldc=1 << 22, lds=1 << 15), -11), (dict(ldc=1 << 22), -11), (dict(lds=1 << 22), -11), (dict(ldc=BIG), -11),
    (dict(rows=1 << 30, ldc=1 << 20), -11),
]


@pytest.mark.parametrize("kw,status", MATRICES)
def test_bad_matrices(kw, status):
    assert quantize(fp8(**kw)) == status and gemm(a=fp8(**kw)) == status
    if "block" not in kw and kw.get("rows", 1) >= 0:
        assert gemm(w=fp8(**dict(dict(rows=130), block=128, **kw) if "rows" not in kw else dict(kw, block=128))) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(dt=7), -3), (dict(ld=256), -4), (dict(ld=276), -4), (dict(x=FAKE + 4), -5), (dict(flags=2), -9),
    (dict(ld=1 << 44), -11), (dict(q=fp8(rows=0, codes=None, scales=None)), 0), (dict(q=fp8(rows=0), x=None), 0),
    (dict(dt=1, ld=274), -4), (dict(q=fp8(rows=(1 << 31) - 1, cols=65536, ldc=65536, lds=512, block=128), ld=65536), -11),
])
def test_bad_quantize(kw, status):
    assert quantize(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), -1), (dict(dt=2), -3), (dict(ld=129), -4), (dict(out=FAKE + 1), -5), (dict(dt=1, out=FAKE + 2), -5),
    (dict(a=fp8(block=128)), -2), (dict(w=fp8(rows=130)), -2), (dict(w=fp8(rows=130, block=128, cols=256)), -2),
    (dict(w=fp8(rows=0, block=128)), -2), (dict(ld=1 << 31), -11), (dict(a=fp8(rows=(1 << 31) - 1), ld=1 << 30), -11),
    (dict(w=fp8(rows=(1 << 31) - 1, block=128), ld=(1 << 31) - 1), -11),
    (dict(ws=None), -8), (dict(wsb=1000), -8), (dict(ws=FAKE + 8), -5),
    (dict(a=fp8(rows=0, codes=None, scales=None), out=None, ws=None), 0),
])
def test_bad_product(kw, status):
    assert gemm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(dt=3), -3), (dict(odt=3), -3), (dict(rows=-1), -2), (dict(rows=1 << 31), -11),
    (dict(ld=256), -4), (dict(ldo=129), -4), (dict(x=FAKE + 8), -5), (dict(ws=FAKE + 8), -5), (dict(ws=None), -8), (dict(wsb=100), -8),
    (dict(w=fp8(rows=130, block=1)), -2), (dict(w=fp8(rows=130, block=128, codes=None)), -1), (dict(rows=0, x=None, out=None, ws=None), 0),
])
def test_bad_linear(kw, status):
    assert linear(**kw) == status


def test_linear_workspace():
    f = nv.nvfp4_fp8_linear_workspace_bytes
    assert f(5, 272) >= 5 * 272 + 5 * 3 * 4 and f(0, 272) > 0
    assert f(-1, 272) == 0 and f(5, 271) == 0 and f(5, 0) == 0 and f(1 << 31, 272) == 0 and f(1 << 30, 1 << 20) == 0 and f(BIG, BIG) == 0
    assert linear(wsb=f(5, 272) - 1) == -8
    f = nv.nvfp4_fp8_gemm_workspace_bytes
    sizes = [f(n) for n in (0, 1, 16, 17, 64, 128, 129, 5000, (1 << 31) - 1)]
    assert sizes == sorted(sizes) and 0 < sizes[0] and sizes[-1] < 59e6 and f(-1) == 0 and f(1 << 31) == 0
    assert gemm(wsb=f(5) - 1) == -8
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_linear_workspace(5, 100, "cpu")


# -------------------------------------------------------- norm and rotation

def rows_of(**kw):
    a = dict(x=FAKE, ld=512, head=128, out=FAKE, ldo=512, heado=128, w=FAKE, heads=4)
    a.update(kw)
    return pack(nv._HEAD_ROWS, a["x"], a["ld"], a["head"], a["out"], a["ldo"], a["heado"], a["w"], a["heads"])


def turn(**kw):
    a = dict(pos=FAKE, ld=10, freq=FAKE, axis=FAKE, axes=3, dim=64, inter=0)
    a.update(kw)
    return pack(nv._ROPE, a["pos"], a["ld"], a["freq"], a["axis"], a["axes"], a["dim"], a["inter"])


def rope(q=None, k=None, dt=0, tokens=10, dim=128, eps=1e-6, offset=0.0, r=None, none=False):
    q = None if none else q or rows_of()
    return nv.load().nvfp4_qk_norm_rope(q, k, dt, tokens, dim, eps, offset, r, None)


@pytest.mark.parametrize("kw,status", [
    (dict(none=True), -1), (dict(dt=5), -3), (dict(dim=96), -2), (dict(tokens=-1), -2), (dict(tokens=1 << 24), -11),
    (dict(eps=0.0), -12), (dict(eps=-1.0), -12), (dict(eps=1e-39), -12), (dict(eps=float("nan")), -12), (dict(eps=float("inf")), -12),
    (dict(offset=float("nan")), -12),
    (dict(tokens=0, q=rows_of(x=None, out=None), r=turn(pos=None, freq=None)), 0),
])
def test_bad_norm(kw, status):
    assert rope(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(heads=0), -2), (dict(heads=4097), -2), (dict(ld=508), -4), (dict(ldo=504), -4),
    (dict(head=120), -4), (dict(heado=132), -4), (dict(head=1400, ld=120), -4), (dict(ld=128, head=9 * 128), -4), (dict(head=-128), -4), (dict(ld=-512), -4), (dict(ld=1 << 31), -11),
    (dict(heado=1 << 40), -11), (dict(x=FAKE + 8), -5), (dict(out=FAKE + 2), -5), (dict(w=FAKE + 2), -5),
])
def test_bad_heads(kw, status):
    assert rope(q=rows_of(**kw)) == status
    assert rope(k=rows_of(**kw)) == status and rope(none=True, k=rows_of(**kw)) == status


def test_in_place_only_with_the_same_strides():
    for kw in (dict(ldo=640), dict(ldo=640, heado=136), dict(ld=1280, heado=144, ldo=1280)):
        assert rope(q=rows_of(**kw)) == -4
    assert rope(tokens=1, q=rows_of(heado=136, ldo=640)) == -4
    # strides that are not used differ: the next check is reached
    assert rope(tokens=1, q=rows_of(ldo=640, w=FAKE + 2)) == -5 and rope(q=rows_of(heads=1, heado=1024, w=FAKE + 2)) == -5


def test_one_row_of_positions_for_all_axes():
    assert rope(r=turn(ld=0, freq=FAKE + 2)) == -5 and rope(r=turn(ld=1)) == -4 and rope(r=turn(ld=-1)) == -4


@pytest.mark.parametrize("kw,status", [
    (dict(pos=None), -1), (dict(freq=None), -1), (dict(dim=0), -2), (dict(dim=8), -2), (dict(dim=72), -2), (dict(dim=144), -2),
    (dict(axes=0), -2), (dict(axes=256), -2), (dict(ld=9), -4), (dict(ld=1 << 50), -11), (dict(pos=FAKE + 4), -5), (dict(freq=FAKE + 2), -5),
])
def test_bad_rotation(kw, status):
    assert rope(r=turn(**kw)) == status


# ------------------------------------------------------------ convolution

def conv(dt=0, none=False, **kw):
    a = dict(x=FAKE, ldx=64, y=2 * FAKE, ldy=64, w=FAKE, bias=FAKE, tokens=12, channels=64, batch=3, width=4, silu=1, starts=FAKE,
             state=FAKE, n=5, lds=192, slots=FAKE, fresh=FAKE)
    a.update(kw)
    c = pack(nv._CONV, a["x"], a["ldx"], a["y"], a["ldy"], a["w"], a["bias"], a["tokens"], a["channels"], a["batch"], a["width"],
                 a["silu"], a["starts"], a["state"], a["n"], a["lds"], a["slots"], a["fresh"])
    return nv.load().nvfp4_causal_conv(None if none else c, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(none=True), -1), (dict(dt=9), -3), (dict(x=None), -1), (dict(y=None), -1), (dict(w=None), -1), (dict(width=1), -2),
    (dict(width=5), -2), (dict(channels=0), -2), (dict(channels=60), -2), (dict(tokens=-1), -2), (dict(batch=-1), -2),
    (dict(n=0), -2), (dict(slots=None, batch=6), -2), (dict(starts=None, batch=5), -2), (dict(lds=191), -4), (dict(lds=196), -4),
    (dict(ldx=56), -4), (dict(ldy=68), -4), (dict(x=FAKE + 8), -5), (dict(y=FAKE + 4), -5), (dict(w=FAKE + 4), -5),
    (dict(bias=FAKE + 1), -5), (dict(starts=FAKE + 2), -5), (dict(state=FAKE + 8), -5), (dict(slots=FAKE + 1), -5),
    (dict(y=FAKE), -12), (dict(tokens=1 << 31), -11), (dict(batch=1 << 31), -11), (dict(channels=1 << 20, ldx=1 << 20, ldy=1 << 20), -11),
    (dict(tokens=1 << 30, channels=64), -11), (dict(n=1 << 31), -11), (dict(lds=1 << 31), -11), (dict(ldx=1 << 31), -11),
    (dict(ldy=1 << 50), -11), (dict(tokens=0, x=None), 0), (dict(batch=0, y=None), 0),
])
def test_bad_convolution(kw, status):
    assert conv(**kw) == status


# ------------------------------------------------------- next tokens

def step(dt=0, odt=0, batch=3, q_len=2, hk=2, hv=4, states=FAKE, n=5, lds=4 * 16384, slots=FAKE, o=FAKE, ldo=512, none=False, **kw):
    a = dict(q=FAKE, ldq=256, k=FAKE, ldk=256, v=FAKE, ldv=512, beta=FAKE, ldb=4, g=FAKE, ldg=4)
    a.update(kw)
    i = pack(nv._GDN_INPUTS, a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["beta"], a["ldb"], a["g"], a["ldg"])
    return nv.load().nvfp4_gdn_step(None if none else i, dt, batch, q_len, hk, hv, 1, states, n, lds, slots, None, o,
                                    odt, ldo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(none=True), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(beta=None), -1), (dict(g=None), -1),
    (dict(states=None), -1), (dict(o=None), -1), (dict(dt=4), -3), (dict(odt=4), -3), (dict(batch=-1), -2), (dict(q_len=0), -2),
    (dict(hk=0), -2), (dict(hk=3), -2), (dict(hv=4100, hk=1), -2), (dict(n=0), -2), (dict(slots=None, batch=6), -2),
    (dict(ldq=248), -4), (dict(ldk=260), -4), (dict(ldv=504), -4), (dict(ldb=3), -4), (dict(ldg=3), -4), (dict(ldo=508), -4),
    (dict(lds=4 * 16384 - 4), -4), (dict(lds=4 * 16384 + 2), -4), (dict(q=FAKE + 8), -5), (dict(beta=FAKE + 1), -5),
    (dict(states=FAKE + 8), -5), (dict(slots=FAKE + 2), -5), (dict(o=FAKE + 1), -5), (dict(batch=1 << 31), -11),
    (dict(batch=1 << 20, q_len=1 << 20), -11), (dict(n=1 << 31), -11), (dict(lds=1 << 31), -11), (dict(ldo=1 << 40), -11),
    (dict(ldg=1 << 40), -11), (dict(batch=0, states=None, q=None), 0),
])
def test_bad_step(kw, status):
    assert step(**kw) == status


# ------------------------------------------------------------ the binding

def refused(f, *args, **kw):
    with pytest.raises(nv.NVFP4Error):
        f(*args, **kw)


def test_the_binding_takes_gpu_tensors_only():
    x = torch.zeros(4, 128)
    q = nv.empty_fp8(4, 128, device="cpu")
    refused(nv.nvfp4_fp8_quantize, x, q)
    refused(nv.fp8_quantize, x, 64)
    refused(nv.fp8_quantize, x[0])
    refused(nv.nvfp4_fp8_gemm, q, nv.empty_fp8(128, 128, 128, "cpu"), x, x)
    refused(nv.fp8_linear, x[0], q)
    refused(nv.nvfp4_qk_norm_rope, None, None, None, None, 64)
    refused(nv.qk_norm_rope, x, x, 64)
    refused(nv.causal_conv, x, torch.zeros(128, 4))
    refused(nv.causal_conv, x[0], torch.zeros(128, 4))
    refused(nv.gdn_step, x, x, x, x, x, 1, 1, torch.zeros(4, 1, 128, 128))
    refused(nv.gdn_step, x, x, x, x, x, 1, 1, torch.zeros(4, 1, 128, 128), q_len=3)


@pytest.mark.parametrize("codes,scales", [
    (torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4, 1)), (torch.zeros(3, 128, dtype=torch.uint8), torch.zeros(4, 1)),
    (torch.zeros(4, 112, dtype=torch.uint8), torch.zeros(4, 1)), (torch.zeros(4, 256, dtype=torch.uint8)[:, ::2], torch.zeros(4, 1)),
    (torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1).double()), (torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 1)),
    (torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 0)), (torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4)),
])
def test_the_binding_checks_matrices(codes, scales):
    refused(nv.FP8Tensor(codes, scales, 4, 128).descriptor)

"""The boundary of the loss calls without a GPU: the library exports what their
header declares, and rejects invalid arguments on the host before any HIP call
(these calls never reach a kernel launch)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import vocab_sharded_embedding_amd as vpe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = 0x10000  # a non-null, 16-byte aligned address that is never dereferenced
F32, BF16, I32, I64 = vpe.VPE_F32, vpe.VPE_BF16, vpe.VPE_I32, vpe.VPE_I64
INF, NAN = float("inf"), float("nan")


def test_header_declares_what_the_library_exports():
    text = open(os.path.join(ROOT, "include", "vpe_loss.h")).read()
    declared = sorted(set(re.findall(r"^\s*vpe_status\s*(vpe_\w+)\s*\(", text, re.M)))
    assert declared == sorted(vpe.LOSS_SYMBOLS)
    lib = vpe.load_library()
    for name in vpe.LOSS_SYMBOLS:
        assert hasattr(lib, name) and hasattr(vpe, name) and name in vpe.__all__
    for name in ("VPE_MAX_LOSS_ROWS", "VPE_MAX_LOSS_DIM", "VPE_MAX_GRAD_TENSORS"):
        assert eval(re.search(rf"#define {name} (.+)", text).group(1)) == getattr(vpe, name)


def test_header_is_c():
    if shutil.which("gcc") is None:
        pytest.skip("no host compiler")
    src = '#include "vpe_loss.h"\nint main(void) { return VPE_OK; }\n'
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-x",
                        "c", "-I", os.path.join(ROOT, "include"), "-"], input=src, text=True,
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    assert r.returncode == 0, r.stdout


def _caller(name, defaults):
    fn = getattr(vpe.load_library(), name)

    def call(**kw):
        unknown = set(kw) - set(defaults)
        assert not unknown, unknown
        return fn(*{**defaults, **kw}.values())
    return call


BAD_SIZES = (dict(m=-1), dict(m=2 ** 21 + 1), dict(dim=0), dict(dim=2 ** 16 + 1), dict(rows=0),
             dict(rows=2 ** 31), dict(rows=2 ** 31 - 1, dim=2 ** 16), dict(bytes=-1))
BAD_SHARDS = (dict(start=-1), dict(start=1), dict(vocab=99), dict(start=2 ** 62, vocab=100))


def test_xent_validation():
    call = _caller("vpe_lmhead_xent", dict(
        x=FAKE, m=4, dim=64, w=FAKE, rows=100, dt=BF16, start=0, vocab=100, t=FAKE, itype=I64,
        lse=FAKE, z=FAKE, ws=FAKE, bytes=1 << 30, stream=None))
    for bad in (dict(dt=5), dict(itype=3)):
        assert call(**bad) == vpe.VPE_ERR_DTYPE, bad
    for bad in (*BAD_SIZES, dict(vocab=0)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in BAD_SHARDS:
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    for name in ("x", "w", "t", "lse", "z", "ws"):
        assert call(**{name: None}) == vpe.VPE_ERR_NULL, name
    for bad in (dict(x=FAKE + 1), dict(w=FAKE + 1), dict(dt=F32, x=FAKE + 2), dict(t=FAKE + 4),
                dict(itype=I32, t=FAKE + 2), dict(lse=FAKE + 2), dict(z=FAKE + 1),
                dict(ws=FAKE + 8)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    need = vpe.vpe_lmhead_xent_workspace(4, 64, 100, BF16)
    assert call(bytes=need - 1) == vpe.VPE_ERR_WORKSPACE
    assert call(m=0, x=None, w=None, t=None, lse=None, z=None, ws=None) == vpe.VPE_OK


def test_xent_loss_validation():
    fn = vpe.load_library().vpe_xent_loss
    arr = (ctypes.c_void_p * 2)(FAKE, FAKE)

    def call(a=arr, b=arr, n=2, m=4, vocab=10, t=FAKE, itype=I32, loss=FAKE, lse=FAKE):
        return fn(a, b, n, m, vocab, t, itype, loss, lse, None)
    assert call(itype=9) == vpe.VPE_ERR_DTYPE
    for bad in (dict(n=0), dict(n=65), dict(m=-1), dict(m=2 ** 21 + 1), dict(vocab=0)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in (dict(a=None), dict(b=None), dict(t=None), dict(loss=None), dict(lse=None),
                dict(a=(ctypes.c_void_p * 2)(FAKE, None))):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(b=(ctypes.c_void_p * 2)(FAKE + 2, FAKE)), dict(t=FAKE + 2),
                dict(loss=FAKE + 1), dict(lse=FAKE + 2)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    assert call(m=0, t=None) == vpe.VPE_OK


def test_xent_grad_validation():
    call = _caller("vpe_lmhead_xent_grad", dict(
        x=FAKE, m=4, dim=64, w=FAKE, rows=100, dt=BF16, start=0, vocab=100, t=FAKE, itype=I64,
        lse=FAKE, g=FAKE, gx=FAKE, gxt=F32, gw=FAKE, gwt=BF16, acc=0, ws=FAKE, bytes=1 << 30,
        stream=None))
    for bad in (dict(dt=5), dict(itype=3), dict(gxt=2), dict(gwt=-1)):
        assert call(**bad) == vpe.VPE_ERR_DTYPE, bad
    for bad in (*BAD_SIZES, dict(vocab=0)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in BAD_SHARDS:
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    for bad in (dict(x=None), dict(w=None), dict(t=None), dict(lse=None), dict(g=None),
                dict(gx=None, gw=None), dict(ws=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(x=FAKE + 1), dict(t=FAKE + 4), dict(lse=FAKE + 2), dict(g=FAKE + 1),
                dict(gx=FAKE + 2), dict(gw=FAKE + 1), dict(ws=FAKE + 8)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    need = vpe.vpe_lmhead_xent_grad_workspace(4, 64, 100, BF16)
    assert call(bytes=need - 1) == vpe.VPE_ERR_WORKSPACE
    assert call(m=0, acc=1, x=None, t=None, lse=None, g=None, ws=None) == vpe.VPE_OK
    assert call(m=0, gw=None, ws=None) == vpe.VPE_OK


def test_head_grad_validation():
    call = _caller("vpe_lmhead_grad", dict(
        d=FAKE, ld=100, col=0, x=FAKE, m=4, dim=64, w=FAKE, rows=100, dt=F32, gx=FAKE, gxt=F32,
        gw=FAKE, gwt=BF16, acc=0, ws=FAKE, bytes=1 << 30, stream=None))
    for bad in (dict(dt=5), dict(gxt=2), dict(gwt=-1)):
        assert call(**bad) == vpe.VPE_ERR_DTYPE, bad
    for bad in (*[b for b in BAD_SIZES if "rows" not in b], dict(rows=0), dict(ld=2 ** 39),
                dict(rows=2 ** 31, ld=2 ** 32)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in (dict(col=-1), dict(col=1), dict(ld=99), dict(ld=0), dict(col=2 ** 62)):
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    for bad in (dict(d=None), dict(x=None), dict(w=None), dict(gx=None, gw=None), dict(ws=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(d=FAKE + 2), dict(x=FAKE + 1), dict(gx=FAKE + 2), dict(gw=FAKE + 1),
                dict(ws=FAKE + 8)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    need = vpe.vpe_lmhead_grad_workspace(4, 64, 100, F32)
    assert call(bytes=need - 1) == vpe.VPE_ERR_WORKSPACE
    assert call(m=0, acc=1, d=None, x=None, ws=None) == vpe.VPE_OK


@pytest.mark.parametrize("fn", [vpe.vpe_lmhead_xent_workspace, vpe.vpe_lmhead_xent_grad_workspace,
                                vpe.vpe_lmhead_grad_workspace])
def test_workspaces_serve_fewer_rows(fn):
    for dt in (F32, BF16):
        for dim, rows in ((1, 1), (64, 4096), (1024, 75968), (999, 50257), (4096, 37984)):
            last = 0
            for m in [*range(0, 300), *range(300, 20000, 701), 10 ** 5, 2 ** 21]:
                need = fn(m, dim, rows, dt)
                assert need >= last and need % 16 == 0, (m, dim, rows)
                last = need
    for bad in ((-1, 8, 8, F32), (1, 0, 8, F32), (1, 8, 0, F32), (1, 8, 2 ** 31, F32),
                (2 ** 22, 8, 8, BF16), (1, 2 ** 17, 8, BF16), (1, 8, 8, 7)):
        with pytest.raises(vpe.VpeError):
            fn(*bad)


def test_clip_validation():
    lib = vpe.load_library()
    one = (ctypes.c_void_p * 1)(FAKE)
    count, f32 = (ctypes.c_int64 * 1)(10), (ctypes.c_int32 * 1)(F32)

    def sumsq(t=one, c=count, d=f32, n=1, s=FAKE, ws=FAKE, b=8):
        return lib.vpe_grad_sumsq(t, c, d, n, s, ws, b, None)

    def clip(t=one, c=count, d=f32, n=1, out=one, s=one, parts=1, most=1.0, norm=FAKE):
        return lib.vpe_grad_clip(t, c, d, n, out, s, parts, most, norm, None)
    for call in (sumsq, clip):
        for bad in (dict(n=-1), dict(n=2 ** 16 + 1), dict(c=(ctypes.c_int64 * 1)(-1)),
                    dict(c=(ctypes.c_int64 * 1)(2 ** 39 + 1))):
            assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
        assert call(d=(ctypes.c_int32 * 1)(4)) == vpe.VPE_ERR_DTYPE
        for bad in (dict(t=None), dict(c=None), dict(d=None), dict(s=None),
                    dict(t=(ctypes.c_void_p * 1)(None))):
            assert call(**bad) == vpe.VPE_ERR_NULL, bad
        assert call(t=(ctypes.c_void_p * 1)(FAKE + 2)) == vpe.VPE_ERR_ALIGN
    assert sumsq(b=7) == vpe.VPE_ERR_WORKSPACE and sumsq(b=-1) == vpe.VPE_ERR_SHAPE
    assert sumsq(ws=None) == vpe.VPE_ERR_NULL
    assert sumsq(s=FAKE + 4) == vpe.VPE_ERR_ALIGN and sumsq(ws=FAKE + 4) == vpe.VPE_ERR_ALIGN
    for bad in (dict(parts=0), dict(parts=65)):
        assert clip(**bad) == vpe.VPE_ERR_SHAPE
    for bad in (-1.0, INF, -INF, NAN):
        assert clip(most=bad) == vpe.VPE_ERR_RANGE
    for bad in (dict(out=None), dict(norm=None), dict(s=(ctypes.c_void_p * 1)(None)),
                dict(out=(ctypes.c_void_p * 1)(None))):
        assert clip(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(out=(ctypes.c_void_p * 1)(FAKE + 1)), dict(norm=FAKE + 2),
                dict(s=(ctypes.c_void_p * 1)(FAKE + 4))):
        assert clip(**bad) == vpe.VPE_ERR_ALIGN, bad
    two = (ctypes.c_int64 * 2)(2 ** 38, 2 ** 38 + 1)
    b = ctypes.c_int64()
    assert lib.vpe_grad_sumsq_workspace(two, 2, ctypes.byref(b)) == vpe.VPE_ERR_SHAPE
    assert lib.vpe_grad_sumsq_workspace(count, 1, None) == vpe.VPE_ERR_NULL
    assert vpe.vpe_grad_sumsq_workspace([0, 0]) == 8 and vpe.vpe_grad_sumsq_workspace([1, 1]) == 16

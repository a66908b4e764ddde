"""The boundary of the training and beam-search calls without a GPU: the library
exports what their headers declare, and rejects invalid arguments on the host
before any HIP call (these calls never reach a kernel launch)."""
import ctypes
import os
import re

import pytest

import vocab_sharded_embedding_amd as vpe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = 0x10000  # a non-null, 16-byte aligned address that is never dereferenced
FAR = 0x7000000000
F32, BF16, I32, I64 = vpe.VPE_F32, vpe.VPE_BF16, vpe.VPE_I32, vpe.VPE_I64
INF, NAN = float("inf"), float("nan")


def _declared(header):
    text = open(os.path.join(ROOT, "include", header)).read()
    return sorted(set(re.findall(r"^\s*vpe_status\s*(vpe_\w+)\s*\(", text, re.M)))


def test_headers_declare_what_the_library_exports():
    lib = vpe.load_library()
    assert _declared("vpe_train.h") == sorted(vpe.TRAIN_SYMBOLS)
    assert _declared("vpe_beam.h") == sorted(vpe.BEAM_SYMBOLS)
    for name in vpe.TRAIN_SYMBOLS + vpe.BEAM_SYMBOLS:
        assert hasattr(lib, name) and hasattr(vpe, name) and name in vpe.__all__


def test_header_constants_match():
    text = open(os.path.join(ROOT, "include", "vpe_train.h")).read()
    text += open(os.path.join(ROOT, "include", "vpe_beam.h")).read()
    for name in ("VPE_MAX_TEACHER_ENTRIES", "VPE_MAX_DISTILL_ROWS", "VPE_MAX_BEAMS",
                 "VPE_MAX_BEAM_PICKS"):
        value = re.search(rf"#define {name} (.+)", text).group(1)
        assert eval(value) == getattr(vpe, name)


def test_headers_are_c():
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no host compiler")
    src = '#include "vpe_train.h"\n#include "vpe_beam.h"\nint main(void) { return VPE_OK; }\n'
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


def test_embed_scaled_validation():
    call = _caller("vpe_embed_scaled", dict(ids=FAKE, itype=I32, n=10, w=FAKE, dt=BF16, rows=100,
                                            dim=64, start=0, scale=2.0, out=FAKE, stream=None))
    assert call(dt=9) == vpe.VPE_ERR_DTYPE
    assert call(itype=5) == vpe.VPE_ERR_DTYPE
    for bad in (dict(n=-1), dict(dim=0), dict(rows=0), dict(n=2 ** 40), dict(rows=2 ** 38)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in (dict(start=-1), dict(start=2 ** 63 - 100), dict(scale=INF), dict(scale=NAN)):
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    for bad in (dict(ids=None), dict(w=None), dict(out=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(ids=FAKE + 2), dict(itype=I64, ids=FAKE + 4), dict(w=FAKE + 1),
                dict(out=FAKE + 1), dict(dt=F32, out=FAKE + 2)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    assert call(n=0, ids=None, w=None, out=None) == vpe.VPE_OK


def test_embed_grad_validation():
    call = _caller("vpe_embed_grad", dict(
        ids=FAKE, itype=I64, n=10, dy=FAKE, dt=BF16, dim=64, start=0, rows=100, scale=1.0, dw=FAKE,
        gdt=F32, acc=0, ws=FAKE, bytes=1 << 30, stream=None))
    for bad in (dict(dt=2), dict(gdt=-1), dict(itype=2)):
        assert call(**bad) == vpe.VPE_ERR_DTYPE, bad
    for bad in (dict(n=-1), dict(n=2 ** 31), dict(dim=0), dict(rows=0), dict(rows=2 ** 31),
                dict(dim=2 ** 20 + 1), dict(rows=2 ** 30, dim=2 ** 10), dict(bytes=-1)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in (dict(start=-1), dict(start=2 ** 63 - 100), dict(scale=-INF), dict(scale=NAN)):
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    for bad in (dict(ids=None), dict(dy=None), dict(dw=None), dict(ws=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(ids=FAKE + 4), dict(dy=FAKE + 1), dict(dw=FAKE + 2), dict(ws=FAKE + 8)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    need = vpe.vpe_embed_grad_workspace(10, 100, 64)
    assert call(bytes=need - 1) == vpe.VPE_ERR_WORKSPACE
    assert call(n=0, acc=1, ids=None, dy=None, dw=None, ws=None) == vpe.VPE_OK
    assert call(n=0, dw=None) == vpe.VPE_ERR_NULL


def test_embed_grad_workspace():
    lib = vpe.load_library()
    b = ctypes.c_int64()
    f = lib.vpe_embed_grad_workspace
    assert f(10, 10, 10, None) == vpe.VPE_ERR_NULL
    for bad in ((-1, 10, 10), (2 ** 31, 10, 10), (10, 0, 10), (10, 2 ** 31, 10), (10, 10, 0),
                (10, 10, 2 ** 20 + 1), (2 ** 30, 10, 2 ** 10)):
        assert f(*bad, ctypes.byref(b)) == vpe.VPE_ERR_SHAPE, bad
    last = 0
    for n in [*range(0, 70), *range(4000, 140000, 997), 10 ** 6, 2 * 10 ** 8]:
        need = vpe.vpe_embed_grad_workspace(n, 1000, 64)
        assert need >= last and need % 16 == 0
        last = need


DISTILL = dict(z=FAKE, ld=1000, col=0, m=4, rows=1000, dt=BF16, start=0, vocab=1000, temp=1.0,
               ids=FAKE, itype=I64, t=FAKE, tdt=F32, k=8, tlse=None)


def _bad_distill(call, shard=True):
    for bad in (dict(itype=7), dict(tdt=7)) + ((dict(dt=7),) if shard else ()):
        assert call(**bad) == vpe.VPE_ERR_DTYPE, bad
    for bad in (dict(m=-1), dict(m=2 ** 21 + 1), dict(k=0), dict(k=1025), dict(vocab=0)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for temp in (0.0, -1.0, INF, NAN, 1e-45, 3e38, 1e-39):
        assert call(temp=temp) == vpe.VPE_ERR_RANGE, temp
    for bad in (dict(ids=None), dict(t=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(ids=FAKE + 4), dict(t=FAKE + 2), dict(tlse=FAKE + 1)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    if shard:
        for bad in (dict(rows=0), dict(rows=2 ** 31), dict(ld=2 ** 39)):
            assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
        for bad in (dict(start=-1), dict(start=1), dict(vocab=999), dict(col=1), dict(col=-1),
                    dict(ld=999), dict(start=2 ** 62, vocab=100)):
            assert call(**bad) == vpe.VPE_ERR_RANGE, bad
        assert call(z=None) == vpe.VPE_ERR_NULL
        assert call(z=FAKE + 1) == vpe.VPE_ERR_ALIGN


def test_distill_shard_validation():
    call = _caller("vpe_distill_shard", dict(**DISTILL, lse=FAKE, dot=FAKE, ws=None, bytes=0,
                                             stream=None))
    _bad_distill(call)
    assert call(dot=None) == vpe.VPE_ERR_NULL
    for bad in (dict(lse=FAKE + 2), dict(dot=FAKE + 1), dict(ws=FAKE + 4)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    assert call(bytes=-1) == vpe.VPE_ERR_SHAPE
    wide = dict(ld=151936, rows=151936, vocab=151936, m=1)
    need = vpe.vpe_distill_workspace(1, 151936)
    assert need > 0
    assert call(**wide) == vpe.VPE_ERR_NULL
    assert call(**wide, ws=FAKE, bytes=need - 1) == vpe.VPE_ERR_WORKSPACE
    assert call(m=0, z=None, ids=None, t=None, lse=None, dot=None) == vpe.VPE_OK


def test_distill_workspace():
    lib = vpe.load_library()
    b = ctypes.c_int64()
    f = lib.vpe_distill_workspace
    assert f(1, 1, None) == vpe.VPE_ERR_NULL
    for bad in ((-1, 5), (2 ** 21 + 1, 5), (5, 0), (5, 2 ** 31)):
        assert f(*bad, ctypes.byref(b)) == vpe.VPE_ERR_SHAPE, bad
    assert vpe.vpe_distill_workspace(0, 10 ** 6) == 0
    assert vpe.vpe_distill_workspace(2 ** 21, 2 ** 31 - 1) >= 0
    sizes = [vpe.vpe_distill_workspace(m, 151936) for m in range(0, 600)]
    assert sizes == sorted(sizes) and sizes[1] > 0


def test_distill_loss_validation():
    arr = (ctypes.c_void_p * 65)(*([FAKE] * 65))
    base = {k: v for k, v in DISTILL.items() if k in ("m", "vocab", "temp", "ids", "itype", "t",
                                                      "tdt", "k", "tlse")}
    call = _caller("vpe_distill_loss", dict(lse_in=arr, dot_in=arr, n=2, **base, loss=FAKE,
                                            lse=FAKE, stream=None))
    _bad_distill(call, shard=False)
    for n in (0, 65, -1):
        assert call(n=n) == vpe.VPE_ERR_SHAPE
    for bad in (dict(lse_in=None), dict(dot_in=None), dict(loss=None), dict(lse=None),
                dict(lse_in=(ctypes.c_void_p * 2)(FAKE, None)),
                dict(dot_in=(ctypes.c_void_p * 2)(None, FAKE))):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(loss=FAKE + 2), dict(lse=FAKE + 1),
                dict(dot_in=(ctypes.c_void_p * 2)(FAKE, FAKE + 2))):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    assert call(m=0, lse_in=None, dot_in=None) == vpe.VPE_OK


def test_distill_grad_validation():
    call = _caller("vpe_distill_grad", dict(**DISTILL, lse=FAKE, go=FAKE, dz=FAR, ld_grad=1000,
                                            gcol=0, stream=None))
    _bad_distill(call)
    for bad in (dict(lse=None), dict(go=None), dict(dz=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(lse=FAKE + 2), dict(go=FAKE + 1), dict(dz=FAR + 1)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    for bad in (dict(ld_grad=999), dict(gcol=1), dict(gcol=-1),
                dict(dz=FAKE, ld_grad=1001), dict(dz=FAKE, ld_grad=1001, gcol=1),
                dict(dz=FAKE + 2), dict(dz=FAKE - 2), dict(dz=FAKE + 2000),
                dict(dz=FAKE + 2 * 3999), dict(dz=FAKE, ld=3000, ld_grad=3000, gcol=999),
                dict(dz=FAKE, ld=3000, ld_grad=3000, col=2000, gcol=1001),
                dict(dz=FAKE - 6000, ld=3000, ld_grad=3000, gcol=500)):
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    assert call(m=0, z=None, dz=None) == vpe.VPE_OK


def test_beam_select_validation():
    call = _caller("vpe_beam_select", dict(
        z=FAKE, ld=1000, col=0, dt=BF16, n=2, beams=4, rows=1000, start=0, vocab=1000, lse=FAKE,
        scores=FAKE, picks=8, keys=FAKE, ws=FAKE, bytes=1 << 20, stream=None))
    assert call(dt=4) == vpe.VPE_ERR_DTYPE
    for bad in (dict(n=-1), dict(n=2 ** 20), dict(beams=0), dict(beams=65), dict(picks=0),
                dict(picks=65), dict(rows=0), dict(rows=2 ** 31), dict(vocab=0), dict(bytes=-1), dict(ld=2 ** 38)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in (dict(start=-1), dict(start=1), dict(vocab=999), dict(vocab=2 ** 30),
                dict(vocab=2 ** 63 - 1), dict(ld=999), dict(col=1), dict(col=-1)):
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    for bad in (dict(z=None), dict(lse=None), dict(scores=None), dict(keys=None), dict(ws=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(z=FAKE + 1), dict(lse=FAKE + 2), dict(scores=FAKE + 1), dict(keys=FAKE + 4),
                dict(ws=FAKE + 4)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    need = vpe.vpe_beam_select_workspace(2, 4, 1000, 8)
    assert call(bytes=need - 1) == vpe.VPE_ERR_WORKSPACE
    assert call(n=0, z=None, lse=None, scores=None, keys=None, ws=None) == vpe.VPE_OK
    b = ctypes.c_int64()
    f = vpe.load_library().vpe_beam_select_workspace
    assert f(1, 1, 1, 1, None) == vpe.VPE_ERR_NULL
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0),
                (1, 1, 1, 65), (2 ** 20, 4, 1, 1), (1, 1, 2 ** 31, 1)):
        assert f(*bad, ctypes.byref(b)) == vpe.VPE_ERR_SHAPE, bad


def test_beam_merge_validation():
    arr = (ctypes.c_void_p * 65)(*([FAKE] * 65))
    call = _caller("vpe_beam_merge", dict(keys=arr, parts=2, n=3, picks=8, vocab=100, score=FAKE,
                                          parent=FAKE, token=FAKE, stream=None))
    for bad in (dict(parts=0), dict(parts=65), dict(n=-1), dict(n=2 ** 21 + 1), dict(picks=0),
                dict(picks=65), dict(vocab=0), dict(vocab=2 ** 32)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in (dict(keys=None), dict(keys=(ctypes.c_void_p * 2)(FAKE, None)), dict(score=None),
                dict(parent=None), dict(token=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    for bad in (dict(keys=(ctypes.c_void_p * 2)(FAKE, FAKE + 4)), dict(score=FAKE + 2),
                dict(parent=FAKE + 4), dict(token=FAKE + 4)):
        assert call(**bad) == vpe.VPE_ERR_ALIGN, bad
    assert call(n=0, keys=None, score=None, parent=None, token=None) == vpe.VPE_OK


def test_beam_reorder_validation():
    call = _caller("vpe_beam_reorder", dict(src=FAKE, outer=2, n=3, b_in=4, bytes=100, parent=FAKE,
                                            ld=4, b_out=4, dst=FAR, stream=None))
    for bad in (dict(outer=-1), dict(n=-1), dict(b_in=0), dict(b_out=0), dict(bytes=0),
                dict(bytes=2 ** 40), dict(n=2 ** 40), dict(outer=2 ** 40), dict(outer=2 ** 30),
                dict(ld=2 ** 40)):
        assert call(**bad) == vpe.VPE_ERR_SHAPE, bad
    for bad in (dict(ld=3), dict(dst=FAKE), dict(dst=FAKE + 2399), dict(dst=FAKE - 2399)):
        assert call(**bad) == vpe.VPE_ERR_RANGE, bad
    for bad in (dict(src=None), dict(parent=None), dict(dst=None)):
        assert call(**bad) == vpe.VPE_ERR_NULL, bad
    assert call(parent=FAKE + 4) == vpe.VPE_ERR_ALIGN
    assert call(outer=0, src=None, parent=None, dst=None) == vpe.VPE_OK
    assert call(n=0, src=None, parent=None, dst=None) == vpe.VPE_OK


def test_binding_rejects_host_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    ids, w = torch.zeros(4, dtype=torch.int64), torch.zeros(8, 16)
    row, t = torch.zeros(4), torch.zeros(4, 3)
    for call in (lambda: vpe.vpe_embed_scaled(ids, w, 0, 1.0),
                 lambda: vpe.vpe_embed_grad(ids, torch.zeros(4, 16), 0, 8),
                 lambda: vpe.vpe_distill_shard(torch.zeros(4, 8), t.long(), t, 0, 8),
                 lambda: vpe.vpe_distill_loss([row], [row], t.long(), t, 8),
                 lambda: vpe.vpe_distill_grad(torch.zeros(4, 8), row, row, t.long(), t, 0, 8),
                 lambda: vpe.vpe_beam_select(torch.zeros(4, 8), row, row, 2, 4, 0, 8),
                 lambda: vpe.vpe_beam_merge([t.long()], 8),
                 lambda: vpe.vpe_beam_reorder(w, t.long(), 2),
                 lambda: vpe.vpe_beam_merge([], 8)):
        with pytest.raises(ValueError):
            call()

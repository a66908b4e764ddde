"""Calls of the training and beam-search boundary that documentation refuses,
each by itself, without a GPU (the calls never reach a kernel launch)."""
import pytest

torch = pytest.importorskip("torch")

import vocab_sharded_embedding_amd as vpe  # noqa: E402

F32, I64 = vpe.VPE_F32, vpe.VPE_I64


def test_temperatures_whose_power_of_two_factor_is_infinite():
    # exponentials are powers of two of z log2(e) / T: the factor has to be finite
    # in fp32, so T past log2(e) / 2^128 = 4.24e-39, and not only 1 / T (2.94e-39).
    # No rows: what is not refused is a no-op.
    lib = vpe.load_library()
    calls = (
        lambda t: lib.vpe_distill_shard(None, 8, 0, 0, 8, F32, 0, 8, t, None, I64, None, F32, 1,
                                        None, None, None, None, 0, None),
        lambda t: lib.vpe_distill_loss(None, None, 1, 0, 8, t, None, I64, None, F32, 1, None, None,
                                       None, None),
        lambda t: lib.vpe_distill_grad(None, 8, 0, 0, 8, F32, 0, 8, t, None, I64, None, F32, 1,
                                       None, None, None, None, 8, 0, None),
    )
    for call in calls:
        for temp in (3e-39, 4e-39, 4.23e-39):
            assert call(temp) == vpe.VPE_ERR_RANGE, temp
        for temp in (4.3e-39, 1e-38, 1.0, 2.0 ** 100):
            assert call(temp) == vpe.VPE_OK, temp


def test_reordered_states_over_their_parents():
    # dst [2, 3 * 4, 100] bytes = 2400; parents: 3 rows of 4 int64, 8 apart
    src, dst, n_parents = 0x10000, 0x7000000000, 2 * 8 + 4
    call = vpe.load_library().vpe_beam_reorder
    for parent in (dst, dst + 2392, dst - 8 * n_parents + 8, dst + 96):
        assert call(src, 2, 3, 4, 100, parent, 8, 4, dst, None) == vpe.VPE_ERR_RANGE, parent


def test_lookup_gradient_over_its_own_inputs():
    # refused before the tensors' device is looked at, so host tensors show it
    n, rows, dim = 12, 6, 8
    need = vpe.vpe_embed_grad_workspace(n, rows, dim)
    pool = torch.zeros(need + 4096, dtype=torch.uint8)

    def at(byte, shape, dtype):
        size = torch.empty(shape, dtype=dtype).nbytes
        return pool[byte:byte + size].view(dtype).view(shape)

    def call(ids=torch.zeros(n, dtype=torch.int64), dy=torch.zeros(n, dim), dw=None, ws=None):
        vpe.vpe_embed_grad(ids, dy, 0, rows, grad_weight=dw, workspace=ws)

    dw = at(16, (rows, dim), torch.float32)  # bytes 16 to 208
    for over in (dict(dy=at(200, (n, dim), torch.float32)), dict(ids=at(192, (n,), torch.int64)),
                 dict(ws=at(0, (need,), torch.uint8)), dict(ws=at(192, (need,), torch.uint8)),
                 dict(dw=at(16, (rows, dim), torch.bfloat16), dy=at(16, (n, dim), torch.float32)),
                 dict(dw=None, ws=at(0, (need,), torch.uint8), dy=at(64, (n, dim), torch.float32)),
                 dict(dw=None, ws=at(0, (need,), torch.uint8),
                      ids=at(need // 8 * 8 - 8, (n,), torch.int64))):
        with pytest.raises(ValueError, match="overlap"):
            call(**{"dw": dw, **over})
    # neighbours, and an empty view inside, are no overlap: the device is what is wrong
    for beside in (dict(dy=at(208, (n, dim), torch.float32)), dict(ws=at(208, (need,), torch.uint8)),
                   dict(ids=pool[32:32].view(torch.int64), dy=pool[64:64].view(torch.float32)
                        .view(0, dim))):
        with pytest.raises(ValueError, match="device|HIP|cuda"):
            call(**{"dw": dw, **beside})


def test_scaled_lookup_over_its_own_inputs():
    rows, dim, n = 10, 8, 4
    pool = torch.zeros(4096)
    weight, out = pool[:rows * dim].view(rows, dim), pool[72:72 + n * dim].view(n, dim)
    ids = pool[100:100 + n].view(torch.int32)  # inside out
    for bad in ((torch.zeros(n, dtype=torch.int32), weight), (ids, torch.zeros(rows, dim))):
        with pytest.raises(ValueError, match="overlap"):
            vpe.vpe_embed_scaled(*bad, 0, 2.0, out=out)
    with pytest.raises(ValueError, match="HIP"):  # neighbours: the device is what is wrong
        vpe.vpe_embed_scaled(pool[112:116].view(torch.int32), weight, 0, 2.0,
                             out=pool[80:80 + n * dim].view(n, dim))

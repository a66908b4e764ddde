"""Which tiles the loss calls take, by the rules that their launchers use (plain C++):
the shapes of the GPU tests reach the kernels that they are there for."""
import os
import shutil
import subprocess
import tempfile

import pytest

from _loss_large import BACKWARD, COPIED, LIVE, ONE_PIECE, PIECES, SMALLER

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "vocab_sharded_embedding_amd", "csrc", "vpe_loss_launch.h")


def _run(body):
    """What a C++ program with `body` as its main, over the launchers' header, prints."""
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    src = f'#include <stdio.h>\n#include "{HEADER}"\nusing namespace vpe;\nint main() {{\n{body}\n}}\n'
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "rules")
        r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-x", "c++", "-", "-o", exe],
                           input=src, text=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        assert r.returncode == 0, r.stdout
        return subprocess.run([exe], text=True, check=True, stdout=subprocess.PIPE).stdout.split()


def _each(shapes, expression):
    body = "".join(f'{{ const int64_t m = {m}, rows = {rows}, dim = {dim}; (void)m, (void)rows, '
                   f'(void)dim; printf("%lld\\n", (long long)({expression})); }}\n'
                   for m, rows, dim in shapes)
    return [int(v) for v in _run(body)]


def test_large_products_are_reached():
    large = PIECES + ONE_PIECE + COPIED + BACKWARD
    assert _each(large, "large_products(m, dim)") == [1] * len(large)
    assert _each(SMALLER, "large_products(m, dim)") == [0] * len(SMALLER)


def test_large_logits_and_pieces_are_reached():
    def pieces(shapes):
        return _each(shapes, "(rows + grad_piece(loss_layout(kLossGrad, m, dim, rows, 1), m, rows, "
                             "1, dim % 8 != 0) - 1) / grad_piece(loss_layout(kLossGrad, m, dim, "
                             "rows, 1), m, rows, 1, dim % 8 != 0)")

    def large(shapes):
        return _each(shapes, "large_logits(m, loss_min(rows, grad_piece(loss_layout(kLossGrad, m, "
                             "dim, rows, 1), m, rows, 1, dim % 8 != 0)))")

    assert all(n >= 3 for n in pieces(PIECES))
    assert all(p[1] % 64 for p in PIECES)  # a ragged last one
    assert pieces(ONE_PIECE) == [1] * len(ONE_PIECE)
    assert pieces(COPIED)[0] < pieces(COPIED)[1]
    assert large(PIECES) == [1] * len(PIECES)
    # few rows: logits in 128 x 128 tiles before products in 256 x 256
    assert large(ONE_PIECE) == [0, 0, 1, 1]
    # the steady loop of a sum has more than four steps of 64
    assert max(d for _, _, d in PIECES) > 512 and max(d for _, _, d in ONE_PIECE) > 512
    assert max(LIVE) == PIECES[0][0]


def test_the_join_of_sums_fits_a_grid():
    """Fewer than 2^32 work-items at every accepted size."""
    sizes = [(m, 1, dim) for m in (1, 4096, 1 << 20, 1 << 21) for dim in (1, 4100, 16384, 1 << 16)]
    groups = _each(sizes, "finish_groups(m, dim)")
    assert all(0 < n and n * 256 < 1 << 32 for n in groups)

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
    src = (f'#include <stdio.h>\n#include "{HEADER}"\nusing namespace vpe;\n'
           f'int main() {{\n{body}\n}}\n')
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
    """Fewer than 2^32 work-items, and 2^16 workgroups, along either dimension at every
    accepted size."""
    sizes = [(m, 1, dim) for m in (1, 4096, 1 << 20, 1 << 21) for dim in (1, 4100, 16384, 1 << 16)]
    wide = _each(sizes, "loss_min(kFinishWidth, finish_groups(m, dim))")
    rows = _each(sizes, "(finish_groups(m, dim) + kFinishWidth - 1) / kFinishWidth")
    for (m, _, dim), x, y in zip(sizes, wide, rows):
        assert 0 < x * 256 < 1 << 32 and 0 < y < 1 << 16
        assert x * y * 256 * 4 >= m * dim and (y == 1 or x * (y - 1) * 256 * 4 < m * (dim + 3))


def test_launches_fit_a_grid():
    """At every accepted size a launch has fewer than 2^32 work-items, and its pieces are
    whole tiles that cover the table and fit their buffers."""
    out = _run("""
  const int64_t sides[] = {1, 3, 33, 64, 65, 200, 1000, 8191, 8192, 1 << 16, (1 << 16) + 1, 1 << 20,
                           (1 << 21) - 63, 1 << 21};
  const int64_t tables[] = {1, 255, 257, 50257, 151936, (1 << 21) + 1, (1 << 24) + 5,
                            (int64_t(1) << 30) + 7, (int64_t(1) << 31) - 1};
  const int64_t limit = int64_t(1) << 32;
  auto tiles = [](int64_t n, int64_t m, int64_t bn, int64_t bm) {
    return loss_up(n, bn) / bn * (loss_up(m, bm) / bm);
  };
  long bad = 0, cases = 0;
  auto check = [&](bool ok, const char *what, int64_t m, int64_t dim, int64_t rows) {
    ++cases;
    if (!ok && bad++ < 20)
      printf("%s:%lld:%lld:%lld\\n", what, (long long)m, (long long)dim, (long long)rows);
  };
  for (int64_t m : sides)
    for (int64_t dim : sides)
      for (int64_t rows : tables) {
        if (dim > 1 << 16 || rows > (int64_t(1) << 39) / dim || rows > (int64_t(1) << 42) / m)
          continue;
        check(launch_rows(dim) >= 256 && launch_rows(dim) % 256 == 0, "rows", m, dim, rows);
        check(tiles(launch_rows(dim), dim, 64, 64) * 512 < limit, "zeros", m, dim, rows);
        for (int dt = 0; dt < 2; ++dt)
          for (int copied = 0; copied < 2; ++copied) {
            const int64_t e = dt ? 2 : 4;
            LossLayout l = loss_layout(kLossForward, m, dim, rows, dt);
            int64_t step = loss_piece(l, m, rows, copied);
            check(step >= loss_min(rows, 256) && (step >= rows || step % 256 == 0), "loss piece", m,
                  dim, rows);
            check((tiles(step, m, 64, 64) + 128) * 512 < limit, "loss", m, dim, rows);
            check(!copied || step <= l.table_rows, "loss copy", m, dim, rows);
            for (int call = 0; call < 4; ++call) {
              const bool given = call > 0, d_copied = call & 1;
              l = loss_layout(given ? kHeadGrad : kLossGrad, m, dim, rows, dt);
              step = given ? head_grad_piece(l, m, rows, dt, d_copied, copied)
                           : grad_piece(l, m, rows, dt, copied);
              check(step >= 256 && step % 256 == 0, "piece", m, dim, rows);
              check(!copied || step <= l.table_rows, "copy", m, dim, rows);
              check((given && !d_copied) ||
                        m * loss_min(step, loss_up(rows, 64)) * e <= l.piece_cap,
                    "buffer", m, dim, rows);
              const int64_t logits = given ? 0 : tiles(step, m, 64, 32);
              for (int gw = 0; gw < 2; ++gw) {
                // the tiles that the products take, and most splits for them
                const int64_t most = loss_most_splits(m, l.dim_pad, rows);
                const bool large = dt && large_products(m, dim);
                const bool small = !dt && small_products(m, dim, step, most, gw);
                const int64_t b = large ? 256 : small ? 64 : 128;
                const int64_t bm = m <= 32 ? 32 : dt && m <= 64 ? 64 : b;
                const int64_t groups =
                    tiles(dim, m, b, bm) * most + (gw ? tiles(dim, step, b, b) : 0);
                check((groups + (large ? logits : 0)) * (large ? 512 : 256) < limit, "products", m,
                      dim, rows);
              }
              check((logits + 128) * 512 < limit, "logits", m, dim, rows);
            }
          }
      }
  printf("%ld %s\\n", cases, bad ? "bad" : "good");
""")
    assert out[-1] == "good" and int(out[-2]) > 10000, out


def test_the_heads_backward_prepares_what_it_reads():
    """An unaligned table is neither copied nor a reason for another path where grad_x is
    not wanted, nor hidden rows where grad_weight is not."""
    out = _run("""
  const auto *even = reinterpret_cast<const char *>(uintptr_t(0x10000)), *odd = even + 4;
  void *out = reinterpret_cast<void *>(uintptr_t(0x20000));
  const auto rows = [&](const char *d, const char *w, const char *x, int64_t m, void *gx,
                        void *gw) {
    const HeadGradRows h = head_grad_rows(
        d, 2000, LossRows{x, m, 136, w, 2000, 1, 0, 2000, nullptr, 0},
        LossGrads{gx, 1, gw, 1, false});
    printf("%d%d%d%d\\n", h.d_copied, h.w_copied, h.x_copied, h.loose);
  };
  const int64_t sizes[] = {128, 300};
  for (int64_t m : sizes) {
    rows(even, even, even, m, out, out);
    rows(even, odd, even, m, out, out);
    rows(even, odd, even, m, out, nullptr);
    rows(even, odd, even, m, nullptr, out);
    rows(even, even, odd, m, out, out);
    rows(even, even, odd, m, nullptr, out);
    rows(even, even, odd, m, out, nullptr);
    rows(odd, odd, odd, m, out, out);
    rows(odd, odd, odd, m, nullptr, out);
    rows(odd, odd, odd, m, out, nullptr);
  }
""")
    assert out[:10] == ["0000", "0001", "0001", "0000", "0010", "0010", "0000", "0001", "0001",
                        "0001"]
    assert out[10:] == ["0000", "0100", "0100", "0000", "0010", "0010", "0000", "1110", "1010",
                        "1100"]

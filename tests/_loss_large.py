"""Shapes, (rows, vocabulary, width), whose bf16 gradients go through products in tiles
of 256 x 256, for the GPU tests that need them and the host test that holds the library
to it."""

# gradients of the loss: several pieces of the vocabulary, the last one ragged (the
# logits of a piece beside the products of the one before); live rows around a tile
PIECES = [(1030, 150001, 136), (1100, 130007, 264), (2047, 70003, 520)]
LIVE = [0, 1, 63, 128, 129, 255, 256, 257, 383, 512, 641, 896, 897, 1023, 1030]
# one piece; the logits through the loop of a long sum
ONE_PIECE = [(192, 70000, 136), (200, 70000, 256), (600, 70000, 1032), (1000, 33000, 520)]
# a table that is copied first, in one piece and in several
COPIED = [(200, 70001, 131), (1030, 140001, 515)]
# the head's backward
BACKWARD = [(192, 3000, 136), (200, 9001, 264), (256, 5000, 1024), (400, 20007, 200),
            (1000, 4096, 520), (1537, 777, 136), (256, 2000, 129)]
# next to them: not in such tiles
SMALLER = [(191, 3000, 136), (512, 3000, 128), (513, 3000, 136), (128, 3000, 264)]

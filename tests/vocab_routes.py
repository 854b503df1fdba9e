"""Sizes of the losses over a vocabulary by the kernels that they run (test
helper), held to the plans by test_vocab_routes.py."""
from __future__ import annotations

from tests.vocab_cases import BF16, F32

# name: dtype, tokens, d, vocab
ROUTES = {
    "tiles, float32": (F32, 300, 256, 1000),
    "tiles": (BF16, 300, 256, 1000),
    "few tokens, float32": (F32, 30, 1024, 20000),
    "few tokens": (BF16, 97, 1280, 28160),
    "rows padded to a tile": (BF16, 166, 768, 41256),
    "256 x 256 tiles, last panel padded": (BF16, 274, 1024, 26351),
    "256 x 256 tiles, last columns on small tiles": (BF16, 399, 544, 66539),
    "256 x 256 tiles, two pieces": (BF16, 2304, 256, 131072),
}
# with lists long enough to be sorted by the wave that holds their logits
# name: dtype, tokens, d, vocab, top
SORTED = {
    "sorted, small tiles, float32": (F32, 600, 512, 3000, 300),
    "sorted, small tiles": (BF16, 1126, 2832, 501, 59),
    "sorted, 256 x 256 tiles": (BF16, 600, 512, 20000, 400),
    "sorted, both": (BF16, 777, 512, 50001, 300),
}
# rows in ranges, the last of fewer than a tile's 256 (its first rows are formed again),
# top = 0: cross entropy
RANGES = {
    "targets": (BF16, 2400, 256, (1 << 21) - 3, 0),
    "lists, as many cells as there can be": (BF16, 2400, 256, 1 << 21, 160),
}
DTYPE = {F32: "f32", BF16: "bf16"}

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
DTYPE = {F32: "f32", BF16: "bf16"}

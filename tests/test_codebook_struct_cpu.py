"""The codebook that a weight's C struct holds is its own, whatever weights were used before it."""
import math

import torch

from bit_nf4_quantized_blockwise_b200 import NF4Weight


def test_a_negative_zero_stays_one():
    books = [tuple((z if j == 7 else (j - 7) / 8.0) for j in range(16)) for z in (0.0, -0.0, 0.0, -0.0)]
    byte = torch.zeros(1, dtype=torch.uint8)
    for book in books:
        w = NF4Weight(byte, None, None, None, 64, 64, book, absmax=torch.ones(64))
        got = list(w.struct().codebook)
        assert got == list(book) and math.copysign(1.0, got[7]) == math.copysign(1.0, book[7])

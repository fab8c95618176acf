"""Channels and tokens of a convolution's prefill, and the tokens of the tile that its kernel takes for them."""

TILED = [(8, 20000, 32), (128, 20000, 32), (192, 20000, 32), (256, 20000, 32), (4096, 3001, 32),
         (8, 80000, 64), (64, 80000, 64), (128, 80000, 64), (192, 80000, 64), (256, 80000, 64), (4096, 9800, 64)]

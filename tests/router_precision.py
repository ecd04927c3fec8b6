"""How far the router's logits may be off, tight enough to see a sum that lost
precision, and shapes whose sums are long enough to lose it.

Tensor cores truncate.  An MMA loses up to one unit in the last place of the sum
that it adds 16 products to, and about as much again where it aligns the
products: up to 2 x 2^-23 of the sum at the worst place in a binade, 0.7 of that
on average over the binade, half of that again on average over what is cut off:
0.7 x 2^-23 of the sum that it reaches, always towards zero.  After 16 MMAs the
kernels add the sum to FP32, rounding to nearest, and begin again at zero.

Products of one sign: the j-th MMA of 16 reaches j / 16 of its sum.  Together
they lose (1 + .. + 16) / 16 = 8.5 times 0.7 x 2^-23: 7.1e-7 of it, and so does
the whole.  Products of both signs: sums grow as the root, the j-th MMA reaches
sqrt(j / 16): 10.9 times 0.7 x 2^-23, 9.1e-7 of each of the sums of 256, whose
losses fall either way as those do: 9.1e-7 of the whole in the root mean square.
The additions in FP32, under 60 of them here, round to nearest by 2^-24 / sqrt(3)
of growing sums: 2^-24 / sqrt(3) x sqrt(60 / 3) = 1.5e-7, apart from the rest.
So the root mean square stays below 1e-6 of that of the logits.

A sum that runs on for n MMAs loses half of n times 0.35 x 2^-23 with products of
one sign, even if the alignment loses nothing: 2.7e-6 for n = 128, as long as
every shape here has them where a kernel does not start again.  A partial sum in
FP16 or BF16 is 2^-13 or 2^-10 off.
"""

import numpy as np

RMS = 1e-6

# (kernel, rows of a small kernel's tile or columns of a tcgen05 one, parts of K, M, E, H): 128 MMAs or more to a part of
# K -- of the warps' kernel, whose 8 warps split K too, to a warp's
LONG = [
    ("tiles", 64, 1, 5000, 40, 2048),
    ("tiles", 64, 2, 5000, 40, 4096),
    ("tiles", 64, 4, 2400, 40, 8192),
    ("tiles", 64, 8, 176, 200, 16384),
    ("tiles", 128, 1, 1300, 1000, 2048),
    ("tiles", 128, 2, 2400, 384, 4096),
    ("tiles", 128, 4, 900, 384, 8192),
    ("tiles", 128, 8, 244, 200, 16384),
    ("tiles", 256, 1, 2400, 1000, 2048),
    ("tiles", 256, 2, 1300, 1000, 4096),
    ("tiles", 256, 4, 700, 700, 8192),
    ("tiles", 256, 8, 193, 200, 16384),
    ("warps", 8, 4, 11, 512, 65536),
    ("warps", 8, 8, 5, 8, 131072),
    ("warps", 32, 1, 9000, 8, 16384),
    ("warps", 32, 2, 4000, 8, 32768),
    ("warps", 32, 4, 108, 128, 65536),
    ("warps", 32, 8, 57, 40, 131072),
    ("few", 1, 8, 1, 256, 16384),
    ("few", 4, 8, 4, 256, 16384),
]


def rms_error(got, want):
    """Root mean square of the errors over that of what is right."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    return float(np.sqrt(np.mean((got - want) ** 2) / np.mean(want ** 2)))

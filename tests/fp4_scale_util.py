"""The 4-bit cache's block scale by its definition, apart from the oracle's and the library's code, and maxima that lie where
the choice of a scale code turns."""

from __future__ import annotations

import numpy as np

#: values of the scale codes 0 to 0x7E
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])
SIXTH = 11184811 * 2.0 ** -26  # the binary32 number nearest to 1/6


def scale_code(amax, g):
    """Code nearest to fl(amax fl(g fl(1/6))), ties to the even code; the products of two binary32 numbers are exact in
    binary64, and so are the middles between codes."""
    factor = np.float32(np.float64(np.float32(g)) * SIXTH)
    x = np.float64(np.float32(np.float64(np.float32(amax)) * np.float64(factor)))
    if x >= E4M3[-1]:
        return len(E4M3) - 1
    low = int(np.searchsorted(E4M3, x, side="right")) - 1
    middle = (E4M3[low] + E4M3[low + 1]) / 2
    return low + int(x > middle or (x == middle and low % 2 == 1))


def middle_maxima(g):
    """For each two codes the binary32 number nearest to the middle between them times 6 / g, and its neighbours."""
    a = ((E4M3[1:] + E4M3[:-1]) / 2 * 6 / np.float64(np.float32(g))).astype(np.float32)
    return np.concatenate([np.nextafter(a, np.float32(0)), a, np.nextafter(a, np.float32(np.inf))])

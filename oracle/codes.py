"""Values held in 8 bits, in float64 from the definition: of each row the largest
magnitude a has the largest code M, the row's scale is a / M, and a value becomes
the code nearest to x M / a, the even one of two as near.  Shares no code with
the CUDA path.  Pinned by ``tests/test_oracle_codes.py`` against exact fractions
and, for e4m3, the list of its 253 numbers."""
import numpy as np

M = {"int8": 127.0, "e4m3": 448.0}


def e4m3_numbers():
    """The value of each byte (0x7f, 0xff: NaN): sign, 4 bits of exponent with bias 7, 3 of fraction."""
    b = np.arange(256)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (8 + f) * 2.0 ** (e - 10), f * 2.0 ** -9) * np.where(b & 128, -1.0, 1.0)
    v[(b & 127) == 127] = np.nan
    return v


def values(codes, fmt):
    """Bytes (int8 array) -> the numbers they stand for."""
    return codes.astype(np.float64) if fmt == "int8" else e4m3_numbers()[codes.view(np.uint8)]


def oracle_encode(x, fmt):
    """x [..., d] float64 (bf16 values) -> codes (int8 bytes), scales float32 [...]."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).max(-1)
    good = np.isfinite(x).all(-1)
    a = np.where(good, a, np.nan)
    with np.errstate(invalid="ignore", divide="ignore"):
        t = np.where(good[..., None] & (a > 0)[..., None], x * M[fmt] / a[..., None], 0.0)   # exact where it is halfway
        scales = np.where(a == 0, np.float32(0), a.astype(np.float32) / np.float32(M[fmt])).astype(np.float32)
    if fmt == "int8":
        return np.rint(t).astype(np.int8), scales
    num = e4m3_numbers()[:127]                          # 0 .. 448, ascending by byte
    m = np.abs(t)
    hi = np.clip(np.searchsorted(num, m), 1, 126)
    lo = hi - 1
    down, up = m - num[lo], num[hi] - m
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    pick = np.where(m == 0, 0, pick).astype(np.uint8)
    return (pick | np.where(np.signbit(t), 128, 0).astype(np.uint8)).view(np.int8), scales

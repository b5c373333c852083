"""float64 oracle of the 4-bit KV cache (include/saga_q4.h): what a row stores and
how it is quantised, from the format's definition. Test infrastructure only;
it shares no code with the CUDA path. Attention over the stored values is the
oracle's own (saga_oracle)."""
import numpy as np

# e2m1: sign, two exponent bits (bias 1), one mantissa bit
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(byte):
    """The value of a scale byte (its sign bit ignored; 0x7f reads as 480)."""
    b = np.asarray(byte, dtype=np.int64) & 0x7F
    e, m = b >> 3, b & 7
    return np.where(e > 0, np.exp2(e - 7.0) * (1 + m / 8.0), m * np.exp2(-9.0))


_E4M3 = e4m3_value(np.arange(127))          # increasing, 0 .. 448


def _nearest_even(grid, x):
    """Index of the grid value nearest to each x >= 0; a tie goes to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def quantise(x, g=1.0):
    """Rows x [..., d] (fp32) -> codes uint8 [..., d/2], scales uint8 [..., d/16].
    g broadcasts over [..., d/16]. The quotients are rounded to fp32 first,
    as the definition says; with g = 1 that never changes a bf16 value's code."""
    f = np.float32
    x = np.nan_to_num(np.asarray(x, dtype=f), nan=0.0, posinf=np.inf, neginf=-np.inf)
    xb = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    g = np.broadcast_to(np.asarray(g, dtype=f), xb.shape[:-1])
    with np.errstate(all="ignore"):
        r = np.minimum(f(448), np.abs(xb).max(-1) / (f(6) * g))
        s = _nearest_even(_E4M3, r.astype(np.float64))
        t = (e4m3_value(s).astype(f) * g)[..., None]
        y = np.abs(xb) / t
    y = np.where(s[..., None] == 0, 0, np.minimum(y, f(6))).astype(np.float64)
    c = _nearest_even(E2M1, y) + 8 * (np.signbit(xb) & (s[..., None] != 0))
    c = c.astype(np.uint8).reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), s.astype(np.uint8)


def values(codes, scales, g=1.0):
    """float64 values of codes [..., d/2] and scales [..., d/16]; g broadcasts
    over [..., d/16]."""
    codes = np.asarray(codes)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], scales.shape[-1], 16)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = e4m3_value(scales) * np.broadcast_to(np.asarray(g, np.float64), scales.shape)
    return (v * s[..., None]).reshape(*codes.shape[:-1], codes.shape[-1] * 2)

"""MX-FP4 rows in plain numpy, from the format's definition in 64 bits (no code shared with the library)."""

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x):
    """float64 [rows][cols] -> codes uint8 [rows][cols/2], scales uint8 [rows][cols/32]."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    m = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    _, ex = np.frexp(m)                       # m = f * 2^ex, f in [1/2, 1): floor(log2 m) = ex - 1
    e = np.where(m > 0, np.clip(ex - 3, -127, 127), -127)
    y = np.where(bad[..., None], 0.0, np.where(np.isfinite(b), b, 0) * np.exp2(-e.astype(np.float64))[..., None])
    a = np.abs(y)
    d = np.abs(a[..., None] - GRID)           # nearest grid value; ties to the even code
    code = d.argmin(-1)
    nxt = np.minimum(code + 1, 7)
    tie = np.take_along_axis(d, nxt[..., None], -1)[..., 0] == np.take_along_axis(d, code[..., None], -1)[..., 0]
    code = np.where(tie & (nxt > code) & (code % 2 == 1), nxt, code)
    code = code + 8 * (y < 0)
    code = code.reshape(rows, cols)
    return ((code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8),
            np.where(bad, 255, e + 127).astype(np.uint8))


def values(codes, scales):
    """codes [..][cols/2], scales [..][>= cols/32] -> float64 [..][cols]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    nb = v.shape[-1] // 32
    s = scales[..., :nb].astype(np.float64)
    unit = np.where(s == 255, np.nan, np.exp2(s - 127))
    return (v.reshape(*v.shape[:-1], nb, 32) * unit[..., None]).reshape(v.shape)

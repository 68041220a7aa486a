"""MXFP4 on the CPU in fp64 numpy, from the format's definition (test helper):
nearest value of the grid by distance, ties to the even code."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(v):
    """(codes [..., K], scale bytes [..., K / 32]) of fp32 values [..., K]."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(*v.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    byte = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2 + 127, 127).clip(0, 254).astype(int)
    a = np.abs(b) / np.exp2(byte[..., None] - 127.0)
    gap = np.abs(a[..., None] - GRID)
    # the even code first among equals: order the candidates by (distance, odd)
    code = np.lexsort((np.broadcast_to(np.arange(8) & 1, gap.shape), gap), axis=-1)[..., 0]
    code = code + 8 * np.signbit(b)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(v.shape).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    return np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)


def values(codes, scales):
    """fp64 values of packed codes [..., K / 2] and scale bytes [..., K / 32]."""
    c = unpack(np.asarray(codes)).astype(int)
    s = np.asarray(scales).astype(float)
    p = np.where(s == 255, np.nan, np.exp2(s - 127))
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(p, 32, -1)

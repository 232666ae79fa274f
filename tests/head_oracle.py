"""Plain forms of the 8-bit head in numpy and 64 bits: quantisation in blocks of 128 and what a quantised matrix stands
for (test infrastructure)."""
import numpy as np
import torch


def e4m3(y):
    """Values |y| <= 448 rounded to the nearest e4m3, ties to the even one."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(y / step) * step


def quantize(x, block_rows, pow2):
    """(values, scales) of x [n, width], the width filled up with zeros to a multiple of 16."""
    x = np.asarray(x, np.float32)
    n, width = x.shape
    cols = -(-width // 16) * 16
    values = np.zeros((n, cols))
    scales = np.ones((-(-n // block_rows), -(-cols // 128)))
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = x[i * block_rows:(i + 1) * block_rows, 128 * j:128 * (j + 1)]
            at = np.s_[i * block_rows:i * block_rows + part.shape[0], 128 * j:128 * j + part.shape[1]]
            if not np.isfinite(part).all():
                scales[i, j] = np.nan
                values[i * block_rows:i * block_rows + part.shape[0], 128 * j:128 * (j + 1)] = np.nan
                continue
            a = float(np.abs(part).max()) if part.size else 0.0
            if a > 0 and pow2:
                e = -126
                while 448.0 * 2.0 ** e < a:
                    e += 1
                scales[i, j] = 2.0 ** e
            elif a > 0:
                scales[i, j] = max(np.float32(a) / np.float32(448), np.float32(2.0 ** -126))
            y = (part / np.float32(scales[i, j])).astype(np.float32)
            values[at] = e4m3(np.clip(y, -448, 448))
    return values, scales


def worth(q, block_rows):
    """What a quantised matrix on the device stands for, in 64 bits."""
    v, s = q["values"].cpu().double(), q["scales"].cpu().float().double()
    s = s.repeat_interleave(block_rows, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
    return v * s


def wide(x, dev):
    """x on the device as the first columns of rows that start 16-byte aligned; what lies between them is NaN."""
    n, V = x.shape
    es = x.element_size()
    w = torch.full((n, -(-V * es // 16) * 16 // es), float("nan"), dtype=x.dtype, device=dev)[:, :V]
    return w.copy_(x)


KINDS = {"f32": torch.float32, "pow2": torch.float8_e8m0fnu}

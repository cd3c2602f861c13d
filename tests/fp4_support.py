"""The microscaled 4-bit form in 64 bits on the host, value by value, for the tests of its kernels."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1])
EPS = 1e-5


def power_of_two(x):
    """2^floor(log2 x), 0 for 0."""
    part, e = np.frexp(x)
    return np.where(x > 0, np.ldexp(1.0, e - 1), 0.0)


def nearest(x, grid):
    """Index of the number of an ascending grid next to x >= 0; a tie goes to the even index."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    below, above = x - grid[i - 1], grid[i] - x
    return np.where((below < above) | ((below == above) & (i % 2 == 1)), i - 1, i)


def kept(x, form):
    """Codes (0..15), scales as stored (bytes), row scales, and the values that fp64 rows x stand for once kept."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        x = np.asarray(x, np.float64)
        rows, cols = x.shape
        n = BLOCK[form]
        blocks = -(-cols // n)
        full = np.zeros((rows, blocks * n))
        full[:, :cols] = x
        b = full.reshape(rows, blocks, n)
        bad = ~np.isfinite(b).all(-1)
        size = np.where(np.isfinite(b), np.abs(b), 0.0)
        top = np.where(bad, 0.0, size.max(-1))
        r = np.ones(rows)
        if form == "mxfp4":
            scale = np.maximum(power_of_two(top) / 4, 2.0 ** -127)
            byte = np.log2(scale).round().astype(int) + 127
            byte[bad] = 255
        else:
            r = np.maximum(power_of_two(size.max((1, 2))) / 1024, 2.0 ** -126)
            byte = nearest(top / (6 * r[:, None]), E4M3)
            scale = E4M3[byte] * r[:, None]
            byte[bad] = 0x7F
        q = np.where(scale[..., None] > 0, size / np.where(scale > 0, scale, 1.0)[..., None], 0.0)
        code = nearest(np.minimum(q, 6.0), LEVELS)
        values = np.where(np.signbit(b), -1, 1) * LEVELS[code] * scale[..., None]
        values[bad] = np.nan
        code = np.where(np.signbit(b), code + 8, code)
        code[bad] = 2
        return (code.reshape(rows, -1)[:, :cols], byte, r, values.reshape(rows, -1)[:, :cols])


def stored(matrix):
    """Codes, scale bytes and row scales of an Fp4Matrix, taken from its bytes by the documented layout."""
    rows, cols, form = matrix.rows, matrix.cols, matrix.format
    data = matrix.data.cpu().numpy()
    stride = (cols + 31) // 32 * 16
    codes = data[:rows * stride].reshape(rows, stride)
    low, high = codes & 15, codes >> 4
    codes = np.stack([low, high], -1).reshape(rows, -1)
    at = (rows * stride + 255) // 256 * 256
    groups = (cols + 255) // 256 * (4 if form == "nvfp4" else 2)
    n_scales = (rows + 127) // 128 * groups * 512
    scales = data[at:at + n_scales].reshape(-1, groups, 512)
    blocks = groups * 4
    r, k = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    scales = scales[r // 128, k // 4, r % 32 * 16 + r % 128 // 32 * 4 + k % 4]
    row_scale = None
    if form == "nvfp4":
        end = at + (n_scales + 255) // 256 * 256
        row_scale = data[end:end + 4 * rows].view(np.float32)
    return codes, scales, row_scale

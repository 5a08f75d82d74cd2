"""fp64 numpy definitions of the layer-side operators: the 8-bit activation format, the
RMS norm with the residual's addition, SwiGLU and the weight gradient, with their
gradients.  Written from the formulas; shares no code with the CUDA path."""
import numpy as np

GROUP = 32
LARGEST = {"e4m3": 448.0, "int8": 127.0}
LOWEST_EXP = -110
HIGHEST_EXP = {"e4m3": 119, "int8": 121}


def e4m3_number(byte):
    """The number an e4m3 byte stands for (1 sign, 4 exponent bits of bias 7, 3 mantissa bits)."""
    b = np.asarray(byte).astype(np.int64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * np.exp2((e - 7).astype(np.float64)), m * 2.0 ** -9)
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


_E4M3 = e4m3_number(np.arange(127))   # non-negative codes in increasing order


def e4m3_code(x):
    """Nearest e4m3 byte of finite x, ties to the even code, saturating at 448."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_E4M3, a), 1, 126)
    lo = hi - 1
    up = (a - _E4M3[lo] > _E4M3[hi] - a) | ((a - _E4M3[lo] == _E4M3[hi] - a) & (hi % 2 == 0))
    c = np.where(a >= 448.0, 126, np.where(up, hi, lo)).astype(np.uint8)
    return np.where(np.signbit(x), c | 128, c).astype(np.uint8)


def scale_exponent(amax, fmt):
    """Smallest e with amax <= L 2^e, within the format's range of e."""
    f, k = np.frexp(np.where(amax > 0, amax, 1.0))    # amax = f 2^k, 1/2 <= f < 1
    fl, kl = np.frexp(LARGEST[fmt])
    e = k - kl + (f > fl)
    return np.clip(np.where(amax > 0, e, LOWEST_EXP), LOWEST_EXP, HIGHEST_EXP[fmt]).astype(np.int64)


def pack(x, fmt):
    """x (rows, cols) -> (codes, scale bytes), uint8, unpadded."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    n = -(-cols // GROUP)
    z = np.zeros((rows, n * GROUP))
    z[:, :cols] = x
    z = z.reshape(rows, n, GROUP)
    bad = ~np.isfinite(z).all(2)
    z = np.where(bad[:, :, None], 0.0, z)
    e = scale_exponent(np.abs(z).max(2), fmt)
    w = z * np.exp2(-e.astype(np.float64))[:, :, None]
    if fmt == "e4m3":
        q = e4m3_code(w)
    else:
        q = np.clip(np.rint(w), -127, 127).astype(np.int8).view(np.uint8)
    return q.reshape(rows, -1)[:, :cols], np.where(bad, 255, e + 127).astype(np.uint8)


def unpack(codes, scales, fmt):
    v = e4m3_number(codes) if fmt == "e4m3" else np.asarray(codes).view(np.int8).astype(np.float64)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, GROUP, 1)[:, :v.shape[1]]


def rmsnorm(x, weight, eps, residual=None):
    """(h, y, xhat, rstd)."""
    h = x if residual is None else x + residual
    rstd = 1 / np.sqrt(np.mean(h * h, 1) + eps)
    xhat = h * rstd[:, None]
    return h, xhat * weight, xhat, rstd


def rmsnorm_grad(dy, xhat, rstd, weight, dres=None):
    """(dh, dweight) of y = xhat weight."""
    w = dy * weight
    dh = rstd[:, None] * (w - xhat * np.mean(w * xhat, 1, keepdims=True))
    return dh if dres is None else dh + dres, np.sum(dy * xhat, 0)


def sigmoid(z):
    return 1 / (1 + np.exp(-np.clip(z, -700, 700)))


def swiglu(gate, up):
    return gate * sigmoid(gate) * up


def swiglu_grad(da, gate, up):
    s = sigmoid(gate)
    return da * up * s * (1 + gate * (1 - s)), da * gate * s


def wgrad(dy, x, col_scale=None, offsets=None):
    g = dy.T @ x if offsets is None else np.stack([dy[a:b].T @ x[a:b] for a, b in zip(offsets, offsets[1:])])
    return g if col_scale is None else g * col_scale

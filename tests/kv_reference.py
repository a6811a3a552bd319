"""64-bit definitions of the KV-cache operators, for the tests: numpy on the
host, written from the formulas, sharing no code with the library."""
import numpy as np

DT = {"f16": (0, 10, 15), "bf16": (1, 7, 127)}


def to_bits(x, dtype):
    """float array -> 16-bit patterns, to nearest even."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float64)).to(torch.float16 if dtype == "f16" else torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def from_bits(b, dtype):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.float16 if dtype == "f16" else torch.bfloat16)
    return t.double().numpy()


def e4m3_values():
    """Value of each of the 256 codes (finite-only form: bias 7, max 448, 0x7f NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 0x7f) == 0x7f] = np.nan
    return np.where(c >= 128, -v, v)


def quantise(x):
    """(..., D) doubles -> codes (uint8), scales (float32)."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(-1)
    top = np.abs(np.where(fine[..., None], x, 0)).max(-1)
    scale = (top / 448.0).astype(np.float32)
    scale = np.where(top > 0, np.maximum(scale, np.float32(2.0 ** -126)), np.float32(0))
    grid = e4m3_values()[:127]
    border = (grid[1:] + grid[:-1]) / 2
    ok = fine & (scale > 0)
    s = np.where(ok, scale, 1).astype(np.float64)[..., None]
    a = np.abs(np.where(ok[..., None], x, 0))
    # compare with border * scale, which is exact in 64 bits
    k = np.zeros(x.shape, np.int64)
    for i, b in enumerate(border):
        up = (a > b * s) | ((a == b * s) & (i % 2 == 1))
        k = np.where(up, i + 1, k)
    codes = (k | np.where(np.signbit(x) & ok[..., None], 128, 0)).astype(np.uint8)
    return codes, np.where(fine, scale, np.float32(np.nan)).astype(np.float32)


def attention(q, K, V, first, scale, window):
    """q: (n, Hq, D), K, V: (L, H, D) doubles, first: position of row 0.
    Returns out, lse, A (the weighted mean of |v|), S (largest sum |q k| * scale)."""
    n, Hq, D = q.shape
    L, H, _ = K.shape
    G = Hq // H
    out = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    A = np.zeros((n, Hq, D))
    S = np.zeros((n, Hq))
    for i in range(n):
        p = first + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0 or lo > p or L == 0:
            continue
        for h in range(H):
            k, v, x = K[lo:p + 1, h], V[lo:p + 1, h], q[i, h * G:(h + 1) * G]
            with np.errstate(invalid="ignore", over="ignore"):
                z = (x @ k.T) * scale
                top = z.max(-1, keepdims=True)
                w = np.exp(z - top)
                tot = w.sum(-1, keepdims=True)
                out[i, h * G:(h + 1) * G] = (w / tot) @ v
                lse[i, h * G:(h + 1) * G] = (top + np.log(tot))[:, 0]
                A[i, h * G:(h + 1) * G] = (w / tot) @ np.abs(v)
                S[i, h * G:(h + 1) * G] = (np.abs(x) @ np.abs(k).T).max(-1) * abs(scale)
    return out, lse, A, S

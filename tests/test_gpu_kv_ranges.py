"""Attention over KV pages where values lie far apart: V rows of very different sizes, seen and unseen;
a key that takes nearly all of the weight; against the 64-bit definition.

Tolerance, beside the terms of test_gpu_kv_ops.py for the output's rounding, the scores and the sums:
  p A           the weights' own rounding, p = 2^-11 for an 8-bit cache (their fp16 values), u for a 16-bit
                cache in the kernel for many rows, 2^-16 in the other; A = sum w |v| / sum w
  8 bits:  n 2^-27 M, M = max_j w_j max_d |v_jd| / sum w over the keys that the row sees: what fp16's least
                step, 2^-24, leaves of weights times V's scales (half of it, of a largest one of 2^2 or more)
  16 bits: n 2^-30 V, V = max |v| over the keys that the row sees: the same of weights whose largest is 2^5
                or more
and 2^-24 (f16) or 2^-126 (bf16) for outputs below the type's normal range.
"""
import math

import numpy as np
import pytest

import gather_lora_paged_b200 as G
import kv_reference as R
from test_gpu_kv_ops import U, Cache, _attend, _dev, _host, _torch

pytestmark = pytest.mark.gpu


def _check(c, b, q, out, lse, hq, scale, window=0, once=False):
    """Rows `out`, `lse` of queries q (n, hq, D) over sequence b."""
    n, D, dtype = q.shape[0], c.D, c.dtype
    L = c.lens[b][1]
    K, V = c.rows(b, 0), c.rows(b, 1)
    want, wl, A, S = R.attention(q, K, V, L - n, scale, window)
    u = U[dtype]
    p = 2.0 ** -11 if c.fmt else u if once else 2.0 ** -16
    kq = np.abs(q).max() * np.abs(K).max() * scale
    e = (D + 6) * 2.0 ** -23 * S[..., None] + 2.0 ** -21
    small = np.zeros(want.shape[:2])
    top = np.abs(V).max(-1)
    for i in range(n):
        a = L - n + i
        lo = max(0, a - window + 1) if window else 0
        for h in range(hq):
            g = h // (hq // c.H)
            if not c.fmt:
                small[i, h] = L * 2.0 ** -30 * top[lo:a + 1, g].max(initial=0)
            elif a >= lo:
                w = np.exp(K[lo:a + 1, g] @ q[i, h] * scale - wl[i, h])
                small[i, h] = L * 2.0 ** -27 * (w * top[lo:a + 1, g]).max()
    tol = (u * np.abs(want) + A * (2 * e + p + 2 * (L + 8) * 2.0 ** -23) + small[..., None]
           + (2.0 ** -24 if dtype == "f16" else 2.0 ** -126))
    if c.fmt and dtype == "bf16":
        tol = tol + A * (2 * D * 2.0 ** -24 * kq)
    got = R.from_bits(_host(out), dtype).reshape(-1, n, hq, D)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], np.broadcast_to(want, got.shape)[bad][:4],
                           np.broadcast_to(tol, got.shape)[bad][:4])
    ltol = e[..., 0] + (L + 8) * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(wl)) + (D * 2.0 ** -24 * kq if c.fmt else 0)
    assert np.all(np.abs(lse.double().cpu().numpy().reshape(-1, n, hq) - wl) <= ltol)


# rows per kv head: few (row tiles of 8, 16 and 48), many
ROWS = [(3, 2), (5, 3), (5, 8), (40, 2), (300, 1)]


@pytest.mark.parametrize("up", [0, 12, 20, 26])
@pytest.mark.parametrize("where", ["newer", "behind the window", "no weight"])
@pytest.mark.parametrize("n,group", ROWS)
def test_a_row_does_not_depend_on_the_size_of_v_rows_without_weight(n, group, where, up):
    """One V row 2^up times the others: unseen by most rows, or seen at a weight of e^-50 or less."""
    H, D, L = 2, 64, n + 130
    window = 100 if where == "behind the window" else 0
    key = {"newer": L - 1, "behind the window": L - n - 99, "no weight": 40}[where]
    c = Cache([(n, L), (1, 20)], H, D, "bf16", 1, 4096, seed=n)

    def spoil(b, part, x):
        if b == 0:
            x[:, :, 0] = 0.0
            if part:
                x[key] *= 2.0 ** up
            elif where == "no weight":
                x[key] = 0.0
                x[key, :, 0] = -128.0
    c.fill(spoil=spoil)
    rng = np.random.default_rng(7)
    q = rng.standard_normal((c.T, H * group, D))
    q[:, :, 0] = 6.0
    q = R.from_bits(R.to_bits(q, "bf16"), "bf16")
    out, lse = _attend(c, _dev(q.reshape(c.T, -1), "bf16"), H * group, window=window, max_rows=n)
    assert c.check()[0] == 0
    _check(c, 0, q[:n], out[:n], lse[:n], H * group, 1 / math.sqrt(D), window)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,group", ROWS)
def test_v_rows_of_every_size(n, group, dtype):
    """V rows whose sizes go up, go down and are mixed, so that the largest product of weight and size moves on."""
    H, D, L = 3, 128, n + 700
    span = 24 if dtype == "f16" else 100
    c = Cache([(n, L), (n, n + 5)], H, D, dtype, 1, 16384, seed=n)
    way = np.stack([np.linspace(-1, 1, L), np.linspace(1, -1, L), np.random.default_rng(1).uniform(-1, 1, L)], 1)

    def spoil(b, part, x):
        if part:
            x *= 2.0 ** (span / 2 * way[:len(x)] - (4 if dtype == "f16" else 0))[..., None]
    c.fill(spoil=spoil)
    q = R.from_bits(R.to_bits(np.random.default_rng(3).standard_normal((c.T, H * group, D)) * 3, dtype), dtype)
    out, lse = _attend(c, _dev(q.reshape(c.T, -1), dtype), H * group, max_rows=n)
    assert c.check()[0] == 0
    for b in (0, 1):
        rows = slice(b * n, b * n + n)
        _check(c, b, q[rows], out[rows], lse[rows], H * group, 1 / math.sqrt(D))


def _one_key_above(L, n, group, dtype, fmt, gap, sink, B, D=64, H=1):
    """B sequences over one cache of L tokens: key 0 is `gap` nats above all others, whose V rows have one sign."""
    torch = _torch()
    c = Cache([(n, L)], H, D, dtype, fmt, 65536, seed=L)

    def spoil(b, part, x):
        if part:
            np.abs(x, out=x)
            x[0] *= sink
        else:
            x *= 0.02
            x[:, :, 0] = 0.0
            x[0] = 0.0
            x[0, :, 0] = 32.0
    c.fill(spoil=spoil)
    rng = np.random.default_rng(gap)
    q = rng.standard_normal((n, H * group, D))
    scale = 1 / math.sqrt(D)
    q[:, :, 0] = gap / scale / 32.0
    q = R.from_bits(R.to_bits(q, dtype), dtype)
    one = c.lens[0]
    c.lens, c.table, c.T = [one] * B, np.repeat(c.table, B, 0), n * B
    c.starts = (np.arange(B + 1) * n).astype(np.int32)
    c.upload()
    dq = _dev(q.reshape(n, -1), dtype).repeat(B, 1)
    out, lse = _attend(c, dq, H * group)
    assert c.check()[0] == 0 and torch.isfinite(out).all()
    return c, q, out, lse, scale


@pytest.mark.parametrize("sink", [0.0, 2.0 ** -7, 1.0])
@pytest.mark.parametrize("gap", [10, 14, 17])
@pytest.mark.parametrize("n,group", [(1, 8), (2, 8), (5, 8)])
def test_many_small_weights_beside_a_large_one_in_8_bits(n, group, gap, sink):
    """8000 keys some 2^-20 below one: in a batch whose items are mostly not cut."""
    c, q, out, lse, scale = _one_key_above(8000, n, group, "f16", 1, gap, sink, 160)
    _check(c, 0, q, out, lse, group, scale)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("gap,sink", [(14, 1.0), (17, 0.0), (18, 0.0), (19, 0.0)])
@pytest.mark.parametrize("n,group", [(40, 2), (4, 8)])
def test_many_small_weights_beside_a_large_one(n, group, gap, sink, fmt):
    """As above for 16-bit caches and for many rows."""
    c, q, out, lse, scale = _one_key_above(6000, n, group, "f16", fmt, gap, sink, 40)
    _check(c, 0, q, out, lse, group, scale, once=n * group > 32)

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


# ---------------------------------------------------------------------------
# values of V that are not finite, and the largest ones


def _set(c, b, part, pos, h, d, bits):
    """The stored bits of one value (16-bit pattern or e4m3 code)."""
    H, D, pt = c.H, c.D, c.pt
    at = ((part * H + h) * pt + pos % pt) * D + d
    pages = c.pool.pages.view(_torch().uint8 if c.fmt else _torch().int16).view(-1, c.pool.desc.page_elems * (2 if c.fmt else 1))
    pages[int(c.table[b, pos // pt]), at] = bits if bits < 0x8000 else bits - 0x10000


def _set_scale(c, b, part, pos, h, value):
    H, D, pt = c.H, c.D, c.pt
    pages = c.pool.pages.view(_torch().float32).view(-1, c.pool.desc.page_elems // 2)
    pages[int(c.table[b, pos // pt]), 2 * H * pt * D // 4 + (part * H + h) * pt + pos % pt] = value


def _odd_bits(c):
    """Bits of infinity, -infinity and NaN (the only one there is in e4m3)."""
    return (0x7f, 0xff, 0x7f) if c.fmt else (0x7f80, 0xff80, 0x7fc0) if c.dtype == "bf16" else (0x7c00, 0xfc00, 0x7e01)


@pytest.mark.parametrize("window", [0, 40, 900])
@pytest.mark.parametrize("dtype,fmt,D", [("bf16", 0, 64), ("f16", 0, 128), ("bf16", 1, 128), ("f16", 1, 64)])
@pytest.mark.parametrize("n,group", [(1, 2), (2, 3), (5, 2), (7, 6), (40, 2), (300, 1), (150, 4)])
def test_infinities_and_nan_among_the_values(n, group, dtype, fmt, D, window):
    """Seen by all rows, by some and by none of an item, of one and of both signs, in items that are cut and not:
    each output is what the definition makes of the keys that its row sees."""
    H, L = 3, n + 1100
    c = Cache([(n, L), (n, n), (n, L)], H, D, dtype, fmt, 16384, seed=n)
    c.fill()
    inf, ninf, nan = _odd_bits(c)
    first = L - n
    odd = [(5, 1, inf), (first - 700, 2, inf), (first - 60, 2, ninf), (first - 41, 3, inf), (first - 39, 4, nan),
           (first, 5, ninf), (first + n // 2, 6, inf), (L - 1, 7, nan), (L - 1, 6, ninf), (first + n // 3, 8, inf),
           (first - 900 + n // 2, 9, inf), (first - 40 + n // 2, 10, ninf)]
    for h in (0, 2):
        for pos, d, bits in odd:
            if pos < L:
                _set(c, 0, 1, pos, h, d + h, bits)
        _set(c, 1, 1, n - 1, h, 20, inf)
        _set(c, 1, 1, n // 2, h, 21, ninf)
    if fmt:  # whole rows: infinite and NaN scales, seen by some
        _set_scale(c, 1, 1, n // 2, 1, math.inf)
        _set_scale(c, 2, 1, first + n // 2, 1, math.nan)
        _set_scale(c, 2, 1, L - 1, 0, -math.inf)
        _set_scale(c, 2, 1, first - 39, 2, math.inf)
    rng = np.random.default_rng(3)
    q = R.from_bits(R.to_bits(rng.standard_normal((c.T, H * group, D)), dtype), dtype)
    out, lse = _attend(c, _dev(q.reshape(c.T, -1), dtype), H * group, window=window)
    assert c.check()[0] == 0
    scale = 1 / math.sqrt(D)
    got = R.from_bits(_host(out), dtype).reshape(-1, H * group, D)
    gl = lse.double().cpu().numpy()
    for b in range(3):
        rows = slice(b * n, b * n + n)
        K, V = c.rows(b, 0), c.rows(b, 1)
        Lb = c.lens[b][1]
        with np.errstate(invalid="ignore"):
            want, wl, _, _ = R.attention(q[rows], K, V, Lb - n, scale, window)
        g = got[rows]
        assert np.array_equal(np.isnan(g), np.isnan(want)), (b, np.argwhere(np.isnan(g) != np.isnan(want))[:6])
        assert np.array_equal(np.isinf(g), np.isinf(want)) and np.array_equal(g[np.isinf(g)], want[np.isinf(want)]), b
        # and where it is finite, the values: V's others with these at zero
        V = np.where(np.isfinite(V), V, 0)
        want, wl, A, S = R.attention(q[rows], K, V, Lb - n, scale, window)
        p = 2.0 ** -11 if fmt else U[dtype] if n * group > 32 else 2.0 ** -16
        tol = U[dtype] * np.abs(want) + A * (2 * ((D + 6) * 2.0 ** -23 * S[..., None] + 2.0 ** -21) + p + 2 * (Lb + 8) * 2.0 ** -23)
        tol = tol + Lb * 2.0 ** -27 * np.abs(V).max(initial=0) + 2.0 ** -24
        if fmt and dtype == "bf16":
            tol = tol + A * (2 * D * 2.0 ** -24 * np.abs(q).max() * np.abs(K).max() * scale)
        fin = np.isfinite(g)
        assert np.all(np.abs(g - want)[fin] <= tol[fin]), b
        assert np.all(np.abs(gl[rows] - wl) <= 2.0 ** -13 * (1 + np.abs(wl))), b


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,group", [(1, 2), (40, 2)])
def test_an_infinity_among_keys_of_next_to_no_weight(n, group, dtype):
    """The first half of a long cache is 75 nats below the rest (2^-108: parts of items that weigh nothing in fp32
    beside the others), and holds infinities: they are what the definition makes of them all the same."""
    H, D, L = 1, 64, 30000
    c = Cache([(n, L)], H, D, dtype, 0, 65536, seed=n)

    def spoil(b, part, x):
        if not part:
            x *= 0.1
            x[:L // 2, :, 0] = -100.0
            x[L // 2:, :, 0] = 0.0
    c.fill(spoil=spoil)
    inf, ninf, _ = _odd_bits(c)
    for pos, d, bits in [(100, 1, inf), (7000, 2, ninf), (100, 3, inf), (9000, 3, ninf)]:
        _set(c, 0, 1, pos, 0, d, bits)
    q = np.random.default_rng(3).standard_normal((n, H * group, D))
    q[:, :, 0] = 6.0
    q = R.from_bits(R.to_bits(q, dtype), dtype)
    out, _ = _attend(c, _dev(q.reshape(n, -1), dtype), H * group)
    assert c.check()[0] == 0
    got = R.from_bits(_host(out), dtype).reshape(n, H * group, D)
    assert np.all(got[..., 1] == np.inf) and np.all(got[..., 2] == -np.inf) and np.isnan(got[..., 3]).all()
    assert np.isfinite(np.delete(got, [1, 2, 3], -1)).all()


def _long(n, group, fmt, L=9000, H=4, D=128):
    """A long sequence beside a short one, filled on the device."""
    torch = _torch()
    c = Cache([(n, L), (1, 700)], H, D, "bf16", fmt, 32768)
    gen = torch.Generator(device="cuda").manual_seed(n)
    if fmt:
        by = c.pool.pages.view(torch.uint8)
        by.copy_(torch.randint(0, 0x70, by.shape, dtype=torch.uint8, generator=gen, device="cuda"))
        by.bitwise_or_(torch.randint(0, 2, by.shape, dtype=torch.uint8, generator=gen, device="cuda") * 128)
        m = 2 * H * c.pt * D // 4
        c.pool.pages.view(torch.float32).view(-1, c.pool.desc.page_elems // 2)[:, m:m + 2 * H * c.pt].fill_(0.01)
    else:
        c.pool.pages.normal_(generator=gen)
    q = torch.randn(c.T, H * group * D, generator=gen, device="cuda").to(torch.bfloat16)
    return c, q


@pytest.mark.parametrize("where", ["seen by all", "newer"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,group", [(1024, 8), (5, 8), (2, 4)])
def test_values_that_are_not_finite_change_nothing_else_and_take_little_time(n, group, fmt, where):
    torch = _torch()
    c, q = _long(n, group, fmt)
    H, D, hq = c.H, c.D, c.H * group
    L = c.lens[0][1]
    # one early key, or the newest one and others in between, so that items have keys that most rows do not see
    keys = [100] if where == "seen by all" else list(range(L - n + 31, L, 32)) + [L - 1]
    for pos in keys:
        for h in range(H):
            _set(c, 0, 1, pos, h, 3, 0)
    ws = torch.empty(G.slora_kv_attention_workspace_bytes(c.pool.h, c.layout, hq, 2, c.T, n), dtype=torch.uint8, device="cuda")
    lse = torch.empty(c.T, hq, device="cuda")

    def timed():
        ms = []
        out = torch.empty_like(q)
        for _ in range(5):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            _attend(c, q, hq, out=out, lse=lse, ws=ws, stream=torch.cuda.current_stream())
            e[1].record()
            torch.cuda.synchronize()
            ms.append(e[0].elapsed_time(e[1]))
        assert c.check()[0] == 0
        return out.view(-1, hq, D), sorted(ms)[2]

    ref, t0 = timed()
    for pos in keys:
        for h in range(H):
            _set(c, 0, 1, pos, h, 3, _odd_bits(c)[0])
    got, t1 = timed()
    sees = torch.arange(n, device="cuda") + L - n >= keys[0]
    odd = got[:n, :, 3].float()
    assert bool((torch.isnan(odd) if fmt else odd == math.inf)[sees].all())
    same = got.view(torch.int16) == ref.view(torch.int16)
    same[:n, :, 3] |= sees[:, None]
    assert bool(same.all())
    assert t1 <= 4 * t0 + 1.0, (t0, t1)


@pytest.mark.parametrize("dtype,fmt", [("bf16", 0), ("f16", 0), ("bf16", 1), ("f16", 1)])
@pytest.mark.parametrize("n,group", [(1, 2), (5, 3), (5, 8), (40, 2), (300, 2)])
def test_the_largest_values(n, group, dtype, fmt):
    """V at the end of the type's range, one sign and equal: the mean is that value, in items that are cut and not."""
    torch = _torch()
    H, D = 2, 64
    top = 65504.0 if dtype == "f16" else R.from_bits(np.array([0x7f7f], np.uint16), "bf16")[0]
    lens = [(n, n + 3000), (n, n), (1, 60)]
    c = Cache(lens, H, D, dtype, fmt, 8192, seed=n)

    def spoil(b, part, x):
        if part:
            x[:] = top
    c.fill(spoil=spoil)
    q = R.from_bits(R.to_bits(np.random.default_rng(3).standard_normal((c.T, H * group, D)) * 3, dtype), dtype)
    out, lse = _attend(c, _dev(q.reshape(c.T, -1), dtype), H * group)
    assert c.check()[0] == 0 and torch.isfinite(lse).all()
    got = R.from_bits(_host(out), dtype)
    # rounding to the type may pass its end where the sums' errors do: half a step there, and no more
    p = 2.0 ** -11 if fmt else U[dtype] if n * group > 32 else 2.0 ** -16
    near = np.abs(got - top) <= top * (U[dtype] + p + 2 * 3100 * 2.0 ** -23)
    assert np.all(near | (got == np.inf))
    # half of it and a quarter: no way past the end
    c2 = Cache(lens, H, D, dtype, fmt, 8192, seed=n)

    def half(b, part, x):
        if part:
            x[:] = top / 2 * np.where(np.arange(len(x)) % 2, 1.0, 0.5)[:, None, None]
    c2.fill(spoil=half)
    out, lse = _attend(c2, _dev(q.reshape(c2.T, -1), dtype), H * group)
    got = R.from_bits(_host(out), dtype).reshape(-1, H * group, D)
    at = 0
    for b, (m, L) in enumerate(lens):
        want, _, _, _ = R.attention(q[at:at + m], c2.rows(b, 0), c2.rows(b, 1) / top, L - m, 1 / math.sqrt(D), 0)
        S = 3 * 9 * math.sqrt(D)  # |q| |k| D / sqrt(D), of values of 3 sigma
        tol = U[dtype] + p + 2 * ((D + 6) * 2.0 ** -23 * S + 2.0 ** -21) + 2 * (L + 8) * 2.0 ** -23 + D * 2.0 ** -22 * S / 8
        assert np.all(np.abs(got[at:at + m] / top - want) <= tol), (b, np.abs(got[at:at + m] / top - want).max(), tol)
        at += m

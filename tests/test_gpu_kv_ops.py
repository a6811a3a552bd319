"""KV-cache operators on the GPU against 64-bit definitions: write (bit for
bit, borders between codes included), read back, attention (ragged batches, windows, odd
head groups and page sizes, rows that see nothing, infinities and NaN in masked
places, bad pages and sequences, strides, graphs, repeat calls), and a run of
them with the LoRA delta as a decode step uses them.

Attention tolerance, per output value o = sum w v / sum w with A = sum w |v| /
sum w, S = max_j scale * sum_d |q_d k_jd|, u = half a step of the output type:
  u |o|                       the one rounding of the output
  2 e A, e = (D + 6) 2^-23 S + 2^-21
                              each score: D products added in fp32 (by truncation
                              at worst), six further roundings; exp2 to 2^-22 and
                              its argument's rounding; in numerator and sum
  p A                         the weights' rounding for the products: 2^-16 as two
                              16-bit halves; u once, where the call may take the
                              kernel for more than 32 rows per kv head; for an 8-bit
                              cache 2^-11, that of their fp16 values (which either
                              kernel multiplies, whole or as three e4m3 values of
                              4 bits each, 11 in all)
  2 (n + 8) 2^-23 A           the two sums over n keys in fp32
  n 2^-25 V                   weights under fp16's normal range, V = max |v|
  D 2^-24 max|q| max|k| scale A (e4m3, bf16): q's fp16 image
"""
import math

import numpy as np
import pytest

import gather_lora_paged_b200 as G
import kv_reference as R

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _torch():
    import torch
    return torch


def _tdt(dtype):
    torch = _torch()
    return torch.float16 if dtype == "f16" else torch.bfloat16


def _dev(x, dtype):
    """float array -> device tensor of the 16-bit type."""
    torch = _torch()
    return torch.from_numpy(R.to_bits(x, dtype).view(np.int16)).cuda().view(_tdt(dtype))


def _host(t):
    torch = _torch()
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Cache:
    """A pool whose pages all hold 0xff bytes (NaN in every format), a batch over
    shuffled pages, and a host copy of what the cache holds."""

    def __init__(self, lens, H, D, dtype="bf16", fmt=0, page_elems=8192, extra_pages=3, max_tokens=8192, seed=0, ldb=None):
        torch = _torch()
        self.lens, self.H, self.D, self.dtype, self.fmt = list(lens), H, D, dtype, fmt
        self.layout = G.make_kv_layout(H, D, fmt)
        probe = G.Pool(0, [64], [64], 1, 0, 1, page_elems, 1, host_only=True)
        self.pt = G.slora_kv_page_tokens(probe.h, self.layout)
        assert self.pt >= 1
        rng = self.rng = np.random.default_rng(seed)
        need = sum(-(-L // self.pt) for _, L in lens)
        self.n_pages = need + extra_pages
        self.pool = G.Pool(G.SLORA_F16 if dtype == "f16" else G.SLORA_BF16, [64], [64], 1, 0, max_tokens, page_elems,
                           self.n_pages)
        self.pool.pages.view(torch.int16).fill_(-1)
        G.slora_pool_set_page_order(self.pool.h, rng.permutation(self.n_pages))
        ids = self.pool.kv_alloc(need)
        self.ldb = ldb or max([1] + [-(-L // self.pt) for _, L in lens])
        self.table = np.full((len(lens), self.ldb), -1, np.int32)
        for b, (_, L) in enumerate(lens):
            k = -(-L // self.pt)
            self.table[b, :k], ids = ids[:k], ids[k:]
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.T = int(self.starts[-1])
        G.slora_kv_check_batch(self.pool.h, self.layout, self.starts, [L for _, L in lens], self.table, self.T)
        self.upload()

    def upload(self):
        torch = _torch()
        self.rs = torch.from_numpy(self.starts).cuda()
        self.kl = torch.tensor([L for _, L in self.lens], dtype=torch.int32).cuda()
        self.bl = torch.from_numpy(self.table).cuda()

    def batch(self):
        return (self.rs, self.kl, self.bl, self.ldb, len(self.lens), self.T)

    def raw(self):
        """The pages on the host: values [page, part, head, slot, D] (bits or codes) and scales."""
        H, D, pt = self.H, self.D, self.pt
        bits = _host(self.pool.pages)[:self.n_pages * self.pool.desc.page_elems].reshape(self.n_pages, -1)
        if self.fmt == 0:
            return bits[:, :2 * H * pt * D].reshape(-1, 2, H, pt, D), None
        by = bits.view(np.uint8)
        n = 2 * H * pt * D
        return by[:, :n].reshape(-1, 2, H, pt, D), by[:, n:n + 8 * H * pt].copy().view(np.float32).reshape(-1, 2, H, pt)

    def rows(self, b, part):
        """Values of sequence b's cached rows (len, H, D) in 64 bits."""
        data, scales = self.raw()
        pos = np.arange(self.lens[b][1])
        pg, sl = np.clip(self.table[b, pos // self.pt], 0, self.n_pages - 1), pos % self.pt
        x = data[pg, part, :, sl]
        if self.fmt == 0:
            return R.from_bits(x, self.dtype)
        return R.e4m3_values()[x] * scales[pg, part, :, sl][..., None].astype(np.float64)

    def fill(self, scale=1.0, spoil=None):
        """Random K and V for every position, placed by the host (not by the operator under test)."""
        torch = _torch()
        H, D, pt = self.H, self.D, self.pt
        bits = _host(self.pool.pages).copy()
        per = self.pool.desc.page_elems
        for b, (_, L) in enumerate(self.lens):
            for part in (0, 1):
                x = self.rng.standard_normal((L, H, D)) * scale * np.exp(0.5 * self.rng.standard_normal((1, H, D)))
                if spoil is not None:
                    spoil(b, part, x)
                pos = np.arange(L)
                pg, sl = self.table[b, pos // pt], pos % pt
                pages = bits[:self.n_pages * per].reshape(self.n_pages, per)
                if self.fmt == 0:
                    view = pages[:, :2 * H * pt * D].reshape(-1, 2, H, pt, D)
                    view = np.lib.stride_tricks.as_strided(pages, (self.n_pages, 2, H, pt, D),
                                                           (per * 2, H * pt * D * 2, pt * D * 2, D * 2, 2))
                    view[pg, part, :, sl] = R.to_bits(x, self.dtype)
                else:
                    codes, sc = R.quantise(R.from_bits(R.to_bits(x, self.dtype), self.dtype))
                    by = pages.view(np.uint8)
                    view = np.lib.stride_tricks.as_strided(by, (self.n_pages, 2, H, pt, D),
                                                           (per * 2, H * pt * D, pt * D, D, 1))
                    view[pg, part, :, sl] = codes
                    sv = np.lib.stride_tricks.as_strided(by[:, 2 * H * pt * D:2 * H * pt * D + 4].view(np.float32),
                                                         (self.n_pages, 2, H, pt), (per * 2, H * pt * 4, pt * 4, 4))
                    sv[pg, part, :, sl] = sc
        self.pool.pages.view(torch.int16).copy_(torch.from_numpy(bits.view(np.int16)))

    def check(self):
        return G.slora_check_device(self.pool.h)


def _attend(c, q, hq, scale=None, window=0, max_rows=None, ldq=None, out=None, lse=None, stream=None, ws=None):
    torch = _torch()
    D = c.D
    scale = scale or 1 / math.sqrt(D)
    out = torch.full((q.shape[0], hq * D), 7.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((q.shape[0], hq), 7.0, device="cuda") if lse is None else lse
    max_rows = max_rows or max(1, max(n for n, _ in c.lens))
    if ws is None:
        size = G.slora_kv_attention_workspace_bytes(c.pool.h, c.layout, hq, len(c.lens), max(c.T, 1), max_rows)
        ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    G.slora_kv_attention(c.pool.h, c.layout, hq, q, ldq or hq * D, out, out.stride(0), lse, *c.batch(), max_rows, scale, window,
                         ws, stream)
    return out, lse


def _compare(c, qv, out, lse, hq, window=0, scale=None, seqs=None, once=False):
    """Every row of the given sequences against the definition, at the tolerance above."""
    D, dtype = c.D, c.dtype
    scale = scale or 1 / math.sqrt(D)
    got = R.from_bits(_host(out), dtype).reshape(-1, hq, D)
    gl = lse.double().cpu().numpy()
    for b, (n, L) in enumerate(c.lens):
        if n == 0 or (seqs is not None and b not in seqs):
            continue
        a = c.starts[b]
        q, K, V = qv[a:a + n].reshape(n, hq, D), c.rows(b, 0), c.rows(b, 1)
        want, wl, A, S = R.attention(q, K, V, L - n, scale, window)
        u = U[dtype]
        fine = lambda x: np.abs(np.where(np.isfinite(x), x, 0))  # noqa: E731
        kq = fine(q).max(initial=0) * fine(K).max(initial=0) * scale
        e = (D + 6) * 2.0 ** -23 * S[..., None] + 2.0 ** -21
        p = 2.0 ** -11 if c.fmt else u if once else 2.0 ** -16
        tol = u * np.abs(want) + A * (2 * e + p + 2 * (L + 8) * 2.0 ** -23) + L * 2.0 ** -25 * fine(V).max(initial=0) + 2.0 ** -24
        if c.fmt and dtype == "bf16":
            tol = tol + A * (2 * D * 2.0 ** -24 * kq)
        ltol = e[..., 0] + (L + 8) * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(wl)) + (D * 2.0 ** -24 * kq if c.fmt else 0)
        g, l = got[a:a + n], gl[a:a + n]
        assert np.array_equal(np.isnan(g), np.isnan(want)), (b, np.argwhere(np.isnan(g) != np.isnan(want))[:4])
        f = np.isfinite(want)
        with np.errstate(invalid="ignore"):
            bad = f & ~(np.abs(g - want) <= tol)
        assert not bad.any(), (b, n, L, np.argwhere(bad)[:4], g[bad][:4], want[bad][:4], np.broadcast_to(tol, g.shape)[bad][:4])
        f = np.isfinite(wl)
        assert np.array_equal(l[~f & ~np.isnan(wl)], wl[~f & ~np.isnan(wl)]), (b, l[~f], wl[~f])
        assert np.all(np.abs(l[f] - wl[f]) <= np.broadcast_to(ltol, l.shape)[f]), (b, np.abs(l[f] - wl[f]).max())


def _q(c, hq, seed=5, scale=1.0):
    rng = np.random.default_rng(seed)
    q = R.from_bits(R.to_bits(rng.standard_normal((max(c.T, 1), hq * c.D)) * scale, c.dtype), c.dtype)
    return q, _dev(q, c.dtype)


# ---------------------------------------------------------------------------
# write and read

LENS_W = [(1, 1), (5, 9), (0, 4), (33, 40), (1, 17), (2, 2)]


@pytest.mark.parametrize("dtype,fmt,H,D,pe", [("bf16", 0, 8, 128, 8192), ("f16", 0, 3, 64, 1024), ("bf16", 1, 8, 128, 8192),
                                               ("f16", 1, 5, 128, 4096), ("f16", 1, 32, 64, 8192), ("bf16", 1, 1, 64, 512),
                                               ("f16", 0, 32, 128, 8192)])
def test_write_is_bit_exact_and_touches_nothing_else(dtype, fmt, H, D, pe):
    torch = _torch()
    c = Cache(LENS_W, H, D, dtype, fmt, pe)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, c.T + 3, H, D)) * np.exp(rng.standard_normal((2, c.T + 3, H, 1)) * 2)
    x[0, 0, 0] = 0.0                      # a zero row
    x[0, 1, 0, :4] = [-0.0, 1e-7, -1e-7, 448.0]
    x = R.from_bits(R.to_bits(x, dtype), dtype)
    # scales that are powers of two and values on the borders between codes
    border = (R.e4m3_values()[1:127] + R.e4m3_values()[:126]) / 2
    x[1, 2, 0, :] = np.resize(border, D)
    x[1, 3, H - 1, :] = -np.resize(border[60:], D) * 2.0 ** -3
    x[1, 2, 0, 0], x[1, 3, H - 1, 0] = 448.0, 448.0 * 2.0 ** -3
    x = R.from_bits(R.to_bits(x, dtype), dtype)
    before, sbefore = (None if a is None else a.copy() for a in c.raw())
    ld = H * D + 24
    k, v = (torch.zeros(c.T + 3, ld, dtype=_tdt(dtype), device="cuda") for _ in range(2))
    k[:, :H * D], v[:, :H * D] = _dev(x[0].reshape(-1, H * D), dtype), _dev(x[1].reshape(-1, H * D), dtype)
    G.slora_kv_write(c.pool.h, c.layout, k, ld, v, ld, c.rs, c.kl, c.bl, c.ldb, len(c.lens), c.T + 3)
    assert c.check()[0] == 0
    want, swant = before, sbefore
    for b, (n, L) in enumerate(c.lens):
        for i in range(n):
            pos = L - n + i
            pg, sl = c.table[b, pos // c.pt], pos % c.pt
            for part in (0, 1):
                row = x[part, c.starts[b] + i]
                if fmt == 0:
                    want[pg, part, :, sl] = R.to_bits(row, dtype)
                else:
                    want[pg, part, :, sl], swant[pg, part, :, sl] = R.quantise(row)
    data, scales = c.raw()
    assert np.array_equal(data, want), np.argwhere(data != want)[:5]
    if fmt:
        assert np.array_equal(scales.view(np.uint32), swant.view(np.uint32))
    # and back
    k2, v2 = (torch.full((c.T + 3, ld), 3.0, dtype=_tdt(dtype), device="cuda") for _ in range(2))
    G.slora_kv_read(c.pool.h, c.layout, k2, ld, v2, ld, c.rs, c.kl, c.bl, c.ldb, len(c.lens), c.T + 3)
    assert c.check()[0] == 0
    for part, t in ((0, k2), (1, v2)):
        assert bool((t[c.T:] == 3.0).all()) and bool((t[:, H * D:] == 3.0).all())
        if fmt == 0:
            assert torch.equal(t[:c.T, :H * D], (k, v)[part][:c.T, :H * D])
        else:
            cd, sc = R.quantise(x[part, :c.T])
            exact = R.e4m3_values()[cd].astype(np.float32) * sc[..., None]   # one fp32 product ...
            assert np.array_equal(_host(t[:c.T, :H * D]), R.to_bits(exact.reshape(c.T, -1), dtype))  # ... one rounding


def test_quotients_next_to_a_border_take_the_exact_code():
    """Scales with long significands and values one 16-bit step around border * scale."""
    torch = _torch()
    H, D, n = 4, 128, 400
    c = Cache([(n, n)], H, D, "f16", 1, 8192)
    rng = np.random.default_rng(11)
    top = R.from_bits(R.to_bits(np.exp(rng.uniform(-3, 6, (n, H))), "f16"), "f16")
    scale = (top / 448.0).astype(np.float32).astype(np.float64)
    grid = R.e4m3_values()[:127]
    border = (grid[1:] + grid[:-1]) / 2
    near = border[rng.integers(0, 126, (n, H, D))] * scale[..., None]
    x = R.from_bits(R.to_bits(near * (1 + rng.integers(-2, 3, (n, H, D)) * 2.0 ** -11), "f16"), "f16")
    x = np.minimum(x, top[..., None]) * rng.choice([-1, 1], (n, H, D))
    x[..., 0] = top
    k = _dev(x.reshape(n, -1), "f16")
    G.slora_kv_write(c.pool.h, c.layout, k, H * D, k, H * D, *c.batch())
    codes, scales = c.raw()
    want, sw = R.quantise(x)
    pos = np.arange(n)
    got = codes[c.table[0, pos // c.pt], 0, :, pos % c.pt]
    assert np.array_equal(scales[c.table[0, pos // c.pt], 1, :, pos % c.pt], sw)
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


def _quantised(rows, dtype):
    """Writes (n, 128) values as one head's K rows; the codes and scales in the pages."""
    n = len(rows)
    c = Cache([(n, n)], 1, 128, dtype, 1, 32768)
    bits = R.to_bits(rows, dtype)
    k = _dev(rows, dtype)
    G.slora_kv_write(c.pool.h, c.layout, k, 128, k, 128, *c.batch())
    assert c.check()[0] == 0
    codes, scales = c.raw()
    pos = np.arange(n)
    pg, sl = c.table[0, pos // c.pt], pos % c.pt
    return R.from_bits(bits, dtype), codes[pg, 1, 0, sl], scales[pg, 1, 0, sl]


@pytest.mark.parametrize("shift", [-20, -138, 90])
def test_every_pair_of_bf16_significands(shift):
    """Each largest significand with every other one, 0 to 17 binades below it: ties where 7 divides either."""
    sig = np.arange(128.0, 256.0)
    rows = np.array([np.minimum(np.append(a * 2.0 ** (e + 1), sig[:127]), a * 2.0 ** (e + 1)) for e in range(18) for a in sig])
    x, codes, scales = _quantised(rows * 2.0 ** shift, "bf16")
    want, sw = R.quantise(x)
    assert np.array_equal(scales, sw) and np.array_equal(codes, want), np.argwhere(codes != want)[:5]


@pytest.mark.parametrize("shift", [-12, -24, 4])
def test_every_largest_fp16_significand(shift):
    """... with values at and around its borders, and random ones."""
    rng = np.random.default_rng(shift + 100)
    top = np.arange(1024.0, 2048.0).repeat(4)[:, None]
    grid = R.e4m3_values()[:127]
    border = ((grid[1:] + grid[:-1]) / 2)[rng.integers(0, 126, (len(top), 64))] * top / 448
    rows = np.concatenate([top, border, rng.uniform(0, 1, (len(top), 63)) * top], 1) * rng.choice([-1, 1], (len(top), 128))
    x, codes, scales = _quantised(rows * 2.0 ** shift, "f16")
    want, sw = R.quantise(x)
    assert np.array_equal(scales, sw) and np.array_equal(codes, want), np.argwhere(codes != want)[:5]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rows_that_are_not_finite_or_tiny(dtype):
    torch = _torch()
    H, D = 2, 64
    c = Cache([(6, 6)], H, D, dtype, 1, 4096)
    x = np.random.default_rng(0).standard_normal((6, H, D))
    x[0, 0, 5], x[1, 0, 9], x[2, 1, 63] = np.inf, -np.inf, np.nan
    tiny = 2.0 ** -24 if dtype == "f16" else 2.0 ** -133
    x[3, 0] = tiny * np.arange(D) / 8
    x[4, 0] = tiny
    x[5, 1] *= 60000 if dtype == "f16" else 1e38
    bits = R.to_bits(x, dtype)
    x = R.from_bits(bits, dtype)
    k = _dev(x.reshape(6, -1), dtype)
    G.slora_kv_write(c.pool.h, c.layout, k, H * D, k, H * D, *c.batch())
    codes, scales = c.raw()
    pos = np.arange(6)
    pg = c.table[0, pos // c.pt]
    want, sw = R.quantise(x)
    assert np.array_equal(codes[pg, 0, :, pos % c.pt], want)
    got = scales[pg, 0, :, pos % c.pt]
    assert np.array_equal(np.isnan(got), np.isnan(sw)) and np.array_equal(got[~np.isnan(sw)], sw[~np.isnan(sw)])
    assert np.array_equal(np.isnan(sw), ~np.isfinite(x).all(-1)) and np.isnan(sw).sum() >= 3
    back = torch.zeros_like(k)
    G.slora_kv_read(c.pool.h, c.layout, back, H * D, torch.zeros_like(k), H * D, *c.batch())
    nan = torch.isnan(back.view(6, H, D)).cpu().numpy()
    assert np.array_equal(nan, np.broadcast_to(np.isnan(sw)[..., None], nan.shape))


def test_write_and_read_skip_what_they_must():
    """Bad sequences and pages are recorded and skipped, negative positions passed over, the rest done."""
    torch = _torch()
    H, D = 2, 64
    lens = [(3, 5), (4, 9), (2, 7), (1, 3)]
    for case, code, info in [("page", 9, 1), ("row", 8, 2), ("len", 8, 1), ("neg", 0, 0), ("low", 9, 3)]:
        c = Cache(lens, H, D, "bf16", 0, 512)
        assert c.pt == 2
        touched = np.ones(c.T, bool)
        if case == "page":
            c.table[1, 4] = c.n_pages      # positions 8, of rows 5..8
            touched[3 + 3] = False
        elif case == "low":
            c.table[3, 1] = -1
            touched[9] = False
        elif case == "row":
            c.starts[3] = c.T + 5          # sequence 2 ends outside; 3 starts there
            touched[7:] = False
        elif case == "len":
            c.lens[1] = (4, c.ldb * c.pt + 1)
            touched[3:7] = False
        else:
            c.lens[0] = (3, 1)             # positions -2, -1, 0
            touched[:2] = False
        c.upload()
        x = torch.randn(c.T, H * D, device="cuda").to(torch.bfloat16)
        G.slora_kv_write(c.pool.h, c.layout, x, H * D, -x, H * D, *c.batch())
        st = c.check()
        assert (st[0] == 6) == (code != 0) and st[1] == code, (case, st)
        if case != "row":
            assert st[2] == (info if code else 0), (case, st)
        k, v = (torch.full_like(x, 5.0) for _ in range(2))
        G.slora_kv_read(c.pool.h, c.layout, k, H * D, v, H * D, *c.batch())
        assert c.check()[1] == code
        for t in range(c.T):
            if touched[t]:
                assert torch.equal(k[t], x[t]) and torch.equal(v[t], -x[t]), (case, t)
            else:
                assert bool((k[t] == 5.0).all()) and bool((v[t] == 5.0).all()), (case, t)


def test_read_of_any_range():
    torch = _torch()
    c = Cache([(0, 50)], 2, 64, "f16", 0, 1024)
    c.fill()
    K, V = c.rows(0, 0), c.rows(0, 1)
    for a, e in [(0, 50), (13, 14), (7, 31), (49, 50), (0, 1)]:
        k, v = (torch.zeros(e - a, 128, dtype=torch.float16, device="cuda") for _ in range(2))
        rs, kl = torch.tensor([0, e - a], dtype=torch.int32).cuda(), torch.tensor([e], dtype=torch.int32).cuda()
        G.slora_kv_read(c.pool.h, c.layout, k, 128, v, 128, rs, kl, c.bl, c.ldb, 1, e - a)
        assert np.array_equal(R.from_bits(_host(k), "f16").reshape(-1, 2, 64), K[a:e])
        assert np.array_equal(R.from_bits(_host(v), "f16").reshape(-1, 2, 64), V[a:e])


# ---------------------------------------------------------------------------
# attention

CASES = [
    # lens, H, G, D, dtype, fmt, page elements, window
    ([(1, 1)], 1, 1, 64, "f16", 0, 512, 0),
    ([(1, 37)], 32, 1, 128, "f16", 0, 8192, 0),
    ([(1, 5), (1, 64), (1, 65), (1, 1), (1, 700), (0, 9), (1, 128)], 8, 4, 128, "bf16", 0, 8192, 0),
    ([(1, 300), (1, 2), (1, 63)], 2, 8, 128, "bf16", 1, 8192, 0),
    ([(1, 300), (1, 2), (1, 63), (1, 4000)], 4, 1, 64, "f16", 1, 16384, 0),
    ([(1, 3000)], 1, 7, 128, "f16", 0, 4096, 0),
    ([(1, 3001)], 2, 3, 64, "bf16", 1, 2048, 0),
    ([(5, 40), (3, 3), (8, 200), (1, 77), (2, 65)], 4, 4, 128, "bf16", 0, 16384, 0),
    ([(5, 40), (3, 3), (8, 200), (1, 77), (2, 65)], 3, 5, 64, "f16", 0, 2048, 0),
    ([(4, 500), (9, 61), (11, 128)], 2, 7, 128, "f16", 1, 8192, 0),
    ([(40, 40), (17, 300), (1, 90), (64, 65)], 2, 4, 128, "bf16", 0, 8192, 0),
    ([(130, 400), (1, 90), (33, 33)], 2, 2, 64, "bf16", 1, 8192, 0),
    ([(1, 500), (6, 300), (70, 200)], 2, 4, 128, "f16", 0, 8192, 100),
    ([(1, 500), (6, 300), (70, 200), (1, 3)], 2, 4, 64, "bf16", 1, 8192, 1),
    ([(1, 700), (20, 640)], 1, 16, 128, "bf16", 0, 8192, 64),
    ([(3, 1), (2, 0), (4, 4), (70, 30)], 2, 2, 128, "bf16", 0, 8192, 0),       # rows before the first token
    ([(1, 40), (2, 90)], 2, 33, 64, "f16", 0, 4096, 0),
    ([(2, 66)], 1, 130, 64, "bf16", 0, 4096, 0),
]


@pytest.mark.parametrize("lens,H,group,D,dtype,fmt,pe,window", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(lens, H, group, D, dtype, fmt, pe, window):
    torch = _torch()
    c = Cache(lens, H, D, dtype, fmt, pe, seed=len(lens))
    c.fill()
    hq = H * group
    qv, q = _q(c, hq)
    out, lse = _attend(c, q, hq, window=window)
    assert c.check()[0] == 0
    _compare(c, qv, out, lse, hq, window, once=max(n for n, _ in lens) * group > 32)
    # the same bits again, and without lse
    again, lse2 = _attend(c, q, hq, window=window)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n,group,D,fmt,B", [(1, 1, 128, 0, 100), (1, 8, 128, 1, 100), (1, 8, 64, 0, 100), (2, 8, 64, 1, 100),
                                             (4, 8, 128, 0, 80), (5, 8, 64, 1, 80), (5, 8, 128, 1, 60), (9, 8, 128, 0, 50),
                                             (9, 8, 64, 1, 50)])
def test_attention_many_short_items_per_cta(n, group, D, fmt, B):
    """Several items of one to three key tiles in each CTA's run, so that all roles are items apart."""
    rng = np.random.default_rng(n * group + D)
    lens = [(n, n + int(np.exp(rng.uniform(0, np.log(330))))) for _ in range(B)]
    H = 6
    c = Cache(lens, H, D, "f16", fmt, 16384)
    c.fill()
    qv, q = _q(c, H * group)
    out, lse = _attend(c, q, H * group)
    assert c.check()[0] == 0
    _compare(c, qv, out, lse, H * group, once=n * group > 32)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows", [4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49])
def test_attention_at_the_borders_of_row_tiles(rows, fmt):
    for n, group in {(1, rows), (rows, 1)}:
        c = Cache([(n, 300), (1, 70)], 2, 64, "bf16", fmt, 4096)
        c.fill()
        qv, q = _q(c, 2 * group)
        out, lse = _attend(c, q, 2 * group)
        assert c.check()[0] == 0
        _compare(c, qv, out, lse, 2 * group, once=rows > 32)


@pytest.mark.parametrize("n,group,D,fmt", [(1, 2, 64, 0), (3, 2, 128, 1), (40, 2, 64, 0)])
def test_attention_one_item_over_every_cta(n, group, D, fmt):
    """A partial from each CTA: more of them than a warp has lanes."""
    c = Cache([(n, 40000)], 1, D, "bf16", fmt, 65536)
    c.fill()
    qv, q = _q(c, group)
    out, lse = _attend(c, q, group)
    assert c.check()[0] == 0
    _compare(c, qv, out, lse, group, once=n * group > 32)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("group", [2, 20])
def test_rows_that_see_nothing_beside_infinities(group, fmt):
    """Rows before the first token get 0 and -inf whatever the item's V rows hold."""
    def spoil(b, part, x):
        if part:
            x[0, :, 3], x[1, 0, 7] = np.inf, np.nan
    c = Cache([(6, 4), (2, 300)], 2, 64, "bf16", fmt, 4096)
    c.fill(spoil=spoil)
    qv, q = _q(c, 2 * group)
    out, lse = _attend(c, q, 2 * group)
    assert bool((out[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())
    _compare(c, qv, out, lse, 2 * group, once=True)


@pytest.mark.parametrize("fmt,D", [(0, 128), (1, 128), (0, 64)])
@pytest.mark.parametrize("lens", [[(1292, 1684), (1377, 1773), (1484, 1893), (1413, 1851)], [(90, 300), (97, 220), (130, 480)] * 5])
def test_chunks_whose_last_row_tile_is_small(lens, fmt, D):
    """Row tiles of 256 rows and one of 14 to 143 in turn, over keys that end inside a tile: one softmax group passes
    over the small ones and comes to the next item before its barriers are there."""
    torch = _torch()
    H, group = 8, 3
    c = Cache(lens, H, D, "bf16", fmt, 2048)
    c.fill()
    qv, q = _q(c, H * group)
    out, lse = _attend(c, q, H * group)
    assert c.check()[0] == 0
    _compare(c, qv, out, lse, H * group, seqs=[0, 2], once=True)
    n = max(n for n, _ in lens)
    ws = torch.empty(G.slora_kv_attention_workspace_bytes(c.pool.h, c.layout, H * group, len(lens), c.T, n), dtype=torch.uint8,
                     device="cuda")
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    for _ in range(30):  # with the cache and the queue warm: nothing but these calls
        _attend(c, q, H * group, out=again, lse=lse2, ws=ws)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1, (1 << 30) - 1])
def test_the_largest_windows_beside_rows_before_the_first_token(window):
    c = Cache([(6, 4), (1, 300), (40, 33)], 2, 64, "bf16", 0, 4096)
    c.fill()
    qv, q = _q(c, 4)
    out, lse = _attend(c, q, 4, window=window)
    assert c.check()[0] == 0
    _compare(c, qv, out, lse, 4, once=True)


@pytest.mark.parametrize("group,n", [(1, 1), (8, 2), (8, 40)])
def test_attention_where_every_sequence_fits_one_tile(group, n):
    """A table of at most 128 positions, at 128 and below: nothing is joined."""
    for longest in (128, 127):
        c = Cache([(n, longest), (1, 1), (n, n)], 2, 128, "f16", 0, 512)
        assert c.pt == 1 or c.ldb * c.pt >= longest
        c.fill()
        qv, q = _q(c, 2 * group)
        out, lse = _attend(c, q, 2 * group)
        assert c.check()[0] == 0
        _compare(c, qv, out, lse, 2 * group, once=n * group > 32)


@pytest.mark.parametrize("fmt", [0, 1])
def test_attention_large_scores_and_values(fmt):
    """Scores of several hundred (all weight on one key), values near the type's largest."""
    c = Cache([(1, 200), (3, 77)], 2, 128, "bf16", fmt, 8192)
    c.fill(scale=30.0)
    qv, q = _q(c, 4, scale=30.0)
    out, lse = _attend(c, q, 4)
    _compare(c, qv, out, lse, 4)
    c = Cache([(1, 200), (3, 77)], 2, 64, "f16", fmt, 8192)
    c.fill(spoil=lambda b, part, x: np.copyto(x, np.sign(x) * 60000.0 if part else x))
    qv, q = _q(c, 4)
    out, lse = _attend(c, q, 4)
    _compare(c, qv, out, lse, 4)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_tiny_values_in_8_bits(dtype):
    """V rows of very different sizes: the weights carry the row scales."""
    c = Cache([(1, 150), (3, 77)], 2, 64, dtype, 1, 8192)
    size = 10.0 ** np.random.default_rng(4).uniform(-4, 3, 200)

    def spoil(b, part, x):
        if part:
            x *= size[:x.shape[0], None, None]
    c.fill(spoil=spoil)
    qv, q = _q(c, 4)
    out, lse = _attend(c, q, 4)
    _compare(c, qv, out, lse, 4)


@pytest.mark.parametrize("lens,window,group", [([(6, 40), (1, 20)], 0, 2), ([(6, 300), (1, 200)], 50, 2), ([(100, 300), (40, 900)], 0, 4),
                                               ([(100, 300), (40, 900)], 70, 4)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_masked_keys_have_no_influence_whatever_they_hold(lens, window, group, fmt):
    """NaN and infinities in K and V at positions that some rows see and others do not."""
    H, D = 2, 64
    c = Cache(lens, H, D, "bf16", fmt, 4096)

    def spoil(b, part, x):
        n, L = lens[b]
        if b == 0:
            x[L - 2, 0, 3] = np.nan if part else 1.0      # seen by the last two rows only
            x[L - 3, 1, 4] = np.inf if part else 1.0
        if window:
            x[max(0, L - n - window)] = np.nan            # just before the first row's window
        if not part and b == 0:
            x[L - 1, 1, 5] = np.nan                       # K: seen by the last row only
    c.fill(spoil=spoil)
    qv, q = _q(c, H * group)
    out, lse = _attend(c, q, H * group, window=window)
    assert c.check()[0] == 0
    got = R.from_bits(_host(out), "bf16").reshape(-1, H * group, D)
    n = lens[0][0]
    assert not np.isnan(got[:n - 3]).any() and np.isnan(got[n - 1, :group, 3]).all()
    _compare(c, qv, out, lse, H * group, window, once=n * group > 32)


def test_bad_sequences_and_pages_are_left_out():
    torch = _torch()
    H, D, hq = 2, 64, 4
    base = [(3, 5), (4, 90), (2, 7), (1, 300), (80, 100)]

    def run(change, code, info, max_rows=None):
        c = Cache(list(base), H, D, "bf16", 0, 2048, ldb=40)
        c.fill()
        qv, q = _q(c, hq)
        change(c)
        c.upload()
        out, lse = _attend(c, q, hq, max_rows=max_rows)
        st = c.check()
        assert st[0] == 6 and st[1] == code and (info is None or st[2] == info), st
        return c, qv, out, lse

    def same(out, lse, a, e):
        return bool((out[a:e] == 7.0).all()) and bool((lse[a:e] == 7.0).all())

    c, qv, out, lse = run(lambda c: c.lens.__setitem__(3, (1, 40 * c.pt + 1)), 8, 3)
    assert same(out, lse, 9, 10)
    _compare(c, qv, out, lse, hq, seqs=[0, 1, 2, 4], once=True)
    c, qv, out, lse = run(lambda c: c.lens.__setitem__(1, (4, -2)), 8, 1)
    assert same(out, lse, 3, 7)
    _compare(c, qv, out, lse, hq, seqs=[0, 2, 3, 4], once=True)
    c, qv, out, lse = run(lambda c: None, 8, 4, max_rows=79)
    assert same(out, lse, 10, 90)
    _compare(c, qv, out, lse, hq, seqs=[0, 1, 2, 3])
    c, qv, out, lse = run(lambda c: c.starts.__setitem__(5, 91), 8, 4)
    assert same(out, lse, 10, 90)
    _compare(c, qv, out, lse, hq, seqs=[0, 1, 2, 3], once=True)
    for bad in (-1, 10 ** 9, -(2 ** 31)):
        def change(c):
            c.table[3, 2] = bad
        c, qv, out, lse = run(change, 9, 3)
        _compare(c, qv, out, lse, hq, seqs=[0, 1, 2, 4], once=True)
        # sequence 3: as if the keys of that page were not there
        K, V = (np.delete(x, np.s_[2 * c.pt:3 * c.pt], 0) for x in (c.rows(3, 0), c.rows(3, 1)))
        want, wl, A, S = R.attention(qv[9:10].reshape(1, hq, D), K, V, K.shape[0] - 1, 1 / math.sqrt(D), 0)
        got = R.from_bits(_host(out[9:10]), "bf16").reshape(1, hq, D)
        assert np.all(np.abs(got - want) <= U["bf16"] * np.abs(want) + A * 2.0 ** -7)


def test_rows_of_no_sequence_are_left_alone_and_nothing_is_nothing():
    torch = _torch()
    c = Cache([(2, 20), (1, 9)], 2, 64, "f16", 0, 2048)
    c.fill()
    c.starts += 3                       # rows 0..2 and the last two belong to nobody
    T = c.T = c.T + 5
    c.upload()
    qv, q = _q(c, 4)
    out, lse = _attend(c, q, 4)
    assert c.check()[0] == 0
    _compare(c, qv, out, lse, 4)
    for rows in (slice(0, 3), slice(6, T)):
        assert bool((out[rows] == 7.0).all()) and bool((lse[rows] == 7.0).all())
    for B, TT in ((0, T), (2, 0)):
        G.slora_kv_attention(c.pool.h, c.layout, 4, q, 256, out, 256, lse, c.rs, c.kl, c.bl, c.ldb, B, TT, 1, 1.0, 0,
                             torch.empty(1 << 26, dtype=torch.uint8, device="cuda"))
        G.slora_kv_write(c.pool.h, c.layout, q, 256, q, 256, c.rs, c.kl, c.bl, c.ldb, B, TT)
    before = out.clone()
    torch.cuda.synchronize()
    assert torch.equal(before, out) and c.check()[0] == 0


@pytest.mark.parametrize("fmt,lens", [(0, [(1, 100), (3, 60)]), (1, [(1, 100), (40, 60)])])
def test_strided_rows_of_a_fused_projection(fmt, lens):
    """q, k, v as slices of one (T, (Hq + 2 H) * D) tensor, out with a stride of its own."""
    torch = _torch()
    H, hq, D = 2, 6, 128
    c = Cache(lens, H, D, "bf16", fmt, 8192)
    c.fill()
    w = (hq + 2 * H) * D
    x = np.random.default_rng(9).standard_normal((c.T, w))
    x = R.from_bits(R.to_bits(x, "bf16"), "bf16")
    qkv = _dev(x, "bf16")
    k, v = qkv[:, hq * D:], qkv[:, (hq + H) * D:]
    G.slora_kv_write(c.pool.h, c.layout, k, w, v, w, *c.batch())
    wide = torch.full((c.T, hq * D + 64), 2.0, dtype=torch.bfloat16, device="cuda")
    out, lse = _attend(c, qkv, hq, ldq=w, out=wide)
    assert c.check()[0] == 0
    assert bool((wide[:, hq * D:] == 2.0).all())
    if fmt == 0:
        a = c.starts[1]
        assert np.array_equal(c.rows(1, 0)[-lens[1][0]:].reshape(-1, H * D), x[a:, hq * D:(hq + H) * D])
    _compare(c, x[:, :hq * D], wide[:, :hq * D].contiguous(), lse, hq, once=lens[1][0] * 3 > 32)


def test_shared_prefix_pages():
    """Two sequences over the same first pages."""
    torch = _torch()
    c = Cache([(1, 40), (2, 40)], 2, 64, "f16", 0, 2048)
    c.fill()
    c.table[1, :3] = c.table[0, :3]
    c.upload()
    qv, q = _q(c, 4)
    out, lse = _attend(c, q, 4)
    _compare(c, qv, out, lse, 4)


def test_offsets_beyond_32_bits():
    """Pages whose element offsets pass 2^32."""
    torch = _torch()
    H, D, pe = 2, 128, 1 << 20
    for fmt in (0, 1):
        c = Cache([(2, 5000), (1, 30)], H, D, "bf16", fmt, pe, extra_pages=4200)
        top = c.n_pages - 1
        used = {int(p): top - i for i, p in enumerate(sorted(set(c.table[c.table >= 0].tolist())))}
        c.table = np.vectorize(lambda p: used.get(int(p), -1))(c.table).astype(np.int32)
        c.upload()
        assert min(used.values()) * pe > 2 ** 32
        rng = np.random.default_rng(1)
        kv = R.from_bits(R.to_bits(rng.standard_normal((2, 5030, H * D)), "bf16"), "bf16")
        k, v = _dev(kv[0], "bf16"), _dev(kv[1], "bf16")
        rs = torch.tensor([0, 5000, 5030], dtype=torch.int32).cuda()
        G.slora_kv_write(c.pool.h, c.layout, k, H * D, v, H * D, rs, c.kl, c.bl, c.ldb, 2, 5030)
        k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
        G.slora_kv_read(c.pool.h, c.layout, k2, H * D, v2, H * D, rs, c.kl, c.bl, c.ldb, 2, 5030)
        qv, q = _q(c, 4)
        out, lse = _attend(c, q, 4)
        assert c.check()[0] == 0
        if fmt == 0:
            assert torch.equal(k, k2) and torch.equal(v, v2)
        cache = [R.from_bits(_host(t), "bf16").reshape(-1, H, D) for t in (k2, v2)]
        if fmt:
            cache = [R.e4m3_values()[cd] * sc[..., None].astype(np.float64)
                     for cd, sc in (R.quantise(x.reshape(-1, H, D)) for x in kv)]
        c.rows = lambda b, part: cache[part][0:5000] if b == 0 else cache[part][5000:5030]
        _compare(c, qv, out, lse, 4)
        c.pool.close()
        del c
        torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", [0, 1])
def test_captured_calls_follow_the_arrays_on_the_device(fmt):
    """One graph of write + attention, replayed as the sequences grow; another graph with a workspace of its own."""
    torch = _torch()
    H, D, hq, B = 2, 64, 4, 3
    c = Cache([(1, 120)] * B, H, D, "bf16", fmt, 2048)
    c.fill()
    kl = torch.tensor([60, 1, 100], dtype=torch.int32).cuda()
    c.kl = kl
    bufs = [torch.zeros(B, n * D, dtype=torch.bfloat16, device="cuda") for n in (hq, H, H, hq)]
    lse = torch.zeros(B, hq, device="cuda")
    size = G.slora_kv_attention_workspace_bytes(c.pool.h, c.layout, hq, B, B, 1)
    work = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()

    def step(ws):
        G.slora_kv_write(c.pool.h, c.layout, bufs[1], H * D, bufs[2], H * D, *c.batch(), s)
        G.slora_kv_attention(c.pool.h, c.layout, hq, bufs[0], hq * D, bufs[3], hq * D, lse, *c.batch(), 1, 0.125, 0, ws, s)

    with torch.cuda.stream(s):
        step(work[0])
    s.synchronize()
    graphs = []
    for ws in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(ws)
        graphs.append(g)
    rng = np.random.default_rng(2)
    for it in range(6):
        new = [rng.standard_normal((B, n * D)) for n in (hq, H, H)]
        for t, x in zip(bufs, new):
            t.copy_(_dev(x, "bf16"))
        kl += torch.tensor([1, 2, 3], dtype=torch.int32).cuda()
        torch.cuda.synchronize()
        graphs[it & 1].replay()
        torch.cuda.synchronize()
        assert c.check()[0] == 0
        c.lens = [(1, int(x)) for x in kl.cpu()]
        qv = R.from_bits(_host(bufs[0]), "bf16")
        _compare(c, qv, bufs[3], lse, hq, scale=0.125)
        if fmt == 0:
            assert np.array_equal(c.rows(2, 1)[-1].reshape(-1), R.from_bits(_host(bufs[2]), "bf16")[2])


def test_calls_side_by_side_on_two_streams():
    torch = _torch()
    c = Cache([(1, 900), (30, 400)], 2, 128, "bf16", 0, 8192)
    c.fill()
    qv, q = _q(c, 8)
    ref, lref = _attend(c, q, 8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    size = G.slora_kv_attention_workspace_bytes(c.pool.h, c.layout, 8, 2, c.T, 30)
    got = []
    for s in streams * 5:
        with torch.cuda.stream(s):
            ws = torch.empty(size, dtype=torch.uint8, device="cuda")
            got.append((*_attend(c, q, 8, stream=s, ws=ws), ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) and torch.equal(l, lref) for o, l, _ in got)


def test_phase_events_bracket_the_calls():
    torch = _torch()
    c = Cache([(1, 100)], 2, 64, "f16", 0, 2048)
    c.fill()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ev:
        e.record()
    _, q = _q(c, 4)
    G.slora_set_phase_events(c.pool.h, ev)
    _attend(c, q, 4, stream=torch.cuda.current_stream())
    G.slora_set_phase_events(c.pool.h, [])
    torch.cuda.synchronize()
    assert 0 < ev[0].elapsed_time(ev[1]) < 1000


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [0, 1])
def test_a_layer_of_decode_with_adapters(fmt):
    """q, k, v deltas -> cache write -> attention -> o delta, over a prompt chunk, decode steps and drafted
    tokens, adapters and KV pages in one pool; each step against the 64-bit definition from the step's own inputs."""
    import oracle
    torch = _torch()
    H, hq, D, dtype, r = 2, 4, 64, "bf16", 8
    hid = 256
    d_in, d_out = [hid] * 3 + [hq * D], [hq * D, H * D, H * D, hid]
    rng = np.random.default_rng(21)
    pool = G.Pool(G.SLORA_BF16, d_in, d_out, 4, r, 64, 4096, 200)
    A_t = [[R.to_bits(rng.standard_normal((r, d)) / math.sqrt(d), dtype) for d in d_in] for _ in range(3)]
    Bm = [[R.to_bits(rng.standard_normal((r, d)) / math.sqrt(r), dtype) for d in d_out] for _ in range(3)]
    for a in range(3):
        pool.register(a, r, 16.0, A_t[a], Bm[a])
    pool.page_in([0, 1, 2])
    layout = G.make_kv_layout(H, D, fmt)
    pt = G.slora_kv_page_tokens(pool.h, layout)
    n_seq, most = 3, 80
    per = -(-most // pt)
    table = np.array(pool.kv_alloc(n_seq * per), np.int32).reshape(n_seq, per)
    bl = torch.from_numpy(table).cuda()
    size = G.slora_kv_attention_workspace_bytes(pool.h, layout, hq, n_seq, 64, 64)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    lens = np.zeros(n_seq, np.int32)
    held = [[np.zeros((0, H, D)) for _ in range(2)] for _ in range(n_seq)]
    for new in ([30, 17, 5], [1, 1, 1], [1, 1, 1], [4, 0, 2], [1, 1, 1]):
        T = sum(new)
        lens += np.array(new, np.int32)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        G.slora_kv_check_batch(pool.h, layout, starts, lens, table, T)
        idx_np = np.repeat(np.arange(n_seq), new).astype(np.int32)
        idx = torch.from_numpy(idx_np).cuda()
        x = rng.standard_normal((T, hid))
        ys = [rng.standard_normal((T, d)) for d in d_out]
        dx = _dev(x, dtype)
        dy = [_dev(y, dtype) for y in ys]
        rs, kl = torch.from_numpy(starts).cuda(), torch.from_numpy(lens.copy()).cuda()
        G.slora_lora_delta(pool.h, [0, 1, 2], [dx] * 3, [hid] * 3, dy[:3], d_out[:3], idx, T)
        batch = (rs, kl, bl, per, n_seq, T)
        G.slora_kv_write(pool.h, layout, dy[1], H * D, dy[2], H * D, *batch)
        att = torch.empty(T, hq * D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, hq, device="cuda")
        G.slora_kv_attention(pool.h, layout, hq, dy[0], hq * D, att, hq * D, lse, *batch, max(new), 1 / math.sqrt(D), 0, ws)
        G.slora_lora_delta(pool.h, [3], [att], [hq * D], [dy[3]], [hid], idx, T)
        k2, v2 = torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
        G.slora_kv_read(pool.h, layout, k2, H * D, v2, H * D, *batch)
        assert G.slora_check_device(pool.h)[0] == 0
        q, k, v = (R.from_bits(_host(t), dtype) for t in dy[:3])
        ref = oracle.lora_delta(1, R.to_bits(x, dtype), idx_np, R.to_bits(ys[1], dtype), np.full(3, r, np.int32),
                                np.full(3, 16.0), [A_t[a][1] for a in range(3)], [Bm[a][1] for a in range(3)])
        assert np.all(np.abs(k - ref) <= 2.0 ** -7 * np.abs(ref).max())
        for b in range(n_seq):
            a, n = starts[b], new[b]
            for part, t in ((0, k), (1, v)):
                rows = t[a:a + n].reshape(n, H, D)
                if fmt:
                    cd, sc = R.quantise(rows)
                    rows = R.e4m3_values()[cd] * sc[..., None].astype(np.float64)
                held[b][part] = np.concatenate([held[b][part], rows])
                back = R.from_bits(_host((k2, v2)[part]), dtype)[a:a + n].reshape(n, H, D)
                assert np.all(np.abs(back - rows) <= 2.0 ** -8 * np.abs(rows) * 1.0001)
            if n:
                want, wl, A, S = R.attention(q[a:a + n].reshape(n, hq, D), *held[b], lens[b] - n, 1 / math.sqrt(D), 0)
                got = R.from_bits(_host(att), dtype)[a:a + n].reshape(n, hq, D)
                e = (D + 6) * 2.0 ** -23 * S[..., None] + 2.0 ** -21
                tol = 2.0 ** -8 * np.abs(want) + A * (2 * e + 2.0 ** -8 + 2.0 ** -14) + 2.0 ** -18
                assert np.all(np.abs(got - want) <= tol)
                assert np.all(np.abs(lse.double().cpu().numpy()[a:a + n] - wl) <= e[..., 0] + 2.0 ** -15 * (1 + np.abs(wl)))
        ref = oracle.lora_delta(1, _host(att), idx_np, R.to_bits(ys[3], dtype), np.full(3, r, np.int32), np.full(3, 16.0),
                                [A_t[a][3] for a in range(3)], [Bm[a][3] for a in range(3)])
        assert np.all(np.abs(R.from_bits(_host(dy[3]), dtype) - ref) <= 2.0 ** -7 * np.abs(ref).max())
    pool.kv_free(table.reshape(-1).tolist())
    pool.close()

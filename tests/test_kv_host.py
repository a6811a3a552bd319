"""KV-cache operators without a GPU: sizes, refusals, and the host-side check
of a batch, on host_only pools; the reference quantiser against torch's e4m3."""
import ctypes

import numpy as np
import pytest

import gather_lora_paged_b200 as G
import kv_reference as R

SIZES = [(8192, 32, 128, 0, 1), (32768, 8, 128, 0, 16), (8192, 8, 128, 1, 7), (32768, 32, 128, 1, 7), (512, 2, 64, 0, 2),
         (512, 1, 64, 1, 7), (16384, 4, 64, 1, 60), (512, 8, 128, 0, 0), (1024, 5, 64, 0, 1)]


def _pool(page_elems=8192, n_pages=64, max_tokens=512, dtype=G.SLORA_BF16):
    return G.Pool(dtype, [64], [64], 4, 8, max_tokens, page_elems, n_pages, host_only=True)


def test_layout_struct_matches_header():
    assert ctypes.sizeof(G.KvLayout) == 32 and G.KvLayout.head_dim.offset == 8


@pytest.mark.parametrize("pe,heads,dim,fmt,want", SIZES)
def test_page_tokens(pe, heads, dim, fmt, want):
    P = _pool(pe)
    assert G.slora_kv_page_tokens(P.h, G.make_kv_layout(heads, dim, fmt)) == want
    row = 2 * dim if fmt == 0 else dim + 4
    assert want * 2 * heads * row <= 2 * pe < (want + 1) * 2 * heads * row


@pytest.mark.parametrize("layout", [(0, 128, 0), (257, 128, 0), (8, 96, 0), (8, 128, 2), (8, 128, -1)])
def test_page_tokens_of_bad_layouts(layout):
    P = _pool()
    assert G.slora_kv_page_tokens(P.h, G.make_kv_layout(*layout)) == 0


GOOD = dict(layout=(8, 128, 0), hq=32, ldk=1024, ldv=1024, ldq=4096, ldo=4096, B=2, T=5, ldb=4, max_rows=3, scale=0.1, window=0,
            k=1 << 20, v=2 << 20, q=3 << 20, out=4 << 20, lse=5 << 20, rs=6 << 20, kl=7 << 20, bl=8 << 20, ws=9 << 20,
            size=1 << 40)


def _call(P, which, a):
    L = G.make_kv_layout(*a["layout"])
    batch = (a["rs"], a["kl"], a["bl"], a["ldb"], a["B"], a["T"])
    if which == "attention":
        return G.lib().slora_kv_attention(P.h, L, a["hq"], a["q"], a["ldq"], a["out"], a["ldo"], a["lse"], *batch,
                                          a["max_rows"], a["scale"], a["window"], a["ws"], a["size"], None)
    f = G.lib().slora_kv_write if which == "write" else G.lib().slora_kv_read
    return f(P.h, L, a["k"], a["ldk"], a["v"], a["ldv"], *batch, None)


@pytest.mark.parametrize("which", ["write", "read", "attention"])
def test_a_good_call_reaches_the_device_check(which):
    P = _pool(32768)
    assert _call(P, which, GOOD) == 9  # host_only: UNSUPPORTED, after every argument check


BAD_ALL = [("layout", (8, 96, 0), 9), ("layout", (0, 128, 0), 1), ("layout", (300, 128, 0), 1), ("layout", (8, 128, 7), 1),
           ("layout", (200, 128, 0), 1), ("B", -1, 1), ("T", -1, 1), ("T", 513, 1), ("ldb", -1, 1), ("rs", None, 1),
           ("kl", None, 1), ("bl", None, 1), ("rs", (6 << 20) + 2, 1), ("kl", (7 << 20) + 1, 1), ("bl", (8 << 20) + 3, 1)]
BAD_ROWS = [("k", None, 1), ("v", None, 1), ("k", (1 << 20) + 8, 1), ("v", (2 << 20) + 2, 1), ("ldk", 1016, 1), ("ldv", 1028, 1)]
BAD_ATT = [("hq", 0, 1), ("hq", 12, 1), ("hq", 2048, 1), ("q", None, 1), ("out", None, 1), ("q", (3 << 20) + 4, 1),
           ("out", 3 << 20, 1), ("ldq", 4088, 1), ("ldo", 4100, 1), ("max_rows", 0, 1), ("max_rows", -1, 1), ("scale", 0.0, 1),
           ("scale", -1.0, 1), ("scale", float("nan"), 1), ("scale", float("inf"), 1), ("window", -1, 1),
           ("lse", (5 << 20) + 2, 1), ("ws", None, 1), ("ws", (9 << 20) + 8, 1), ("size", 100, 1)]


@pytest.mark.parametrize("which,name,value,status",
                         [(w, *b) for w in ("write", "read", "attention") for b in BAD_ALL] +
                         [(w, *b) for w in ("write", "read") for b in BAD_ROWS] + [("attention", *b) for b in BAD_ATT])
def test_refusals(which, name, value, status):
    P = _pool(32768)
    assert _call(P, which, {**GOOD, name: value}) == status
    assert len(G.slora_last_error(P.h)) > 10


def test_null_pool_and_layout():
    P = _pool(32768)
    assert G.lib().slora_kv_write(None, G.make_kv_layout(8, 128), 16, 1024, 16, 1024, 4, 4, 4, 1, 1, 1, None) == 1
    assert G.lib().slora_kv_write(P.h, None, 16, 1024, 16, 1024, 4, 4, 4, 1, 1, 1, None) == 1
    assert G.lib().slora_kv_page_tokens(None, G.make_kv_layout(8, 128)) == 0


def test_a_pool_of_too_many_rows():
    P = _pool(1 << 20, n_pages=1 << 19)   # 2^39 elements: 2^33 rows of 64
    st = _call(P, "write", {**GOOD, "layout": (8, 64, 0)})
    assert st == 9 and "2^32" in G.slora_last_error(P.h)


def test_workspace_bytes():
    P = _pool(32768)
    L = G.make_kv_layout(8, 128)
    need = G.slora_kv_attention_workspace_bytes(P.h, L, 32, 2, 5, 3)
    assert need > 0
    assert _call(P, "attention", {**GOOD, "size": need}) == 9 and _call(P, "attention", {**GOOD, "size": need - 1}) == 1
    for bad in [(0, 2, 5, 3), (12, 2, 5, 3), (32, 0, 5, 3), (32, 2, 0, 3), (32, 2, 5, 0), (32, -1, 5, 3)]:
        assert G.slora_kv_attention_workspace_bytes(P.h, L, *bad) == 0
    # never less for more: one workspace serves every smaller step
    sizes = [G.slora_kv_attention_workspace_bytes(P.h, L, 32, b, t, m) for b, t, m in
             [(1, 1, 1), (2, 64, 1), (2, 64, 32), (64, 300, 40), (64, 512, 512)]]
    assert sizes == sorted(sizes)


def test_check_batch_knows_the_held_pages():
    P = _pool(32768, n_pages=16)
    L = G.make_kv_layout(8, 128)          # 16 tokens per page
    kv = P.kv_alloc(6)
    bl = np.full((2, 4), -1, np.int32)
    bl[0, :3], bl[1, :2] = kv[:3], kv[3:5]
    good = ([0, 4, 5], [40, 32], bl, 5)
    G.slora_kv_check_batch(P.h, L, *good)

    def refused(rs=good[0], kl=good[1], blocks=bl, T=5, word=""):
        with pytest.raises(G.SloraError) as e:
            G.slora_kv_check_batch(P.h, L, rs, kl, blocks, T)
        assert e.value.status == 1 and word in e.value.message

    refused(rs=[0, 6, 5], word="sequence 0")
    refused(rs=[0, 4, 6], word="sequence 1")
    refused(rs=[-1, 4, 5], word="sequence 0")
    refused(kl=[40, 65], word="sequence 1")
    refused(kl=[-1, 32], word="sequence 0")
    refused(kl=[49, 32], word="page -1")     # a fourth page that the table does not have
    other = bl.copy()
    other[1, 0] = next(i for i in range(16) if i not in kv)
    refused(blocks=other, word="not a held KV page")
    other[1, 0] = 16
    refused(blocks=other, word="page 16")
    P.kv_free([kv[4]])
    refused(word=f"page {kv[4]}")
    G.slora_kv_check_batch(P.h, L, [0, 4, 5], [40, 16], bl, 5)  # not used any more
    G.slora_kv_check_batch(P.h, L, [0], [], np.zeros((0, 4), np.int32), 0)
    with pytest.raises(ValueError):
        G.slora_kv_check_batch(P.h, L, [0, 1], [1, 2], bl, 5)


def test_reference_quantiser_against_torch():
    import torch
    rng = np.random.default_rng(7)
    x = R.from_bits(R.to_bits(rng.standard_normal((200, 64)) * np.exp(rng.standard_normal((200, 1)) * 4), "bf16"), "bf16")
    x[:, 0] = 448 * 2.0 ** rng.integers(-20, 20, 200)   # scales that are powers of two ...
    x[:, 1:] = np.clip(x[:, 1:], -np.abs(x[:, :1]), np.abs(x[:, :1]))
    codes, scale = R.quantise(x)
    q = torch.from_numpy(x / scale[:, None].astype(np.float64)).float()  # ... so that the quotient is exact in 32 bits
    want = q.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    vals = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(vals, nan=-1), np.nan_to_num(R.e4m3_values(), nan=-1))

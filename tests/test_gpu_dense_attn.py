"""basiskv_dense_attn against the formula in 64 bits, over shapes, lengths and masks."""
import math

import pytest
import torch

from tests.serving_reference import Cache, assert_attention, attention

pytestmark = pytest.mark.gpu

from long_context_decode_basiskv_b200 import binding as bk  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
SHAPES = {  # Hq, Hkv, d, r, P, dtype
    "8b": (32, 8, 128, 64, 16, BF),
    "wide": (8, 1, 128, 96, 64, BF),
    "d64": (4, 2, 64, 48, 32, BF),
    "mha": (2, 2, 128, 128, 16, BF),
    "r80": (16, 2, 128, 80, 16, BF),
    "r16": (8, 2, 64, 16, 32, BF),
    "tiny": (8, 2, 64, 16, 32, F32),
    "f32": (4, 4, 128, 40, 16, F32),
    "r24": (8, 1, 128, 24, 16, BF),     # bf16 rows that are not swizzled
}


def cfg_of(name):
    hq, hkv, d, r, P, dt = SHAPES[name]
    return bk.Config(hq, hkv, d, r, 8, P, 512, 8, dt)


def queries(cfg, B, n, seed, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((B, n, cfg.num_q_heads, cfg.head_dim), generator=g, device="cuda") * scale).to(cfg.dtype)


def options(cfg, B, softcap=0.0, window=0, slopes=False, prefix=None, scale=0.0):
    s = p = None
    if slopes:
        s = torch.pow(2.0, -8.0 * (torch.arange(cfg.num_q_heads, device="cuda") + 1.0) / cfg.num_q_heads)
    if prefix is not None:
        p = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    return bk.AttnOptions(scale, softcap, window, s, p)


def run(cfg, cache, q, opt, ws=None):
    B, n = q.shape[:2]
    o = torch.full((B, n, cfg.num_q_heads, cfg.rank_v), float("nan"), device="cuda")
    lse = torch.full((B, n, cfg.num_q_heads), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = bk.alloc_dense_workspace(cfg, B, n, cache.max_pages) if ws is None else ws
    bk.dense_attn(cfg, cache.paged, q, o, ws, err, opt, lse)
    return o, lse, int(err.item()), ws


def check(name, lengths, n, seed=1, max_pages=None, **kw):
    cfg = cfg_of(name)
    cache = Cache(cfg, lengths, seed, max_pages)
    B = len(lengths)
    q = queries(cfg, B, n, seed)
    opt = options(cfg, B, **kw)
    o, lse, err, ws = run(cfg, cache, q, opt)
    assert err == 0
    scale = kw.get("scale") or 1 / math.sqrt(cfg.head_dim)
    for b, L in enumerate(lengths):
        pre = max(0, min(L, kw["prefix"][b])) if kw.get("prefix") is not None else 0
        want = attention(cache.K[b], cache.C[b], q[b], scale, opt.softcap, opt.window, opt.slopes, pre)
        assert_attention(o[b], lse[b], *want, f"{name} n={n} L={L} {kw}")
    o2, lse2, _, _ = run(cfg, cache, q, opt, ws)         # the workspace as the first call left it
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


MASKS = [dict(), dict(softcap=30.0), dict(slopes=True), dict(window=7), dict(window=64, softcap=20.0, slopes=True),
         dict(prefix="third"), dict(prefix="third", window=5, slopes=True), dict(scale=0.2, window=1)]


def filled(mask, lengths):
    m = dict(mask)
    if m.get("prefix") == "third":
        m["prefix"] = [[L // 3, L + 9, -4, L][b % 4] for b, L in enumerate(lengths)]
    return m


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("mask", range(len(MASKS)))
def test_single_token(name, mask):
    lengths = [1, 16, 17, 0, 500, 129, 64, 2]
    check(name, lengths, 1, **filled(MASKS[mask], lengths))


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("n", [2, 5, 17, 40])
@pytest.mark.parametrize("mask", range(len(MASKS)))
def test_few_tokens(name, n, mask):
    lengths = [n, n + 1, 0, 333, n + 127]
    check(name, lengths, n, **filled(MASKS[mask], lengths))


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("n,lengths", [(130, [130, 700]), (300, [300]), (257, [1500, 257, 258])])
@pytest.mark.parametrize("mask", [0, 4, 6])
def test_prompts(name, n, lengths, mask):
    check(name, lengths, n, **filled(MASKS[mask], lengths))


@pytest.mark.parametrize("name", ["8b", "wide", "tiny", "r24", "mha"])
@pytest.mark.parametrize("n", [1, 4, 33])
@pytest.mark.parametrize("window", [0, 3000])
def test_long_contexts(name, n, window):
    check(name, [20011, 4097, n], n, window=window)


@pytest.mark.parametrize("name,n,batch", [("8b", 130, 7), ("wide", 40, 80), ("r80", 40, 40), ("8b", 96, 13)])
@pytest.mark.parametrize("mask", [dict(), dict(softcap=30.0, prefix=4000), dict(slopes=True), dict(window=900)])
def test_more_row_tiles_than_fit_at_once(name, n, batch, mask):
    """Row tiles in more than one wave, most of them short, the last sequences' long."""
    lengths = [n + b % 5 for b in range(batch - 4)] + [8200, 700, 8197, 8207]
    if mask.get("prefix"):
        mask = dict(mask, prefix=[mask["prefix"]] * batch)
    check(name, lengths, n, **mask)


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("n", [1, 3, 17, 130])
@pytest.mark.parametrize("slope", [0.1, -0.1])
def test_scores_that_rise_or_fall_along_the_keys(name, n, slope):
    """40 nats from the first key to the last, either way: references are raised, or stand, in every tile."""
    cfg = cfg_of(name)
    L = [400, n, 399]
    cache = Cache(cfg, L, 11)
    q = queries(cfg, 3, n, 11, 0.5)
    s = torch.full((cfg.num_q_heads,), slope, device="cuda")
    o, lse, err, _ = run(cfg, cache, q, bk.AttnOptions(slopes=s))
    assert err == 0
    for b in range(3):
        want = attention(cache.K[b], cache.C[b], q[b], 1 / math.sqrt(cfg.head_dim), slopes=s)
        assert_attention(o[b], lse[b], *want, f"{name} n={n} slope={slope}")


@pytest.mark.parametrize("name", ["8b", "tiny"])
def test_block_table_wider_than_the_cache(name):
    """Splits are planned for the table's width; most of them have nothing to do here."""
    check(name, [90, 5], 1, max_pages=2000)
    check(name, [90, 35], 35, max_pages=2000)


@pytest.mark.parametrize("name", ["8b", "wide", "tiny", "r24"])
@pytest.mark.parametrize("n", [1, 30])
def test_pages_outside_every_window_are_not_read(name, n):
    cfg = cfg_of(name)
    cache = Cache(cfg, [1000], 3)
    q = queries(cfg, 1, n, 3)
    opt = options(cfg, 1, window=50, prefix=[20])
    o, lse, err, _ = run(cfg, cache, q, opt)
    assert err == 0
    P = cfg.page_size
    first = (1000 - n - 50 + 1) // P                      # the window's first page; page 0 (1) holds the prefix
    keep = -(-20 // P)
    cache.paged.block_table[0, keep:first] = -1
    o2, lse2, err, _ = run(cfg, cache, q, opt)
    assert err == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("name", ["8b", "r24", "tiny"])
@pytest.mark.parametrize("n", [1, 30])
def test_non_finite_values_in_unseen_tokens(name, n):
    """Tokens that no new token sees: infinities and NaN in their keys and latents change nothing."""
    cfg = cfg_of(name)
    cache = Cache(cfg, [200], 4)
    q = queries(cfg, 1, n, 4)
    opt = options(cfg, 1, window=9)
    o, lse, _, _ = run(cfg, cache, q, opt)
    P = cfg.page_size
    lo = 200 - n - 9 + 1                                  # the first seen token; its page holds unseen ones too
    page, slot = lo // P, lo % P
    id = int(cache.paged.block_table[0, page])
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(cfg.dtype).min):
        cache.paged.k_raw[id, :, :slot] = bad
        cache.paged.c_lat[id, :, :slot] = bad
        o2, lse2, err, _ = run(cfg, cache, q, opt)
        assert err == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("name", ["8b", "wide", "tiny", "r24"])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_faults_are_reported(name, n):
    cfg = cfg_of(name)
    lengths = [300, 200, 400]
    cache = Cache(cfg, lengths, 5)
    q = queries(cfg, 3, n, 5)
    cache.paged.block_table[1, 1] = cache.paged.num_phys_pages      # one bad page: its tokens are not seen
    cache.paged.seq_len[2] = cache.max_pages * cfg.page_size + 1
    o, lse, err, ws = run(cfg, cache, q, None)
    assert err == bk.DEVERR_BLOCK_TABLE | bk.DEVERR_SEQ_LEN
    P, scale = cfg.page_size, 1 / math.sqrt(cfg.head_dim)
    assert_attention(o[0], lse[0], *attention(cache.K[0], cache.C[0], q[0], scale), "beside a fault")
    want = attention(cache.K[1], cache.C[1], q[1], scale, hidden_keys=range(P, 2 * P))
    assert_attention(o[1], lse[1], *want, "bad page")
    assert (o[2] == 0).all() and (lse[2] == -math.inf).all()
    if n > 1:
        cache.paged.seq_len[2] = n - 1                    # cannot hold the new tokens
        o, lse, err, _ = run(cfg, cache, q, None, ws)
        assert err & bk.DEVERR_SEQ_LEN and (o[2] == 0).all()


def test_nan_score_reaches_its_row():
    cfg = cfg_of("8b")
    cache = Cache(cfg, [100], 6)
    q = queries(cfg, 1, 1, 6)
    q[0, 0, 3, 5] = float("nan")
    o, lse, err, _ = run(cfg, cache, q, None)
    assert torch.isnan(o[0, 0, 3]).all() and torch.isnan(lse[0, 0, 3])
    assert torch.isfinite(o[0, 0, 4:]).all() and torch.isfinite(o[0, 0, :3]).all()


@pytest.mark.parametrize("n", [1, 64])
def test_captured_and_on_two_streams(n):
    """Two calls at once (own workspaces), and a captured one that is replayed on new queries."""
    cfg = cfg_of("8b")
    cache = Cache(cfg, [3000, 1000], 7)
    q = [queries(cfg, 2, n, s) for s in (1, 2)]
    want = [run(cfg, cache, x, None)[:2] for x in q]
    st = [torch.cuda.Stream() for _ in q]
    ws = [bk.alloc_dense_workspace(cfg, 2, n, cache.max_pages) for _ in q]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = [torch.empty_like(w[0]) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for x in (0, 1):
            bk.dense_attn(cfg, cache.paged, q[x], o[x], ws[x], err, stream=st[x])
    torch.cuda.synchronize()
    for x in (0, 1):
        assert torch.equal(o[x], want[x][0])
    qin, out = q[0].clone(), torch.empty_like(o[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bk.dense_attn(cfg, cache.paged, qin, out, ws[0], err)
    for x in (1, 0):
        qin.copy_(q[x])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[x][0])
    assert int(err.item()) == 0


def test_padded_batch_and_untouched_memory():
    """Rows past the batch stay as they were; empty sequences give zeros."""
    cfg = cfg_of("8b")
    cache = Cache(cfg, [50, 0, 0], 8)
    q = queries(cfg, 3, 1, 8)
    big = torch.full((5, 1, cfg.num_q_heads, cfg.rank_v), 3.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = bk.alloc_dense_workspace(cfg, 3, 1, cache.max_pages)
    bk.dense_attn(cfg, cache.paged, q, big[:3], ws, err)
    assert int(err.item()) == 0
    assert (big[3:] == 3).all() and (big[1:3] == 0).all() and (big[0] != 0).any()
    e = torch.empty((0, 1, cfg.num_q_heads, cfg.head_dim), dtype=cfg.dtype, device="cuda")
    sub = bk.PagedCache.__new__(bk.PagedCache)
    sub.__dict__.update(cache.paged.__dict__)
    sub.block_table = cache.paged.block_table[:0]
    bk.dense_attn(cfg, sub, e, big[:0], ws, err)


def test_lse_joins_two_halves():
    """Attention over two halves of a context, joined by their lse, is attention over the whole."""
    cfg = cfg_of("8b")
    cache = Cache(cfg, [1024], 9)
    q = queries(cfg, 1, 1, 9)
    o, lse, _, _ = run(cfg, cache, q, None)
    part = []
    for lo, hi in ((0, 512), (512, 1024)):
        sub = bk.PagedCache.__new__(bk.PagedCache)
        sub.__dict__.update(cache.paged.__dict__)
        sub.block_table = cache.paged.block_table[:, lo // 16:hi // 16].contiguous()
        sub.seq_len = torch.tensor([hi - lo], dtype=torch.int32, device="cuda")
        c = Cache.__new__(Cache)
        c.__dict__.update(paged=sub, max_pages=sub.max_pages)
        part.append(run(cfg, c, q, None)[:2])
    w = torch.stack([p[1] for p in part]).softmax(0)
    joined = sum(w[x][..., None] * part[x][0] for x in (0, 1))
    assert (joined - o).norm() <= 2.0 ** -15 * o.norm()
    assert (torch.logsumexp(torch.stack([p[1] for p in part]), 0) - lse).abs().max() <= 2.0 ** -15


@pytest.mark.parametrize("name,n,L,kw", [("r80", 130, 9000, dict(softcap=30.0, prefix=[8900])),
                                         ("8b", 130, 9000, dict(window=2000, prefix=[3000]))])
def test_no_wait_gives_up_over_many_calls(name, n, L, kw):
    """Calls behind one another, C tiles copied by either of the two roles that copy them (or by one of them
    throughout): no wait misses its phase, and the results stay bit for bit the same."""
    cfg = cfg_of(name)
    cache = Cache(cfg, [L] * 4, 5)
    kw = {k: v * 4 if k == "prefix" else v for k, v in kw.items()}
    q, opt = queries(cfg, 4, n, 5), options(cfg, 4, **kw)
    o, lse, err, ws = run(cfg, cache, q, opt)
    assert err == 0
    again, flag = torch.empty_like(o), torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(200):
        bk.dense_attn(cfg, cache.paged, q, again, ws, flag, opt)
    assert int(flag.item()) == 0
    assert torch.equal(o, again)

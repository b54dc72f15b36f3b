"""basiskv_dense_attn where its kernels change course: CTAs without keys, and what else the shapes and masks of
test_gpu_dense_attn.py do not reach."""
import math

import pytest
import torch

from tests.serving_reference import Cache, assert_attention, attention, swizzle
from tests.test_gpu_dense_attn import F32, SHAPES, cfg_of, check, options, queries, run

pytestmark = pytest.mark.gpu

from long_context_decode_basiskv_b200 import binding as bk  # noqa: E402


@pytest.mark.parametrize("name", ["8b", "wide", "mha", "d64"])
@pytest.mark.parametrize("n,empty,pages", [(33, 200, None), (130, 200, None), (33, 3, 4000), (300, 1, 4000)])
def test_many_ctas_without_keys(name, n, empty, pages):
    """Empty sequences, and shares of a key axis that is short in a wide block table: CTAs whose copy and MMA
    warps have nothing to do and end at once, among CTAs that work, call after call."""
    cfg = cfg_of(name)
    lengths = [0] * empty + [n + 65, 0]
    cache = Cache(cfg, lengths, 12, pages)
    q = queries(cfg, len(lengths), n, 12)
    o, lse, err, ws = run(cfg, cache, q, None)
    assert err == 0
    assert (o[:empty] == 0).all() and (o[-1] == 0).all()
    assert (lse[:empty] == -math.inf).all() and (lse[-1] == -math.inf).all()
    want = attention(cache.K[empty], cache.C[empty], q[empty], 1 / math.sqrt(cfg.head_dim))
    assert_attention(o[empty], lse[empty], *want, f"{name} n={n} beside {empty} empty ones")
    again, flag = torch.empty_like(o), torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(50):
        bk.dense_attn(cfg, cache.paged, q, again, ws, flag)
    assert int(flag.item()) == 0 and torch.equal(o, again)


# ---------------------------------------------------------------------------
# one workspace, many shapes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("calls", [
    # (shape, new tokens, lengths): few CTAs and many, shares of long key axes, in turn
    [("8b", 1, [9000]), ("8b", 1, [300] * 64), ("8b", 3, [5000, 700]), ("8b", 1, [40] * 200)],
    [("tiny", 1, [6000]), ("tiny", 1, [300] * 40), ("r24", 2, [5000]), ("f32", 1, [900] * 9)],
    [("8b", 1, [9000]), ("wide", 130, [4000]), ("8b", 40, [3000]), ("mha", 300, [2000] * 3), ("r80", 1, [500] * 70)],
    [("wide", 40, [9000]), ("tiny", 1, [2000] * 3), ("8b", 1, [2000] * 30), ("d64", 64, [70] * 50), ("r24", 64, [900])],
])
def test_one_workspace_for_many_shapes(calls):
    """A workspace that holds the largest of several shapes serves them in any order, without being cleared."""
    cases = []
    for x, (name, n, lengths) in enumerate(calls):
        cfg = cfg_of(name)
        cache = Cache(cfg, lengths, 20 + x)
        q = queries(cfg, len(lengths), n, 20 + x)
        o, lse, err, _ = run(cfg, cache, q, None)          # a workspace of its own
        assert err == 0
        cases.append((cfg, cache, q, o, lse, bk.dense_workspace_bytes(cfg, len(lengths), n, cache.max_pages)))
    ws = torch.zeros(max(c[-1] for c in cases), dtype=torch.uint8, device="cuda")
    for turn in range(3):
        for x in (range(len(cases)) if turn != 1 else reversed(range(len(cases)))):
            cfg, cache, q, o, lse, _ = cases[x]
            o2, lse2, err, _ = run(cfg, cache, q, None, ws)  # (o2 and lse2 start as NaN)
            assert err == 0
            assert torch.equal(o, o2) and torch.equal(lse, lse2), (turn, calls[x])


# ---------------------------------------------------------------------------
# scores past their cap, references that rise
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("n", [1, 3, 17, 130])
@pytest.mark.parametrize("mask", [dict(softcap=1.0), dict(softcap=2.0, window=100, prefix="third"),
                                  dict(softcap=0.5, slopes=True), dict(softcap=1.0, window=9, slopes=True)])
def test_scores_around_and_past_their_cap(name, n, mask):
    """Scores of about 1.2 nats under caps of 0.5 to 2: some far below the cap, some far above, of both signs, in
    every tile; tiles that are seen whole and tiles that are not."""
    lengths = [n + 400, n, n + 127]
    mask = dict(mask)
    if mask.get("prefix"):
        mask["prefix"] = [L // 3 for L in lengths]
    check(name, lengths, n, seed=31, **mask)


def refill(cache, b, K):
    """Other keys for sequence b, in the pages it has."""
    cfg, L = cache.cfg, cache.lengths[b]
    P, H, n = cfg.page_size, cfg.num_kv_heads, -(-L // cfg.page_size)
    on = cfg.dtype == torch.bfloat16 and cfg.head_dim % 16 == 0 and cfg.rank_v % 16 == 0
    full = torch.full((n * P, H, cfg.head_dim), float("nan"), dtype=cfg.dtype, device="cuda")
    full[:L] = K
    cache.paged.k_raw[cache.paged.block_table[b, :n].long()] = swizzle(
        full.reshape(n, P, H, -1).transpose(1, 2).contiguous(), on)
    cache.K[b] = K


# The tiles of keys are taken from the last to the first; of the tiles that all rows see whole, the one `at` tiles
# before the last has its scores raised by 10 nats from its 32-key group `group` on, and so have all keys before.
RISES = [((1, 4, 6), (0, 0, 0)), ((1, 4, 6), (1, 2, 3)), ((2, 3, 4), (3, 3, 3)), ((4, 5, 8), (2, 0, 1)), ((1, 2, 3), (3, 1, 2))]


def levels(L, n, rises):
    """Nats of every key: 0 at the end, 30 at the start."""
    lv = torch.zeros(L)
    last = (L - 1) // 128                                   # tiles are 128 keys from key 0
    whole = (L - n) // 128 - 1                              # the last tile that every row sees whole
    for at, group in zip(*rises):
        t = min(whole, last - 1) - at
        lv[128 * t + 32 * group:128 * (t + 1)] += 10
        lv[:128 * t] += 10
    return lv


@pytest.mark.parametrize("name,n", [("8b", 17), ("8b", 130), ("wide", 17), ("wide", 40), ("mha", 40), ("mha", 300),
                                    ("d64", 130), ("r80", 33), ("8b", 3), ("wide", 1), ("r24", 17), ("f32", 20)])
@pytest.mark.parametrize("rises", range(len(RISES)))
@pytest.mark.parametrize("mod", [dict(), dict(slopes=True), dict(softcap=12.0)])
def test_scores_that_pass_the_reference_inside_a_tile(name, n, rises, mod):
    """Keys along one direction, ever longer towards the start: scores of 30 nats that pass the rows' references
    by 10 at a time, at each of the four column groups, in tiles whose products start a sum and in others; for half
    of the heads by less, so that rows of a warp differ.  Uncapped and unbiased, biased, and under a cap that the
    second rise passes.

    The bounds of assert_attention hold: |s| < 32 nats and sum |q k| scale < 40 (below, the noise adds a nat or
    two), a score's error is the tensor cores' 8 cut-off sums of at most 2^-23 32 each (or 128 fp32 roundings, fewer in the root of their squares), 2^-15, and scale, reference
    and exponent add 2^-17; the weights' 2^-16 and the sums' 2^-18 stay: 0.94 2^-14 together."""
    cfg = cfg_of(name)
    L = 1500 + n
    cache = Cache(cfg, [L, 64 + n], 41)
    g = torch.Generator(device="cuda").manual_seed(41)
    H, d, Hq = cfg.num_kv_heads, cfg.head_dim, cfg.num_q_heads
    scale = 1 / math.sqrt(d)
    u = torch.randn((H, d), generator=g, device="cuda").sign() / math.sqrt(d)      # a unit vector of each KV head
    size = math.sqrt(30 / scale)
    lv = levels(L, n, RISES[rises]).cuda() / 30
    K = lv[:, None, None] * size * u + 0.1 * torch.randn((L, H, d), generator=g, device="cuda")
    refill(cache, 0, K.to(cfg.dtype))
    part = torch.where(torch.arange(Hq, device="cuda") % 2 == 0, 1.0, 0.5)[:, None]
    q = part * size * u.repeat_interleave(Hq // H, 0) + 0.1 * torch.randn((2, n, Hq, d), generator=g, device="cuda")
    q = q.to(cfg.dtype)
    opt = options(cfg, 2, **mod)
    if opt.slopes is not None:
        opt.slopes *= 2.0 ** -8                              # a bias that leaves the rises as they are
    o, lse, err, _ = run(cfg, cache, q, opt)
    assert err == 0
    for b in range(2):
        want = attention(cache.K[b], cache.C[b], q[b], scale, opt.softcap, 0, opt.slopes)
        assert_attention(o[b], lse[b], *want, f"{name} n={n} {RISES[rises]} {mod}")


# ---------------------------------------------------------------------------
# bounds of the kernels that keep 24 bits of a weight
# ---------------------------------------------------------------------------
# Few keys, so that no error averages out, and scores that fp32 holds exactly before they are scaled: one element of
# a query and of a key is not zero, their product has 16 bits.  With |s| < 2 nats (2.9 in log 2 units), relative to
# sum w |C| (half steps of fp32: 2^-24):
#   a score: the factor scale log2(e), its product and the reference taken off, 3 2^-24 2.9 ln 2 < 2^-21.4;  2^x: 2^-22
#   both in numerator and denominator: 2 (2^-21.4 + 2^-22) < 2^-19.7
#   three bf16 terms: 2^-24;  products added on tensor cores (each addition cut off, 2^-23, three terms and the tile
#   onto the sum before): 4 2^-23;  the sum of weights over lanes: 5 2^-24;  a merge of two shares (its two weights,
#   products and sums): 2^-21;  the division: 2^-23
# Together below 2^-19.7 + 2^-21 + 2^-20.4 < 2^-18.5.  Two bf16 terms leave 2^-16 of a weight at worst.  The CUDA cores
# add key by key: 2^-24 for each.  lse: score and 2^x 2^-20.7, the sum of weights 2^-21.4, log2, its sum with the
# reference (below 16) and the factor ln 2 3 2^-21: below 2^-19.
TIGHT = 2.0 ** -18.5


def tight_case(cfg, lengths, n, seed):
    cache = Cache(cfg, lengths, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, d, Hq = cfg.num_kv_heads, cfg.head_dim, cfg.num_q_heads
    for b, L in enumerate(lengths):
        K = torch.zeros((L, H, d), device="cuda")
        K[:, :, 5] = torch.rand((L, H), generator=g, device="cuda") * 2 - 1        # |k| < 1
        refill(cache, b, K.to(cfg.dtype))
    q = torch.zeros((len(lengths), n, Hq, d), device="cuda")
    q[..., 5] = (torch.rand((len(lengths), n, Hq), generator=g, device="cuda") + 1) * math.sqrt(d)   # |s| < 2
    return cache, q.bfloat16().to(cfg.dtype)                                       # 8 bits in fp32 too


def two_terms(w):
    hi = w.float().bfloat16().float()
    return (hi + (w.float() - hi).bfloat16().float()).double()


@pytest.mark.parametrize("name,n", [("8b", 1), ("8b", 3), ("mha", 1), ("mha", 9), ("r80", 2), ("d64", 5), ("r16", 1),
                                    ("wide", 1), ("tiny", 1), ("tiny", 30), ("f32", 1), ("f32", 200), ("r24", 1)])
def test_weights_keep_24_bits(name, n):
    """Up to 16 rows, and the CUDA cores: within a bound that weights of 16 bits break."""
    cfg = cfg_of(name)
    lengths = [n + b % 7 for b in range(40)]
    cache, q = tight_case(cfg, lengths, n, 51)
    if cfg.dtype == F32:                                                           # 8-bit keys: exact products
        for b in range(len(lengths)):
            refill(cache, b, cache.K[b].bfloat16().float())
    on = cfg.dtype != F32 and cfg.rank_v % 16 == 0                                 # tensor cores
    bound = TIGHT + (0 if on else max(lengths)) * 2.0 ** -24
    scale = 1 / math.sqrt(cfg.head_dim)
    o, lse, err, _ = run(cfg, cache, q, None)
    assert err == 0
    worst = coarse = 0.0
    for b in range(len(lengths)):
        want, want_lse, size = attention(cache.K[b], cache.C[b], q[b], scale)
        size = size.clamp(min=1e-9)
        worst = max(worst, float(((o[b].double() - want).abs() / size).max()))
        assert ((lse[b].double() - want_lse).abs() <= 2.0 ** -19).all()
        G = cfg.group
        for h in range(cfg.num_q_heads):                                           # what two terms would give
            s = q[b, -1, h].double() @ cache.K[b][:, h // G].double().T * scale
            w = torch.exp(s - s.max())
            C = cache.C[b][:, h // G].double()
            diff = (two_terms(w) - w) @ C / w.sum()
            coarse = max(coarse, float((diff.abs() / size[-1, h]).max()))
    assert worst <= bound, math.log2(worst)
    assert coarse > bound or n > 9, math.log2(coarse)                              # over many keys errors average out

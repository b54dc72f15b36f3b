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

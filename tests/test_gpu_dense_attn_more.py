"""basiskv_dense_attn where its kernels change course: CTAs without keys, and what else the shapes and masks of
test_gpu_dense_attn.py do not reach."""
import math

import pytest
import torch

from tests.serving_reference import Cache, assert_attention, attention
from tests.test_gpu_dense_attn import cfg_of, options, queries, run

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

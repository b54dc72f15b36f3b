"""The binding's own checks, on the host: what it hands out, and what it refuses before the library is called."""
import copy
import pickle

import pytest
import torch

from long_context_decode_basiskv_b200 import binding as bk


def config(**kw):
    base = dict(num_q_heads=8, num_kv_heads=2, head_dim=64, rank_v=16, rank_k=8, page_size=16, hidden=512, top_k=8,
                dtype=torch.float32)
    base.update(kw)
    return bk.Config(**base)


def test_a_config_hands_out_structs_of_its_own():
    """Writing to a struct that c() gave changes neither the next one nor what the calls pass."""
    cfg = config()
    mine = cfg.c()
    mine.page_size = 64
    assert cfg.c().page_size == 16
    passed = cfg._ref()._obj
    assert passed.page_size == 16 and passed is not mine
    cfg.c().head_dim = 128
    assert cfg._ref()._obj.head_dim == 64
    for other in (copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):     # after a call has made the struct
        assert other == cfg and other._ref()._obj.page_size == 16

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


class Stand:
    """What the binding asks of a tensor before it calls the library, without a GPU."""

    def __init__(self, shape, device=0):
        self.shape, self.at = torch.Size(shape), device
        self.device = f"cuda:{device}" if device >= 0 else "cpu"

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.at

    def data_ptr(self):
        return 256


@pytest.fixture
def no_library(monkeypatch):
    calls = []
    monkeypatch.setattr(bk, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(bk, "_stream", lambda s: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or bk.OK
    monkeypatch.setattr(bk, "lib", Library)
    return calls


def cache_of_stands(**at):
    cache = bk.PagedCache.__new__(bk.PagedCache)
    cache.num_phys_pages = 4
    for name, shape in (("k_raw", (4, 2, 16, 64)), ("c_lat", (4, 2, 16, 16)), ("r_res", (4, 2, 16, 8)),
                        ("summary", (4, 2, 64)), ("block_table", (1, 4)), ("seq_len", (1,))):
        setattr(cache, name, Stand(shape, at.get(name, 0)))
    return cache


@pytest.mark.parametrize("name", ["k_raw", "c_lat", "block_table", "seq_len"])
@pytest.mark.parametrize("device", [1, -1])
def test_attention_over_a_cache_on_another_device(no_library, name, device):
    args = Stand((1, 8, 64)), Stand((1, 8, 16)), Stand((4096,)), Stand((1,))
    bk.dense_attn(config(), cache_of_stands(), *args)
    assert no_library == ["basiskv_dense_attn"]
    with pytest.raises(ValueError, match="others are on cuda:0"):
        bk.dense_attn(config(), cache_of_stands(**{name: device}), *args)
    assert len(no_library) == 1

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


@pytest.fixture
def passed(no_library, monkeypatch):
    """The arguments of the library's calls."""
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append(a) or bk.OK
    monkeypatch.setattr(bk, "lib", Library)
    return seen


@pytest.mark.parametrize("window,want", [(5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                         (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 7, 2 ** 31 - 1), (-3, -1), (-2 ** 32, -1)])
def test_a_window_past_32_bits_is_no_smaller_one(passed, window, want):
    args = Stand((1, 8, 64)), Stand((1, 8, 16)), Stand((4096,)), Stand((1,))
    bk.dense_attn(config(), cache_of_stands(), *args, bk.AttnOptions(window=window))
    assert passed[0][5]._obj.window == want


@pytest.mark.parametrize("opt", [dict(scale=1e-50), dict(softcap=1e-60), dict(scale=-1e-50)])
def test_options_that_fp32_makes_zero_are_refused(passed, opt):
    """Zero stands for the default scale, or for no cap."""
    args = Stand((1, 8, 64)), Stand((1, 8, 16)), Stand((4096,)), Stand((1,))
    with pytest.raises(ValueError, match="fp32"):
        bk.dense_attn(config(), cache_of_stands(), *args, bk.AttnOptions(**opt))
    assert not passed


def test_counts_past_32_bits_are_not_cut_off(passed):
    i = Stand((1,))
    bk.assign_pages(config(), Stand((1, 4)), i, i, Stand((2 ** 32 + 5,)), i, i, i, Stand((1, 2 ** 32 + 8)), i)
    assert passed[0][3] == passed[0][12] == 2 ** 31 - 1
    bk.release_pages(config(), Stand((1, 4)), i, i, Stand((2 ** 32 + 5,)), i, i, i, i)
    assert passed[1][3] == 2 ** 31 - 1

"""The serving operators as they are used together: pages for the new tokens,
rotary, append, attention over the whole cache, out-projection, step after
step, against the fp64 oracle's stored cache and the 64-bit attention formula."""
import math

import numpy as np
import pytest
import torch

from oracle import basiskv_oracle as O
from tests.harness import F32_REL_L2, BF16_REL_L2, OracleCase, close_report, to64
from tests.serving_reference import attention, rotate

pytestmark = pytest.mark.gpu

from long_context_decode_basiskv_b200 import binding as bk  # noqa: E402
from long_context_decode_basiskv_b200.engine import DecodeEngine  # noqa: E402
from long_context_decode_basiskv_b200.workloads import WORKLOADS, make_case, shrink  # noqa: E402


def stored(x, storage):
    return x if storage == "f32" else torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("base,kw", [
    ("tiny_fp32", dict(batch=3, ragged=(1, 700))),
    ("llama3_8b_32k", dict(batch=5, ragged=(1, 900), top_k=16)),
    ("llama3_70b_64k", dict(batch=2, ragged=(300, 400), top_k=16)),
])
@pytest.mark.parametrize("roped", [False, True])
def test_dense_decode_step(base, kw, roped):
    """DecodeEngine with dense attention, its pages from a pool, with and without rotary positions:
    o_lat and y against 64 bits on the rounded cache; the graph and the host-buffer step give its bits."""
    wl = shrink(WORKLOADS[base], name="dense_" + base, **kw)
    case = make_case(wl, "cuda")
    storage = "f32" if wl.dtype == "f32" else "bf16"
    cfg = bk.Config(wl.num_q_heads, wl.num_kv_heads, wl.head_dim, wl.rank_v, wl.rank_k, wl.page_size, wl.hidden,
                    wl.top_k, wl.torch_dtype)
    rope = bk.Rope(cfg, base=500000.0, scaling="llama3", factor=8.0, original_len=256) if roped else None
    keys = [k.clone() for k in case.keys]
    eng = DecodeEngine(case, attention="dense", rope=rope, paging="pool",
                       options=bk.AttnOptions(softcap=30.0, window=200))
    y = eng.step()
    torch.cuda.synchronize()
    assert int(eng.err.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(keys, case.keys))      # the case keeps its keys
    oc = OracleCase(case)
    tol = F32_REL_L2 if storage == "f32" else BF16_REL_L2
    for b, L in enumerate(case.lengths):
        K, q = case.keys[b], case.q[b].unsqueeze(0)
        if roped:
            K = rotate(K, torch.arange(L, device="cuda"), rope.inv_freq, rope.mscale, "half")[0].to(K.dtype)
            q = rotate(q, torch.tensor([L - 1], device="cuda"), rope.inv_freq, rope.mscale, "half")[0].to(q.dtype)
        cache = O.prefill(to64(K), to64(case.values[b]), oc.A, oc.P, oc.E, wl.page_size, storage, capacity=L)
        C = torch.from_numpy(np.ascontiguousarray(np.swapaxes(cache.C[:, :L], 0, 1))).cuda()
        o, _, _ = attention(K, C, q, 1 / math.sqrt(wl.head_dim), 30.0, 200)
        want_y = O.out_projection(o[0].cpu().numpy(), oc.G)
        for got, want in ((eng.o_lat[b], o[0]), (y[b], torch.from_numpy(want_y))):
            assert close_report(to64(got), to64(want))[1] <= tol
    ref = eng.o_lat.clone(), y.clone()
    eng.o_lat.zero_()
    assert torch.equal(eng.graph_step(), ref[1]) and torch.equal(eng.o_lat, ref[0])
    host_in, host_y = eng.input_buffer().cpu().pin_memory(), torch.empty_like(y, device="cpu").pin_memory()
    eng.graph_step_host(host_in, host_y)
    torch.cuda.synchronize()
    assert torch.equal(host_y, ref[1].cpu())


def test_routed_step_with_rope():
    """Rotary in front of the routed step: both overlaps give what rotated inputs give without it."""
    wl = shrink(WORKLOADS["llama3_8b_32k"], batch=2, context=16 * 60 + 5, top_k=8, name="routed_rope")
    case = make_case(wl, "cuda")
    cfg = DecodeEngine(case).cfg
    rope = bk.Rope(cfg, base=500000.0)
    turned = make_case(wl, "cuda")
    for b, L in enumerate(case.lengths):
        plain = case.keys[b].contiguous()
        k, q = torch.empty_like(plain), torch.empty_like(case.q[b])
        pos = torch.arange(L, dtype=torch.int32, device="cuda")
        bk.rotary(cfg, rope, None, plain[None], None, k[None], positions=pos[None])
        bk.rotary(cfg, rope, case.q[b][None, None], None, q[None, None], None, positions=pos[None, -1:].contiguous())
        turned.keys[b], turned.q[b] = k, q
    turned.A, turned.P, turned.E = case.A, case.P, case.E
    want = DecodeEngine(turned)
    want.step()
    for overlap in ("pdl", "streams"):
        eng = DecodeEngine(case, rope=rope, overlap=overlap)
        eng.step()
        torch.cuda.synchronize()
        assert int(eng.err.item()) == 0
        assert torch.equal(eng.sel, want.sel) and torch.equal(eng.y, want.y)


def test_prompt_then_steps_from_one_pool():
    """A prompt (prefill and its attention), then single tokens, every page from the pool: the rows of the
    prompt's attention and of the steps are the rows of one long prompt's."""
    wl = shrink(WORKLOADS["llama3_8b_32k"], batch=1, context=300, top_k=16, name="prompt_chain")
    case = make_case(wl, "cuda")
    cfg = bk.Config(32, 8, 128, 64, 32, 16, 4096, 16, torch.bfloat16)
    from long_context_decode_basiskv_b200.pages import PagePool
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    factors = bk.Factors(case.A.contiguous(), case.P.contiguous(), case.E.contiguous(), case.A)
    q = (torch.randn((1, 300, 32, 128), device="cuda") * 1.5).to(torch.bfloat16)
    rope = bk.Rope(cfg)
    k, v = case.keys[0][None].contiguous(), case.values[0][None].contiguous()

    def pieces(cuts):
        pool = PagePool(cfg, 40, 1, 20)
        cache = bk.PagedCache(cfg, 40, pool.block_table, pool.seq_len)
        cache.block_table, cache.seq_len = pool.block_table, pool.seq_len
        out = []
        for a, b in zip(cuts[:-1], cuts[1:]):
            n = b - a
            pool.extend(torch.tensor([n], dtype=torch.int32, device="cuda"), err)
            qr, kr = torch.empty_like(q[:, a:b].contiguous()), torch.empty_like(k[:, a:b].contiguous())
            bk.rotary(cfg, rope, q[:, a:b].contiguous(), k[:, a:b].contiguous(), qr, kr, seq_len=pool.seq_len)
            bk.append(cfg, cache, factors, kr, v[:, a:b].contiguous(), err)
            o = torch.empty((1, n, 32, 64), device="cuda")
            bk.dense_attn(cfg, cache, qr, o, bk.alloc_dense_workspace(cfg, 1, n, 20), err)
            out.append(o)
        return torch.cat(out, 1)
    whole = pieces([0, 300])
    parts = pieces([0, 200, 201, 202, 206, 250] + list(range(251, 301)))
    assert int(err.item()) == 0
    assert (whole - parts).norm() <= 2.0 ** -14 * whole.norm()

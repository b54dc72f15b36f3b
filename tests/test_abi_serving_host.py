"""Host-side checks of the serving entry points (pages, rotary, attention over
the whole cache): what they refuse, and the frequencies they compute, in a
process that sees no GPU (made-up addresses that no kernel may receive)."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

from long_context_decode_basiskv_b200 import binding as bk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GPU_VISIBLE = os.environ.get("CUDA_VISIBLE_DEVICES") != "" and torch.cuda.is_available()


def test_serving_checks_in_a_process_without_gpu():
    if not GPU_VISIBLE:
        pytest.skip("no GPU visible: the checks run in this process")
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.abspath(__file__)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.fixture(scope="module")
def L():
    if GPU_VISIBLE:
        pytest.skip("a GPU is visible: these calls run in a child process")
    if not os.path.exists(bk.LIB_PATH):
        from long_context_decode_basiskv_b200 import build
        build.build()
    return bk.lib()


def _cfg(**kw):
    base = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, rank_v=64, rank_k=32, page_size=16,
                hidden=4096, top_k=128, dtype=bk.BF16)
    base.update(kw)
    return bk.CConfig(*[base[f] for f, _ in bk.CConfig._fields_])


BAD, UNS, WS = bk.ERR_INVALID_ARG, bk.ERR_UNSUPPORTED, bk.ERR_WORKSPACE


def test_assign_pages_refusals(L):
    def call(cfg=None, batch=2, mp=10, phys=40, seq=256, add=512, table=1024, free=2048, cnt=4096, so=8192, co=8448,
             slots=16384, cols=8, err=32768):
        return L.basiskv_assign_pages(ctypes.byref(cfg or _cfg()), batch, mp, phys, seq, add, table, free, cnt, so, co,
                                      slots, cols, err, None)
    assert call(batch=0) == bk.OK
    assert call(batch=-1) == BAD
    assert call(cfg=_cfg(page_size=8)) == UNS
    assert call(mp=0) == BAD and call(phys=0) == BAD
    assert call(mp=49153) == UNS and call(phys=1 << 24) == UNS and call(batch=16385) == UNS
    for name in ("seq", "add", "table", "free", "cnt", "so", "co", "err"):
        assert call(**{name: None}) == BAD, name
    assert call(cols=0) == BAD                       # slots without columns
    assert call(so=512) == BAD and call(co=256) == BAD and call(so=4096) == BAD and call(so=8448) == BAD


def test_release_pages_refusals(L):
    def call(batch=2, mp=10, phys=40, seq=256, rel=512, table=1024, free=2048, cnt=4096, so=8192, co=8448, err=32768):
        return L.basiskv_release_pages(ctypes.byref(_cfg()), batch, mp, phys, seq, rel, table, free, cnt, so, co, err,
                                       None)
    assert call(batch=0) == bk.OK
    assert call(batch=-1) == BAD and call(mp=0) == BAD and call(batch=16385) == UNS
    for name in ("seq", "rel", "table", "free", "cnt", "so", "co", "err"):
        assert call(**{name: None}) == BAD, name
    assert call(so=512) == BAD and call(co=8192) == BAD


def _params(**kw):
    base = dict(layout=0, rotary_dim=128, scaling=0, base=10000.0, factor=8.0, original_len=8192.0, beta_fast=32.0,
                beta_slow=1.0, low_freq_factor=1.0, high_freq_factor=4.0)
    base.update(kw)
    return bk.CRopeParams(*[base[f] for f, _ in bk.CRopeParams._fields_])


@pytest.mark.parametrize("bad", [
    dict(layout=2), dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=130), dict(scaling=5), dict(scaling=-1),
    dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(scaling=1, factor=0.5),
    dict(scaling=2, factor=math.nan), dict(scaling=3, original_len=0.0), dict(scaling=3, beta_fast=1.0),
    dict(scaling=3, beta_slow=0.0), dict(scaling=4, high_freq_factor=1.0), dict(scaling=4, low_freq_factor=-1.0),
])
def test_rope_init_refusals(L, bad):
    rope = bk.CRope()
    assert L.basiskv_rope_init(ctypes.byref(rope), ctypes.byref(_params(**bad))) == BAD
    assert L.basiskv_rope_init(None, ctypes.byref(_params())) == BAD
    assert L.basiskv_rope_init(ctypes.byref(rope), None) == BAD


def test_rope_frequencies(L):
    """Every scaling against its definition, worked out here pair by pair."""
    D, base, F, N = 128, 10000.0, 8.0, 8192.0
    plain = [base ** (-2 * i / D) for i in range(D // 2)]

    def of(**kw):
        rope = bk.CRope()
        assert L.basiskv_rope_init(ctypes.byref(rope), ctypes.byref(_params(**kw))) == bk.OK
        return list(rope.inv_freq)[:D // 2], rope.mscale

    def same(got, want):
        assert got == pytest.approx(want, rel=1e-13)

    f, m = of()
    same(f, plain)
    assert m == 1.0
    same(of(scaling=1)[0], [x / F for x in plain])
    same(of(scaling=2)[0], [(base * F ** (D / (D - 2))) ** (-2 * i / D) for i in range(D // 2)])
    # yarn: turns over the original context decide; the ramp runs over whole pairs
    f, m = of(scaling=3)
    assert m == pytest.approx(0.1 * math.log(F) + 1)
    turns = [N * x / (2 * math.pi) for x in plain]
    lo = max(i for i in range(D // 2) if turns[i] >= 32)     # the last pair with at least beta_fast turns
    hi = min(i for i in range(D // 2) if turns[i] <= 1)      # the first with at most beta_slow
    want = [plain[i] if i <= lo else plain[i] / F if i >= hi else
            plain[i] * (1 - (i - lo) / (hi - lo)) + plain[i] / F * (i - lo) / (hi - lo) for i in range(D // 2)]
    same(f, want)
    # llama3: by wavelength
    f, m = of(scaling=4)
    assert m == 1.0
    want = []
    for x in plain:
        wave = 2 * math.pi / x
        if wave < N / 4:
            want.append(x)
        elif wave > N / 1:
            want.append(x / F)
        else:
            t = (N / wave - 1) / (4 - 1)
            want.append((1 - t) * x / F + t * x)
    same(f, want)


def test_rotary_refusals(L):
    rope = bk.CRope()
    L.basiskv_rope_init(ctypes.byref(rope), ctypes.byref(_params()))

    def call(cfg=None, rp=rope, q=256, qs=4096, k=65536, ks=1024, qo=131072, ko=262144, pos=None, seq=512, batch=1, n=2):
        return L.basiskv_rotary(ctypes.byref(cfg or _cfg()), ctypes.byref(rp) if rp else None, q, qs, k, ks, qo, ko, pos,
                                seq, batch, n, None)
    assert call(batch=0) == bk.OK and call(n=0) == bk.OK
    assert call(batch=-1) == BAD and call(n=-1) == BAD
    assert call(rp=None) == BAD
    assert call(cfg=_cfg(head_dim=64)) == BAD                 # 128 rotated elements of 64
    assert call(q=None) == BAD and call(ko=None) == BAD       # one of a pair
    assert call(q=None, qo=None, k=None, ko=None) == BAD
    assert call(pos=512) == BAD and call(seq=None) == BAD     # both, neither
    assert call(qs=4095) == BAD and call(ks=1000) == BAD
    assert call(qo=256, qs=6144) == BAD                       # in place with gaps
    assert call(q=257) == BAD
    assert call(cfg=_cfg(page_size=8)) == UNS
    bad = bk.CRope(layout=3, rotary_dim=64)
    assert call(rp=bad) == BAD


def test_dense_attn_refusals(L):
    good = bk.CCache(256, 256, None, None, 256, 256, 10, 10)   # no residuals, no summaries: they are not read

    def call(cfg=None, cache=good, q=256, batch=1, n=1, opt=None, o=256, ws=256, nws=1 << 40, err=256):
        return L.basiskv_dense_attn(ctypes.byref(cfg or _cfg()), ctypes.byref(cache) if cache else None, q, batch, n,
                                    ctypes.byref(opt) if opt else None, o, None, ws, nws, err, None)
    assert call(batch=0) == bk.OK and call(n=0) == bk.OK
    assert call(batch=-1) == BAD and call(n=-1) == BAD
    assert call(batch=65536) == UNS
    assert call(cache=None) == BAD
    assert call(cache=bk.CCache(0, 256, None, None, 256, 256, 10, 10)) == BAD
    assert call(cache=bk.CCache(256, 264, None, None, 256, 256, 10, 10)) == BAD
    assert call(cache=bk.CCache(256, 256, None, None, 256, 256, 10, 49153)) == UNS
    assert call(q=None) == BAD and call(q=264) == BAD and call(o=None) == BAD and call(o=260) == BAD
    assert call(err=None) == BAD
    assert call(ws=None) == WS and call(nws=0) == WS and call(ws=264) == WS
    assert call(n=161) == BAD                                  # more than the block table holds
    assert call(cfg=_cfg(head_dim=96)) == UNS and call(cfg=_cfg(dtype=7)) == BAD
    for bad in (dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(softcap=-2.0),
                dict(softcap=math.inf), dict(softcap=math.nan), dict(window=-1)):
        assert call(opt=bk.CAttnOptions(**bad)) == BAD, bad


def test_counts_past_32_bits_are_refused(L):
    big = dict(phys=1 << 20, mp=49152)
    args = (256, 512, 1024, 2048, 4096, 8192, 8448)
    for cols, want in (((1 << 30) + 1, UNS), ((1 << 31) - 1, UNS)):
        assert L.basiskv_assign_pages(ctypes.byref(_cfg()), 1, big["mp"], big["phys"], *args, 16384, cols, 32768,
                                      None) == want
    rope = bk.CRope()
    L.basiskv_rope_init(ctypes.byref(rope), ctypes.byref(_params()))
    assert L.basiskv_rotary(ctypes.byref(_cfg()), ctypes.byref(rope), 256, 4096, None, 0, 131072, None, None, 512,
                            1 << 16, 1 << 15, None) == UNS
    c = _cfg(page_size=64)
    for batch, n, mp in ((65535, 1, 49152), (65535, 4096, 64)):  # tiles of the tables, rows of the call
        cache = bk.CCache(256, 256, None, None, 256, 256, 1 << 20, mp)
        assert L.basiskv_dense_attn(ctypes.byref(c), ctypes.byref(cache), 256, batch, n, None, 256, None, 256, 1 << 60,
                                    256, None) == UNS
        assert L.basiskv_dense_attn_workspace_bytes(ctypes.byref(c), batch, n, mp) == 0
    assert L.basiskv_dense_attn_workspace_bytes(ctypes.byref(c), 8192, 1, 49152) > 0


@pytest.mark.parametrize("opt", [dict(softcap=1e-44), dict(softcap=3e38), dict(scale=3e38),
                                 dict(scale=1e-42), dict(scale=1e-30, softcap=1e20)])
def test_dense_attn_refuses_scores_that_fp32_does_not_hold(L, opt):
    """scale / softcap, softcap log2(e) and scale log2(e) are fp32 factors in the kernels."""
    cache = bk.CCache(256, 256, None, None, 256, 256, 10, 10)
    assert L.basiskv_dense_attn(ctypes.byref(_cfg()), ctypes.byref(cache), 256, 1, 1,
                                ctypes.byref(bk.CAttnOptions(**opt)), 256, None, 256, 1 << 40, 256, None) == BAD


def test_dense_workspace_bytes(L):
    c = ctypes.byref(_cfg())
    assert L.basiskv_dense_attn_workspace_bytes(c, 8, 1, 2048) > 0
    for args in ((0, 1, 10), (1, 0, 10), (1, 1, 0), (1, 161, 10), (65536, 1, 10), (1, 1, 49153)):
        assert L.basiskv_dense_attn_workspace_bytes(c, *args) == 0, args
    assert L.basiskv_dense_attn_workspace_bytes(ctypes.byref(_cfg(head_dim=96)), 1, 1, 10) == 0
    assert L.basiskv_dense_attn_workspace_bytes(None, 1, 1, 10) == 0


def test_binding_refuses_host_tensors_and_bad_arguments(L):
    cfg = bk.Config(8, 2, 64, 16, 8, 16, 512, 8, torch.float32)
    i = torch.zeros(1, dtype=torch.int32)
    t2 = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bk.assign_pages(cfg, t2, i, i, t2[0], i, i, i, None, i)
    with pytest.raises(ValueError, match="max_pages"):
        bk.release_pages(cfg, i, i, i, t2[0], i, i, i, i)
    with pytest.raises(ValueError, match="layout"):
        bk.Rope(cfg, layout="both")
    with pytest.raises(ValueError, match="scaling"):
        bk.Rope(cfg, scaling="longer")
    with pytest.raises(ValueError, match="rotary_dim"):
        bk.Rope(cfg, rotary_dim=66)
    with pytest.raises(bk.BasisKVError):
        bk.Rope(cfg, rotary_dim=7)
    rope = bk.Rope(cfg, rotary_dim=32)
    assert len(rope.inv_freq) == 16 and rope.mscale == 1.0
    q = torch.zeros((1, 1, 8, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        bk.rotary(cfg, rope, q, None, q, None, seq_len=i)
    with pytest.raises(ValueError, match="neither"):
        bk.rotary(cfg, rope, None, None, None, None, seq_len=i)
    with pytest.raises(ValueError, match="together"):
        bk.rotary(cfg, rope, q, None, None, None, seq_len=i)

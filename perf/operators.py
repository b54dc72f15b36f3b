"""The serving operators around the paged cache, as cases to be measured.

``run`` computes each one either in its plain form (elementary torch
operations, 32 bits, no fused library call) or, where ``own`` is set, with the
framework's calls.  Four operators, used in this order by a decode step or a
prompt: pages for the new tokens (``assign``, and ``release`` for requests that
end), rotary positions for the new queries and keys (``rotary``), and
attention of the new tokens over the whole paged cache (``attn``).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _pages(name, op, batch, page, max_pages, lo, hi, add_lo, add_hi, share=0.0):
    return dict(name=name, op=op, batch=batch, page=page, max_pages=max_pages, lo=lo, hi=hi,
                add_lo=add_lo, add_hi=add_hi, share=share)


def _rotary(name, batch, n_new, hq, hkv, d, rot, layout, scaling, dtype, far, packed):
    return dict(name=name, op="rotary", batch=batch, n_new=n_new, hq=hq, hkv=hkv, d=d, rot=rot, layout=layout,
                scaling=scaling, dtype=dtype, far=far, packed=packed)


def _attn(name, batch, n_new, lo, hi, hq, hkv, d, r, page, dtype, window=0, softcap=0.0, slopes=False, prefix=0,
          qscale=2.0):
    return dict(name=name, op="attn", batch=batch, n_new=n_new, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, r=r, page=page,
                dtype=dtype, window=window, softcap=softcap, slopes=slopes, prefix=prefix, qscale=qscale)


def listed():
    return [
        # one decode step of a serving batch: every request grows by a token, some need a page
        _pages("pages-decode-64", "assign", 64, 16, 2049, 2048, 32768, 1, 1),
        # a batch of prompts comes in: whole block tables and the slot of every token
        _pages("pages-prompts-64", "assign", 64, 16, 2048, 0, 0, 2048, 32768),
        # half of the batch's requests end and give their pages back
        _pages("pages-release-64", "release", 64, 16, 2048, 2048, 32768, 0, 0, 0.5),
        # the decode step's queries and keys far into long contexts, frequencies scaled by band
        _rotary("rotary-decode-64", 64, 1, 32, 8, 128, 128, "half", "llama3", "bf16", 131072, False),
        # a whole 32K prompt out of a packed projection, scaled by ramp
        _rotary("rotary-prompt-32k", 1, 32767, 32, 8, 128, 128, "half", "yarn", "bf16", 32767, True),
        # the small fp32 layer with a part of each head rotated in interleaved pairs
        _rotary("rotary-partial-fp32", 3, 1999, 8, 2, 64, 32, "interleaved", "linear", "f32", 4096, False),
        # decode of the small fp32 layer: a call that is all latency
        _attn("attn-decode-tiny-fp32", 1, 1, 2048, 2048, 8, 2, 64, 16, 32, "f32"),
        # decode of eight 32K contexts
        _attn("attn-decode-8x32k", 8, 1, 32768, 32768, 32, 8, 128, 64, 16, "bf16"),
        # decode of a ragged batch in a layer with a sliding window and capped scores
        _attn("attn-decode-ragged-window", 64, 1, 2048, 32768, 32, 8, 128, 64, 16, "bf16", window=4096, softcap=50.0),
        # decode of one very long context, distance bias
        _attn("attn-decode-131k-bias", 1, 1, 131071, 131071, 32, 8, 128, 64, 64, "bf16", slopes=True),
        # a whole prompt
        _attn("attn-prompt-8k", 1, 8192, 8192, 8192, 32, 8, 128, 64, 16, "bf16"),
        # a chunk of a longer prompt of the wide layer: capped scores, a prefix that sees itself
        _attn("attn-chunk-1k-of-16k", 1, 1021, 16381, 16381, 64, 8, 128, 96, 16, "bf16", softcap=30.0, prefix=15900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "release", "rotary", "decode", "decode", "chunk", "chunk", "plain"])
    if op in ("assign", "release"):
        page = rng.choice([16, 32, 64])
        longest = _log(rng, 64, 32000)
        batch = _log(rng, 1, max(2, min(256, 2000000 // longest)))
        if op == "release":
            return {k: v for k, v in _pages("", op, batch, page, longest // page + 2, longest // 3, longest, 0, 0,
                                            rng.choice([0.1, 0.5, 1.0])).items() if k != "name"}
        add = _log(rng, 1, longest)
        return {k: v for k, v in _pages("", op, batch, page, (longest + add) // page + 2, longest // 3, longest,
                                        rng.choice([0, 1]), add).items() if k != "name"}
    if op == "rotary":
        d = rng.choice([64, 128])
        tokens = _log(rng, 1, 30000)
        n_new = rng.choice([1, tokens, max(1, tokens // 3)])
        hkv = rng.choice([1, 2, 8])
        c = _rotary("", max(1, min(512, tokens // n_new)), n_new, hkv * rng.choice([1, 2, 4]), hkv, d,
                    rng.choice([d, d // 2, d // 4, d - 12]), rng.choice(["half", "interleaved"]),
                    rng.choice(["none", "linear", "ntk", "yarn", "llama3"]), rng.choice(["bf16", "bf16", "f32"]),
                    n_new + _log(rng, 1, 500000), rng.choice([False, True]))
        return {k: v for k, v in c.items() if k != "name"}
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    softcap = rng.choice([0.0, 0.0, 30.0])
    slopes = rng.choice([False, False, True])
    if op == "plain":  # fp32, and ranks that are no multiple of 16
        hkv = rng.choice([1, 2])
        n_new = rng.choice([1, 1, _log(rng, 2, 300)])
        hi = n_new + _log(rng, 1, 6000)
        c = _attn("", rng.choice([1, 3]), n_new, max(n_new, hi // 2), hi, hkv * rng.choice([1, 4]), hkv,
                  rng.choice([64, 128]), rng.choice([16, 24, 40]), rng.choice([16, 32]), rng.choice(["f32", "bf16"]),
                  window, softcap, slopes, rng.choice([0, hi // 3]))
        return {k: v for k, v in c.items() if k != "name"}
    hkv, g = rng.choice([1, 2, 8]), rng.choice([1, 2, 4, 8])
    d, r = rng.choice([(64, 16), (64, 48), (128, 32), (128, 64), (128, 96), (128, 128)])
    if op == "decode":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 40, min(131072, 400000 // batch))
        n_new = rng.choice([1, 1, 1, 2, 5])
        c = _attn("", batch, n_new, max(n_new, hi // 4), hi, hkv * g, hkv, d, r, rng.choice([16, 32, 64]), "bf16",
                  window, softcap, slopes, 0)
    else:
        batch = rng.choice([1, 1, 2])
        n_new = _log(rng, 17, 2000) // batch + 1
        hi = n_new + rng.choice([0, _log(rng, 1, 5000)])
        c = _attn("", batch, n_new, max(n_new, hi - 300), hi, hkv * g, hkv, d, r,
                  rng.choice([16, 32, 64]), "bf16", window, softcap, slopes, rng.choice([0, 0, hi // 2]))
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _lengths(rng, lo, hi, batch):
    return rng.integers(lo, hi, size=batch, endpoint=True).astype(np.int32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _prepare_pages(case, seed):
    rng = np.random.default_rng(seed)
    B, P, mp = case["batch"], case["page"], case["max_pages"]
    assign = case["op"] == "assign"
    seq = _lengths(rng, case["lo"], case["hi"], B)
    add = _lengths(rng, case["add_lo"], case["add_hi"], B)
    have = -(-seq // P)
    total = int(have.sum())
    phys = B * (-(-(case["hi"] + case["add_hi"]) // P) + 1)  # a pool that holds every request at its longest
    spare = phys - total
    perm = rng.permutation(phys).astype(np.int32)
    table = np.full((B, mp), -1, np.int32)
    table[np.arange(mp)[None, :] < have[:, None]] = perm[:total]
    free = np.full(phys, -1, np.int32)
    free[:spare] = perm[total:]
    st = dict(op=case["op"], page=P, phys=phys, table=_dev(table), seq=_dev(seq), free=_dev(free),
              count=_dev(np.array([spare], np.int32)), seq_out=_dev(seq), count_out=_dev(np.array([0], np.int32)))
    if assign:
        st["add"] = _dev(add)
        st["slots"] = torch.empty((B, max(1, int(case["add_hi"]))), dtype=torch.int32, device=DEV)
    else:
        st["release"] = _dev((rng.random(B) < case["share"]).astype(np.int32))
    if own:
        from long_context_decode_basiskv_b200 import binding as bk
        st.update(bk=bk, cfg=bk.Config(32, 8, 128, 64, 32, P, 4096, 128, torch.bfloat16),
                  err=torch.zeros(1, dtype=torch.int32, device=DEV))
    return st


_ORIG = 8192  # context the frequencies were made for, where they are scaled


def _scaling_of(case):
    return dict(kind=case["scaling"], factor=8.0, original=_ORIG, beta_fast=32.0, beta_slow=1.0, low=1.0, high=4.0)


def _frequencies(case):
    """Radians per position of each pair (64 bits) and the factor on cos and sin."""
    rot, base, s = case["rot"], 500000.0, _scaling_of(case)
    i = torch.arange(rot // 2, dtype=torch.float64)
    if s["kind"] == "ntk" and rot > 2:
        base = base * s["factor"] ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    m = 1.0
    if s["kind"] == "linear":
        f = f / s["factor"]
    elif s["kind"] == "llama3":
        wave = 2 * math.pi / f
        mix = ((s["original"] / wave - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        f = (1 - mix) * f / s["factor"] + mix * f
    elif s["kind"] == "yarn":
        def at(turns):
            return rot * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(s["beta_fast"])), 0), min(math.ceil(at(s["beta_slow"])), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / s["factor"] * ramp + f * (1 - ramp)
        m = 0.1 * math.log(s["factor"]) + 1.0
    return f, m


def _prepare_rotary(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, n, hq, hkv, d, td = case["batch"], case["n_new"], case["hq"], case["hkv"], case["d"], _dtype(case)
    if case["packed"]:  # one row of the fused projection per token: queries, keys, values
        x = torch.randn((B, n, hq + 2 * hkv, d), generator=gen, device=DEV).to(td)
        q, k = x[:, :, :hq], x[:, :, hq:hq + hkv]
    else:
        q = torch.randn((B, n, hq, d), generator=gen, device=DEV).to(td)
        k = torch.randn((B, n, hkv, d), generator=gen, device=DEV).to(td)
    f, m = _frequencies(case)
    st = dict(op="rotary", q=q, k=k, seq=_dev(_lengths(rng, n, max(n, case["far"]), B)), freq=f.to(DEV), m=m,
              rot=case["rot"], layout=case["layout"])
    if own:
        from long_context_decode_basiskv_b200 import binding as bk
        cfg = bk.Config(hq, hkv, d, 16, 8, 16, 512, 8, td)
        s = _scaling_of(case)
        st.update(bk=bk, cfg=cfg,
                  rope=bk.Rope(cfg, base=500000.0, rotary_dim=case["rot"], layout=case["layout"], scaling=s["kind"],
                               factor=s["factor"], original_len=s["original"], beta_fast=s["beta_fast"],
                               beta_slow=s["beta_slow"], low_freq_factor=s["low"], high_freq_factor=s["high"]),
                  q_out=torch.empty((B, n, hq, d), dtype=td, device=DEV),
                  k_out=torch.empty((B, n, hkv, d), dtype=td, device=DEV))
    return st


def _prepare_attn(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, n, hq, hkv, d, r, P = (case[x] for x in ("batch", "n_new", "hq", "hkv", "d", "r", "page"))
    td = _dtype(case)
    seq = _lengths(rng, case["lo"], case["hi"], B)
    have = -(-seq // P)
    mp, phys = int(have.max()), int(have.sum())
    table = np.full((B, mp), -1, np.int32)
    table[np.arange(mp)[None, :] < have[:, None]] = rng.permutation(phys).astype(np.int32)
    # keys and latents of the size that the decode workloads give them; queries sharp enough that
    # a row's weights are far from uniform
    k = torch.randn((phys, hkv, P, d), generator=gen, device=DEV).mul_(0.8).to(td)
    c = torch.randn((phys, hkv, P, r), generator=gen, device=DEV).to(td)
    q = torch.randn((B, n, hq, d), generator=gen, device=DEV).mul_(case["qscale"]).to(td)
    slopes = None
    if case["slopes"]:
        slopes = torch.pow(2.0, -8.0 * (torch.arange(hq, device=DEV, dtype=torch.float32) + 1) / hq)
    prefix = None
    if case["prefix"]:
        prefix = torch.full((B,), case["prefix"], dtype=torch.int32, device=DEV)
    st = dict(op="attn", k=k, c=c, q=q, table=_dev(table), seq=_dev(seq), window=case["window"],
              softcap=case["softcap"], slopes=slopes, prefix=prefix, page=P)
    if own:
        from long_context_decode_basiskv_b200 import binding as bk
        cfg = bk.Config(hq, hkv, d, r, 8, P, 512, 8, td)
        cache = bk.PagedCache(cfg, phys, st["table"], st["seq"])
        cache.k_raw, cache.c_lat = k, c  # the pages made above
        st.update(bk=bk, cfg=cfg, cache=cache,
                  opts=bk.AttnOptions(softcap=case["softcap"], window=case["window"], slopes=slopes, prefix_len=prefix),
                  o=torch.empty((B, n, hq, r), dtype=torch.float32, device=DEV),
                  lse=torch.empty((B, n, hq), dtype=torch.float32, device=DEV),
                  ws=bk.alloc_dense_workspace(cfg, B, n, mp), err=torch.zeros(1, dtype=torch.int32, device=DEV))
    return st


def prepare(case, seed):
    if case["op"] == "rotary":
        return _prepare_rotary(case, seed)
    if case["op"] == "attn":
        return _prepare_attn(case, seed)
    return _prepare_pages(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_assign(s):
    P, table, seq, add, count = s["page"], s["table"], s["seq"].long(), s["add"].long(), s["count"].long()
    have, want = (seq + P - 1) // P, (seq + add + P - 1) // P
    off = torch.cumsum(want - have, 0) - (want - have)
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    new = (j >= have[:, None]) & (j < want[:, None])
    at = (count - 1 - (off - have)[:, None] - j).clamp(0, s["phys"] - 1)
    table = torch.where(new, s["free"][at], table)
    t = torch.arange(s["slots"].shape[1], device=DEV)[None, :]
    pos = seq[:, None] + t
    page = torch.gather(table, 1, (pos // P).clamp(max=table.shape[1] - 1)).long()
    slots = torch.where(t < add[:, None], page * P + pos % P, -1)
    return table, (seq + add).int(), (count - (want - have).sum()).int(), slots.int()


def _plain_release(s):
    P, table, seq, count = s["page"], s["table"], s["seq"].long(), s["count"].long()
    gone = s["release"] != 0
    n = torch.where(gone, (seq + P - 1) // P, 0)
    off = torch.cumsum(n, 0) - n
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    to = torch.where(j < n[:, None], count + off[:, None] + j, s["phys"])  # the last place takes what is not pushed
    free = torch.cat([s["free"], s["free"][:1]]).scatter(0, to.reshape(-1), table.reshape(-1))[:-1]
    return free, torch.where(gone, 0, seq).int(), (count + n.sum()).int()


def _plain_rotary(s):
    n, rot = s["q"].shape[1], s["rot"]
    pos = (s["seq"].long() - n)[:, None] + torch.arange(n, device=DEV)
    a = pos.double()[:, :, None] * s["freq"]
    cos, sin = (a.cos() * s["m"]).float()[:, :, None], (a.sin() * s["m"]).float()[:, :, None]

    def turn(x):
        y = x.float()
        if s["layout"] == "half":
            u, v = y[..., :rot // 2], y[..., rot // 2:rot]
            out = torch.cat([u * cos - v * sin, v * cos + u * sin, y[..., rot:]], -1)
        else:
            u, v = y[..., 0:rot:2], y[..., 1:rot:2]
            out = torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), y[..., rot:]], -1)
        return out.to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _rows(pages, table, columns):
    """[batch][heads][tokens][columns] in token order, 32 bits: the pages of every sequence, with
    the order of 16-byte chunks that bf16 pages are stored in undone."""
    x = pages[table.clamp(min=0).long()]                      # [B][pages][heads][P][columns]
    x = x.permute(0, 2, 1, 3, 4)
    if columns is not None:
        x = x.gather(4, columns.expand(x.shape))
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4]).float()


def _chunk_columns(x, other):
    """Where each column of a page's rows is stored, [P][columns], or None where rows are plain."""
    if x.dtype != torch.bfloat16 or x.shape[3] % 16 or other.shape[3] % 16:
        return None
    chunks = x.shape[3] // 8
    mask = 7 if chunks % 8 == 0 else 3 if chunks % 4 == 0 else 1
    row, col = torch.arange(x.shape[2], device=DEV)[:, None], torch.arange(x.shape[3], device=DEV)[None, :]
    return ((col // 8) ^ (row & mask)) * 8 + col % 8


def _plain_attn(s):
    q, seq = s["q"], s["seq"].long()
    B, n, hq, d = q.shape
    hkv, r = s["c"].shape[1], s["c"].shape[3]
    k, c = _rows(s["k"], s["table"], _chunk_columns(s["k"], s["c"])), _rows(s["c"], s["table"],
                                                                        _chunk_columns(s["c"], s["k"]))
    qh = q.float().permute(0, 2, 1, 3).reshape(B, hkv, -1, d)          # rows: head of the group, then token
    x = (qh @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).reshape(B, hq, n, -1)
    if s["softcap"]:
        x = torch.tanh(x.div_(s["softcap"])).mul_(s["softcap"])
    i = (seq - n)[:, None, None] + torch.arange(n, device=DEV)[:, None]    # [B][n][1]
    j = torch.arange(x.shape[3], device=DEV)
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * (i - j).abs()[:, None].float()
    see = j <= i
    if s["window"]:
        see = see & (i - j < s["window"])
    if s["prefix"] is not None:
        see = see | (j < torch.minimum(s["prefix"].long(), seq)[:, None, None])
    x = x.masked_fill(~see[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0.0, top)
    w = x.sub_(base).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.reshape(B, hkv, -1, w.shape[3]) @ c).reshape(B, hq, n, r)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (base + total.log())[..., 0]
    return o.transpose(1, 2).contiguous(), lse.transpose(1, 2).contiguous()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        bk = s["bk"]
        if s["op"] == "assign":
            bk.assign_pages(s["cfg"], s["table"], s["seq"], s["add"], s["free"], s["count"], s["seq_out"],
                            s["count_out"], s["slots"], s["err"])
            return s["table"], s["seq_out"], s["count_out"], s["slots"]
        if s["op"] == "release":
            bk.release_pages(s["cfg"], s["table"], s["seq"], s["release"], s["free"], s["count"], s["seq_out"],
                             s["count_out"], s["err"])
            return s["free"], s["seq_out"], s["count_out"]
        if s["op"] == "rotary":
            bk.rotary(s["cfg"], s["rope"], s["q"], s["k"], s["q_out"], s["k_out"], seq_len=s["seq"])
            return s["q_out"], s["k_out"]
        bk.dense_attn(s["cfg"], s["cache"], s["q"], s["o"], s["ws"], s["err"], options=s["opts"], lse=s["lse"])
        return s["o"], s["lse"]
    return {"assign": _plain_assign, "release": _plain_release, "rotary": _plain_rotary, "attn": _plain_attn}[s["op"]](s)


# ---------------------------------------------------------------------------
# floors
# ---------------------------------------------------------------------------
def _expected_pairs(case, L):
    """Query-key pairs that one head of a sequence of L tokens scores, and the keys that any row sees."""
    n, w, pre = case["n_new"], case["window"], min(case["prefix"], L)
    i = np.arange(L - n, L, dtype=np.int64)
    lo = np.maximum(0, i - w + 1) if w else np.zeros_like(i)
    pairs = np.where(pre > i, pre, i + 1 - lo + np.minimum(pre, lo))
    first = int(lo[0])
    return int(pairs.sum()), L - first + min(pre, first)


def work(case):
    B = case["batch"]
    if case["op"] in ("assign", "release"):
        P, mid = case["page"], (case["lo"] + case["hi"]) / 2
        if case["op"] == "release":
            pages = case["share"] * B * mid / P
            return {"bytes": 8.0 * pages + 12 * B + 8, "flops": 0.0}
        add = (case["add_lo"] + case["add_hi"]) / 2
        return {"bytes": 8.0 * B * add / P + 4.0 * B * max(1, case["add_hi"]) + 16 * B + 8, "flops": 0.0}
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotary":
        tokens = B * case["n_new"] * (case["hq"] + case["hkv"])
        return {"bytes": 2.0 * tokens * case["d"] * e + 4 * B, "flops": 3.0 * tokens * case["rot"]}
    L = (case["lo"] + case["hi"]) // 2
    pairs, keys = _expected_pairs(case, L)
    new = B * case["n_new"] * case["hq"]
    return {"bytes": float(B * keys * case["hkv"] * (case["d"] + case["r"]) * e + new * (case["d"] * e + case["r"] * 4 + 4)),
            "flops": 2.0 * B * case["hq"] * pairs * (case["d"] + case["r"])}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotary(case, s):
    """Each pair as a complex number times m exp(i angle)."""
    n, rot = case["n_new"], case["rot"]
    f, m = _frequencies(case)
    out = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        for b in range(case["batch"]):
            first = int(s["seq"][b]) - n
            pos = torch.arange(first, first + n, dtype=torch.float64, device=DEV)
            spin = torch.polar(torch.full((n, 1, rot // 2), m, dtype=torch.float64, device=DEV),
                               (pos[:, None] * f.to(DEV)[None, :])[:, None, :])
            if case["layout"] == "half":
                z = torch.complex(y[b, ..., :rot // 2], y[b, ..., rot // 2:rot]) * spin
                y[b, ..., :rot // 2], y[b, ..., rot // 2:rot] = z.real, z.imag
            else:
                z = torch.view_as_complex(y[b, ..., :rot].reshape(*y.shape[1:-1], rot // 2, 2).contiguous()) * spin
                y[b, ..., :rot] = torch.view_as_real(z).flatten(-2)
        out.append(y)
    return tuple(out)


def _exact_attn(case, s):
    B, n, hq, hkv, d, r, P = (case[x] for x in ("batch", "n_new", "hq", "hkv", "d", "r", "page"))
    swizzled = case["dtype"] == "bf16" and d % 16 == 0 and r % 16 == 0

    def stored(page_rows, width):  # [pages * P][width]: chunk c of row j sits at chunk c ^ (j & mask)
        if not swizzled:
            return page_rows
        x = page_rows.reshape(-1, P, width // 8, 8)
        chunks = width // 8
        mask = 7 if chunks % 8 == 0 else 3 if chunks % 4 == 0 else 1
        y = torch.empty_like(x)
        for j in range(P):
            y[:, j] = x[:, j, [c ^ (j & mask) for c in range(chunks)]]
        return y.reshape(-1, width)

    o = torch.zeros((B, n, hq, r), dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, hq), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        L = int(s["seq"][b])
        pages = s["table"][b, :-(-L // P)].long()
        pre = min(int(s["prefix"][b]), L) if s["prefix"] is not None else 0
        for g in range(hkv):
            K = stored(s["k"][pages, g].reshape(-1, d), d)[:L].double()
            C = stored(s["c"][pages, g].reshape(-1, r), r)[:L].double()
            step = max(1, (1 << 26) // L)
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                for t0 in range(0, n, step):
                    i = torch.arange(L - n + t0, L - n + min(n, t0 + step), device=DEV)[:, None]
                    j = torch.arange(L, device=DEV)[None, :]
                    x = s["q"][b, t0:t0 + step, h].double() @ K.T / math.sqrt(d)
                    if case["softcap"]:
                        x = case["softcap"] * torch.tanh(x / case["softcap"])
                    if s["slopes"] is not None:
                        x = x - s["slopes"][h].double() * (i - j).abs()
                    hidden = j > i
                    if case["window"]:
                        hidden = hidden | (j <= i - case["window"])
                    hidden = hidden & (j >= pre)
                    x[hidden] = -math.inf
                    z = torch.logsumexp(x, 1)
                    lse[b, t0:t0 + step, h] = z
                    o[b, t0:t0 + step, h] = torch.exp(x - z[:, None]).nan_to_num(0.0) @ C
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    if case["op"] == "attn":
        return _exact_attn(case, s)
    return None  # whole numbers: compared as they are

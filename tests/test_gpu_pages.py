"""basiskv_assign_pages and basiskv_release_pages against a plain loop on the host."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from long_context_decode_basiskv_b200 import binding as bk  # noqa: E402
from long_context_decode_basiskv_b200.pages import PagePool  # noqa: E402


def cfg_of(page):
    return bk.Config(32, 8, 128, 64, 32, page, 4096, 128, torch.bfloat16)


def assign_plain(P, seq, add, table, free, count, cols):
    table, seq, slots = table.copy(), seq.astype(np.int64), np.full((len(seq), cols), -1, np.int64)
    for b in range(len(seq)):
        for t in range(int(add[b])):
            pos = int(seq[b]) + t
            if pos % P == 0:
                count -= 1
                table[b, pos // P] = free[count]
            if t < cols:
                slots[b, t] = int(table[b, pos // P]) * P + pos % P
    return table, (seq + add).astype(np.int32), count, slots


def release_plain(P, seq, rel, table, free, count):
    free, seq = free.copy(), seq.copy()
    for b in range(len(seq)):
        if rel[b]:
            for x in range(-(-int(seq[b]) // P)):
                free[count] = table[b, x]
                count += 1
            seq[b] = 0
    return free, seq, count


def state(rng, B, P, lo, hi, extra_pages, spare):
    seq = rng.integers(lo, hi, B, endpoint=True).astype(np.int32)
    have = -(-seq // P)
    mp = int(have.max()) + extra_pages
    phys = int(have.sum()) + spare
    perm = rng.permutation(phys).astype(np.int32)
    table = np.full((B, mp), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    free = np.full(phys, -9, np.int32)
    free[:spare] = perm[at:]
    return seq, table, free, spare


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(x):
    return torch.tensor([x], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,P,lo,hi,add_lo,add_hi,cols", [
    (1, 16, 0, 0, 1, 1, 1),
    (1, 64, 63, 64, 0, 130, 130),
    (5, 32, 0, 100, 0, 0, 4),                 # nothing to add
    (64, 16, 100, 900, 1, 1, 1),              # a decode step
    (64, 16, 100, 900, 1, 1, None),           # ... without slots
    (37, 16, 0, 200, 0, 700, 701),            # odd rows of slots (single stores)
    (37, 16, 0, 200, 0, 700, 640),            # fewer columns than tokens, vector stores
    (33, 64, 1, 5000, 0, 3000, 3000),         # a cluster
    (3000, 16, 0, 40, 0, 40, 8),              # several requests per thread
    (1025, 32, 0, 70, 0, 3, 3),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_assign(B, P, lo, hi, add_lo, add_hi, cols, in_place):
    rng = np.random.default_rng(B + P + hi)
    add = rng.integers(add_lo, add_hi, B, endpoint=True).astype(np.int32)
    seq, table, free, count = state(rng, B, P, lo, hi, add_hi // P + 1, int((add // P + 1).sum()) + 2)
    want = assign_plain(P, seq, add, table, free, count, cols or 1)
    s, c, t, err = cu(seq), i32(count), cu(table), i32(0)
    so, co = (s, c) if in_place else (torch.full_like(s, 77), i32(88))
    slots = None if cols is None else torch.full((B, cols), 55, dtype=torch.int32, device="cuda")
    bk.assign_pages(cfg_of(P), t, s, cu(add), cu(free), c, so, co, slots, err)
    assert int(err.item()) == 0
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert np.array_equal(so.cpu().numpy(), want[1])
    assert int(co.item()) == want[2]
    if cols:
        assert np.array_equal(slots.cpu().numpy(), want[3])


@pytest.mark.parametrize("B,P,lo,hi", [(1, 16, 0, 0), (1, 16, 1, 1), (64, 16, 100, 9000), (2000, 32, 0, 200)])
@pytest.mark.parametrize("share", [0.0, 0.5, 1.0])
def test_release(B, P, lo, hi, share):
    rng = np.random.default_rng(B + P)
    seq, table, free, count = state(rng, B, P, lo, hi, 2, 5)
    rel = (rng.random(B) < share).astype(np.int32) * 3           # any nonzero value
    want = release_plain(P, seq, rel, table, free, count)
    s, c, f, err = cu(seq), i32(count), cu(free), i32(0)
    bk.release_pages(cfg_of(P), cu(table), s, cu(rel), f, c, s, c, err)
    assert int(err.item()) == 0
    assert np.array_equal(f.cpu().numpy(), want[0])
    assert np.array_equal(s.cpu().numpy(), want[1])
    assert int(c.item()) == want[2]


@pytest.mark.parametrize("B", [3, 200])
@pytest.mark.parametrize("fault,bit", [
    ("few", bk.DEVERR_PAGES), ("count", bk.DEVERR_PAGES), ("negative_count", bk.DEVERR_PAGES),
    ("add", bk.DEVERR_SEQ_LEN), ("seq", bk.DEVERR_SEQ_LEN), ("wide", bk.DEVERR_SEQ_LEN),
    ("overflow", bk.DEVERR_SEQ_LEN), ("free_id", bk.DEVERR_BLOCK_TABLE), ("last_page", bk.DEVERR_BLOCK_TABLE),
])
def test_assign_faults_change_nothing(B, fault, bit):
    P, cols = 16, 64
    rng = np.random.default_rng(5)
    add = np.full(B, 40, np.int32)
    seq, table, free, count = state(rng, B, P, 17, 30, 4, 4 * B)
    if fault == "few":
        count = 2 * B - 1
    elif fault == "count":
        count = free.size + 1
    elif fault == "negative_count":
        count = -1
    elif fault == "add":
        add[B - 1] = -1
    elif fault == "seq":
        seq[1] = -16
    elif fault == "wide":
        add[0] = table.shape[1] * P - seq[0] + 1
    elif fault == "overflow":
        add[0] = 2**31 - 1
    elif fault == "free_id":
        free[count - 2] = free.size
    else:
        table[B - 1, seq[B - 1] // P] = -1
    s, c, t, err, f = cu(seq), i32(count), cu(table), i32(0), cu(free)
    so, co = torch.zeros_like(s), i32(0)
    slots = torch.full((B, cols), 55, dtype=torch.int32, device="cuda")
    bk.assign_pages(cfg_of(P), t, s, cu(add), f, c, so, co, slots, err)
    assert int(err.item()) & bit
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(f.cpu().numpy(), free)
    assert np.array_equal(so.cpu().numpy(), seq) and int(co.item()) == count
    assert (slots == -1).all()


@pytest.mark.parametrize("fault,bit", [("full", bk.DEVERR_PAGES), ("id", bk.DEVERR_BLOCK_TABLE),
                                       ("long", bk.DEVERR_SEQ_LEN)])
def test_release_faults_change_nothing(fault, bit):
    P, B = 16, 90
    rng = np.random.default_rng(6)
    seq, table, free, count = state(rng, B, P, 100, 300, 1, 4)
    if fault == "full":
        count = free.size - 3
    elif fault == "id":
        table[50, 2] = free.size + 1
    else:
        seq[3] = table.shape[1] * P + 1
    s, c, f, err = cu(seq), i32(count), cu(free), i32(0)
    bk.release_pages(cfg_of(P), cu(table), s, torch.ones_like(s), f, c, s, c, err)
    assert int(err.item()) & bit
    assert np.array_equal(f.cpu().numpy(), free) and np.array_equal(s.cpu().numpy(), seq) and int(c.item()) == count


def test_pool_over_many_steps_in_a_graph():
    """Requests grow and end for a while, the growth replayed from a captured graph: no page is ever
    held twice, and all of them come back."""
    B, P, mp = 20, 16, 30
    pool = PagePool(cfg_of(P), B * mp, B, mp)
    err, add = i32(0), torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.zeros((B, 32), dtype=torch.int32, device="cuda")
    pool.extend(add, err, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.extend(add, err, slots)
    rng = np.random.default_rng(0)
    for step in range(40):
        add.copy_(cu(rng.integers(0, 33, B).astype(np.int32)))
        rel = ((pool.seq_len + add) > P * mp).int()
        pool.release(rel, err)
        g.replay()
        L, t = pool.seq_len.cpu().numpy(), pool.block_table.cpu().numpy()
        held = np.concatenate([t[b, :-(-int(L[b]) // P)] for b in range(B)])
        free = pool.free_pages[:int(pool.free_count.item())].cpu().numpy()
        assert int(err.item()) == 0
        assert np.array_equal(np.sort(np.concatenate([held, free])), np.arange(B * mp))
        used = slots[slots >= 0].cpu().numpy()
        assert len(np.unique(used)) == used.size == int(add.sum())
    pool.release(torch.ones_like(add), err)
    assert int(pool.free_count.item()) == B * mp and int(pool.seq_len.sum()) == 0


def test_empty_batch():
    e, err = torch.zeros(0, dtype=torch.int32, device="cuda"), i32(0)
    t, f, c = torch.zeros((0, 4), dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), i32(4)
    bk.assign_pages(cfg_of(16), t, e, e, f, c, e, c, None, err)
    bk.release_pages(cfg_of(16), t, e, e, f, c, e, c, err)
    assert int(c.item()) == 4 and int(err.item()) == 0

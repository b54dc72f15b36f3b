"""DecodeEngine built and stepped on a stream of the caller's, with that stream far behind the current one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from long_context_decode_basiskv_b200 import binding as bk  # noqa: E402
from long_context_decode_basiskv_b200.engine import DecodeEngine, config_of  # noqa: E402
from long_context_decode_basiskv_b200.workloads import WORKLOADS, make_case, shrink  # noqa: E402

BEHIND = 200_000_000  # cycles: 0.1 s, longer than the host takes to enqueue a build and a step


@pytest.mark.parametrize("behind", ["side", "current"])
@pytest.mark.parametrize("kw", [dict(), dict(paging="pool", roped=True), dict(paging="pool", roped=True, attention="dense"),
                                dict(prefill_mode="tc", roped=True)])
def test_built_on_a_stream(kw, behind):
    """What a build makes on the way (lengths, rotated keys, a pool's free list) is neither read before it is
    there nor written over while the stream may still read it."""
    wl = shrink(WORKLOADS["llama3_8b_32k"], name="streams", batch=6, ragged=(40, 600), top_k=8)
    case = make_case(wl, "cuda")
    kw = dict(kw)
    rope = bk.Rope(config_of(case), base=500000.0) if kw.pop("roped", False) else None
    want = DecodeEngine(case, rope=rope, **kw)
    want.step()
    torch.cuda.synchronize()
    assert int(want.err.item()) == 0
    side = torch.cuda.Stream()
    other = torch.cuda.Stream()
    late = side if behind == "side" else other
    with torch.cuda.stream(other):                  # the current stream of the build
        with torch.cuda.stream(late):
            torch.cuda._sleep(BEHIND)
        eng = DecodeEngine(case, rope=rope, stream=side, **kw)
        eng.step(side)
    torch.cuda.synchronize()
    assert int(eng.err.item()) == 0
    assert torch.equal(eng.cache.seq_len, want.cache.seq_len)
    for b in range(wl.batch):
        assert torch.equal(eng.logical(eng.cache.k_raw, b), want.logical(want.cache.k_raw, b)), b
        assert torch.equal(eng.logical(eng.cache.c_lat, b), want.logical(want.cache.c_lat, b)), b
    assert torch.equal(eng.o_lat, want.o_lat) and torch.equal(eng.y, want.y)


def test_prefill_again_on_a_stream_that_is_behind():
    wl = shrink(WORKLOADS["llama3_8b_32k"], name="streams", batch=6, ragged=(40, 600), top_k=8)
    case = make_case(wl, "cuda")
    eng = DecodeEngine(case, rope=bk.Rope(config_of(case)))
    eng.step()
    torch.cuda.synchronize()
    k, y = [eng.logical(eng.cache.k_raw, b).clone() for b in range(wl.batch)], eng.y.clone()
    eng.cache.k_raw.zero_()
    eng.cache.c_lat.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(BEHIND)
    eng.prefill(side)
    eng.step(side)
    torch.cuda.synchronize()
    assert int(eng.err.item()) == 0
    assert all(torch.equal(eng.logical(eng.cache.k_raw, b), k[b]) for b in range(wl.batch))
    assert torch.equal(eng.y, y)

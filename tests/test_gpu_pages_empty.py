"""Page calls for a batch of no requests: every output is what it would be if the calls did nothing."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from long_context_decode_basiskv_b200 import binding as bk  # noqa: E402


@pytest.mark.parametrize("stream", [False, True])
def test_empty_batch(stream):
    cfg = bk.Config(32, 8, 128, 64, 32, 16, 4096, 128, torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    none, table, free = torch.zeros(0, **i32), torch.zeros((0, 5), **i32), torch.arange(7, **i32)
    err, count = torch.zeros(1, **i32), torch.full((1,), 6, **i32)
    st = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    for call in (lambda out: bk.assign_pages(cfg, table, none, none, free, count, none, out, None, err, st),
                 lambda out: bk.assign_pages(cfg, table, none, none, free, count, none, out,
                                             torch.zeros((0, 3), **i32), err, st),
                 lambda out: bk.release_pages(cfg, table, none, none, free, count, none, out, err, st)):
        out = torch.full((4,), -1, **i32)[3:]          # (no alignment beyond the type's)
        torch.cuda.synchronize()
        call(out)
        call(count)                                    # in place
        torch.cuda.synchronize()
        assert out.tolist() == [6] and count.tolist() == [6]
    assert free.tolist() == list(range(7)) and err.tolist() == [0]

"""basiskv_rotary against the formula in 64 bits.

Bound of an element with pair (u, v): the angle's fraction of a turn is rounded
to fp32 (pi 2^-24 of angle), sincospi is off by at most 2 units in the last
place (2^-23), mscale, two products and a sum add 4 x 2^-24: together below
12 x 2^-24 (|u| + |v|) mscale; then the storage type's half step of the value."""
import pytest
import torch

from tests.serving_reference import rotate

pytestmark = pytest.mark.gpu

from long_context_decode_basiskv_b200 import binding as bk  # noqa: E402


def cfg_of(hq, hkv, d, dtype):
    return bk.Config(hq, hkv, d, 16, 8, 16, 512, 8, dtype)


def check(got, x, pos, rope, layout, dtype):
    want, size = rotate(x, pos, rope.inv_freq, rope.mscale, layout)
    rot = 2 * len(rope.inv_freq)
    half_step = torch.finfo(dtype).eps / 2
    err = (got.double() - want).abs()
    assert (err <= 12 * 2.0 ** -24 * size + half_step * want.abs() + 1e-37).all()
    assert torch.equal(got[..., rot:], x[..., rot:])


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=16.0, original_len=4096), dict(scaling="llama3", factor=8.0, original_len=8192)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hkv,d,rot,B,n", [
    (32, 8, 128, 128, 3, 1), (8, 2, 64, 32, 2, 33), (2, 1, 128, 100, 1, 7), (4, 4, 64, 2, 5, 3), (1, 1, 64, 52, 1, 1),
    (8, 8, 128, 64, 1, 2000),
])
@pytest.mark.parametrize("scaling", range(len(SCALINGS)))
def test_rotary(dtype, layout, hq, hkv, d, rot, B, n, scaling):
    cfg = cfg_of(hq, hkv, d, dtype)
    rope = bk.Rope(cfg, base=500000.0, rotary_dim=rot, layout=layout, **SCALINGS[scaling])
    g = torch.Generator(device="cuda").manual_seed(n + rot)
    q = torch.randn((B, n, hq, d), generator=g, device="cuda").to(dtype)
    k = torch.randn((B, n, hkv, d), generator=g, device="cuda").to(dtype)
    seq = torch.tensor([n + x for x in (0, 131072, 7, 1000003, 12)[:B]], dtype=torch.int32, device="cuda")
    qo, ko = torch.full_like(q, 9), torch.full_like(k, 9)
    bk.rotary(cfg, rope, q, k, qo, ko, seq_len=seq)
    for b in range(B):
        pos = int(seq[b]) - n + torch.arange(n, device="cuda")
        check(qo[b], q[b], pos, rope, layout, dtype)
        check(ko[b], k[b], pos, rope, layout, dtype)
    # explicit positions, in place: the same bits
    pos = (seq[:, None] - n + torch.arange(n, device="cuda", dtype=torch.int32)).contiguous()
    q2, k2 = q.clone(), k.clone()
    bk.rotary(cfg, rope, q2, k2, q2, k2, positions=pos)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    # keys alone
    k3 = torch.empty_like(k)
    bk.rotary(cfg, rope, None, k, None, k3, seq_len=seq)
    assert torch.equal(k3, ko)


@pytest.mark.parametrize("dtype,pad", [(torch.bfloat16, 0), (torch.float32, 0), (torch.bfloat16, 3)])
def test_packed_projection(dtype, pad):
    """Queries and keys as slices of one projection's rows (pad: rows whose stride is no multiple of 16 bytes)."""
    hq, hkv, d, B, n = 8, 2, 64, 2, 19
    cfg = cfg_of(hq, hkv, d, dtype)
    rope = bk.Rope(cfg)
    width = (hq + 2 * hkv) * d + pad
    x = torch.randn((B, n, width), device="cuda").to(dtype)
    v = x[:, :, :width - pad].unflatten(2, (hq + 2 * hkv, d))
    q, k = v[:, :, :hq], v[:, :, hq:hq + hkv]
    seq = torch.tensor([n, 5000], dtype=torch.int32, device="cuda")
    out = [torch.empty((B, n, h, d), dtype=dtype, device="cuda") for h in (hq, hkv, hq, hkv)]
    bk.rotary(cfg, rope, q, k, out[0], out[1], seq_len=seq)
    bk.rotary(cfg, rope, q.contiguous(), k.contiguous(), out[2], out[3], seq_len=seq)
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    with pytest.raises(ValueError, match="evenly spaced"):
        bk.rotary(cfg, rope, q.transpose(2, 3).contiguous().transpose(2, 3), None, out[0], None, seq_len=seq)


def test_positions_and_empty_calls():
    cfg = cfg_of(4, 2, 64, torch.float32)
    rope = bk.Rope(cfg, layout="interleaved")
    q = torch.randn((1, 3, 4, 64), device="cuda")
    pos = torch.tensor([[0, -5, 2**24]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    bk.rotary(cfg, rope, q, None, out, None, positions=pos)
    check(out[0], q[0], pos[0], rope, "interleaved", torch.float32)
    assert torch.equal(out[0, 0], q[0, 0])                # position 0 turns nothing
    e = torch.empty((0, 3, 4, 64), device="cuda")
    bk.rotary(cfg, rope, e, None, e, None, positions=pos[:0])
    e = torch.empty((2, 0, 4, 64), device="cuda")
    bk.rotary(cfg, rope, e, None, e, None, seq_len=torch.zeros(2, dtype=torch.int32, device="cuda"))


def test_other_stream():
    cfg = cfg_of(4, 2, 64, torch.float32)
    rope = bk.Rope(cfg)
    q = torch.randn((1, 300, 4, 64), device="cuda")
    seq = torch.tensor([300], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    bk.rotary(cfg, rope, q, None, a, None, seq_len=seq)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    bk.rotary(cfg, rope, q, None, b, None, seq_len=seq, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a, b)

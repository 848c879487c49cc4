"""What the attention binding refuses on the device, before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import attention
    return attention


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def i32(*shape):
    return z(*shape, dtype=torch.int32)


def u8(*shape):
    return z(*shape, dtype=torch.uint8)


def refused(f, *a, error=ValueError, **k):
    with pytest.raises(error):
        f(*a, **k)


def test_rope(att):
    x, pos, f = z(4, 2, 32), i32(2, 4), z(16, dtype=torch.float32)
    att.rope_axes(x, pos, f, (8, 8))
    for bad in ((x.float(), pos, f, (8, 8)), (x[0], pos, f, (8, 8)), (x.cpu(), pos, f, (8, 8)), (x.transpose(0, 1), pos, f, (8, 8)), (x[..., ::2], pos, f, (8,)),
                (x, pos.long(), f, (8, 8)), (x, i32(4, 2), f, (8, 8)), (x, i32(1, 4), f, (8, 8)), (x, pos.cpu(), f, (8, 8)), (x, pos, f[:8], (8, 8)),
                (x, pos, f.double(), (8, 8)), (x, i32(5, 4), f, (4, 4, 4, 2, 2)), (None, pos, f, (8, 8))):
        refused(att.rope_axes, *bad)
    refused(att.rope_axes, x, pos, f, (8, 8), out=z(4, 2, 48))
    refused(att.rope_axes, x, pos, f, (8, 8), out=z(4, 2, 32, dtype=torch.float16))
    refused(att.rope_axes, x, pos, f, (8, 5), error=RuntimeError)
    refused(att.rope_axes, x, i32(0, 4), f, (), error=(ValueError, RuntimeError))
    refused(att.rope_axes, z(4, 2, 24), pos, f, (4, 4), error=RuntimeError)
    refused(att.rope_axes, z(0, 2, 32), i32(2, 0), f, (8, 8), error=RuntimeError)


def test_cache_rows(att):
    kv, sf, gs = u8(3, 2, 2, 16, 32), u8(3, 2, 2, 4, 16), torch.ones(2, device="cuda")
    k, slots = z(5, 2, 64), torch.arange(5, dtype=torch.int32, device="cuda")
    att.nvfp4_kv_append(k, k, slots, gs, kv, sf)
    for bad in ((k.float(), k, slots, gs, kv, sf), (k, z(5, 3, 64), slots, gs, kv, sf), (k, z(4, 2, 64), slots, gs, kv, sf), (k, k, slots.long(), gs, kv, sf),
                (k, k, slots[:4], gs, kv, sf), (k, k, slots, gs[:1], kv, sf), (k, k, slots, gs.double(), kv, sf), (k, k, slots, gs, kv.short(), sf),
                (k, k, slots, gs, kv[0], sf), (k, k, slots, gs, kv, sf.transpose(3, 4)), (k, k, slots, gs, kv.transpose(2, 3), sf), (k, k, slots, gs, kv, sf.cpu()),
                (k, k, slots, gs, kv, None), (k, k, None, gs, kv, sf), (k.transpose(1, 2).contiguous().transpose(1, 2), k, slots, gs, kv, sf)):
        refused(att.nvfp4_kv_append, *bad)
    refused(att.nvfp4_kv_append, z(5, 2, 64), z(5, 2, 64), slots, gs, u8(3, 2, 2, 48, 32), u8(3, 2, 2, 4, 48), error=RuntimeError)
    refused(att.nvfp4_kv_append, z(5, 2, 272), z(5, 2, 272), slots, gs, u8(3, 2, 2, 16, 136), u8(3, 2, 2, 17, 16), error=RuntimeError)
    att.nvfp4_kv_read(slots, gs, kv, sf)
    refused(att.nvfp4_kv_read, slots, gs, kv, sf, k=z(4, 2, 64))
    refused(att.nvfp4_kv_read, slots, gs, kv, sf, v=z(5, 2, 64, dtype=torch.float16))
    refused(att.nvfp4_kv_read, slots.long(), gs, kv, sf)


def test_decode(att):
    kv, sf, gs = u8(3, 2, 2, 16, 32), u8(3, 2, 2, 4, 16), torch.ones(2, device="cuda")
    q, table, lens = z(2, 1, 4, 64), i32(2, 1), i32(2)
    att.nvfp4_attention_decode(q, kv, sf, gs, table, lens)
    for bad in ((q.float(), kv, sf, gs, table, lens), (q[0], kv, sf, gs, table, lens), (z(2, 1, 5, 64), kv, sf, gs, table, lens), (z(2, 1, 4, 32), kv, sf, gs, table, lens),
                (q, kv, sf, gs, i32(3, 1), lens), (q, kv, sf, gs, i32(2), lens), (q, kv, sf, gs, table.long(), lens), (q, kv, sf, gs, table, i32(1)),
                (q, kv, sf, gs, table, lens.long()), (q.transpose(2, 3).contiguous().transpose(2, 3), kv, sf, gs, table, lens), (q.cpu(), kv, sf, gs, table, lens),
                (z(2, 3, 4, 64).transpose(0, 1).contiguous().transpose(0, 1), kv, sf, gs, table, lens)):
        refused(att.nvfp4_attention_decode, *bad)
    ok = (q, kv, sf, gs, table, lens)
    refused(att.nvfp4_attention_decode, *ok, out=z(2, 1, 4, 32))
    refused(att.nvfp4_attention_decode, *ok, out=z(2, 2, 4, 64)[:, :1])
    refused(att.nvfp4_attention_decode, *ok, lse=z(7, dtype=torch.float32))
    refused(att.nvfp4_attention_decode, *ok, workspace=u8(1000))
    refused(att.nvfp4_attention_decode, *ok, workspace=7)
    refused(att.nvfp4_attention_decode, *ok, scale=0.0, error=RuntimeError)
    refused(att.nvfp4_attention_decode, z(2, 65, 4, 64), *ok[1:], error=RuntimeError)


def test_decode_takes_rows_of_a_projection(att):
    """q as a part of a wider tensor gives what its copy gives."""
    g = torch.Generator(device="cuda").manual_seed(0)
    kv = torch.randint(0, 256, (8, 2, 2, 16, 32), device="cuda", generator=g, dtype=torch.uint8)
    sf = torch.randint(0, 0x60, (8, 2, 2, 4, 16), device="cuda", generator=g, dtype=torch.uint8)
    gs = torch.tensor([300.0, 200.0], device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    lens = torch.tensor([32, 7, 0, 20], dtype=torch.int32, device="cuda")
    qkv = torch.randn(12, 8, 64, device="cuda", generator=g).bfloat16()
    for t in (1, 3):
        wide = qkv[: 4 * t].view(4, t, 8, 64)
        part = wide[:, :, 2:6]
        assert torch.equal(att.nvfp4_attention_decode(part, kv, sf, gs, table, lens), att.nvfp4_attention_decode(part.contiguous(), kv, sf, gs, table, lens))
    one = qkv[:3].view(1, 3, 8, 64)[:, 1:2, 4:8]
    assert torch.equal(att.nvfp4_attention_decode(one, kv, sf, gs, table[:1], lens[:1]), att.nvfp4_attention_decode(one.contiguous(), kv, sf, gs, table[:1], lens[:1]))


def test_prefill_without_rows(att):
    q, k, cu = z(5, 2, 64), z(5, 2, 64), torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    refused(att.attention_prefill, z(0, 2, 64), k, k, cu, error=RuntimeError)
    refused(att.attention_prefill, q, z(0, 2, 64), z(0, 2, 64), cu, error=RuntimeError)
    refused(att.attention_prefill, z(5, 0, 64), k, k, cu, error=RuntimeError)
    refused(att.attention_prefill, q, z(5, 0, 64), z(5, 0, 64), cu)
    refused(att.attention_prefill, q, k, k, cu[:1], error=RuntimeError)
    long = z(4000, 2, 64)
    assert att.attention_prefill_ws_bytes(5, 4000, 2, 2, 1, 64) > 0
    cu_k = torch.tensor([0, 4000], dtype=torch.int32, device="cuda")
    refused(att.attention_prefill, q, long, long, cu, cu_k, workspace=u8(100))
    refused(att.attention_prefill, q, long, long, cu, cu_k, workspace=torch.empty(1 << 26, dtype=torch.uint8))
    refused(att.attention_prefill, q, long, long, cu, cu_k, workspace=u8(1 << 26)[4:], error=RuntimeError)


def test_prefill(att):
    q, k, cu = z(6, 4, 64), z(6, 2, 64), torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    att.attention_prefill(q, k, k, cu)
    for bad in ((q.float(), k, k, cu), (q, k.float(), k, cu), (q, k, z(5, 2, 64), cu), (q, z(6, 3, 64), z(6, 3, 64), cu), (q, z(6, 2, 32), z(6, 2, 32), cu),
                (q, k, k, cu.long()), (q, k, k, cu.cpu()), (q, k, k, cu, cu[:2].contiguous()), (q[0], k, k, cu), (q.transpose(0, 1), k, k, cu), (q.cpu(), k, k, cu)):
        refused(att.attention_prefill, *bad)
    refused(att.attention_prefill, q, k, k, cu, out=z(6, 4, 32))
    refused(att.attention_prefill, q, k, k, cu, lse=z(3, dtype=torch.float32))
    refused(att.attention_prefill, q, k, k, cu[:1].contiguous(), error=RuntimeError)
    refused(att.attention_prefill, q, k, k, cu, scale=-1.0, error=RuntimeError)
    refused(att.attention_prefill, z(6, 4, 24), z(6, 2, 24), z(6, 2, 24), cu, error=RuntimeError)

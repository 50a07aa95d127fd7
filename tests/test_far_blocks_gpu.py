"""Caches of more than 2^32 bytes: the sliding calls and the normed append on blocks whose
byte offsets pass 32 bits, checked on a copy of those blocks in a small cache."""
import pytest
import torch

pytestmark = pytest.mark.gpu
HKV, G, D, WINDOW, SINKS = 8, 4, 128, 100, 20


@pytest.fixture(scope="module")
def far():
    """(blocks of a cache above 4 GB per plane, one byte an element; far block ids)"""
    num = (5 << 30) // (HKV * 16 * D)
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("no room for the caches")
    return num, torch.arange(num - 60, num - 1, dtype=torch.int32)


def planes(far_ids, num, dtype, dev, g):
    """A near cache of 60 blocks, and the far one that holds the same at far_ids."""
    out = []
    for _ in range(2):
        if dtype == torch.int8:
            near = torch.randint(-127, 128, (60, HKV, 16, D), generator=g, dtype=dtype).to(dev)
        else:
            near = torch.randn(60, HKV, 16, D, generator=g).to(dtype).to(dev)
        big = torch.zeros(num, HKV, 16, D, dtype=dtype, device=dev)
        big.view(torch.uint8 if dtype != torch.bfloat16 else torch.int16)[far_ids.long().to(dev)] = \
            near.view(torch.uint8 if dtype != torch.bfloat16 else torch.int16)[:len(far_ids)]
        out.append((near, big))
    return out


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_decode(cuda_device, far, kind):
    import paged_kv_decode_25_gb300 as mi
    num, ids = far
    dev, g = cuda_device, torch.Generator().manual_seed(96)
    dtype = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[kind]
    (kn, kf), (vn, vf) = planes(ids, num, dtype, dev, g)
    lens = torch.tensor([300, 17, 240], dtype=torch.int32, device=dev)
    near = torch.randperm(len(ids), generator=g)[:57].view(3, 19).to(torch.int32)
    q = torch.randn(3, HKV * G, D, generator=g).to(torch.bfloat16).to(dev)
    fn = {"bf16": mi.mi_paged_decode_attention_sliding, "fp8": mi.mi_paged_decode_attention_sliding_fp8,
          "int8": mi.mi_paged_decode_attention_sliding_int8}[kind]
    outs = []
    for k, v, tables, blocks in ((kn, vn, near, 60), (kf, vf, ids[near.long()], num)):
        extra = []
        if kind == "fp8":
            extra = [torch.ones(HKV, device=dev)] * 2
        elif kind == "int8":
            extra = [torch.ones(blocks, HKV, device=dev)] * 2
        d = mi.dims(3, HKV * G, HKV, D, blocks, 19)
        ws = torch.empty(mi.mi_paged_sliding_workspace_bytes(d, WINDOW, SINKS), dtype=torch.uint8, device=dev)
        out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device=dev)
        mi.check(fn(d, q, k, v, *extra, tables.to(dev), lens, WINDOW, SINKS, D ** -0.5, out, ws, dev_err=err))
        assert err.item() == 0
        outs.append(out)
    assert torch.count_nonzero(outs[0].float()) > 0 and same(*outs)


def test_append_and_prefill(cuda_device, far):
    import paged_kv_decode_25_gb300 as mi
    num, ids = far
    dev, g = cuda_device, torch.Generator().manual_seed(97)
    (kn, kf), (vn, vf) = planes(ids, num, torch.bfloat16, dev, g)
    near = torch.randperm(len(ids), generator=g)[:50].view(2, 25).to(torch.int32)
    lens, news = [400, 260], [100, 260]
    x = torch.randn(360, (HKV * G + 2 * HKV) * D, generator=g).to(torch.bfloat16).to(dev)
    q, k, v = x.split([HKV * G * D, HKV * D, HKV * D], 1)
    w = torch.rand(D, generator=g).to(torch.bfloat16).to(dev)
    st, rope = mi.mi_rope_table(1e6, D, 400)
    mi.check(st)
    rope = torch.from_numpy(rope).to(dev)
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, news)]).to(torch.int32)
    seq = torch.cat([torch.full((m,), s) for s, m in enumerate(news)])
    results = []
    for kc, vc, tables, blocks in ((kn, vn, near, 60), (kf, vf, ids[near.long()], num)):
        slots = (tables[seq, (pos // 16).long()] * 16 + pos % 16).to(torch.int32)
        d = mi.dims(360, HKV * G, HKV, D, blocks, 25)
        q_out = torch.empty(360, HKV * G, D, dtype=torch.bfloat16, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        mi.check(mi.mi_paged_kv_append_norm(d, q, k, v, w, w, 1e-6, pos.to(dev), slots.to(dev), rope, 400, q_out, kc, vc, err))
        out = torch.empty_like(q_out)
        mi.check(mi.mi_paged_prefill_attention_sliding(
            mi.dims(2, HKV * G, HKV, D, blocks, 25), 360, 260, q_out, kc, vc, tables.to(dev),
            torch.tensor(lens, dtype=torch.int32, device=dev), torch.tensor([0, 100, 360], dtype=torch.int32, device=dev),
            WINDOW, SINKS, D ** -0.5, out, err))
        assert err.item() == 0
        results.append((q_out, out, kc[slots.long().to(dev) // 16, :, slots.long().to(dev) % 16]))
    for a, b in zip(*results):
        assert torch.count_nonzero(a.float()) > 0 and same(a, b)

"""INT8 decode over long units that one warp, or one block, sums up alone: no rounding
may go the same way in every step. The sums of the outputs run over hundreds of
blocks, and tensor cores cut each towards zero, so whatever fills an accumulator
beside the outputs themselves shows as an error of one sign."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def signed_error(dev, Hq, Hkv, d, n, window, spread, seed):
    """Mean of (out - ref) over the mean of |ref|, of a few requests of a batch with more
    units than an SM has warps, times all SMs: none of them is split."""
    import paged_kv_decode_25_gb300 as mi
    warps = 12 * torch.cuda.get_device_properties(dev).multi_processor_count
    B, pool, W, G = -(-warps // Hkv) + 5, 500, -(-n // 16), Hq // Hkv
    g = torch.Generator(device=dev).manual_seed(seed)
    tables = torch.randint(0, pool, (B, W), generator=g, device=dev, dtype=torch.int32)
    k, v = (torch.randint(-127, 128, (pool, Hkv, 16, d), generator=g, device=dev, dtype=torch.int8) for _ in range(2))
    ka, va = (1 + torch.rand(pool, Hkv, generator=g, device=dev) for _ in range(2))
    q = (spread * torch.randn(B, Hq, d, generator=g, device=dev)).to(torch.bfloat16)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev)
    out, err = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device=dev)
    D = mi.dims(B, Hq, Hkv, d, pool, W)
    if window:
        ws = torch.empty(mi.mi_paged_sliding_workspace_bytes(D, window, 0), dtype=torch.uint8, device=dev)
        mi.check(mi.mi_paged_decode_attention_sliding_int8(D, q, k, v, ka, va, tables, lens, window, 0, d ** -0.5, out, ws,
                                                           dev_err=err))
    else:
        ws = torch.empty(mi.mi_paged_decode_workspace_bytes(D), dtype=torch.uint8, device=dev)
        mi.check(mi.mi_paged_decode_attention_int8(D, q, k, v, ka, va, tables, lens, d ** -0.5, out, ws, dev_err=err))
    assert err.item() == 0
    t = torch.arange(max(0, n - window) if window else 0, n, device=dev)
    errors, refs = [], []
    for s in range(0, B, B // 8):
        blk = tables[s, t // 16].long()
        for h in range(Hkv):
            kk, vv = (c[blk, h, t % 16].double() * a[blk, h].double()[:, None] / 127 for c, a in ((k, ka), (v, va)))
            ref = torch.softmax(q[s, h * G:(h + 1) * G].double() @ kk.T * d ** -0.5, -1) @ vv
            errors.append(out[s, h * G:(h + 1) * G].double() - ref)
            refs.append(ref.abs())
    return float(torch.stack(errors).mean() / torch.stack(refs).mean())


# An output's rounding to bf16 is at most 2^-8 of it, to either side: over N outputs its
# mean has a deviation of at most 2^-8 / sqrt(3 N), here N >= 8,192 and so 2^-8 / 157, and
# the weights' roundings (2^-11) are averaged once more over the tokens. 2^-8 / 16 is ten
# such deviations.
BOUND = 2.0 ** -8 / 16


@pytest.mark.parametrize("spread", [1.0, 0.1])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 8, 128), (8, 4, 64)])
def test_long_windows(cuda_device, Hq, Hkv, d, spread):
    for window in (4096, 8192):
        assert abs(signed_error(cuda_device, Hq, Hkv, d, 9000, window, spread, 80)) <= BOUND, window


@pytest.mark.parametrize("spread", [1.0, 0.1])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 8, 128), (8, 4, 64)])
def test_long_contexts(cuda_device, Hq, Hkv, d, spread):
    for n in (8192, 24000):
        assert abs(signed_error(cuda_device, Hq, Hkv, d, n, 0, spread, 81)) <= BOUND, n

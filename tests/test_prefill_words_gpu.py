"""Prefill over lengths and starts that are no lengths and starts: words near the ends
of 32 bits, whose sums and differences would wrap. The request is reported, its rows
stay as they were (bad starts) or are zero (no tokens), and the others are right."""
import pytest
import torch

from paged_ref import Batch, attention_ref

pytestmark = pytest.mark.gpu
LEAST, MOST = -2 ** 31, 2 ** 31 - 1


def call(mi, dev, b, q, lens, starts, most, Hq, variant, window=70, sinks=5):
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    D = mi.dims(len(lens), Hq, b.Hkv, b.d, b.num_blocks, b.tables.shape[1])
    args = (D, q.shape[0], most, q.to(dev), b.k.to(dev), b.v.to(dev), b.tables.to(dev), i32(lens), i32(starts))
    if variant == "sliding":
        mi.check(mi.mi_paged_prefill_attention_sliding(*args, window, sinks, b.d ** -0.5, out, err))
    else:
        mi.check(mi.mi_paged_prefill_attention_variant(*args, b.d ** -0.5, out, dev_err=err, variant=variant))
    torch.cuda.synchronize()
    return out.cpu(), err.item()


def right(b, s, q, out, n, variant, window=70, sinks=5):
    m, G = q.shape[0], q.shape[1] // b.Hkv
    for i in range(m):
        t = torch.arange(n - m + i + 1)
        if variant == "sliding":
            t = t[(t < sinks) | (t > n - m + i - window)]
        for h in range(b.Hkv):
            k, v = (b.tokens(c, s, h)[t] for c in (b.k, b.v))
            ref, tol = attention_ref(q[i, h * G:(h + 1) * G].double(), k, v, b.d ** -0.5)
            assert torch.all((out[i, h * G:(h + 1) * G].double() - ref).abs() <= tol), (i, h)


@pytest.mark.parametrize("variant", [0, 1, 2, 3, "sliding"])
@pytest.mark.parametrize("n", [LEAST, LEAST + 3, LEAST + 4, -1])
def test_lengths(cuda_device, variant, n):
    import paged_kv_decode_25_gb300 as mi
    b = Batch([200, 90], 2, 64, 91)
    q = b.queries(4 + 9, 8)
    out, err = call(mi, cuda_device, b, q, [n, 90], [0, 4, 13], 9, 8, variant)
    assert err == mi.MI_DEVERR_BAD_QUERY
    assert torch.count_nonzero(out[:4].float()) == 0
    right(b, 1, q[4:], out[4:], 90, variant)


@pytest.mark.parametrize("variant", [0, 1, 2, 3, "sliding"])
@pytest.mark.parametrize("a,z", [(MOST, LEAST), (MOST - 9, LEAST + 40), (64, LEAST + 63), (64, LEAST + 64)])
def test_starts(cuda_device, variant, a, z):
    """Request 0 begins past all rows and ends far before them, 1 begins there; 2 is good."""
    import paged_kv_decode_25_gb300 as mi
    b = Batch([200, 200, 90], 2, 64, 92)
    q = b.queries(60, 8)
    out, err = call(mi, cuda_device, b, q, [200, 200, 90], [a, z, 51, 60], 60, 8, variant)
    assert err == mi.MI_DEVERR_BAD_QUERY
    assert torch.all(out[:51] == 7.0)
    right(b, 2, q[51:], out[51:], 90, variant)

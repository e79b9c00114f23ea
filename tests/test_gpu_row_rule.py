"""Rows of an e4m3 cache are the same whoever writes them: kv_cache_write, or kv_cache_append, whose
values are not rotated."""
import math

import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import TYPES, ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("typ", ["bf16", "fp16"])
def test_the_same_codes_and_scales(cuda_device, typ, d):
    """Every exponent of the type as a row's largest, on both sides of the border 1.75 2^E; zeros,
    subnormals, infinities and NaN."""
    t = TYPES[typ]
    g = torch.Generator().manual_seed(d)
    exponents = range(-133, 128) if typ == "bf16" else range(-24, 16)
    tops = [m * 2.0 ** e for e in exponents for m in (1.0, 1.75, 1.7578125, 1.9921875)]
    rows = torch.rand((len(tops), d), generator=g, dtype=torch.float64) * 2 - 1
    rows = (rows * torch.tensor(tops, dtype=torch.float64)[:, None]).to(t)
    rows[:, 7] = torch.tensor(tops, dtype=torch.float64).to(t)
    odd = torch.zeros((5, d), dtype=t)
    odd[1] = -0.0
    odd[2, 3], odd[3, 60], odd[4, 0] = math.inf, -math.inf, math.nan
    x = torch.cat([rows, odd])[:, None].cuda()
    n = x.shape[0]
    slots = torch.randperm(-(-n // 16) * 16, generator=g)[:n].cuda()
    still = torch.cat([torch.ones(1, d // 2), torch.zeros(1, d // 2)], 1).cuda()
    got = []
    for append in (False, True):
        shape = (-(-n // 16), 1, 16, d)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                for _ in range(2))
        ks, vs = (torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2))
        if append:
            fat.kv_cache_append(None, x, x, k, v, slots, slots * 0, still, k_scale=ks, v_scale=vs)
        else:
            fat.kv_cache_write(x, x, k, v, slots, k_scale=ks, v_scale=vs)
        got.append((v.view(torch.uint8), vs))
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
    assert all(torch.equal(a, b) for a, b in zip(*got))
    # and they are what the definition gives
    codes, e = got[0]
    at = slots.cpu()
    held = codes.cpu()[at // 16, 0, at % 16].view(torch.float8_e4m3fn).double()
    e = e.cpu()[at // 16, 0, at % 16]
    for r in range(0, n, 7):
        values, byte = ref.quantise_row(x[r, 0].double().cpu().numpy())
        assert int(e[r]) == byte, r
        if byte != 255:
            assert torch.equal(held[r] * 2.0 ** (byte - 127), torch.as_tensor(values)), r
    assert e[-3:].tolist() == [255] * 3 and e[-5:-3].tolist() == [127] * 2

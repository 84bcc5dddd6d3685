"""Rotated appending to an 8-bit cache: an infinity or a NaN changes nothing but its own block and head."""
import pytest
import torch

import sparse_head_attention_gb300 as ea
from cache_reference import tokens
from gpu_helpers import gpu_device
from tree_reference import inv_freq

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("T", [100, 12])
def test_a_non_finite_value_stays_in_its_block(dtype, T):
    dev = gpu_device()
    f = torch.from_numpy(inv_freq(128)).to(dev)
    K, V = tokens((1, T, 2, 128), 1).to(dev), tokens((1, T, 2, 128), 2).to(dev)
    start = torch.tensor([24], dtype=torch.int32, device=dev)
    first = tokens((1, 24, 2, 128), 3).to(dev)
    out = []
    for bad in (False, True):
        c = ea.kv_cache(1, 128, 2, dtype=dtype, scale_block=32, device=dev)
        ea.ea_cache_write_rope(c, first, first, f)
        k, v = K.clone(), V.clone()
        if bad:
            k[0, T - 2, 1, 5], v[0, 10, 0, 127] = float("inf"), float("nan")
        ea.ea_cache_write_rope(c, k, v, f, start=start)
        out.append(c)
    good, bad = out
    for x, y, scales, h, row in ((good.K, bad.K, (good.k_scale, bad.k_scale), 1, 24 + T - 2), (good.V, bad.V, (good.v_scale, bad.v_scale), 0, 34)):
        j = row // 32
        nan = torch.isnan(scales[1])
        assert nan[0, h, j] and int(nan.sum()) == 1
        same = torch.ones(1, 128, 2, dtype=torch.bool, device=dev)
        same[0, 32 * j : 32 * j + 32, h] = False
        assert torch.equal(x.view(torch.uint8)[same], y.view(torch.uint8)[same])
        assert torch.equal(scales[0][~nan], scales[1][~nan])

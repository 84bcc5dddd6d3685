"""The operators for drafted tokens in the bounds-checked build (libea_checked.so): odd
sizes, every mode, ragged lengths and counts; the error word stays clear and the results
match the plain forms.  And caches whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
import test_rope_gpu as rope
import test_tree_attn_gpu as attn
import test_tree_gpu as tree
from gpu_helpers import check_no_device_error, gpu_device
from sparse_head_attention_gb300 import build as ea_build

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16


@pytest.fixture(scope="module")
def checked():
    d = gpu_device()
    prev = ea.use_library(ea_build.build(checked=True))
    yield d
    ea.use_library(prev)


@pytest.mark.parametrize("dtype,sb,page", [(BF16, 64, 0), (BF16, 64, 192), (E4M3, 32, 192), (INT8, 16, 0)])
def test_attention(checked, dtype, sb, page):
    lens, n, T = [700, 0, 1, 129, 640], [41, 41, 7, 0, 13], 41
    cap = 768
    bm = attn.blocks(5, 3, cap, 2, 0.4)
    modes = [[(b + h) % 3 for h in range(3)] for b in range(5)]
    attn.check(checked, attn.make_cache(5, cap, 3, dtype, sb, page, 1), 15, 3, T, lens, n, modes, sink=20, window=90, bm=bm, seed=3)


@pytest.mark.parametrize("dtype,sb,page", [(BF16, 64, 64), (E4M3, 32, 0), (INT8, 64, 128)])
def test_append(checked, dtype, sb, page):
    rope.check_append(checked, dtype, sb, page, 3, 70, [5, 63, 0, 100], [70, 1, 0, 33], Hq=9, rot=96, interleaved=True)


def test_plan_and_accept(checked):
    tree.test_plan_and_accept(checked, "forest", 5, 77)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_offsets_beyond_32_bits(dtype):
    """Pages at the far end of a pool of more than 2^32 bytes (2^31 elements) a tensor."""
    dev = gpu_device()
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    page, Hkv, T, Hq = 64, 8, 3, 16
    pages = (1 << 32) // (page * Hkv * 128 * (2 if dtype == BF16 else 1)) + 9
    K = torch.empty(pages, page, Hkv, 128, dtype=dtype, device=dev)
    V = torch.empty_like(K)
    sc = [None, None] if dtype == BF16 else [torch.empty(pages, Hkv, 1, device=dev) for _ in range(2)]
    table = torch.tensor([[pages - 1, pages - 2, 0], [1, pages - 3, pages - 4]], dtype=torch.int32, device=dev)
    far = ea.KVCache(K, V, *sc, block_table=table)
    # the same in a small pool
    at = table.flatten().sort().values
    near_table = torch.searchsorted(at, table.flatten()).view(2, 3).to(torch.int32)
    k, v = torch.zeros(6, page, Hkv, 128, dtype=dtype, device=dev), torch.zeros(6, page, Hkv, 128, dtype=dtype, device=dev)
    s2 = [None, None] if dtype == BF16 else [torch.zeros(6, Hkv, 1, device=dev) for _ in range(2)]
    near = ea.KVCache(k, v, *s2, block_table=near_table)
    g = torch.Generator(device=dev).manual_seed(1)
    kn, vn = (torch.randn(2, 150, Hkv, 128, generator=g, device=dev).to(BF16) for _ in range(2))
    f = torch.from_numpy(rope.inv_freq(128)).to(dev)
    start = torch.tensor([20, 0], dtype=torch.int32, device=dev)
    zero = torch.zeros(2, dtype=torch.int32, device=dev)
    ws = ea.cache_workspace(dev)
    for c in (far, near):
        ea.ea_cache_write_rope(c, kn[:, :20], vn[:, :20], f, start=zero, workspace=ws)
        ea.ea_cache_write_rope(c, kn, vn, f, start=start, workspace=ws)
    check_no_device_error(ws)
    Q, Kd, Vd = (torch.randn(2, T, h, 128, generator=g, device=dev).to(BF16) for h in (Hq, Hkv, Hkv))
    depth, mask = ea.ea_tree_plan(torch.tensor([[-1, 0, 1]] * 2, dtype=torch.int32, device=dev))
    m = torch.zeros(2, Hkv, dtype=torch.uint8, device=dev)
    out = [ea.ea_hybrid_attn_tree(Q, Kd, Vd, c, start + 150, depth, mask, m, sink=0, window=1) for c in (far, near)]
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1]) and np.isfinite(out[0][1].cpu().numpy()).all()

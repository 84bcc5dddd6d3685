"""The KV cache operators in the bounds-checked build (libea_checked.so): odd
sizes, every mode, ragged lengths; the error word stays clear and the results
match the plain forms."""
import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
import test_cache_ops_gpu as ops
import test_decode_q8_gpu as dec
import test_key_weights_gpu as kw
from gpu_helpers import gpu_device
from sparse_head_attention_gb300 import build as ea_build
from sparse_head_attention_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    d = gpu_device()
    prev = ea.use_library(ea_build.build(checked=True))
    yield d
    ea.use_library(prev)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("page,num_splits", [(0, 0), (64, 0), (192, 5)])
def test_decode(dev, dtype, page, num_splits):
    lens = [700, 0, 1, 129, 640]
    cap = 768 if page == 192 else 704
    c = ops.make_cache(len(lens), cap, 3, dtype, 32, page, seed=1)
    bm = wl.block_mask(len(lens), 3, cap, density=0.4, seed=2).numpy()
    dec.check(dev, c, ops.tokens((len(lens), 9, 128), seed=3), lens, dec.all_modes(len(lens), 3), 20, 90, bm, num_splits)


@pytest.mark.parametrize("dtype", [E4M3, INT8, BF16])
def test_write_select_compact(dev, dtype):
    ops.test_write_appends_at_any_row(dev, dtype, 32, 64)
    ops.test_select_keeps_the_heaviest(dev, 4097, 2048, 1, 0)
    ops.test_compact_gathers_and_requantises(dev, dtype, INT8, (128, 256))


def test_key_weights(dev):
    lens = [701, 0, 1, 129, 640]
    for Tq in (1, 33, 300):
        bm = wl.block_mask(len(lens), 3, 701, density=0.3, seed=Tq).numpy()
        kw.check(dev, len(lens), Tq, 701, 9, 3, kw.all_modes(len(lens), 3), 30, 77, lens, bm, seed=Tq)

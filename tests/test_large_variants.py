"""The kernel variants that only large calls take, at the sizes where they begin: runs of eight features in the norm and rotation
(from 2^17 rows on), and four rows a thread in a cache's read (from eight rows a thread of every SM on)."""
import numpy as np
import pytest
import torch

from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from oracle import kv_cache as kv_ref
from oracle import set_rows as rows_ref
from tests import test_rope
from tests.test_cache_write import fill
from tests.test_rope import case

# 2 x 513 tokens (not a multiple of a block's 32 or 64) of 128 heads: 131328 rows
BIG = dict(B=2, S=513, Hq=96, Hkv=32)
ROPE = {
    "half": case(**BIG, D=128, rot=128, seed=40),
    "half_d64_part": case(**BIG, D=64, rot=48, layout="bshd", strided=True, norm="f32", seed=41),
    "interleaved": case(**BIG, D=128, rot=128, interleaved=True, norm="f32", factor=1.2, seed=42),
    "interleaved_d64": case(**BIG, D=64, rot=64, interleaved=True, layout="bshd", strided=True, seed=43),
    "part": case(**BIG, D=128, rot=16, far=100000, seed=44),
    "rotation_alone": case(**BIG, D=128, rot=96, norm=None, layout="bshd", seed=45),
    "norm_alone": case(**BIG, D=64, rot=0, seed=46),
    "runs_of_four": case(**BIG, D=128, rot=24, seed=47),           # 12 pairs are no whole runs of eight
    "runs_of_four_f32": case(B=2, S=513, Hq=96, Hkv=32, D=64, rot=32, dtype=torch.float32, interleaved=True, seed=48),
    "below": case(B=2, S=511, Hq=96, Hkv=32, D=128, rot=128, seed=49),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ROPE)
def test_norm_and_rotation_of_many_rows(name, monkeypatch):
    monkeypatch.setitem(test_rope.CASES, name, ROPE[name])
    test_rope.test_forward_matches_oracle(name)
    test_rope.test_backward_matches_oracle(name)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [5, 1861])
@pytest.mark.parametrize("layout", ["bhsd", "bshd"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
def test_reads_of_many_rows(fmt, D, dtype, layout, n):
    """Heads shorter than a block's step and heads that no step divides; an odd number of rows in all, so that the last block
    is in part empty."""
    step = 256 // ((D // 2 if fmt == "q4_0" else D) // (8 if dtype == torch.bfloat16 else 4))
    many = 8 * step * torch.cuda.get_device_properties(0).multi_processor_count
    H, begin = 7, 3
    B = -(-many // (H * n)) | 1
    planes = fill(B, H, n + begin + 1, D, fmt, 8)
    got = kv.cache_read(*planes, begin, n, dtype=dtype, layout=layout)
    torch.cuda.synchronize()
    assert ft.device_status() == 0
    for i, x in enumerate(got):
        want = kv_ref.values(planes[2 * i].cpu().numpy(), planes[2 * i + 1].cpu().numpy())[:, :, begin:begin + n]
        want = want.astype(np.float32)   # exact: at most 11 + 8 bits
        if dtype == torch.bfloat16:
            want = rows_ref.to_bf16_bits(want)
        x = x if layout == "bhsd" else x.transpose(1, 2)
        np.testing.assert_array_equal(x.float().cpu().numpy(), want)

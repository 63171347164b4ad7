"""What the serving calls' outputs hold beyond the common bounds: bf16 rows that are the f32 rows rounded."""
import numpy as np
import pytest
import torch

from test_gpu_q8 import attn, q8_batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,keys,hq,hkv,d", [([1, 1], [700, 2000], 8, 2, 128),  # decode, partials and merge
                                                ([1, 1, 1], [37, 70, 120], 8, 2, 64),  # decode, one split
                                                ([5, 16], [900, 2100], 16, 2, 256),  # tcgen05, partials and merge
                                                ([9, 2], [700, 130], 32, 8, 128),
                                                ([5, 20], [90, 128], 16, 2, 256),  # tcgen05, one split
                                                ([40, 3], [90, 60], 4, 4, 64),
                                                ([3, 5], [200, 333], 24, 2, 128)])  # the general kernel
def test_bf16_rows_are_the_f32_rows_rounded_once(kind, rows, keys, hq, hkv, d):
    """One computation whatever the output's type: the bf16 rows equal the f32 rows rounded to nearest, bit for bit,
    and a call repeats itself."""
    b, _, c = q8_batch(kind, 15, rows=rows, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32)
    wide, flags, st = attn(c, b, kind)
    assert st == 0 and (flags == 0).all()
    want = torch.from_numpy(wide).to(torch.bfloat16).float().numpy()
    for _ in range(3):
        got, _, st = attn(c, b, kind, out_dtype=torch.bfloat16)
        assert st == 0
        assert (got == want).all(), f"{np.mean(got != want):.1%} of the elements differ"
        again, _, _ = attn(c, b, kind)
        assert (again == wide).all()

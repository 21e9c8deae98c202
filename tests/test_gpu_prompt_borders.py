"""w4_prompt_attention of heads of up to 64 around the sizes at which its steps change from 128 keys to 64, on the GPU."""
from __future__ import annotations

import pytest

from test_gpu_attention import check_prompt, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,hq,hk,dim", [([500] * 14 + [130], 16, 4, 64), ([500] * 14 + [1], 15, 15, 64), ([257] * 30, 20, 4, 40), ([100, 1, 0, 63] * 30, 24, 8, 64),
                                            ([5000], 24, 2, 64), ([4096], 30, 2, 48), ([4095, 1], 32, 2, 64)])
def test_on_either_side_of_the_border(lens, hq, hk, dim, dtype):
    T = sum(lens)
    check_prompt(*(randn(i, T, h, dim, dtype=dtype) for i, h in ((1, hq), (2, hk), (3, hk))), lens)

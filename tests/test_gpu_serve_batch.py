"""What a sequence gets does not depend on the other sequences of its batch: the kernel and the row tiles go by the
batch's longest draft, the precision must not."""

import pytest
import torch

from tests import serve_ref as R
from tests.test_gpu_serve import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


class Fine(Batch):
    """Held to two bf16 halves of a weight whatever the batch (e4m3: f16)."""

    def p_half(self):
        return {"bf16": R.HALF["bf16"] ** 2, "e4m3": R.HALF["f16"], "f32": 0.0}[self.dtype]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("hq,hkv,lens,qlens", [
    (32, 8, (300, 900, 65), (1, 1, 1)),          # few rows each
    (32, 8, (300, 900, 65), (1, 5, 1)),          # one of 20 rows moves them to the wide kernel
    (32, 8, (300, 900, 65), (1, 64, 1)),         # one of 256 rows
    (16, 2, (700, 90, 400), (7, 17, 64)),        # 56, 136 and 512 rows
    (8, 1, (640,), (64,)),
])
def test_precision_does_not_depend_on_the_batch(dtype, d, hq, hkv, lens, qlens):
    for gain in (1.0, 3.0):                      # many weights that count, and few
        b = Fine(dtype, d, hq, hkv, 64, lens, qlens, "tree", seed=33, gain=gain)
        b.attend()
        b.check()

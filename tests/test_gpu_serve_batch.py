"""What a sequence gets does not depend on the other sequences of its batch: the kernel and the row tiles go by the
batch's longest draft, the precision must not."""

import pytest
import torch

from tests import serve_ref as R
from tests.test_gpu_serve import Batch, _status, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


def _half(b, r):
    """Half a step of the weights of sequence r, from its own rows: bf16 twice (hi + lo) up to 128, once above; f16."""
    if b.dtype == "e4m3":
        return R.HALF["f16"]
    return R.HALF["bf16"] ** 2 if b.qlens[r] * b.hq // b.hkv <= 128 else R.HALF["bf16"]


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
        b = Batch(dtype, d, hq, hkv, 64, lens, qlens, "tree", seed=33, gain=gain)
        b.attend()
        assert _status(b.scratch) == (0, 0)
        for r, n in enumerate(lens):
            c = slice(b.cu[r], b.cu[r + 1])
            o, l, mag, top = R.attend(*b.values(r), b.scale, b.vis[r])
            b_out, b_lse = R.attend_bounds(o, l, mag, top, d, n, _half(b, r))
            _within(R.f64(b.out[c]), o, b_out, f"out of sequence {r}")
            _within(R.f64(b.lse[:, c]), l, b_lse, f"lse of sequence {r}")

"""Values that are not finite, in places where a weight or a factor of the softmax is zero or nothing."""

import pytest
import torch

from tests import serve_ref as R
from tests.test_gpu_serve import _status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


class Two:
    """Contiguous cache of one sequence whose keys score either far above or far below each other: q = 8, k = +-8 in
    every place, so that scores differ by 1000 and more and the low keys' weights underflow to 0.  V is 1."""

    def __init__(self, dtype, d, hq, hkv, n, qlen, high):
        from block_sparse_long_pooled_b200 import fp2
        self.k = torch.where(high.cuda()[None, :, None, None], 8.0, -8.0).expand(1, n, hkv, d).contiguous().to(R.TORCH[dtype])
        self.v = torch.ones((1, n, hkv, d), device="cuda").to(R.TORCH[dtype])
        self.q = torch.full((qlen, hq, d), 8.0, device="cuda").to(R.TORCH[dtype])
        self.kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.handle = fp2.make_decode(self.q, fp2.make_cache(self.k, self.v), [0, qlen], self.kv_len, n)
        self.scratch = fp2.alloc_scratch(fp2.fp2_decode_workspace(self.handle), "cuda")
        self.out = torch.empty((qlen, hq, d), dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
        self.lse = torch.empty((hq, qlen), device="cuda")

    def attend(self):
        from block_sparse_long_pooled_b200 import fp2
        fp2.fp2_tree_attend(self.handle, self.out, self.lse, self.scratch)
        assert _status(self.scratch) == (0, 0)


@pytest.mark.parametrize("dtype,d,value", [("bf16", 128, "nan"), ("bf16", 64, "inf"), ("bf16", 128, "-inf"),
                                           ("e4m3", 128, "nan"), ("f32", 64, "nan"), ("f32", 64, "inf")])
@pytest.mark.parametrize("hq,hkv,n,qlen", [
    (1, 1, 20001, 1),       # 296 pieces: the join takes 32 at a time
    (4, 1, 20001, 3),
    (8, 1, 20001, 5),       # more than 16 rows: two streams
    (32, 8, 3000, 5),
    (16, 2, 2000, 40),      # more than 128 rows
    (4, 4, 100, 3),
])
def test_a_seen_value_that_is_not_finite_shows_whatever_its_weight(dtype, d, value, hq, hkv, n, qlen):
    """The key's weight underflows to 0 in every row; its element still becomes infinite or NaN, and no other does."""
    tile = torch.arange(n) // 64
    for j in (0, 70, n // 2, n - qlen - 1, n - qlen):    # (the last one is the first drafted key: all tokens see it)
        last = torch.zeros(n, dtype=torch.bool)
        last[n - qlen - 1 if j < n - qlen - 1 else 3] = True
        later = torch.zeros(n, dtype=torch.bool)         # of 296 pieces in four runs, not among the first 32
        later[n // 7 + (j == n // 7)] = True
        for high in (tile % 2 != tile[j] % 2, last, later):
            b = Two(dtype, d, hq, hkv, n, qlen, high)
            if dtype == "e4m3":
                b.v.view(torch.uint8)[0, j, 0, 5] = 0x7F
            else:
                b.v[0, j, 0, 5] = float(value)
            b.attend()
            bad = ~torch.isfinite(b.out.float())
            want = torch.zeros_like(bad)
            want[:, :hq // hkv, 5] = True
            assert torch.equal(bad, want), (j, int(high.sum()))
            assert torch.isfinite(b.lse).all()
            assert (b.out.float()[~want] - 1).abs().max() <= 2.0 ** -20      # n equal weights of 1: their sum is exact


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("f32", 64)])
@pytest.mark.parametrize("hq,hkv,n,qlen", [(1, 1, 20001, 1), (4, 1, 20001, 3), (8, 1, 20001, 5), (32, 8, 3000, 5),
                                           (16, 2, 2000, 40), (4, 4, 300, 3)])
def test_a_score_that_is_nan_makes_row_and_lse_nan(dtype, d, hq, hkv, n, qlen):
    """NaN in K, of one key or of whole tiles that every token sees, before and after finite ones."""
    for j0, j1 in ((0, 1), (0, 64), (0, 200), (77, 78), (n // 2, n // 2 + 100), (n - qlen - 1, n - qlen)):
        b = Two(dtype, d, hq, hkv, n, qlen, torch.arange(n) % 3 == 0)
        if dtype == "e4m3":
            b.k.view(torch.uint8)[0, j0:j1, 0] = 0xFF
        else:
            b.k[0, j0:j1, 0] = float("nan")
        b.attend()
        g = hq // hkv
        assert torch.isnan(b.lse[:g]).all() and torch.isfinite(b.lse[g:]).all(), (j0, j1)
        assert torch.isnan(b.out[:, :g].float()).all() and torch.isfinite(b.out[:, g:].float()).all(), (j0, j1)


def test_small_weights_beside_a_large_one_whose_value_is_zero():
    """e4m3, more than 16 rows: weights are f16, and what the small ones add up to has to keep its bits too."""
    from tests.test_gpu_serve import Batch
    b = Batch("e4m3", 128, 160, 5, 128, (3, 8, 1, 8, 9), (3, 8, 1, 8, 9), "tree", seed=602286, rows_over=7, joined=True, gain=4.0)
    b.attend()
    b.check()

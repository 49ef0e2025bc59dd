"""Device status of the serving calls: where it stands, what it covers, and who reads it."""

import pytest
import torch

from tests.test_gpu_serve import Batch, _status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


def test_a_lone_status_word_is_read_alone():
    """fp2_rotate's word, whatever lies behind it: here what the head of a decode call's scratch would hold."""
    from block_sparse_long_pooled_b200 import fp2
    words = torch.zeros(256, dtype=torch.int32, device="cuda")
    words[1] = 0x5E000000 | 100
    words[64:164] = fp2.FP2_DEV_TIMEOUT
    k = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    h = fp2.make_rotate(None, k, None, None, None, None, torch.empty_like(k), None,
                        slots=torch.tensor([0, 2], device="cuda"))
    assert _status(words) == (fp2.FP2_OK, 0)
    fp2.fp2_rotate(h, words[:1])
    assert _status(words) == (fp2.FP2_ERR_DEVICE_BOUNDS, fp2.FP2_DEV_SLOT_OOB)
    assert words[0] == fp2.FP2_DEV_SLOT_OOB


def test_bits_added_to_a_call_s_scratch_are_read_with_its_own():
    from block_sparse_long_pooled_b200 import fp2
    b = Batch("bf16", 128, 8, 2, 16, (100, 90), (2, 2), None, seed=4)
    b.attend()
    k = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    h = fp2.make_rotate(None, k, None, None, None, None, torch.empty_like(k), None,
                        slots=torch.tensor([0, 2], device="cuda"))
    assert _status(b.scratch) == (fp2.FP2_OK, 0)
    fp2.fp2_rotate(h, b.scratch[:4].view(torch.int32))
    assert _status(b.scratch) == (fp2.FP2_ERR_DEVICE_BOUNDS, fp2.FP2_DEV_SLOT_OOB)
    b.table_dev[1, 2] = -1
    b.attend()
    assert _status(b.scratch) == (fp2.FP2_ERR_DEVICE_BOUNDS, fp2.FP2_DEV_PAGE_OOB)


def test_a_scratch_holds_the_status_of_its_last_call():
    """The attention meets a page that is out of range, the weights after it do not."""
    from block_sparse_long_pooled_b200 import fp2
    b = Batch("bf16", 128, 8, 2, 16, (100, 90), (2, 2), None, seed=4)
    own = fp2.alloc_scratch(fp2.fp2_decode_workspace(b.handle), "cuda")
    mass = torch.zeros((2, 2, b.max_len), device="cuda")
    page = int(b.table[1, 2])

    def step(mass_scratch):
        b.table_dev[1, 2] = -1
        b.attend()
        b.table_dev[1, 2] = page
        fp2.fp2_key_mass(b.handle, b.lse, None, mass, mass_scratch)

    step(own)
    assert _status(b.scratch) == (fp2.FP2_ERR_DEVICE_BOUNDS, fp2.FP2_DEV_PAGE_OOB) and _status(own) == (0, 0)
    step(b.scratch)
    assert _status(b.scratch) == (0, 0)

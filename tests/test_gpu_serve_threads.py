"""Serving calls from threads of their own, as a server makes them."""

import threading

import pytest
import torch

from tests.test_gpu_serve import Batch, _status
from tests.test_gpu_serve_rings import check_all

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


def _in_threads(*works):
    errors = []

    def guarded(work):
        try:
            work()
        except Exception as e:      # noqa: BLE001  (told to the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("dtype,d,qlen", [("bf16", 128, 1), ("bf16", 64, 40), ("e4m3", 128, 2), ("f32", 64, 2)])
def test_the_first_call_of_a_thread(dtype, d, qlen):
    """A thread that has not used the GPU yet has no context of its own when the call makes its tensor maps."""
    from block_sparse_long_pooled_b200 import fp2
    b = Batch(dtype, d, 8, 2, 16, (300, 77), (qlen, 3), "tree", seed=11)
    mass = torch.zeros((2, 2, b.max_len), device="cuda")
    torch.cuda.synchronize()
    _in_threads(b.attend)
    check_all(b)
    _in_threads(lambda: fp2.fp2_key_mass(b.handle, b.lse, None, mass, b.scratch))
    check_all(b, mass)


def test_one_handle_on_two_streams_and_two_threads():
    """The handle holds nothing of a call's: with scratch and outputs of their own, calls on it may overlap."""
    from block_sparse_long_pooled_b200 import fp2
    b = Batch("bf16", 128, 8, 2, 16, (3000, 700, 64), (5, 1, 40), "tree", seed=10)
    b.attend()
    check_all(b)
    sides = [(torch.cuda.Stream(), torch.zeros_like(b.out), torch.zeros_like(b.lse), torch.empty_like(b.scratch))
             for _ in range(2)]
    torch.cuda.synchronize()

    def work(stream, out, lse, scratch):
        for _ in range(50):
            fp2.fp2_tree_attend(b.handle, out, lse, scratch, stream=stream)

    _in_threads(*(lambda s=s: work(*s) for s in sides))
    torch.cuda.synchronize()
    for _, out, lse, scratch in sides:
        assert torch.equal(out, b.out) and torch.equal(lse, b.lse) and _status(scratch) == (0, 0)

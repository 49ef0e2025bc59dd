"""The binding's structs hold addresses: they have to keep what is there alive."""

import gc
import weakref

import torch

from block_sparse_long_pooled_b200 import build as B
from block_sparse_long_pooled_b200 import fp2


def test_pooled_and_index_structs_keep_their_tensors():
    """`pooled, _ = alloc_pooled(...)` and then another `_`: the buffers must not go back to the allocator, which would
    hand them out again under the next call's outputs."""
    B.build()
    q, k, v = (torch.zeros((300, h, 128), dtype=torch.bfloat16) for h in (8, 2, 2))
    prob, params = fp2.make_problem(q, k, v, [0, 300], 2), fp2.make_params(128)
    ws = fp2.fp2_workspace_query(prob, params)
    pooled, tensors = fp2.alloc_pooled(ws, prob, "cpu")
    index, more = fp2.alloc_index(ws, "cpu")
    where = [weakref.ref(t) for t in (*tensors.values(), *more.values())]
    addresses = [t.data_ptr() for t in tensors.values()]
    del tensors, more
    gc.collect()
    assert all(w() is not None for w in where)
    assert [getattr(pooled, f) for f in ("qbar", "kbar", "vbar", "kbar_mma", "vbar_mma")] == addresses
    del pooled, index
    gc.collect()
    assert all(w() is None for w in where)

"""The ends of what the serving calls take: the longest caches, the most sequences and heads, layouts of the cache that
other cases leave out."""

import numpy as np
import pytest
import torch

from tests import serve_ref as R
from tests.test_gpu_serve import Batch, _evict_case, _gen, _status, _within
from tests.test_gpu_serve_rings import _attend_and_weigh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


@pytest.mark.parametrize("dtype,d,hq,hkv,page,qlen", [
    ("bf16", 128, 4, 1, 64, 1), ("bf16", 64, 8, 2, 16, 2), ("e4m3", 128, 8, 1, 0, 1), ("bf16", 128, 8, 1, 128, 9),
    ("e4m3", 128, 4, 1, 16, 40), ("f32", 64, 4, 1, 64, 2),
])
def test_the_longest_cache(dtype, d, hq, hkv, page, qlen):
    from block_sparse_long_pooled_b200 import fp2
    _attend_and_weigh(Batch(dtype, d, hq, hkv, page, (fp2.FP2_MAX_CACHE_LEN,), (qlen,), "tree", seed=1))


def test_eviction_from_and_to_the_longest_cache():
    from block_sparse_long_pooled_b200 import fp2
    n = fp2.FP2_MAX_CACHE_LEN
    mass = torch.floor(torch.randn((1, 1, n), generator=_gen(3)).abs() * 3)
    _evict_case("bf16", 64, 1, 64, (n,), 4000, 4, 100, mass=mass)
    # a budget of all but one key: the lightest one, the last of its equals, goes
    k = torch.randint(-30000, 30000, (1, n, 1, 64), dtype=torch.int16, generator=_gen(4)).cuda().view(torch.bfloat16)
    ko, vo = torch.zeros_like(k), torch.zeros_like(k)
    kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
    mo, kept = torch.zeros((1, 1, n - 1), device="cuda"), torch.zeros((1, 1, n - 1), dtype=torch.int32, device="cuda")
    lo = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = fp2.make_evict(fp2.make_cache(k, k.clone()), kv_len, n, mass.cuda(), n - 1, 0, 0, fp2.make_cache(ko, vo), mo, kept, lo)
    scratch = fp2.alloc_scratch(fp2.fp2_evict_workspace(h), "cuda")
    fp2.fp2_evict(h, scratch)
    assert _status(scratch) == (0, 0)
    m = mass[0, 0].numpy()
    gone = int(np.flatnonzero(m == m.min())[-1])
    keep = torch.cat([torch.arange(gone), torch.arange(gone + 1, n)])
    assert torch.equal(kept[0, 0].cpu().long(), keep) and torch.equal(mo[0, 0].cpu(), mass[0, 0, keep])
    bits = k.view(torch.int16)[0, keep.cuda()]
    for o in (ko, vo):
        assert torch.equal(o.view(torch.int16)[0, :n - 1], bits) and (o.view(torch.int16)[0, n - 1] == 0).all()


@pytest.mark.parametrize("dtype,d,hq,hkv,most", [("bf16", 128, 4, 4, 3), ("e4m3", 128, 8, 1, 64), ("bf16", 64, 12, 4, 64),
                                                 ("f32", 64, 2, 2, 9)])
def test_as_many_sequences_as_there_can_be(dtype, d, hq, hkv, most):
    """512 of 0 to 400 keys, some without tokens, some with nothing but their tokens."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 400, 512)]
    qlens = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, most + 1, 512))]
    lens[7], qlens[7], lens[511], qlens[511] = most, most, 399, most
    _attend_and_weigh(Batch(dtype, d, hq, hkv, 16, lens, qlens, "tree", seed=2))


@pytest.mark.parametrize("group", [1, 20])
def test_as_many_heads_as_there_can_be(group):
    from block_sparse_long_pooled_b200 import fp2
    hkv, d, n = 65536, 64, 5
    b = Batch("bf16", d, hkv * group, hkv, 0, (n,), (1,), None, seed=3)
    _attend_and_weigh(b)
    if group > 1:
        return
    # rotated in place, and three of the five keys kept
    x = torch.randn((1, hkv, d), generator=_gen(4)).to(torch.bfloat16).cuda()
    y, rope = torch.empty_like(x), fp2.make_rope(fp2.rope_frequencies(d)[0])
    pos = torch.tensor([77], dtype=torch.int32, device="cuda")
    fp2.fp2_rotate(fp2.make_rotate(x, x, x, pos, rope, y, torch.empty_like(x), torch.empty_like(x)))
    want, mag = R.rotate(R.f64(x), np.array([77]), rope.inv_freq, False, 1.0)
    _within(y, want, R.rotate_bound(want, mag, "bf16"), "heads")
    _evict_case("bf16", d, 64, 16, (n, 4) * 100, 3, 0, 1)


def test_eviction_within_one_pool_of_pages():
    """Source and destination pages lie in the same pool, in any order."""
    from block_sparse_long_pooled_b200 import fp2
    g = _gen(8)
    lens, budget, page, hkv, d = (700, 90, 333), 100, 16, 2, 128
    need, got = [-(-n // page) for n in lens], -(-budget // page)
    order = torch.randperm(sum(need) + 3 * got, generator=g).to(torch.int32)
    table, table_o, at = torch.full((3, max(need)), -1, dtype=torch.int32), torch.empty((3, got), dtype=torch.int32), 0
    for r, x in enumerate(need):
        table[r, :x] = order[at:at + x]
        table_o[r] = order[at + x:at + x + got]
        at += x + got
    k, v = (torch.randn((len(order), page, hkv, d), generator=g).to(torch.bfloat16) for _ in "kv")
    kd, vd = k.cuda(), v.cuda()
    mass = torch.rand((3, hkv, 700), generator=g)
    mo, kept = torch.zeros((3, hkv, budget), device="cuda"), torch.zeros((3, hkv, budget), dtype=torch.int32, device="cuda")
    lo = torch.zeros(3, dtype=torch.int32, device="cuda")
    h = fp2.make_evict(fp2.make_cache(kd, vd, table.cuda()), torch.tensor(lens, dtype=torch.int32, device="cuda"), 700,
                       mass.cuda(), budget, 4, 20, fp2.make_cache(kd, vd, table_o.cuda()), mo, kept, lo)
    scratch = fp2.alloc_scratch(fp2.fp2_evict_workspace(h), "cuda")
    fp2.fp2_evict(h, scratch)
    assert _status(scratch) == (0, 0)
    for r, n in enumerate(lens):
        for hh in range(hkv):
            j = torch.from_numpy(R.evict(mass[r, hh].numpy(), n, budget, 4, 20))
            assert torch.equal(kept[r, hh, :len(j)].cpu().long(), j)
            i = torch.arange(len(j))
            for old, new in ((k, kd.cpu()), (v, vd.cpu())):
                assert torch.equal(new[table_o[r, i // page].long(), i % page, hh], old[table[r, j // page].long(), j % page, hh])
        for old, new in ((k, kd.cpu()), (v, vd.cpu())):           # the source's rows are as they were
            pages = table[r, :need[r]].long()
            assert torch.equal(new[pages], old[pages])


@pytest.mark.parametrize("dtype,d,qlen", [("bf16", 128, 1), ("bf16", 64, 40), ("e4m3", 128, 9), ("f32", 64, 2)])
def test_pages_that_hold_k_and_v_side_by_side(dtype, d, qlen):
    """[pages, 2, page_size, Hkv, d]: the strides between pages are twice a page."""
    from block_sparse_long_pooled_b200 import fp2
    b = Batch(dtype, d, 8, 2, 32, (500, 77), (qlen, 3), "tree", seed=9)
    both = torch.stack((b.k.view(torch.uint8), b.v.view(torch.uint8)), 1).view(b.k.dtype)
    b.cache = fp2.make_cache(both[:, 0], both[:, 1], b.table_dev)
    b.handle = fp2.make_decode(b.q, b.cache, b.cu, b.kv_len, b.max_len, b.hkv, tree_mask=b.words_dev, **b.descale)
    _attend_and_weigh(b)


@pytest.mark.parametrize("tokens,hq,hkv,inter", [(5, 8, 2, False), (300, 32, 8, True), (5000, 3, 1, False), (20000, 8, 2, True)])
def test_rotate_in_place_inside_one_projection(tokens, hq, hkv, inter):
    """Q in its own place, a view of the projection's output, while K and V go to the slots of a cache; then all three
    in place.  The same bits as into buffers of their own, and nothing else of the projection changes."""
    from block_sparse_long_pooled_b200 import fp2
    g, d = _gen(12), 128
    x = torch.randn((tokens, hq + 2 * hkv + 1, d), generator=g).to(torch.bfloat16).cuda()
    cut = lambda t: (t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:hq + 2 * hkv])  # noqa: E731
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 1 << 17, (tokens,), generator=g).to(torch.int32).cuda()
    rope = fp2.make_rope(fp2.rope_frequencies(64)[0], inter)
    slots = torch.randperm(tokens + 7, generator=g)[:tokens].cuda()
    rows = lambda: torch.zeros((tokens + 7, hkv, d), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    own = [torch.zeros((tokens, hq, d), dtype=torch.bfloat16, device="cuda"), rows(), rows()]
    fp2.fp2_rotate(fp2.make_rotate(*cut(x), pos, rope, *own, slots=slots, q_norm=w, k_norm=w))
    y, k, v = x.clone(), rows(), rows()
    fp2.fp2_rotate(fp2.make_rotate(*cut(y), pos, rope, cut(y)[0], k, v, slots=slots, q_norm=w, k_norm=w))
    assert torch.equal(cut(y)[0], own[0]) and torch.equal(k, own[1]) and torch.equal(v, own[2])
    assert torch.equal(y[:, hq:], x[:, hq:])
    y = x.clone()
    fp2.fp2_rotate(fp2.make_rotate(*cut(y), pos, rope, *cut(y), q_norm=w, k_norm=w))
    for got, want in zip(cut(y), (own[0], own[1][slots], own[2][slots])):
        assert torch.equal(got, want)
    assert torch.equal(y[:, -1], x[:, -1])

"""Serving kernels over so many tiles that every ring of barriers goes round three times and more, and loads that land
out of order.  The 64-bit forms are computed on the GPU here, in float64, with serve_ref's bounds."""

import numpy as np
import pytest
import torch

from tests import serve_ref as R
from tests.test_gpu_serve import Batch, _evict_case, _gen, _status, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


def _sequence(b, r):
    """Q, K, V of sequence r as float64 on the GPU (K and V of keys that nobody sees as zeros), and what is seen."""
    c, n = slice(b.cu[r], b.cu[r + 1]), b.lens[r]
    vis = torch.from_numpy(b.vis[r]).cuda()
    out = [b.qc[c].cuda().to(torch.float32).double() * b.ds[0]]
    for x, s in ((b.kc, b.ds[1]), (b.vc, b.ds[2])):
        if b.table is None:
            rows = x[r, :n]
        else:
            j = torch.arange(n)
            rows = x.view(torch.uint8 if x.element_size() == 1 else torch.int16)[b.table[r].long()[j // b.page], j % b.page]
            rows = rows.view(x.dtype)
        rows = rows.cuda().to(torch.float32).double() * s
        out.append(torch.where(vis.any(0)[:, None, None], rows, 0.0).transpose(0, 1))    # [Hkv, n, d]
    return out, vis


def check_all(b, mass=None):
    """Every sequence's rows (and, given the call's mass without an old one, its keys' weights)."""
    assert _status(b.scratch) == (0, 0)
    G = b.hq // b.hkv
    for r in range(len(b.lens)):
        if b.qlens[r] == 0:
            continue
        c, n, Q = slice(b.cu[r], b.cu[r + 1]), b.lens[r], b.qlens[r]
        (q, k, v), vis = _sequence(b, r)
        q = q.view(Q, b.hkv, G, b.d).permute(1, 2, 0, 3).reshape(b.hkv, G * Q, b.d)
        see = vis.repeat(G, 1)[None]
        s = (q @ k.transpose(1, 2) * b.scale).masked_fill(~see, -np.inf)
        m = (q.abs() @ k.abs().transpose(1, 2) * b.scale).masked_fill(~see, 0.0)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[..., None])
        back = lambda x: x.view(b.hkv, G, Q, -1).permute(2, 0, 1, 3).reshape(Q, b.hq, -1).cpu().numpy()  # noqa: E731
        rows = lambda x: x.reshape(b.hq, Q).cpu().numpy()  # noqa: E731
        o, mag, l, top = back(p @ v), back(p @ v.abs()), rows(lse), rows(m.amax(-1))
        b_out, b_lse = R.attend_bounds(o, l, mag, top, b.d, n, b.p_half())
        _within(R.f64(b.out[c]), o, b_out, f"out of sequence {r}")
        _within(R.f64(b.lse[:, c]), l, b_lse, f"lse of sequence {r}")
        if mass is None:
            continue
        # from the LSE that the call was given, as R.key_mass
        given = b.lse[:, c].double().reshape(b.hkv, G * Q, 1)
        w = torch.where(see, torch.exp(s - given), 0.0)
        e = R.score_error(m, b.d) + (torch.where(see, s.abs(), 0.0) + given.abs() + 4) * 4 * R.U + (Q * G + 16) * 2 * R.U
        want, bound = w.sum(1).cpu().numpy(), (w * e).sum(1).cpu().numpy()
        _within(R.f64(mass[r, :, :n]), want, bound + 3 * R.U * want + 1e-37, f"mass of sequence {r}")


def _attend_and_weigh(b):
    from block_sparse_long_pooled_b200 import fp2
    b.attend()
    assert _status(b.scratch) == (0, 0)
    mass = torch.zeros((len(b.lens), b.hkv, b.max_len), device="cuda")
    fp2.fp2_key_mass(b.handle, b.lse, None, mass, b.scratch)
    check_all(b, mass)


INSTANCES = [("e4m3", 128), ("bf16", 64), ("bf16", 128)]


@pytest.mark.parametrize("dtype,d", INSTANCES)
@pytest.mark.parametrize("qlen", [1, 5, 64])      # the few-rows kernel; both streams on one row tile; a row tile each
def test_rings_go_round_on_one_sequence(dtype, d, qlen):
    # 938 tiles of 64 keys and 469 of 128 over 18 CTAs a KV head (37 of the few-rows kernel): 26 and more each, of
    # rings of up to 8; an odd number of tiles, the last one in part
    _attend_and_weigh(Batch(dtype, d, 32, 8, 64, (60001,), (qlen,), "tree", seed=70 + qlen))


@pytest.mark.parametrize("dtype,d", INSTANCES)
@pytest.mark.parametrize("page", [0, 16, 128])
def test_rings_go_round_across_pieces(dtype, d, page):
    """Sequences of one, two and more row tiles in one batch: streams that change between sharing a row tile and
    having one each, several passes of the weights, NaN in every row that no token may see."""
    b = Batch(dtype, d, 16, 4, page, (9000, 131, 12007, 2560, 3001, 77, 15000, 64, 1), (64, 5, 33, 64, 1, 7, 40, 64, 1),
              "tree", seed=80, holes=True, rows_over=5)
    _attend_and_weigh(b)
    # 74 KV heads: two CTAs each, that walk all of a batch
    b = Batch(dtype, d, 74, 74, page, (700, 1031, 64, 300, 65, 900), (20, 64, 17, 33, 1, 30), "tree", seed=81, holes=True)
    _attend_and_weigh(b)


@pytest.mark.parametrize("dtype,d", INSTANCES)
@pytest.mark.parametrize("hq,hkv,lens,qlens", [(32, 8, (20001,), (5,)), (32, 8, (20001,), (64,)),
                                               (16, 4, (3000, 8001, 131), (64, 6, 40))])
def test_a_v_tile_that_lands_late_changes_nothing(dtype, d, hq, hkv, lens, qlens):
    """A V tile that is loaded after the two behind it, some 50 us later: the same bits.  (The checked build has the
    hook, and runs this below; the normal one ignores it.)"""
    from block_sparse_long_pooled_b200 import fp2
    b = Batch(dtype, d, hq, hkv, 64, lens, qlens, "tree", seed=90)
    b.attend()
    check_all(b)
    want = b.out.clone(), b.lse.clone()
    try:
        for tile in range(10):
            fp2.fp2_debug_set(fp2.FP2_DEBUG_LATE_V_TILE, tile)
            b.out.fill_(7.0)
            b.attend()
            assert _status(b.scratch) == (0, 0)
            assert torch.equal(b.out, want[0]) and torch.equal(b.lse, want[1]), tile
    finally:
        fp2.fp2_debug_set(fp2.FP2_DEBUG_LATE_V_TILE, -1)


@pytest.mark.parametrize("page,dst_page", [(64, 64), (0, 16)])
def test_evict_from_sequences_whose_weights_are_read_again(page, dst_page):
    """More keys than a cluster's threads hold (16 x 512 x 16), and weights of a few values: ties everywhere."""
    lens = (200000, 131073, 131072, 140011)
    g = _gen(60)
    mass = torch.floor(torch.randn((4, 1, lens[0]), generator=g).abs() * 2)
    mass[3, 0, ::7] = torch.rand((lens[0] + 6) // 7, generator=g) * 4
    _evict_case("bf16", 64, 1, page, lens, 1200, 5, 70, mass=mass, dst_page=dst_page)


def test_ring_cases_pass_under_the_checked_build():
    import os
    import subprocess
    import sys
    from block_sparse_long_pooled_b200 import build, fp2
    if fp2.fp2_build_flags() == fp2.FP2_BUILD_CHECKED:
        pytest.skip("this is that run")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        "tests/test_gpu_serve_rings.py", "-k", "rings_go_round or lands_late"], cwd=root,
                       env=dict(os.environ, FP2_LIBRARY=build.build(checked=True)), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]

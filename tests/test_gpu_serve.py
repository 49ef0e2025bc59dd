"""The serving operators on the GPU against their 64-bit forms (tests/serve_ref.py has the bounds)."""

import numpy as np
import pytest
import torch

from tests import serve_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _store(x, dtype):
    return x.clamp(-448, 448).to(R.TORCH[dtype]) if dtype == "e4m3" else x.to(R.TORCH[dtype])


def _within(got, want, bound, what):
    got = R.f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {want[bad][0]}, bound {np.broadcast_to(bound, bad.shape)[bad][0]}"


def _status(scratch):
    from block_sparse_long_pooled_b200 import fp2
    torch.cuda.synchronize()
    return fp2.fp2_get_device_status(scratch)


# ------------------------------------------------------------------ rotate

@pytest.mark.parametrize("src,dst,d,rot,inter,norm,tokens,hq,hkv,page", [
    ("bf16", "bf16", 128, 128, False, False, 1, 8, 2, 16),
    ("bf16", "bf16", 128, 64, True, True, 37, 5, 1, 64),
    ("bf16", "bf16", 64, 16, False, True, 130, 3, 3, 0),
    ("bf16", "e4m3", 128, 128, False, True, 513, 32, 4, 64),
    ("bf16", "e4m3", 128, 32, True, False, 9, 7, 7, 0),
    ("bf16", "e4m3", 64, 64, False, False, 21, 2, 1, 16),
    ("f32", "f32", 64, 32, True, False, 257, 8, 2, 0),
    ("f32", "f32", 64, 64, False, True, 2, 1, 1, 128),
    ("f32", "f32", 128, 128, False, True, 66, 4, 2, 16),
    ("f32", "e4m3", 64, 48, False, False, 19, 4, 4, 16),
    ("bf16", "bf16", 128, 0, False, True, 40, 4, 2, 0),        # norms only
    ("bf16", "bf16", 128, 112, False, False, 3000, 9, 1, 64),  # warps that walk several heads
    # so many tokens that a warp has several
    ("bf16", "e4m3", 128, 128, False, True, 9601, 3, 1, 16),
    ("bf16", "bf16", 128, 48, True, False, 9474, 1, 2, 0),
    ("bf16", "bf16", 64, 64, False, True, 18949, 1, 1, 64),
    ("f32", "f32", 64, 32, True, True, 19001, 2, 1, 0),
    ("f32", "e4m3", 64, 64, False, False, 18947, 1, 1, 128),
    ("bf16", "bf16", 64, 32, True, True, 16401, 8, 1, 16),
])
def test_rotate(src, dst, d, rot, inter, norm, tokens, hq, hkv, page):
    from block_sparse_long_pooled_b200 import fp2
    g = _gen(7)
    qkv = (torch.randn((tokens, hq + 2 * hkv, d), generator=g) * 1.5).to(R.TORCH[src]).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g).to(torch.int32)
    pos[0] = 2 ** 31 - 1
    freq = None if rot == 0 else fp2.rope_frequencies(rot, 500000.0, "llama3", 8.0)[0]
    rope = None if rot == 0 else fp2.make_rope(freq, inter, 1.25)
    wq = (1 + 0.3 * torch.randn(d, generator=g)).to(R.TORCH[src]).cuda() if norm else None
    wk = (1 + 0.3 * torch.randn(d, generator=g)).to(R.TORCH[src]).cuda() if norm else None
    de = dict(q_descale=0.5, k_descale=0.25, v_descale=0.125) if dst == "e4m3" else {}
    slots = None
    shape = (tokens, hkv, d)
    if page:
        pages = -(-tokens // page) + 1
        shape = (pages, page, hkv, d)
        slots = torch.randperm(pages * page, generator=g)[:tokens].clone()
        if tokens > 1:
            slots[tokens // 2] = -1
    mark = _store(torch.full((1,), 3.0), dst)
    qo = mark.cuda().expand(tokens * hq * d).clone().view(tokens, hq, d)
    ko = mark.cuda().expand(int(np.prod(shape))).clone().view(shape)
    vo = ko.clone()
    h = fp2.make_rotate(q, k, v, pos.cuda(), rope, qo, ko, vo, slots=None if slots is None else slots.cuda(),
                        q_norm=wq, k_norm=wk, norm_eps=1e-5, **de)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp2.fp2_rotate(h, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for x, out, w, scale, where in ((q, qo, wq, de.get("q_descale", 1.0), None), (k, ko, wk, de.get("k_descale", 1.0), slots),
                                    (v, vo, None, de.get("v_descale", 1.0), slots)):
        turns = out is not vo
        want, mag = R.rotate(R.f64(x), pos.numpy(), freq if turns else None, inter, 1.25,
                             None if w is None else R.f64(w), 1e-5)
        bound = R.rotate_bound(want, mag, dst, scale)
        if dst == "e4m3":
            lim = 448 * scale
            want = np.clip(want, -lim, lim)
        got = R.f64(out) * scale
        if where is None:
            _within(got.reshape(want.shape), want, bound, "rows")
            continue
        flat = got.reshape(-1, hkv, d)
        use = where.numpy() >= 0
        _within(flat[where.numpy()[use]], want[use], bound[use], "slots")
        rest = np.ones(len(flat), bool)
        rest[where.numpy()[use]] = False
        assert (flat[rest] == 3.0 * scale).all()    # rows that no slot names are left alone


def test_rotate_in_place_and_partial_inputs():
    from block_sparse_long_pooled_b200 import fp2
    g = _gen(8)
    q = torch.randn((70, 6, 128), generator=g).to(torch.bfloat16).cuda()
    k = torch.randn((70, 2, 128), generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(70, dtype=torch.int32, device="cuda")
    rope = fp2.make_rope(fp2.rope_frequencies(128)[0])
    a, b = torch.empty_like(q), torch.empty_like(k)
    fp2.fp2_rotate(fp2.make_rotate(q, k, None, pos, rope, a, b, None))
    c, d = torch.empty_like(q), torch.empty_like(k)
    fp2.fp2_rotate(fp2.make_rotate(q, None, None, pos, rope, c, None, None))
    fp2.fp2_rotate(fp2.make_rotate(None, k, None, pos, rope, None, d, None))
    assert torch.equal(a, c) and torch.equal(b, d)
    fp2.fp2_rotate(fp2.make_rotate(q, k, None, pos, rope, q, k, None))
    assert torch.equal(a, q) and torch.equal(b, k)


def test_rotate_reports_a_slot_out_of_range():
    from block_sparse_long_pooled_b200 import fp2
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    out, out2 = (torch.zeros((4, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 4, 0], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = fp2.make_rope(fp2.rope_frequencies(64)[0])
    fp2.fp2_rotate(fp2.make_rotate(None, k, k, pos, rope, None, out, out2, slots=slots), status)
    assert int(status) == fp2.FP2_DEV_SLOT_OOB
    for o in (out, out2):
        assert torch.equal(o[:, 0, 0].cpu(), torch.tensor([1.0, 0, 0, 1.0], dtype=torch.bfloat16))


# ------------------------------------------------------------------ decode

class Batch:
    """A decode batch on the GPU.  `holes`: everything that no token may see is NaN (K and V)."""

    def __init__(self, dtype, d, hq, hkv, page, lens, qlens, mask="tree", seed=0, holes=False, rows_over=0, joined=False,
                 gain=1.0):
        from block_sparse_long_pooled_b200 import fp2
        g = _gen(seed)
        self.dtype, self.d, self.hq, self.hkv, self.page = dtype, d, hq, hkv, page
        self.lens, self.qlens = list(lens), list(qlens)
        n, T = len(lens), sum(qlens)
        self.max_len = max(max(lens), max(qlens), 1) + rows_over
        if page:
            need = [-(-x // page) for x in lens]
            most, total = max(-(-self.max_len // page), 1), sum(need) + 3
            order = torch.randperm(total, generator=g).to(torch.int32)
            self.table = torch.full((n, most), -7, dtype=torch.int32)
            at = 0
            for r, x in enumerate(need):
                self.table[r, :x] = order[at:at + x]
                at += x
            shape = (total, page, hkv, d)
        else:
            self.table, shape = None, (n, self.max_len, hkv, d)
        self.descale = dict(q_descale=1 / 16, k_descale=1 / 32, v_descale=1 / 64) if dtype == "e4m3" else {}
        ds = [self.descale.get(w + "_descale", 1.0) for w in "qkv"]
        k = _store(torch.randn(shape, generator=g) / ds[1], dtype)
        v = _store(torch.randn(shape, generator=g) / ds[2], dtype)
        q = _store(torch.randn((T, hq, d), generator=g) * gain / ds[0], dtype)
        self.cu = [0]
        for x in qlens:
            self.cu.append(self.cu[-1] + x)
        words = None
        if mask == "tree":
            words = torch.zeros(T, dtype=torch.int64)
            for r, x in enumerate(qlens):
                own = []
                for i in range(x):
                    up = int(torch.randint(max(0, i - 3), i, (1,), generator=g)) if i else None
                    w = (own[up] if i else 0) | (1 << i)
                    own.append(w)
                    words[self.cu[r] + i] = w - (1 << 64) if w >> 63 else w
        elif mask == "none":       # no drafted key is seen; with no earlier keys the row is empty
            words = torch.zeros(T, dtype=torch.int64)
        elif mask == "all":        # bits past the sequence's tokens mean nothing
            words = torch.full((T,), -1, dtype=torch.int64)
        self.words = words
        self.vis = [R.visible(x, m, None if words is None else words[self.cu[r]:self.cu[r] + x].numpy())
                    if x <= m else np.zeros((x, max(m, 0)), bool) for r, (x, m) in enumerate(zip(qlens, lens))]
        if holes:
            bad = torch.full((hkv, d), float("nan")).to(R.TORCH[dtype])
            used = np.zeros(shape[:2], bool)
            for r, m in enumerate(lens):
                see = self.vis[r].any(0) if qlens[r] else np.zeros(m, bool)
                for j in range(m):
                    at = (r, j) if self.table is None else (int(self.table[r, j // page]), j % page)
                    used[at] = see[j]
            w = torch.from_numpy(~used)
            for x in (k, v):
                bits = {"e4m3": torch.uint8, "bf16": torch.int16, "f32": torch.int32}[dtype]
                xb, bb = x.view(bits), bad.view(bits)
                xb[w] = bb
        self.kc, self.vc, self.qc = k, v, q
        if joined:    # K and V interleaved token by token, Q a view of a wider tensor
            both = torch.empty((shape[0], shape[1], 2, hkv, d), dtype=k.dtype)
            both.view(torch.uint8)[:, :, 0] = k.view(torch.uint8)
            both.view(torch.uint8)[:, :, 1] = v.view(torch.uint8)
            both = both.cuda()
            self.k, self.v = both[:, :, 0], both[:, :, 1]
            wide = torch.zeros((T, hq + 3, d), dtype=q.dtype).cuda()
            self.q = wide[:, 2:2 + hq]
            self.q.view(torch.uint8).copy_(q.view(torch.uint8).cuda())
        else:
            self.k, self.v, self.q = k.cuda(), v.cuda(), q.cuda()
        self.table_dev = None if self.table is None else self.table.cuda()
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.words_dev = None if words is None else words.cuda()
        self.cache = fp2.make_cache(self.k, self.v, self.table_dev)
        self.scale = 1.0 / np.sqrt(d)
        self.handle = fp2.make_decode(self.q, self.cache, self.cu, self.kv_len, self.max_len, hkv,
                                      tree_mask=self.words_dev, **self.descale)
        self.scratch = fp2.alloc_scratch(fp2.fp2_decode_workspace(self.handle), "cuda")
        self.out = torch.full((T, hq, d), 7.0, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
        self.lse = torch.full((hq, T), 7.0, device="cuda")
        self.ds = ds

    def values(self, r):
        n, c = self.lens[r], slice(self.cu[r], self.cu[r + 1])
        table = None if self.table is None else self.table.numpy()
        return (R.f64(self.qc[c]) * self.ds[0], R.cache_rows(self.kc, table, r, n) * self.ds[1],
                R.cache_rows(self.vc, table, r, n) * self.ds[2])

    def attend(self, stream=None):
        from block_sparse_long_pooled_b200 import fp2
        fp2.fp2_tree_attend(self.handle, self.out, self.lse, self.scratch, stream=stream)

    def p_half(self):
        # e4m3: weights are f16.  bf16: two bf16 halves when no sequence has over 128 rows per KV head, else one.
        if self.dtype == "e4m3":
            return R.HALF["f16"]
        if self.dtype == "f32":
            return 0.0
        rows = max(self.qlens) * self.hq // self.hkv
        return R.HALF["bf16"] ** 2 if rows <= 128 else R.HALF["bf16"]

    def check(self):
        assert _status(self.scratch) == (0, 0)
        out, lse = R.f64(self.out), R.f64(self.lse)
        for r in range(len(self.lens)):
            if self.qlens[r] == 0:
                continue
            c = slice(self.cu[r], self.cu[r + 1])
            q, k, v = self.values(r)
            o, l, mag, top = R.attend(q, k, v, self.scale, self.vis[r])
            b_out, b_lse = R.attend_bounds(o, l, mag, top, self.d, self.lens[r], self.p_half(),
                                            "f32" if self.dtype == "f32" else "bf16")
            _within(out[c], o, b_out, f"out of sequence {r}")
            empty = ~np.isfinite(l)
            assert (lse[:, c][empty] == -np.inf).all() and (out[c].transpose(1, 0, 2)[empty] == 0).all()
            _within(lse[:, c][~empty], l[~empty], b_lse[~empty], f"lse of sequence {r}")


TREE = [
    # dtype, d, hq, hkv, page, lens, qlens, mask
    ("bf16", 128, 32, 8, 0, (1,), (1,), None),
    ("bf16", 128, 32, 8, 64, (300, 1, 65, 64, 63), (1, 1, 1, 1, 1), None),
    ("bf16", 128, 8, 2, 16, (1000, 33, 17), (3, 7, 1), "tree"),
    ("bf16", 128, 5, 1, 128, (777, 130), (5, 6), "tree"),
    ("bf16", 64, 8, 8, 16, (200, 64, 7), (7, 64, 7), "tree"),
    ("bf16", 64, 8, 1, 0, (513, 100), (4, 2), None),
    ("bf16", 64, 16, 2, 64, (900, 40), (9, 40), "tree"),
    ("bf16", 128, 16, 2, 64, (700, 64, 5000), (64, 64, 33), "tree"),
    ("bf16", 128, 64, 2, 64, (70, 300), (64, 20), None),           # 32 heads a KV head: 2048 rows
    ("bf16", 128, 4, 4, 64, (20000,), (2,), "tree"),
    ("e4m3", 128, 32, 8, 64, (129, 64, 1, 1000), (1, 1, 1, 1), None),
    ("e4m3", 128, 8, 1, 16, (50, 400, 7), (4, 3, 7), "tree"),
    ("e4m3", 128, 10, 2, 128, (600, 90), (13, 64), "tree"),
    ("e4m3", 128, 8, 8, 0, (64, 3000, 31), (1, 64, 31), "all"),
    ("bf16", 128, 8, 2, 16, (40, 6, 0, 9), (6, 6, 0, 0), "none"),  # rows without a key, sequences without a token
    ("e4m3", 128, 8, 2, 16, (40, 5, 0, 9), (6, 5, 0, 0), "none"),
    ("f32", 64, 8, 2, 16, (300, 1, 65, 64), (1, 1, 1, 1), None),
    ("f32", 64, 10, 2, 0, (700, 64), (5, 33), "tree"),
    ("f32", 64, 4, 4, 64, (9000, 3), (64, 3), "all"),
    ("f32", 64, 4, 1, 128, (40, 6, 0, 9), (6, 6, 0, 0), "none"),
    ("f32", 64, 16, 2, 16, (300, 64), (64, 20), "tree"),
    # one sequence in 74 pieces or more
    ("bf16", 64, 4, 1, 16, (20001,), (3,), "tree"),
    ("e4m3", 128, 4, 1, 0, (12000,), (11,), "tree"),
    ("f32", 64, 4, 1, 64, (8200,), (2,), None),
]


@pytest.mark.parametrize("dtype,d,hq,hkv,page,lens,qlens,mask", TREE)
@pytest.mark.parametrize("holes", [False, True])
def test_tree_attend(dtype, d, hq, hkv, page, lens, qlens, mask, holes):
    b = Batch(dtype, d, hq, hkv, page, lens, qlens, mask, seed=len(lens) + d, holes=holes, rows_over=13 if holes else 0)
    b.attend()
    b.check()


def test_tree_attend_strided_inputs_and_large_scores():
    for dtype, d in (("bf16", 128), ("e4m3", 128), ("f32", 64)):
        b = Batch(dtype, d, 8, 2, 16, (500, 77), (3, 1), "tree", seed=5, joined=True, gain=6.0)
        b.attend()
        b.check()


@pytest.mark.parametrize("qlen", [1, 40])
def test_a_value_that_only_some_tokens_see(qlen):
    """An infinite or NaN V row of a drafted key reaches exactly the rows that see the key."""
    for dtype, d, bad in (("bf16", 128, float("inf")), ("bf16", 128, float("nan")), ("e4m3", 128, float("nan")),
                          ("f32", 64, float("inf"))):
        b = Batch(dtype, d, 8, 2, 64, (200,), (qlen + 2,), "tree", seed=11)
        words = b.words.clone()
        words[:] = 1                       # every token sees drafted key 0
        words[qlen] |= 1 << (qlen + 1)     # token qlen also sees the last one
        b.words_dev.copy_(words)
        n = 200
        j = n - 1
        page = int(b.table[0, j // 64])
        b.v[page, j % 64] = torch.tensor(bad).to(b.v.dtype) if dtype != "e4m3" else b.v[page, j % 64]
        if dtype == "e4m3":
            b.v.view(torch.uint8)[page, j % 64] = 0x7F
        b.attend()
        torch.cuda.synchronize()
        fin = torch.isfinite(b.out.float()).all(-1).all(-1).cpu()
        assert not fin[qlen] and fin[:qlen].all() and fin[qlen + 1:].all()


@pytest.mark.parametrize("qlen", [1, 40])
def test_a_value_that_is_not_finite_stays_in_its_element(qlen):
    """NaN in V of a key that every token sees: NaN there, in every token of the group's heads, and nowhere else."""
    for dtype, d in (("bf16", 128), ("e4m3", 128), ("f32", 64)):
        b = Batch(dtype, d, 8, 2, 64, (300,), (qlen,), None, seed=12)
        page = int(b.table[0, 1])
        if dtype == "e4m3":
            b.v.view(torch.uint8)[page, 7, 1, 37] = 0xFF
        else:
            b.v[page, 7, 1, 37] = float("nan")
        b.attend()
        torch.cuda.synchronize()
        bad = torch.isnan(b.out.float()).cpu()
        want = torch.zeros_like(bad)
        want[:, 4:, 37] = True
        assert torch.equal(bad, want) and torch.isfinite(b.lse).all()


def test_a_cache_whose_offsets_pass_32_bits():
    """Pages at the end of caches of 2.3e9 values (K, V and the eviction's)."""
    from block_sparse_long_pooled_b200 import fp2
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    g = _gen(40)
    pages, hkv, d = 140000, 2, 128
    k, v, ko, vo = (torch.empty((pages, 64, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    assert k.numel() > 1 << 31
    table = torch.arange(pages - 5, pages, dtype=torch.int32, device="cuda")[None].contiguous()
    n = 300
    kk, vv = (torch.randn((5 * 64, hkv, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    slots = (pages - 5) * 64 + torch.arange(n, device="cuda")
    fp2.fp2_rotate(fp2.make_rotate(None, kk[:n], vv[:n], pos, None, None, k, v, slots=slots))
    q = torch.randn((3, 4, d), generator=g).to(torch.bfloat16).cuda()
    cache = fp2.make_cache(k, v, table)
    kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
    dec = fp2.make_decode(q, cache, [0, 3], kv_len, n)
    scratch = fp2.alloc_scratch(fp2.fp2_decode_workspace(dec), "cuda")
    out, lse = torch.empty_like(q), torch.empty((4, 3), device="cuda")
    fp2.fp2_tree_attend(dec, out, lse, scratch)
    vis = R.visible(3, n, None)
    want, wl, mag, top = R.attend(R.f64(q), R.f64(kk[:n]), R.f64(vv[:n]), d ** -0.5, vis)
    bo, bl = R.attend_bounds(want, wl, mag, top, d, n, R.HALF["bf16"] ** 2)
    _within(out, want, bo, "out")
    mass = torch.zeros((1, hkv, n), device="cuda")
    fp2.fp2_key_mass(dec, lse, None, mass, scratch)
    new, bound = R.key_mass(R.f64(q), R.f64(kk[:n]), d ** -0.5, vis, R.f64(lse))
    _within(mass[0], new, bound + 3 * R.U * new + 1e-37, "mass")
    mo, kept = torch.empty((1, hkv, 64), device="cuda"), torch.empty((1, hkv, 64), dtype=torch.int32, device="cuda")
    lo = torch.empty(1, dtype=torch.int32, device="cuda")
    ev = fp2.make_evict(cache, kv_len, n, mass, 64, 4, 8, fp2.make_cache(ko, vo, table[:, 4:].contiguous()), mo, kept, lo)
    es = fp2.alloc_scratch(fp2.fp2_evict_workspace(ev), "cuda")
    fp2.fp2_evict(ev, es)
    assert _status(es) == (0, 0)
    for h in range(hkv):
        idx = R.evict(mass[0, h].cpu().numpy(), n, 64, 4, 8)
        assert np.array_equal(kept[0, h].cpu().numpy(), idx)
        assert torch.equal(ko[pages - 1, :, h], kk[idx, h]) and torch.equal(vo[pages - 1, :, h], vv[idx, h])


def test_tree_attend_is_repeatable_and_lse_is_optional():
    from block_sparse_long_pooled_b200 import fp2
    b = Batch("bf16", 128, 16, 4, 64, (9000, 100, 4000), (5, 1, 8), "tree", seed=3)
    b.attend()
    first = b.out.clone()
    for _ in range(3):
        fp2.fp2_tree_attend(b.handle, b.out, None, b.scratch)
        assert torch.equal(first, b.out)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_tree_attend_bad_lengths_and_pages(dtype, d):
    from block_sparse_long_pooled_b200 import fp2
    b = Batch(dtype, d, 8, 2, 16, (100, 90, 80), (2, 2, 2), None, seed=4)
    b.kv_len.copy_(torch.tensor([100, b.max_len + 1, 1]))   # above the bound; below its tokens
    b.attend()
    st, bits = _status(b.scratch)
    assert st == fp2.FP2_ERR_DEVICE_BOUNDS and bits == fp2.FP2_DEV_LEN_OOB
    assert (b.out[2:] == 0).all() and (b.lse[:, 2:] == -float("inf")).all()
    want, lse, _, _ = R.attend(*b.values(0), b.scale, b.vis[0])
    assert np.abs(R.f64(b.out[:2]) - want).max() < 0.05
    # a page id out of range: its keys drop out, the rest is attended
    b.kv_len.copy_(torch.tensor([100, 90, 80]))
    for wrong in (-1, b.k.shape[0]):
        keep = int(b.table[1, 2])
        b.table_dev[1, 2] = wrong
        b.attend()
        st, bits = _status(b.scratch)
        assert st == fp2.FP2_ERR_DEVICE_BOUNDS and bits == fp2.FP2_DEV_PAGE_OOB
        q, k, v = b.values(1)
        vis = b.vis[1].copy()
        vis[:, 32:48] = False
        want, lse, mag, top = R.attend(q, k, v, b.scale, vis)
        _within(b.out[2:4], want, R.attend_bounds(want, lse, mag, top, d, 90, b.p_half(), dtype)[0], "the other pages")
        b.table_dev[1, 2] = keep
    b.attend()
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("qlen", [1, 64])
def test_decode_waits_are_bounded(dtype, qlen):
    """A load that never arrives ends in a status bit; the next call is unaffected."""
    from block_sparse_long_pooled_b200 import fp2
    b = Batch(dtype, 128, 8, 2, 64, (900, 300), (qlen, qlen), None, seed=9)
    mass = torch.zeros((2, 2, b.max_len), device="cuda")
    b.attend()
    b.check()
    try:
        fp2.fp2_debug_set(fp2.FP2_DEBUG_WAIT_LIMIT_NS, 2_000_000)
        fp2.fp2_debug_set(fp2.FP2_DEBUG_WITHHOLD_K_TILE, 0)
        b.attend()
        st, bits = _status(b.scratch)
        assert st == fp2.FP2_ERR_TIMEOUT and bits & fp2.FP2_DEV_TIMEOUT
        fp2.fp2_key_mass(b.handle, torch.zeros_like(b.lse), None, mass, b.scratch)
        st, bits = _status(b.scratch)
        assert st == fp2.FP2_ERR_TIMEOUT and bits & fp2.FP2_DEV_TIMEOUT
    finally:
        fp2.fp2_debug_set(fp2.FP2_DEBUG_WITHHOLD_K_TILE, -1)
        fp2.fp2_debug_set(fp2.FP2_DEBUG_WAIT_LIMIT_NS, 0)
    b.attend()
    b.check()


# ------------------------------------------------------------------ key mass

@pytest.mark.parametrize("dtype,d,hq,hkv,page,lens,qlens,mask", TREE)
@pytest.mark.parametrize("in_place", [False, True])
def test_key_mass(dtype, d, hq, hkv, page, lens, qlens, mask, in_place):
    from block_sparse_long_pooled_b200 import fp2
    b = Batch(dtype, d, hq, hkv, page, lens, qlens, mask, seed=len(lens) + d, holes=in_place)
    b.attend()
    g = _gen(21)
    n, stride = len(lens), b.max_len + 5
    mass = torch.rand((n, hkv, stride), generator=g)
    had = torch.tensor([max(0, x - y) for x, y in zip(lens, qlens)], dtype=torch.int32)
    mass_in = mass.cuda()
    out = mass_in if in_place else torch.full((n, hkv, stride), -5.0, device="cuda")
    fp2.fp2_key_mass(b.handle, b.lse, mass_in, out, b.scratch, decay=0.75, mass_len=had.cuda() if in_place else None)
    assert _status(b.scratch) == (0, 0)
    got, lse = R.f64(out), R.f64(b.lse)
    for r in range(n):
        old = mass[r].double().numpy()
        rest = old if in_place else np.full_like(old, -5.0)
        assert (got[r, :, lens[r]:] == rest[:, lens[r]:]).all()
        keep = old[:, :lens[r]] * 0.75
        if in_place:
            keep[:, int(had[r]):] = 0
        if qlens[r] == 0:
            new, bound = np.zeros_like(keep), np.zeros_like(keep)
        else:
            c = slice(b.cu[r], b.cu[r + 1])
            q, k, _ = b.values(r)
            new, bound = R.key_mass(q, k, b.scale, b.vis[r], lse[:, c])
        # the decayed sum and its sum with the new weight: a rounding each
        _within(got[r, :, :lens[r]], keep + new, bound + 3 * R.U * (np.abs(keep) + new) + 1e-37, f"mass of sequence {r}")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_key_mass_without_any_token_decays(dtype, d):
    from block_sparse_long_pooled_b200 import fp2
    b = Batch(dtype, d, 8, 2, 16, (200, 0, 33), (0, 0, 0), None, seed=13)
    mass = torch.rand((3, 2, b.max_len), generator=_gen(1)).cuda()
    out = torch.full_like(mass, -1.0)
    fp2.fp2_key_mass(b.handle, b.lse, mass, out, b.scratch, decay=0.5)
    assert _status(b.scratch) == (0, 0)
    for r, n in enumerate(b.lens):
        assert torch.equal(out[r, :, :n], mass[r, :, :n] * 0.5) and (out[r, :, n:] == -1).all()
    b.attend()     # no rows: nothing to do, and no stale status
    assert _status(b.scratch) == (0, 0)


def test_key_mass_sums_to_the_rows():
    from block_sparse_long_pooled_b200 import fp2
    b = Batch("bf16", 128, 8, 2, 64, (3000, 64), (9, 64), "tree", seed=2)
    b.attend()
    mass = torch.zeros((2, 2, b.max_len), device="cuda")
    fp2.fp2_key_mass(b.handle, b.lse, None, mass, b.scratch)
    total = mass.double().sum(-1).cpu()
    assert torch.allclose(total, torch.tensor([[36.0, 36.0], [256.0, 256.0]], dtype=torch.float64), rtol=1e-4)


# ------------------------------------------------------------------ evict

def _evict_case(dtype, d, hkv, page, lens, budget, sink, window, mass=None, seed=1, dst_page=None):
    from block_sparse_long_pooled_b200 import fp2
    g = _gen(seed)
    n, L = len(lens), max(max(lens), 1)
    dst_page = page if dst_page is None else dst_page

    def cache(sizes, page, fill):
        if page:
            need = [-(-x // page) for x in sizes]
            total = sum(need) + 2
            order = torch.randperm(total, generator=g).to(torch.int32)
            table = torch.full((n, max(max(need), 1)), -3, dtype=torch.int32)
            at = 0
            for r, x in enumerate(need):
                table[r, :x] = order[at:at + x]
                at += x
            shape = (total, page, hkv, d)
        else:
            table, shape = None, (n, max(max(sizes), 1), hkv, d)
        mk = lambda: torch.randint(0, 120, shape + (R.TORCH[dtype].itemsize,), generator=g, dtype=torch.uint8).view(R.TORCH[dtype])[..., 0] if fill else torch.zeros(shape).to(R.TORCH[dtype])  # noqa: E731,E501
        return mk().contiguous().cuda(), mk().contiguous().cuda(), table

    k, v, table = cache(lens, page, True)
    ko, vo, table_o = cache([min(x, budget) for x in lens], dst_page, False)
    if mass is None:
        mass = torch.randn((n, hkv, L), generator=g).mul_(2.5).exp_() * (torch.rand((n, hkv, L), generator=g) > 0.3)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mo = torch.full((n, hkv, budget), -1.0, device="cuda")
    kept = torch.full((n, hkv, budget), -9, dtype=torch.int32, device="cuda")
    lo = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    h = fp2.make_evict(fp2.make_cache(k, v, dev(table)), kv_len, L, mass.cuda(), budget, sink, window,
                       fp2.make_cache(ko, vo, dev(table_o)), mo, kept, lo)
    scratch = fp2.alloc_scratch(fp2.fp2_evict_workspace(h), "cuda")
    fp2.fp2_evict(h, scratch)
    assert _status(scratch) == (0, 0)
    raw = lambda t: t.view(torch.uint8).cpu().numpy().reshape(*t.shape[:3], -1)  # noqa: E731
    rk, rv, rko, rvo = raw(k), raw(v), raw(ko), raw(vo)
    at = lambda t, x, r, j: x[r, j] if t is None else x[int(t[r, j // x.shape[1]]), j % x.shape[1]]  # noqa: E731
    for r, m in enumerate(lens):
        N = min(m, budget)
        assert int(lo[r]) == N
        for hh in range(hkv):
            want = R.evict(mass[r, hh].numpy(), m, budget, sink, window)
            assert np.array_equal(kept[r, hh, :N].cpu().numpy(), want), (r, hh)
            assert (kept[r, hh, N:] == -1).all() and (mo[r, hh, N:] == 0).all()
            assert np.array_equal(mo[r, hh, :N].cpu().numpy(), mass[r, hh].numpy()[want], equal_nan=True)
            for i, j in enumerate(want):
                assert np.array_equal(at(table_o, rko, r, i)[hh], at(table, rk, r, int(j))[hh])
                assert np.array_equal(at(table_o, rvo, r, i)[hh], at(table, rv, r, int(j))[hh])
    if table_o is None:
        for r, m in enumerate(lens):
            assert (rko[r, min(m, budget):] == 0).all() and (rvo[r, min(m, budget):] == 0).all()


@pytest.mark.parametrize("dtype,d,hkv,page,lens,budget,sink,window", [
    ("bf16", 128, 2, 16, (100, 40, 0, 1, 64, 65), 64, 4, 16),
    ("bf16", 64, 1, 0, (500, 33), 32, 0, 0),
    ("e4m3", 128, 3, 64, (2000, 129, 128), 128, 0, 128),         # the window is the whole budget
    ("f32", 64, 1, 16, (300,), 1, 0, 0),
    ("bf16", 128, 1, 64, (5000, 4999), 600, 100, 37),            # a cluster per row
    ("e4m3", 128, 1, 128, (20000,), 1000, 4, 64),
    ("bf16", 128, 2, 0, (300, 70), 1000, 10, 10),                # everything fits
])
def test_evict(dtype, d, hkv, page, lens, budget, sink, window):
    _evict_case(dtype, d, hkv, page, lens, budget, sink, window)


def test_evict_to_another_page_size_and_odd_weights():
    L = 400
    mass = torch.zeros((2, 2, L))
    mass[0, 0] = 1.0                                   # all equal: the lowest indexes
    mass[0, 1, 100:200] = -0.0
    mass[0, 1, 300] = float("nan")
    mass[0, 1, 5] = float("inf")
    mass[1, 0] = torch.arange(L).float() - 200         # negative ones too
    mass[1, 1] = torch.arange(L).float().flip(0) * 1e-42   # subnormal
    _evict_case("bf16", 128, 2, 64, (L, L - 3), 50, 3, 5, mass=mass, dst_page=16)
    _evict_case("bf16", 128, 2, 64, (L, L - 3), 50, 0, 0, mass=mass, dst_page=0)


def test_evict_bad_lengths_and_pages():
    from block_sparse_long_pooled_b200 import fp2
    k = torch.ones((8, 16, 1, 128), dtype=torch.bfloat16, device="cuda")
    ko, vo = torch.zeros_like(k), torch.zeros_like(k)
    table = torch.tensor([[0, 1, 9], [3, 4, 5]], dtype=torch.int32, device="cuda")
    table_o = torch.tensor([[0, 1], [-1, 3]], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([48, 48], dtype=torch.int32, device="cuda")
    mass = torch.arange(48, device="cuda").float().expand(2, 1, 48).contiguous()
    mo = torch.zeros((2, 1, 32), device="cuda")
    kept = torch.zeros((2, 1, 32), dtype=torch.int32, device="cuda")
    lo = torch.zeros(2, dtype=torch.int32, device="cuda")
    h = fp2.make_evict(fp2.make_cache(k, k.clone(), table), kv_len, 48, mass, 32, 0, 0, fp2.make_cache(ko, vo, table_o),
                       mo, kept, lo)
    scratch = fp2.alloc_scratch(fp2.fp2_evict_workspace(h), "cuda")
    fp2.fp2_evict(h, scratch)
    assert _status(scratch) == (fp2.FP2_ERR_DEVICE_BOUNDS, fp2.FP2_DEV_PAGE_OOB)
    assert torch.equal(kept[0, 0].cpu(), torch.arange(16, 48, dtype=torch.int32))
    assert (ko[0] == 1).all() and (ko[1] == 0).all()     # old keys 32 .. 47 are on no page
    assert (ko[3] == 1).all() and (ko[2] == 0).all()     # new rows 0 .. 15 of the second sequence neither
    kv_len.copy_(torch.tensor([49, -1]))
    ko.zero_()
    fp2.fp2_evict(h, scratch)
    assert _status(scratch) == (fp2.FP2_ERR_DEVICE_BOUNDS, fp2.FP2_DEV_LEN_OOB)
    assert (lo == 0).all() and (kept == -1).all() and (mo == 0).all() and (ko == 0).all()


# ------------------------------------------------------------------ as they are used

def test_decode_captured_in_a_graph_follows_the_lengths():
    """One graph, replayed while the cache grows; a second one with scratch of its own beside it."""
    b = Batch("bf16", 128, 8, 2, 16, (400, 90), (1, 1), None, seed=6)
    c = Batch("e4m3", 128, 8, 2, 16, (300, 90), (3, 2), "tree", seed=7)
    graphs = []
    for x in (b, c):
        x.attend()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            x.attend()
        graphs.append(gr)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for lens in ((400, 90), (377, 1), (16, 17)):
        b.lens = list(lens)
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        b.vis = [R.visible(1, n, None) for n in lens]
        b.out.fill_(7.0)
        torch.cuda.synchronize()
        for s, gr in ((s1, graphs[0]), (s2, graphs[1])):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        b.check()
        c.check()


def test_calls_that_overlap_on_two_streams():
    """Eager and captured decode, mass and eviction on two streams at once, with scratch of their own."""
    from block_sparse_long_pooled_b200 import fp2
    sides = []
    for i, (dtype, qlens) in enumerate((("bf16", (1, 1, 1)), ("e4m3", (40, 5, 64)))):
        b = Batch(dtype, 128, 8, 2, 16, (3000, 700, 64), qlens, "tree", seed=50 + i)
        mass = torch.zeros((3, 2, b.max_len), device="cuda")
        ko, vo = (torch.zeros((3, 64, 2, 128), dtype=b.k.dtype, device="cuda") for _ in range(2))
        mo, kept = torch.zeros((3, 2, 64), device="cuda"), torch.zeros((3, 2, 64), dtype=torch.int32, device="cuda")
        lo = torch.zeros(3, dtype=torch.int32, device="cuda")
        ev = fp2.make_evict(b.cache, b.kv_len, b.max_len, mass, 64, 2, 8, fp2.make_cache(ko, vo), mo, kept, lo)
        es = fp2.alloc_scratch(fp2.fp2_evict_workspace(ev), "cuda")

        def step(b=b, mass=mass, ev=ev, es=es):
            b.attend()
            fp2.fp2_key_mass(b.handle, b.lse, None, mass, b.scratch)
            fp2.fp2_evict(ev, es)

        step()
        torch.cuda.synchronize()
        b.check()
        want = [t.clone() for t in (b.out, b.lse, mass, ko.view(torch.uint8), vo.view(torch.uint8), mo, kept, lo)]
        have = (b.out, b.lse, mass, ko.view(torch.uint8), vo.view(torch.uint8), mo, kept, lo)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        sides.append((step, graph, torch.cuda.Stream(), want, have, b, es))
    for turn in range(6):
        for have in (sides[0][4], sides[1][4]):
            for t in have[:3]:
                t.zero_()
        torch.cuda.synchronize()
        for i, (step, graph, stream, _, _, _, _) in enumerate(sides):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay() if (turn + i) % 2 else step()
        torch.cuda.synchronize()
        for _, _, _, want, have, b, es in sides:
            assert all(torch.equal(x, y) for x, y in zip(want, have))    # the same bits every time
            assert _status(b.scratch) == (0, 0) and _status(es) == (0, 0)


def test_serving_loop_from_prompt_to_evicted_cache():
    """Rotate a prompt into a paged cache, prefill it, decode a drafted tree, accumulate the keys' weights, evict,
    and decode on the smaller cache: every step against its 64-bit form on the buffers of the step before."""
    from block_sparse_long_pooled_b200 import fp2
    g = _gen(31)
    hq, hkv, d, page, L, extra = 8, 2, 128, 64, 1000, 5
    freq, scale = fp2.rope_frequencies(d, 1e6, "yarn", 4.0, 32768)
    rope = fp2.make_rope(freq, False, scale)
    pages = -(-(L + extra) // page)
    table = torch.randperm(pages + 2, generator=g)[:pages].to(torch.int32)[None].contiguous()
    kc, vc = (torch.zeros((pages + 2, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def append(tokens, first, seed):
        x = torch.randn((tokens, hq + 2 * hkv, d), generator=_gen(seed)).to(torch.bfloat16).cuda()
        j = torch.arange(first, first + tokens)
        slots = table[0].long()[j // page] * page + j % page
        q = torch.empty((tokens, hq, d), dtype=torch.bfloat16, device="cuda")
        fp2.fp2_rotate(fp2.make_rotate(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], j.to(torch.int32).cuda(), rope, q,
                                       kc, vc, slots=slots.cuda()))
        return q

    q = append(L, 0, 1)
    prob = fp2.make_problem(q, kc, vc, [0, L], hkv, page_table=table.cuda())
    params = fp2.make_params(64, alpha=0.0)                   # dense: the prompt's exact attention
    ws = fp2.fp2_workspace_query(prob, params)
    scratch = fp2.alloc_scratch(ws.prefill_scratch_bytes, "cuda")
    out = torch.empty_like(q)
    lse = torch.empty((hq, L), device="cuda")
    fp2.fp2_prefill(prob, params, out, lse, scratch)
    assert _status(scratch) == (0, 0)
    t = table.numpy()
    k64, v64 = R.cache_rows(kc, t, 0, L), R.cache_rows(vc, t, 0, L)
    last = slice(L - 3, L)
    want, wl, _, _ = R.attend(R.f64(q[last]), k64, v64, d ** -0.5, R.visible(3, L, None))
    assert np.abs(R.f64(out[last]) - want).max() < 2e-2        # the prefill's own tolerance
    # the prefill's last tokens through the decode path: their weights start the keys' sums
    tail = fp2.make_decode(q[last], fp2.make_cache(kc, vc, table.cuda()), [0, 3],
                           torch.tensor([L], dtype=torch.int32, device="cuda"), L, hkv)
    ds = fp2.alloc_scratch(fp2.fp2_decode_workspace(tail), "cuda")
    mass = torch.zeros((1, hkv, L + extra), device="cuda")
    fp2.fp2_key_mass(tail, lse[:, last].contiguous(), None, mass, ds)
    # a drafted tree of five tokens
    q2 = append(extra, L, 2)
    words = torch.tensor([1, 3, 5, 11, 16], dtype=torch.int64)
    n = torch.tensor([L + extra], dtype=torch.int32, device="cuda")
    cache = fp2.make_cache(kc, vc, table.cuda())
    dec = fp2.make_decode(q2, cache, [0, extra], n, L + extra, hkv, tree_mask=words.cuda())
    ds = fp2.alloc_scratch(fp2.fp2_decode_workspace(dec), "cuda")
    o2, l2 = torch.empty_like(q2), torch.empty((hq, extra), device="cuda")
    fp2.fp2_tree_attend(dec, o2, l2, ds)
    k64, v64 = R.cache_rows(kc, t, 0, L + extra), R.cache_rows(vc, t, 0, L + extra)
    vis = R.visible(extra, L + extra, words.numpy())
    want, wl, mag, top = R.attend(R.f64(q2), k64, v64, d ** -0.5, vis)
    bo, bl = R.attend_bounds(want, wl, mag, top, d, L + extra, R.HALF["bf16"] ** 2)
    _within(o2, want, bo, "tree")
    _within(l2, wl, bl, "lse")
    before = mass.cpu().double().numpy()[0]
    fp2.fp2_key_mass(dec, l2, mass, mass, ds, decay=0.5, mass_len=torch.tensor([L], dtype=torch.int32, device="cuda"))
    new, bound = R.key_mass(R.f64(q2), k64, d ** -0.5, vis, R.f64(l2))
    before[:, L:] = 0
    _within(mass[0], before * 0.5 + new, bound + 3 * R.U * (before + new) + 1e-37, "mass")
    # keep 256 keys, go on with one token on the small cache
    budget, sink, window = 256, 4, 32
    po = -(-(budget + 1) // page)
    to = torch.arange(po - 1, -1, -1, dtype=torch.int32)[None].contiguous()
    ko, vo = (torch.zeros((po, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mo, kept = torch.zeros((1, hkv, budget), device="cuda"), torch.zeros((1, hkv, budget), dtype=torch.int32, device="cuda")
    lo = torch.zeros(1, dtype=torch.int32, device="cuda")
    small = fp2.make_cache(ko, vo, to.cuda())
    ev = fp2.make_evict(cache, n, L + extra, mass, budget, sink, window, small, mo, kept, lo)
    es = fp2.alloc_scratch(fp2.fp2_evict_workspace(ev), "cuda")
    fp2.fp2_evict(ev, es)
    assert _status(es) == (0, 0)
    m = mass.cpu().numpy()
    keep = np.stack([R.evict(m[0, h], L + extra, budget, sink, window) for h in range(hkv)])
    assert np.array_equal(kept.cpu().numpy()[0], keep) and int(lo) == budget
    x = torch.randn((1, hq + 2 * hkv, d), generator=_gen(3)).to(torch.bfloat16).cuda()
    q3 = torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([int(to[0, budget // page]) * page + budget % page], device="cuda")
    fp2.fp2_rotate(fp2.make_rotate(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:],
                                   torch.tensor([L + extra], dtype=torch.int32, device="cuda"), rope, q3, ko, vo, slots=slot))
    fin = fp2.make_decode(q3, small, [0, 1], lo + 1, budget + 1, hkv)
    fs = fp2.alloc_scratch(fp2.fp2_decode_workspace(fin), "cuda")
    o3, l3 = torch.empty_like(q3), torch.empty((hq, 1), device="cuda")
    fp2.fp2_tree_attend(fin, o3, l3, fs)
    assert _status(fs) == (0, 0)
    tk, tv = R.cache_rows(ko, to.numpy(), 0, budget + 1), R.cache_rows(vo, to.numpy(), 0, budget + 1)
    for h in range(hkv):
        assert np.array_equal(tk[:budget, h], k64[keep[h], h]) and np.array_equal(tv[:budget, h], v64[keep[h], h])
    want, wl, mag, top = R.attend(R.f64(q3), tk, tv, d ** -0.5, np.ones((1, budget + 1), bool))
    bo, bl = R.attend_bounds(want, wl, mag, top, d, budget + 1, R.HALF["bf16"] ** 2)
    _within(o3, want, bo, "decode")
    _within(l3, wl, bl, "decode lse")


def test_serving_cases_pass_under_the_checked_build():
    """The same sources with device-side checks of the rows and positions written: no check may fire."""
    import os
    import subprocess
    import sys
    from block_sparse_long_pooled_b200 import build, fp2
    if fp2.fp2_build_flags() == fp2.FP2_BUILD_CHECKED:
        pytest.skip("this is that run")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        "tests/test_gpu_serve.py", "-k", "tree or rotate or mass or evict"], cwd=root,
                       env=dict(os.environ, FP2_LIBRARY=build.build(checked=True)), capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]

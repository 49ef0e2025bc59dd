"""Steps of a serving loop back to back, with nothing between them.  The kernels start while the ones before them still
run and wait before they touch memory; every step here works on what the step before wrote into the same buffers, and
has to come out as it does when each call is waited for."""

import pytest
import torch

from tests import serve_ref as R
from tests.test_gpu_serve import _gen, _status, _store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_long_pooled_b200 import build
    build.build()


class Loop:
    """Rotation and append, attention, weights and eviction, STEPS times, in buffers that every step uses again.  The new
    tokens overwrite the last rows of each sequence; the weights decay into themselves; the kept lengths go round two
    words.  What each step wrote is kept apart for comparison by the outputs only."""

    STEPS = 24

    def __init__(self, dtype, d, hq, hkv, lens, tokens, page=16):
        from block_sparse_long_pooled_b200 import fp2
        g, n, T = _gen(20), len(lens), len(lens) * tokens
        src = "f32" if dtype == "f32" else "bf16"
        most = max(lens)
        need = [-(-x // page) for x in lens]
        order = torch.randperm(sum(need), generator=g).to(torch.int32)
        table, at = torch.full((n, max(need)), -1, dtype=torch.int32), 0
        for r, x in enumerate(need):
            table[r, :x] = order[at:at + x]
            at += x
        ds = dict(q_descale=1 / 16, k_descale=1 / 32, v_descale=1 / 64) if dtype == "e4m3" else {}
        shape = (sum(need), page, hkv, d)
        self.first = [_store(torch.randn(shape, generator=g) * (20 if ds else 1), dtype).cuda() for _ in "kv"]
        self.k, self.v = (x.clone() for x in self.first)
        j = torch.cat([torch.arange(x - tokens, x) for x in lens])
        row = torch.arange(n).repeat_interleave(tokens)
        slots = (table[row, j // page].long() * page + j % page).cuda()
        self.q = torch.zeros((T, hq, d), dtype=self.k.dtype, device="cuda")
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cache = fp2.make_cache(self.k, self.v, table.cuda())
        rope = fp2.make_rope(fp2.rope_frequencies(d)[0])
        dec = fp2.make_decode(self.q, cache, list(range(0, T + 1, tokens)), self.kv_len, most, hkv, **ds)
        self.scratch = [fp2.alloc_scratch(fp2.fp2_decode_workspace(dec), "cuda") for _ in range(2)]
        self.mass0 = torch.rand((n, hkv, most), generator=g).cuda()
        self.mass = self.mass0.clone()
        budget = max(1, min(lens) // 2)
        ko, vo = (torch.zeros((n, budget, hkv, d), dtype=self.k.dtype, device="cuda") for _ in "kv")
        small = fp2.make_cache(ko, vo)
        new = lambda *s, t=torch.float32: torch.zeros((self.STEPS,) + s, dtype=t, device="cuda")  # noqa: E731
        wide = torch.float32 if dtype == "f32" else torch.bfloat16
        self.out, self.lse, self.out2, self.lse2 = new(T, hq, d, t=wide), new(hq, T), new(n, hq, d, t=wide), new(hq, n)
        self.mass_out, self.kept = new(n, hkv, budget), new(n, hkv, budget, t=torch.int32)
        self.len_out = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.x = [(torch.randn((T, hq + 2 * hkv, d), generator=g)).to(R.TORCH[src]).cuda() for _ in range(self.STEPS)]
        pos = [(j + i).to(torch.int32).cuda() for i in range(self.STEPS)]
        q2 = self.q[:n]
        dec2 = fp2.make_decode(q2, small, list(range(n + 1)), self.len_out, budget, hkv, **ds)
        self.scratch += [fp2.alloc_scratch(fp2.fp2_decode_workspace(dec2), "cuda")]
        calls = []
        for i in range(self.STEPS):
            x = self.x[i]
            rot = fp2.make_rotate(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos[i], rope, self.q, self.k, self.v,
                                  slots=slots, **ds)
            ev = fp2.make_evict(cache, self.kv_len, most, self.mass, budget, 1 % budget, 0, small, self.mass_out[i], self.kept[i],
                                self.len_out)
            if i == 0:
                self.scratch += [fp2.alloc_scratch(fp2.fp2_evict_workspace(ev), "cuda")]
            calls += [lambda rot=rot: fp2.fp2_rotate(rot),
                      lambda i=i: fp2.fp2_tree_attend(dec, self.out[i], self.lse[i], self.scratch[0]),
                      lambda i=i: fp2.fp2_key_mass(dec, self.lse[i], self.mass, self.mass, self.scratch[1], decay=0.5),
                      lambda ev=ev: fp2.fp2_evict(ev, self.scratch[3]),
                      lambda i=i: fp2.fp2_tree_attend(dec2, self.out2[i], self.lse2[i], self.scratch[2])]
        self.calls = calls

    def reset(self):
        for x, y in zip((self.k, self.v), self.first):
            x.copy_(y)
        self.mass.copy_(self.mass0)
        for t in (self.out, self.lse, self.out2, self.lse2, self.mass_out, self.kept):
            t.zero_()
        torch.cuda.synchronize()

    def results(self):
        torch.cuda.synchronize()
        assert all(_status(s) == (0, 0) for s in self.scratch)
        return [t.clone() for t in (self.out, self.lse, self.out2, self.lse2, self.mass_out, self.kept, self.mass,
                                    self.k.view(torch.uint8), self.v.view(torch.uint8))]


@pytest.mark.parametrize("dtype,d,hq,hkv,lens,tokens", [
    ("bf16", 128, 32, 8, (300, 90, 64), 1),
    ("bf16", 128, 32, 8, (300, 90, 64), 5),       # the wide kernel
    ("bf16", 64, 16, 2, (2000, 700), 40),
    ("e4m3", 128, 32, 8, (129, 64, 1000), 1),
    ("e4m3", 128, 8, 1, (500, 65, 64), 9),
    ("f32", 64, 8, 2, (300, 64, 77), 2),
])
def test_a_chain_of_steps_sees_what_the_step_before_wrote(dtype, d, hq, hkv, lens, tokens):
    b = Loop(dtype, d, hq, hkv, lens, tokens)
    b.reset()
    for call in b.calls:
        call()
        torch.cuda.synchronize()
    want = b.results()
    assert not torch.equal(want[0][0], want[0][1]) and not torch.equal(want[5][0], want[5][-1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in b.calls:
            call()
    for turn in range(12):
        b.reset()
        if turn % 3:
            graph.replay()
        else:
            for call in b.calls:
                call()
        for i, (x, y) in enumerate(zip(b.results(), want)):
            assert torch.equal(x, y), (turn, i)

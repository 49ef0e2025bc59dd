"""The serving operators around the prefill, as cases to be measured.

rotate  head norms and rotary positions of Q and K, K and V written to their cache slots
tree    attention of drafted tokens (one token: a decode step) over a cache
mass    attention weight that each cached key receives, accumulated
evict   the heaviest keys of a cache, moved to another cache

``run`` computes them in elementary torch operations; with ``own`` it calls the library.
"""

import math
import random

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_ELT = {"f32": 4, "bf16": 2, "e4m3": 1}
_E4M3_DESCALE = {"q": 1 / 16, "k": 1 / 32, "v": 1 / 64}   # stored = value / descale


def listed():
    return [
        # one decode step of eight requests, K/V appended to a paged cache: latency
        dict(name="rotate step", op="rotate", tokens=8, hq=32, hkv=8, d=128, rot=128, inter=False, norm=False,
             scaling="llama3", src="bf16", dst="bf16", page=64),
        # an odd chunk of an fp32 model with a partly rotated head and interleaved pairs
        dict(name="rotate f32 chunk", op="rotate", tokens=1537, hq=8, hkv=2, d=64, rot=32, inter=True, norm=False,
             scaling="none", src="f32", dst="f32", page=0),
        # a 64K prompt of the GQA-8 layer: head norms, long-context frequencies, FP8 out for the FP8 prefill
        dict(name="rotate fp8 prompt", op="rotate", tokens=65536, hq=32, hkv=4, d=128, rot=128, inter=False, norm=True,
             scaling="yarn", src="bf16", dst="e4m3", page=64),
        # three short requests, one new token each: latency
        dict(name="decode small", op="tree", seqs=3, lo=190, hi=1000, mix=1, qlo=1, qhi=1, hq=32, hkv=8, d=128,
             dtype="bf16", page=0),
        # a serving batch of ragged requests, one new token each, paged
        dict(name="decode batch", op="tree", seqs=64, lo=500, hi=16384, mix=2, qlo=1, qhi=1, hq=32, hkv=8, d=128,
             dtype="bf16", page=64),
        # one request at 128K, a drafted tree of seven tokens
        dict(name="tree long", op="tree", seqs=1, lo=131072, hi=131072, mix=3, qlo=7, qhi=7, hq=32, hkv=8, d=128,
             dtype="bf16", page=64),
        # wide drafted trees over an FP8 cache, eight query heads per KV head
        dict(name="tree wide fp8", op="tree", seqs=8, lo=9000, hi=32768, mix=4, qlo=33, qhi=64, hq=32, hkv=4, d=128,
             dtype="e4m3", page=64),
        # the keys' weights after a decode step of a ragged FP8 batch
        dict(name="mass step fp8", op="mass", seqs=32, lo=200, hi=8192, mix=5, qlo=1, qhi=1, hq=32, hkv=8, d=128,
             dtype="e4m3", page=64),
        # the weights that the last 32 prompt tokens give a 64K prompt's keys
        dict(name="mass window", op="mass", seqs=1, lo=65536, hi=65536, mix=6, qlo=32, qhi=32, hq=32, hkv=8, d=128,
             dtype="bf16", page=0),
        # a few short requests cut to small caches
        dict(name="evict small", op="evict", seqs=5, lo=150, hi=2048, mix=7, budget=512, sink=4, window=64, hkv=8,
             d=128, dtype="bf16", page=16),
        # a 128K prompt cut to 8K keys
        dict(name="evict long", op="evict", seqs=1, lo=131072, hi=131072, mix=8, budget=8192, sink=128, window=512,
             hkv=8, d=128, dtype="bf16", page=64),
        # a ragged FP8 batch, most of it over the budget
        dict(name="evict batch fp8", op="evict", seqs=24, lo=900, hi=32768, mix=9, budget=2048, sink=4, window=256,
             hkv=4, d=128, dtype="e4m3", page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rotate", "tree", "mass", "evict"))
    hkv = rng.choice((1, 2, 4, 8))
    g = rng.choice((1, 2, 4, 5, 8))
    page = rng.choice((0, 16, 64, 128))
    mix = rng.randrange(1 << 20)
    if op == "rotate":
        src, dst = rng.choice((("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")))
        d = 64 if src == "f32" else rng.choice((64, 128)) if dst == "bf16" else 128
        rot = rng.choice((d, d // 2, d // 4))
        most = (1 << 30) // ((hkv * g + 2 * hkv) * d * (_ELT[src] + _ELT[dst]))
        return dict(op=op, tokens=_log(rng, 1, min(65536, most)), hq=hkv * g, hkv=hkv, d=d, rot=rot, inter=rng.random() < 0.5,
                    norm=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "llama3", "yarn")), src=src,
                    dst=dst, page=page)
    dtype = rng.choice(("bf16", "e4m3"))
    d = 128 if dtype == "e4m3" else rng.choice((64, 128))
    seqs = _log(rng, 1, 48)
    hi = _log(rng, 20, min(130000, 262144 // seqs))
    lo = _log(rng, 1, hi)
    if op == "evict":
        budget = _log(rng, 16, max(16, hi))
        sink = rng.randrange(0, budget // 2)
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, mix=mix, budget=budget, sink=sink,
                    window=rng.randrange(0, budget - sink + 1), hkv=hkv, d=d, dtype=dtype, page=page)
    most = max(1, min(64, (8 << 20) // (seqs * hi * hkv * g // 4 + 1)))
    qhi = min(_log(rng, 1, most), lo)
    return dict(op=op, seqs=seqs, lo=lo, hi=hi, mix=mix, qlo=rng.randint(1, qhi), qhi=qhi, hq=hkv * g, hkv=hkv, d=d,
                dtype=dtype, page=page)


# ---------------------------------------------------------------- sizes that follow from a case

def _lens(case):
    r = random.Random(case["mix"])
    lens = [_log(r, case["lo"], case["hi"]) for _ in range(case["seqs"])]
    lens[-1] = case["lo"]
    lens[0] = case["hi"]
    if "qlo" not in case:
        return lens, None
    return lens, [r.randint(case["qlo"], case["qhi"]) for _ in range(case["seqs"])]


def _inv_freq(case):
    """Inverse frequencies [rot / 2] in 64 bits and the factor on cos and sin."""
    r, base = case["rot"], 500000.0 if case["scaling"] == "llama3" else 1000000.0
    f = base ** (-np.arange(0, r, 2, dtype=np.float64) / r)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "llama3":       # factor 8, low 1, high 4, trained at 8192
        turns = 8192 * f / (2 * np.pi)
        t = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f * ((1 - t) / 8.0 + t), 1.0
    if case["scaling"] == "yarn":         # factor 4, beta 32 / 1, trained at 32768
        dim = lambda beta: r * math.log(32768 / (beta * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), r - 1)
        t = np.clip((np.arange(r // 2) - low) / max(high - low, 0.001), 0.0, 1.0)
        return f * (1 - t + t / 4.0), 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def work(case):
    if case["op"] == "rotate":
        n = case["tokens"] * (case["hq"] + 2 * case["hkv"]) * case["d"]
        rotated = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": n * (_ELT[case["src"]] + _ELT[case["dst"]]) + case["tokens"] * 12,
                "flops": rotated * (3 * case["rot"] + (4 * case["d"] if case["norm"] else 0))}
    lens, qlens = _lens(case)
    e, hkv, d = _ELT[case["dtype"]], case["hkv"], case["d"]
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": hkv * (sum(lens) * 4 + kept * (4 * d * e + 8)), "flops": 0}
    hq, rows, pairs = case["hq"], sum(qlens), sum(a * b for a, b in zip(lens, qlens))
    if case["op"] == "tree":
        return {"bytes": sum(lens) * hkv * d * e * 2 + rows * hq * (d * (e + 2) + 4) + rows * 8,
                "flops": 4 * d * hq * pairs}
    return {"bytes": sum(lens) * hkv * (d * e + 8) + rows * hq * (d * e + 4), "flops": 2 * d * hq * pairs}


# ---------------------------------------------------------------- inputs

class _State:
    pass


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _stored(x, dtype, which):
    if dtype == "e4m3":
        return (x.float() / _E4M3_DESCALE[which]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return x.to(_DT[dtype])


def _pages(lens, page, gen):
    """A page table [seqs, most pages] of scattered pages (-1: no page), and the number of pages."""
    need = [-(-n // page) for n in lens]
    total = sum(need)
    order = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
    need_t = torch.tensor(need, device="cuda")
    slot = torch.arange(max(need), device="cuda")[None]
    first = (torch.cumsum(need_t, 0) - need_t)[:, None]
    table = torch.where(slot < need_t[:, None], order[(first + slot).clamp(max=total - 1)], -1)
    return table.to(torch.int32).contiguous(), total


def _cache_shape(lens, case, gen):
    """(page table or None, shape of K and of V)."""
    if case["page"] == 0:
        return None, (len(lens), max(lens), case["hkv"], case["d"])
    table, total = _pages(lens, case["page"], gen)
    return table, (total, case["page"], case["hkv"], case["d"])


def _row_of(table, page, n, L):
    """Row of the flattened cache that holds token j of sequence r: [n, L]."""
    j = torch.arange(L, device="cuda")
    if table is None:
        return torch.arange(n, device="cuda")[:, None] * L + j[None]
    return table.long().clamp(min=0)[:, j // page] * page + j % page


def _prepare_rotate(case, seed):
    s, g = _State(), _gen(seed)
    T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    # one projection's output [T, Hq + 2 Hkv, d], of which Q, K and V are views
    qkv = torch.randn((T, hq + 2 * hkv, d), device="cuda", generator=g) * 1.5
    qkv = qkv.to(_DT[case["src"]])
    s.q, s.k, s.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s.norms = [None, None]
    if case["norm"]:
        s.norms = [(1.0 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(_DT[case["src"]]) for _ in range(2)]
    s.eps = 1e-6
    if T <= 64:   # new tokens of requests of any length, else one prompt's chunk
        s.pos = torch.randint(0, 131072, (T,), device="cuda", generator=g).to(torch.int32)
    else:
        s.pos = torch.arange(T, device="cuda", dtype=torch.int32) + int(seed) % 4096
    s.inv_freq, s.factor = _inv_freq(case)
    if case["page"]:
        rows = -(-T // case["page"]) * case["page"]
        cache = (rows // case["page"], case["page"], hkv, d)
        s.slots = torch.randperm(rows, device="cuda", generator=g)[:T].contiguous()
        if T > 64:
            order = torch.randperm(rows // case["page"], device="cuda", generator=g)
            j = torch.arange(T, device="cuda")
            s.slots = order[j // case["page"]] * case["page"] + j % case["page"]
        if T > 1:
            s.slots[T // 2] = -1    # a padding token
    else:
        cache, s.slots = (T, hkv, d), None
    dst = _DT[case["dst"]]
    s.q_out = torch.zeros((T, hq, d), device="cuda").to(dst)
    s.k_out, s.v_out = torch.zeros(cache, device="cuda").to(dst), torch.zeros(cache, device="cuda").to(dst)
    if own:
        from block_sparse_long_pooled_b200 import fp2
        rope = fp2.make_rope(s.inv_freq, interleaved=case["inter"], scale=s.factor)
        s.handle = fp2.make_rotate(s.q, s.k, s.v, s.pos, rope, s.q_out, s.k_out, s.v_out, slots=s.slots,
                                   q_norm=s.norms[0], k_norm=s.norms[1], norm_eps=s.eps)
    else:
        s.freq = torch.from_numpy(s.inv_freq).cuda()
    return s


def _prepare_decode(case, seed):
    s, g = _State(), _gen(seed)
    lens, qlens = _lens(case)
    n, hq, hkv, d = len(lens), case["hq"], case["hkv"], case["d"]
    s.table, shape = _cache_shape(lens, case, g)
    # a direction per KV head that queries lean to and one key in 64 carries
    u = torch.randn((hkv, d), device="cuda", generator=g)
    u = u / u.norm(dim=-1, keepdim=True) * math.sqrt(d)
    k = torch.randn(shape, device="cuda", generator=g)
    k += (torch.rand(shape[:3], device="cuda", generator=g) < 1 / 64)[..., None] * 0.6 * u
    s.k = _stored(k, case["dtype"], "k")
    del k
    s.v = _stored(torch.randn(shape, device="cuda", generator=g), case["dtype"], "v")
    T = sum(qlens)
    q = torch.randn((T, hkv, hq // hkv, d), device="cuda", generator=g) + 0.5 * u[None, :, None]
    s.q = _stored(q.view(T, hq, d), case["dtype"], "q")
    s.kv_len = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s.cu = [0]
    for x in qlens:
        s.cu.append(s.cu[-1] + x)
    s.max_len, s.scale = max(lens), 1.0 / math.sqrt(d)
    s.descale = [_E4M3_DESCALE[w] if case["dtype"] == "e4m3" else 1.0 for w in "qkv"]
    # drafted trees: token i hangs under an earlier one, and sees it and what it sees; one token sees itself
    s.mask = None
    if case["qhi"] > 1 and case["op"] == "tree":
        r = random.Random(seed)
        bits = []
        for x in qlens:
            m = []
            for i in range(x):
                m.append((m[r.randrange(max(0, i - 4), i)] if i else 0) | (1 << i))
            bits += [b - (1 << 64) if b >> 63 else b for b in m]
        s.mask = torch.tensor(bits, device="cuda", dtype=torch.int64)
    # rows of the padded batch that the plain form works on
    s.qlen = torch.tensor(qlens, device="cuda")
    s.q_row = (torch.tensor(s.cu[:-1], device="cuda")[:, None]
               + torch.arange(max(qlens), device="cuda")[None]).clamp(max=T - 1)
    s.q_used = torch.arange(max(qlens), device="cuda")[None] < s.qlen[:, None]
    s.out = torch.empty((T, hq, d), device="cuda", dtype=torch.bfloat16)
    s.lse = torch.empty((hq, T), device="cuda")
    if case["op"] == "mass":
        s.mass = torch.empty((n, hkv, s.max_len), device="cuda").exponential_(generator=g)
        s.mass_out = torch.zeros_like(s.mass)
        s.decay = 0.9375
        sc, vis, _ = _scores(s, case)
        s.lse = torch.empty((hq, T), device="cuda")
        s.lse[:, s.q_row[s.q_used]] = torch.logsumexp(sc.masked_fill(~vis, -math.inf), -1).permute(1, 0, 2)[:, s.q_used]
        del sc, vis
    if own:
        from block_sparse_long_pooled_b200 import fp2
        cache = fp2.make_cache(s.k, s.v, s.table)
        s.handle = fp2.make_decode(s.q, cache, s.cu, s.kv_len, s.max_len, hkv, tree_mask=s.mask,
                                   q_descale=s.descale[0], k_descale=s.descale[1], v_descale=s.descale[2])
        s.scratch = fp2.alloc_scratch(fp2.fp2_decode_workspace(s.handle), "cuda")
    return s


def _prepare_evict(case, seed):
    s, g = _State(), _gen(seed)
    lens, _ = _lens(case)
    n, hkv = len(lens), case["hkv"]
    s.table, shape = _cache_shape(lens, case, g)
    s.k = _stored(torch.randn(shape, device="cuda", generator=g), case["dtype"], "k")
    s.v = _stored(torch.randn(shape, device="cuda", generator=g), case["dtype"], "v")
    s.kv_len = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s.max_len, s.budget = max(lens), case["budget"]
    # heavy-tailed weights, an eighth of them with no weight at all: ties
    mass = torch.randn((n, hkv, s.max_len), device="cuda", generator=g).mul_(2.5).exp_()
    s.mass = mass * (torch.rand(mass.shape, device="cuda", generator=g) > 0.125)
    s.table_out, shape = _cache_shape([case["budget"]] * n, case, g)
    s.k_out = torch.zeros(shape, device="cuda").to(_DT[case["dtype"]])
    s.v_out = torch.zeros(shape, device="cuda").to(_DT[case["dtype"]])
    s.mass_out = torch.zeros((n, hkv, case["budget"]), device="cuda")
    s.kept = torch.zeros((n, hkv, case["budget"]), device="cuda", dtype=torch.int32)
    s.len_out = torch.zeros(n, device="cuda", dtype=torch.int32)
    if own:
        from block_sparse_long_pooled_b200 import fp2
        s.handle = fp2.make_evict(fp2.make_cache(s.k, s.v, s.table), s.kv_len, s.max_len, s.mass, case["budget"],
                                  case["sink"], case["window"], fp2.make_cache(s.k_out, s.v_out, s.table_out),
                                  s.mass_out, s.kept, s.len_out)
        s.scratch = fp2.alloc_scratch(fp2.fp2_evict_workspace(s.handle), "cuda")
    return s


def prepare(case, seed):
    s = {"rotate": _prepare_rotate, "tree": _prepare_decode, "mass": _prepare_decode,
         "evict": _prepare_evict}[case["op"]](case, seed)
    s.case = case
    return s


# ---------------------------------------------------------------- the plain forms

def _turn(x, cos, sin, rot, inter):
    """Rotate the first `rot` values of each head of x [T, H, d]."""
    a, rest = x[..., :rot], x[..., rot:]
    if inter:
        x1, x2 = a[..., 0::2], a[..., 1::2]
    else:
        x1, x2 = a[..., :rot // 2], a[..., rot // 2:]
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if inter else torch.cat((y1, y2), -1)
    return torch.cat((y, rest), -1)


def _run_rotate(s):
    c = s.case
    angle = s.pos.double()[:, None, None] * s.freq
    cos, sin = (torch.cos(angle) * s.factor).float(), (torch.sin(angle) * s.factor).float()
    dst = s.q_out.dtype

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s.eps) * w.float()
        return _turn(x, cos, sin, c["rot"], c["inter"])

    def narrow(x):
        return (x.clamp(-448.0, 448.0) if dst == torch.float8_e4m3fn else x).to(dst)

    s.q_out.copy_(narrow(one(s.q, s.norms[0])))
    k, v = narrow(one(s.k, s.norms[1])), narrow(s.v.float())
    if s.slots is None:
        s.k_out.copy_(k)
        s.v_out.copy_(v)
        return s.q_out, s.k_out, s.v_out
    # the row past the end takes the padding tokens
    rows = s.k_out.shape[0] * s.k_out.shape[1]
    at = torch.where(s.slots < 0, rows, s.slots)
    for out, x in ((s.k_out, k), (s.v_out, v)):
        byte = out.view(rows, -1).view(torch.uint8)
        wide = torch.cat((byte, byte[:1]))
        wide[at] = x.reshape(x.shape[0], -1).view(torch.uint8)
        byte.copy_(wide[:rows])
    return s.q_out, s.k_out, s.v_out


def _gathered(s, x, descale):
    """[n, Hkv, L, d] in 32 bits; rows that hold no key of the sequence are zero."""
    L = s.max_len
    rows = _row_of(s.table, s.case["page"], s.kv_len.shape[0], L)
    flat = x.view(-1, *x.shape[2:])
    y = flat.view(torch.uint8)[rows].view(x.dtype).float() * descale
    used = torch.arange(L, device="cuda")[None] < s.kv_len[:, None]
    return torch.where(used[:, :, None, None], y, 0.0).permute(0, 2, 1, 3)


def _scores(s, case):
    """Scaled scores [n, Hq, rows, L] of the padded batch, which of them are visible, and the sizes."""
    n, L, hq, hkv, d = s.kv_len.shape[0], s.max_len, case["hq"], case["hkv"], case["d"]
    s.case = case
    Q = s.q_row.shape[1]
    q = s.q.view(torch.uint8)[s.q_row].view(s.q.dtype).float() * s.descale[0]          # [n, Q, Hq, d]
    q = q.view(n, Q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    k = _gathered(s, s.k, s.descale[1])
    sc = (torch.matmul(q, k.transpose(-1, -2)) * s.scale).view(n, hq, Q, L)
    j = torch.arange(L, device="cuda")[None, None]
    i = torch.arange(Q, device="cuda")[None, :, None]
    b = j - (s.kv_len.long() - s.qlen)[:, None, None]      # index of a drafted key, below 0 for the others
    if s.mask is None:
        vis = b <= i
    else:
        vis = (b < 0) | ((s.mask[s.q_row][:, :, None] >> b.clamp(0, 63)) & 1).bool()
    vis = vis & (j < s.kv_len[:, None, None]) & s.q_used[:, :, None]
    return sc, vis[:, None], (n, L, hq, hkv, d, Q)


def _run_tree(s):
    sc, vis, (n, L, hq, hkv, d, Q) = _scores(s, s.case)
    sc = sc.masked_fill(~vis, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isinf(m), 0.0, m))
    total = p.sum(-1, keepdim=True)
    v = _gathered(s, s.v, s.descale[2])
    o = torch.matmul(p.view(n, hkv, -1, L), v).view(n, hq, Q, d) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total))[..., 0]
    s.out[s.q_row[s.q_used]] = o.permute(0, 2, 1, 3)[s.q_used].to(s.out.dtype)
    s.lse[:, s.q_row[s.q_used]] = lse.permute(1, 0, 2)[:, s.q_used]
    return s.out, s.lse


def _run_mass(s):
    sc, vis, (n, L, hq, hkv, d, Q) = _scores(s, s.case)
    lse = s.lse[:, s.q_row].permute(1, 0, 2)[..., None]                                # [n, Hq, Q, 1]
    p = torch.where(vis, torch.exp(sc - lse), 0.0)
    new = s.mass * s.decay + p.view(n, hkv, -1, L).sum(2)
    used = torch.arange(L, device="cuda")[None, None] < s.kv_len[:, None, None]
    s.mass_out.copy_(torch.where(used, new, s.mass_out))
    return s.mass_out


def _run_evict(s):
    c = s.case
    n, hkv, L, B = s.kv_len.shape[0], c["hkv"], s.max_len, s.budget
    j = torch.arange(L, device="cuda")[None, None]
    length = s.kv_len[:, None, None]
    forced = (j < c["sink"]) | (j >= length - c["window"])
    key = torch.where(forced, math.inf, s.mass).masked_fill(j >= length, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :B]
    short = torch.arange(order.shape[-1], device="cuda")[None, None]
    order = torch.where(short < length, order, L)                # L: no key
    order = torch.sort(order, dim=-1).values
    if order.shape[-1] < B:
        order = torch.cat((order, order.new_full((n, hkv, B - order.shape[-1]), L)), -1)
    there = order < L
    s.kept.copy_(torch.where(there, order, -1))
    s.mass_out.copy_(torch.where(there, torch.gather(s.mass, 2, order.clamp(max=L - 1)), 0.0))
    s.len_out.copy_(s.kv_len.clamp(max=B))
    src = _row_of(s.table, c["page"], n, L)
    dst = _row_of(s.table_out, c["page"], n, B)
    r, h, i = torch.nonzero(there, as_tuple=True)
    from_row, to_row = src[r, order[r, h, i]], dst[r, i]
    for x, y in ((s.k, s.k_out), (s.v, s.v_out)):
        flat = lambda t: t.view(-1, *t.shape[2:]).view(torch.uint8)  # noqa: E731
        flat(y)[to_row, h] = flat(x)[from_row, h]
    return s.k_out, s.v_out, s.mass_out, s.kept, s.len_out


def run(s):
    op = s.case["op"]
    if not own:
        return {"rotate": _run_rotate, "tree": _run_tree, "mass": _run_mass, "evict": _run_evict}[op](s)
    from block_sparse_long_pooled_b200 import fp2
    if op == "rotate":
        fp2.fp2_rotate(s.handle)
        return s.q_out, s.k_out, s.v_out
    if op == "tree":
        fp2.fp2_tree_attend(s.handle, s.out, s.lse, s.scratch)
        return s.out, s.lse
    if op == "mass":
        fp2.fp2_key_mass(s.handle, s.lse, s.mass, s.mass_out, s.scratch, decay=s.decay)
        return s.mass_out
    fp2.fp2_evict(s.handle, s.scratch)
    return s.k_out, s.v_out, s.mass_out, s.kept, s.len_out


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _exact_rotate(s):
    c = s.case
    T, r = c["tokens"], c["rot"]
    out = []
    turn = torch.polar(torch.full((T, r // 2), s.factor, dtype=torch.float64, device="cuda"),
                       torch.outer(s.pos.double(), torch.from_numpy(s.inv_freq).cuda()))[:, None]
    for x, w in ((s.q, s.norms[0]), (s.k, s.norms[1])):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + s.eps) * w.double()
        head = x[..., :r].reshape(T, -1, r // 2, 2) if c["inter"] else x[..., :r].reshape(T, -1, 2, r // 2).mT
        z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
        x[..., :r] = (z if c["inter"] else z.mT).reshape(T, -1, r)
        out.append(x)
    out.append(s.v.double())
    if c["dst"] == "e4m3":
        out = [x.clamp(-448, 448) for x in out]
    if s.slots is None:
        return out
    for i in (1, 2):
        cache = torch.zeros(s.k_out.shape, dtype=torch.float64, device="cuda")
        use = s.slots >= 0
        cache.view(-1, c["hkv"], c["d"])[s.slots[use]] = out[i][use]
        out[i] = cache
    return out


def _exact_rows(s, case, r, g):
    """(scores, visible, values) of sequence r and KV head g, rows token-major then head."""
    lens, qlens = _lens(case)
    L, Q, G = lens[r], qlens[r], case["hq"] // case["hkv"]
    j = torch.arange(L, device="cuda")
    rows = (r * s.max_len + j) if s.table is None else s.table[r].long()[j // case["page"]] * case["page"] + j % case["page"]
    at = lambda x: x.view(-1, case["hkv"], case["d"])[:, g].view(torch.uint8)[rows].view(x.dtype).double()  # noqa: E731
    k, v = at(s.k) * s.descale[1], at(s.v) * s.descale[2]
    t0 = s.cu[r]
    q = s.q[t0:t0 + Q, g * G:(g + 1) * G].double().reshape(Q * G, -1) * s.descale[0]
    seen = torch.ones((Q, L), dtype=torch.bool, device="cuda")
    for i in range(Q):
        bits = (1 << (i + 1)) - 1 if s.mask is None else int(s.mask[t0 + i])
        seen[i, L - Q:] = torch.tensor([bool(bits >> b & 1) for b in range(Q)], device="cuda")
    return q @ k.T / math.sqrt(case["d"]), seen.repeat_interleave(G, 0), v


def _exact_decode(s, case):
    lens, qlens = _lens(case)
    G, mass = case["hq"] // case["hkv"], case["op"] == "mass"
    out = torch.zeros(s.out.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s.lse.shape, dtype=torch.float64, device="cuda")
    new = s.mass_out.double() if mass else None
    for r in range(len(lens)):
        t0, Q, L = s.cu[r], qlens[r], lens[r]
        for g in range(case["hkv"]):
            sc, seen, v = _exact_rows(s, case, r, g)
            if mass:
                given = s.lse[g * G:(g + 1) * G, t0:t0 + Q].T.reshape(-1, 1).double()
                new[r, g, :L] = s.mass[r, g, :L].double() * s.decay + (torch.exp(sc - given) * seen).sum(0)
                continue
            sc[~seen] = -math.inf
            z = torch.logsumexp(sc, -1)
            out[t0:t0 + Q, g * G:(g + 1) * G] = (torch.exp(sc - z[:, None]) @ v).view(Q, G, -1)
            lse[g * G:(g + 1) * G, t0:t0 + Q] = z.view(Q, G).T
    return new if mass else (out, lse)


def _exact_evict(s):
    c = s.case
    lens, _ = _lens(c)
    B = c["budget"]
    k, v = (torch.zeros(s.k_out.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    w = np.zeros(tuple(s.mass_out.shape))
    kept = np.full(w.shape, -1, dtype=np.int32)
    mass = s.mass.double().cpu().numpy()
    for r, L in enumerate(lens):
        N = min(L, B)
        for g in range(c["hkv"]):
            rank = mass[r, g, :L].copy()
            rank[:c["sink"]] = np.inf
            rank[max(0, L - c["window"]):] = np.inf
            idx = np.sort(np.lexsort((np.arange(L), -rank))[:N])
            kept[r, g, :N], w[r, g, :N] = idx, mass[r, g, idx]
            i, j = torch.from_numpy(idx).cuda(), torch.arange(N, device="cuda")
            for x, y in ((s.k, k), (s.v, v)):
                if s.table is None:
                    y[r, j, g] = x[r, :, g].double()[i]
                else:
                    P = c["page"]
                    rows = x.view(-1, c["hkv"], c["d"])[:, g].view(torch.uint8)[s.table[r].long()[i // P] * P + i % P]
                    y.view(-1, c["hkv"], c["d"])[s.table_out[r].long()[j // P] * P + j % P, g] = rows.view(x.dtype).double()
    return k, v, w, kept, np.minimum(lens, B).astype(np.int32)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s)
    return _exact_evict(s) if case["op"] == "evict" else _exact_decode(s, case)

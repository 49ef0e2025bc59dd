"""The serving operators without a GPU: struct layouts, frequencies, and what the calls refuse (every check runs
on the host before anything is launched)."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from block_sparse_long_pooled_b200 import build as B
from block_sparse_long_pooled_b200 import fp2
from tests import serve_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, SMALL = fp2.FP2_ERR_INVALID_ARG, fp2.FP2_ERR_UNSUPPORTED, fp2.FP2_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def test_struct_layouts_match_the_header(tmp_path):
    names = ("fp2_cache", "fp2_rotation", "fp2_decode", "fp2_eviction")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fp2.h"', "int main(void) {"]
    for n in names:
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
        lines += [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in getattr(fp2, n)._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        name, value = line.split()
        s, _, f = name.partition(".")
        c = getattr(fp2, s)
        assert (getattr(c, f).offset if f else ctypes.sizeof(c)) == int(value), name


def test_rope_frequencies():
    f, s = fp2.rope_frequencies(128, 10000.0)
    assert s == 1.0 and f[0] == 1.0 and np.isclose(f[-1], 10000.0 ** (-126 / 128), rtol=1e-14)
    g, _ = fp2.rope_frequencies(128, 10000.0, "linear", 4.0)
    assert np.allclose(g * 4, f, rtol=1e-14)
    g, _ = fp2.rope_frequencies(128, 10000.0, "ntk", 4.0)
    assert g[0] == 1.0 and np.isclose(g[-1], f[-1] / 4, rtol=1e-12)
    f, _ = fp2.rope_frequencies(128, 500000.0)
    g, s = fp2.rope_frequencies(128, 500000.0, "llama3", 8.0, 8192, 1.0, 4.0)
    turns = 8192 * f / (2 * np.pi)
    assert s == 1.0 and np.array_equal(g[turns >= 4], f[turns >= 4])
    assert np.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((g < f) & (g > f / 8))[mid].all()
    f, _ = fp2.rope_frequencies(128, 1e6)
    g, s = fp2.rope_frequencies(128, 1e6, "yarn", 4.0, 32768)
    assert np.isclose(s, 0.1 * np.log(4) + 1) and np.isclose(g[0], f[0]) and np.isclose(g[-1], f[-1] / 4)
    assert (np.diff(g / f) <= 1e-15).all()
    for bad in (dict(rotary_dim=7), dict(rotary_dim=64, scaling="cubic"), dict(rotary_dim=64, factor=0.0)):
        with pytest.raises(ValueError):
            fp2.rope_frequencies(**bad)


def _rotation(T=4, hq=4, hkv=2, d=64, src="bf16", dst="bf16", **over):
    q, k, v = (torch.zeros((T, h, d), dtype=R.TORCH[src]) for h in (hq, hkv, hkv))
    qo, ko, vo = (torch.zeros((T, h, d), dtype=R.TORCH[dst]) for h in (hq, hkv, hkv))
    h = fp2.make_rotate(q, k, v, torch.zeros(T, dtype=torch.int32), fp2.make_rope(fp2.rope_frequencies(d)[0]), qo, ko, vo)
    for name, value in over.items():
        setattr(h.struct, name, value)
    return h


@pytest.mark.parametrize("over,code", [
    (dict(head_dim=96), UNS), (dict(rotary_dim=24), UNS), (dict(rotary_dim=80), UNS), (dict(rotary_dim=-16), UNS),
    (dict(in_dtype=fp2.FP2_E4M3), UNS), (dict(out_dtype=fp2.FP2_F32), UNS), (dict(tokens=-1), INV),
    (dict(num_q_heads=-1), INV), (dict(num_q_heads=0, num_kv_heads=0), INV), (dict(q=None), INV), (dict(q_out=None), INV),
    (dict(k_out=None), INV), (dict(v_out=None), INV), (dict(positions=None), INV), (dict(inv_freq_host=None), INV),
    (dict(q_stride_tok=8), INV), (dict(kv_out_stride_tok=129), INV), (dict(num_slots=3), INV),
    (dict(rope_scale=float("nan")), INV), (dict(q_descale=0.0), INV), (dict(k_descale=2.0), INV),
])
def test_rotate_refusals(over, code):
    h = _rotation(**over)
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_rotate(h, stream=0)
    assert e.value.status == code and fp2.fp2_last_error()


def test_rotate_refuses_odd_pointers_and_infinite_frequencies():
    h = _rotation()
    h.struct.k += 2
    with pytest.raises(fp2.FP2Error):
        fp2.fp2_rotate(h, stream=0)
    f = fp2.rope_frequencies(64)[0]
    f[3] = np.inf
    z = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(fp2.FP2Error):
        fp2.fp2_rotate(fp2.make_rotate(z, None, None, torch.zeros(1, dtype=torch.int32), fp2.make_rope(f), z, None, None),
                       stream=0)
    assert fp2.fp2_rotate(_rotation(T=0), stream=0) is None      # nothing to do is no error


def test_make_rotate_checks_shapes():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    pos, rope = z(4, t=torch.int32), fp2.make_rope(fp2.rope_frequencies(64)[0])
    good = dict(q=z(4, 4, 64), k=z(4, 2, 64), v=z(4, 2, 64), positions=pos, rope=rope, q_out=z(4, 4, 64),
                k_out=z(4, 2, 64), v_out=z(4, 2, 64))
    fp2.make_rotate(**good)
    for bad in (dict(q=z(3, 4, 64)), dict(k=z(4, 2, 64, t=torch.float32)), dict(v=z(4, 1, 64)), dict(q_out=z(4, 4, 32)),
                dict(k_out=z(4, 3, 64)), dict(v_out=None), dict(positions=pos.long()), dict(slots=pos),
                dict(q_norm=z(32)), dict(k_norm=z(64, t=torch.float32)), dict(q=z(4, 4, 128)[..., ::2]),
                dict(k=None), dict(k_out=z(2, 8, 2, 64)[:, :4], v_out=z(2, 8, 2, 64)[:, :4])):
        with pytest.raises(ValueError):
            fp2.make_rotate(**{**good, **bad})


def _decode(n=2, qlen=3, hq=4, hkv=2, d=128, dtype="bf16", page=16, most=100, paged=True, **over):
    T = n * qlen
    shape = (20, page, hkv, d) if paged else (n, most, hkv, d)
    k = torch.zeros(shape, dtype=R.TORCH[dtype])
    table = torch.zeros((n, -(-most // page)), dtype=torch.int32) if paged else None
    h = fp2.make_decode(torch.zeros((T, hq, d), dtype=R.TORCH[dtype]), fp2.make_cache(k, k.clone(), table),
                        np.arange(n + 1) * qlen, torch.zeros(n, dtype=torch.int32), most)
    for name, value in over.items():
        where = h.struct.cache if name in [f for f, _ in fp2.fp2_cache._fields_] else h.struct
        setattr(where, name, value)
    return h


@pytest.mark.parametrize("kw,code", [
    (dict(qlen=65), UNS), (dict(most=2), INV), (dict(max_kv_len=524289), UNS), (dict(max_kv_len=-1), INV),
    (dict(max_kv_len=113), INV),                              # more pages than the table has
    (dict(paged=False, max_kv_len=101), INV), (dict(paged=False, num_outer=1), INV),
    (dict(page=24), UNS), (dict(page=8), UNS), (dict(rows=0), INV), (dict(num_outer=0), INV),
    (dict(num_q_heads=3), INV), (dict(num_q_heads=66), UNS), (dict(head_dim=96), UNS), (dict(dtype="f32", d=128), UNS),
    (dict(dtype="e4m3", d=64), UNS), (dict(softmax_scale=-1.0), INV), (dict(k_descale=0.0), INV), (dict(q=None), INV),
    (dict(softmax_scale=1e-39), INV), (dict(softmax_scale=1e38, q_descale=100.0), INV), (dict(v_descale=3e37), INV),
    (dict(num_kv_heads=65537, num_q_heads=65537), UNS),
    (dict(kv_len=None), INV), (dict(k=None), INV), (dict(stride_tok=252), INV), (dict(stride_outer=4095), INV),
    (dict(q_stride_tok=500), INV), (dict(num_seqs=0), UNS), (dict(num_seqs=513), UNS), (dict(cu_seqlens_q_host=None), INV),
])
def test_decode_refusals(kw, code):
    h = _decode(**kw)
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_decode_workspace(h)
    assert e.value.status == code and fp2.fp2_last_error()


def test_sizes_that_a_c_int_cannot_hold():
    with pytest.raises(ValueError):
        fp2.make_decode(torch.zeros((1, 4, 64), dtype=torch.bfloat16),
                        fp2.make_cache(torch.zeros((1, 50, 2, 64), dtype=torch.bfloat16)), [0, 1],
                        torch.zeros(1, dtype=torch.int32), 2 ** 32 + 50)


def test_decode_calls_check_scratch_and_outputs():
    h = _decode()
    need = fp2.fp2_decode_workspace(h)
    raw = torch.zeros(need + 512, dtype=torch.uint8)
    off = -raw.data_ptr() % 256
    out, lse = torch.zeros((6, 4, 128), dtype=torch.bfloat16), torch.zeros((4, 6))
    mass = torch.zeros((2, 2, 100))
    for scratch, code in ((raw[off:off + need - 1], SMALL), (raw[off + 16:off + 16 + need], INV)):
        for call in (lambda: fp2.fp2_tree_attend(h, out, lse, scratch, stream=0),
                     lambda: fp2.fp2_key_mass(h, lse, None, mass, scratch, stream=0)):
            with pytest.raises(fp2.FP2Error) as e:
                call()
            assert e.value.status == code
    ok = raw[off:off + need]
    with pytest.raises(ValueError):
        fp2.fp2_tree_attend(h, out.float(), lse, ok, stream=0)
    with pytest.raises(ValueError):
        fp2.fp2_tree_attend(h, out[:5], lse, ok, stream=0)
    with pytest.raises(ValueError):
        fp2.fp2_tree_attend(h, out, lse.t().contiguous(), ok, stream=0)
    with pytest.raises(fp2.FP2Error):
        fp2.fp2_key_mass(h, lse, None, mass[..., :99].contiguous(), ok, stream=0)
    with pytest.raises(fp2.FP2Error):
        fp2.fp2_key_mass(h, None, None, mass, ok, stream=0)
    with pytest.raises(fp2.FP2Error):
        fp2.fp2_key_mass(h, lse, None, mass, ok, decay=float("inf"), stream=0)
    no_v = fp2.make_decode(torch.zeros((2, 4, 128), dtype=torch.bfloat16),
                           fp2.make_cache(torch.zeros((2, 50, 2, 128), dtype=torch.bfloat16)), [0, 1, 2],
                           torch.zeros(2, dtype=torch.int32), 50)
    with pytest.raises(ValueError):
        fp2.fp2_tree_attend(no_v, out[:2], None, ok, stream=0)


def test_make_decode_and_cache_check_shapes():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    cache = fp2.make_cache(z(2, 50, 2, 128), z(2, 50, 2, 128))
    good = dict(q=z(3, 4, 128), cache=cache, cu_seqlens=[0, 1, 3], kv_len=z(2, t=torch.int32), max_kv_len=50)
    fp2.make_decode(**good)
    for bad in (dict(q=z(3, 4, 64)), dict(q=z(3, 4, 128, t=torch.float32)), dict(cu_seqlens=[0, 1, 2]),
                dict(kv_len=z(3, t=torch.int32)), dict(kv_len=z(2, t=torch.int64)), dict(tree_mask=z(3, t=torch.int32)),
                dict(num_kv_heads=4)):
        with pytest.raises(ValueError):
            fp2.make_decode(**{**good, **bad})
    for k, v, t in ((z(2, 50, 128), None, None), (z(2, 50, 2, 128), z(2, 49, 2, 128), None),
                    (z(2, 50, 2, 128), z(2, 50, 2, 128, t=torch.float32), None),
                    (z(4, 16, 2, 128), z(4, 16, 2, 128), z(2, 2, t=torch.int64)),
                    (z(2, 50, 2, 256)[..., ::2], None, None)):
        with pytest.raises(ValueError):
            fp2.make_cache(k, v, t)
    with pytest.raises(ValueError):        # one row of pages for two sequences
        fp2.make_decode(**{**good, "cache": fp2.make_cache(z(4, 64, 2, 128), z(4, 64, 2, 128), z(1, 2, t=torch.int32))})


def _evict(n=2, hkv=2, d=128, most=100, budget=40, sink=4, window=8, paged_out=False, **over):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    src = fp2.make_cache(z(n, most, hkv, d), z(n, most, hkv, d))
    dst = fp2.make_cache(z(n * 3, 16, hkv, d), z(n * 3, 16, hkv, d), z(n, 3, t=torch.int32)) if paged_out else \
        fp2.make_cache(z(n, budget, hkv, d), z(n, budget, hkv, d))
    h = fp2.make_evict(src, z(n, t=torch.int32), most, z(n, hkv, most, t=torch.float32), budget, sink, window, dst,
                       z(n, hkv, budget, t=torch.float32), z(n, hkv, budget, t=torch.int32), z(n, t=torch.int32))
    for name, value in over.items():
        part, _, field = name.partition("__")
        setattr(getattr(h.struct, part) if field else h.struct, field or name, value)
    return h


@pytest.mark.parametrize("kw,code", [
    (dict(sink=20, window=21), INV), (dict(sink=-1), INV), (dict(window=-1), INV), (dict(mass_stride=99), INV),
    (dict(max_kv_len=101), INV), (dict(max_kv_len=-1), INV), (dict(dst__rows=39), INV), (dict(dst__num_outer=1), INV),
    (dict(paged_out=True, dst__max_pages_per_seq=2), INV), (dict(dst__head_dim=64), INV), (dict(dst__num_kv_heads=1), INV),
    (dict(dst__dtype=fp2.FP2_E4M3), INV), (dict(kept=None), INV), (dict(mass=None), INV), (dict(kv_len_out=None), INV),
    (dict(dst__v=None), INV), (dict(src__stride_tok=255), INV), (dict(num_seqs=0), UNS), (dict(src__head_dim=80), UNS),
])
def test_evict_refusals(kw, code):
    h = _evict(**kw)
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_evict_workspace(h)
    assert e.value.status == code and fp2.fp2_last_error()


def test_evict_refuses_a_budget_above_the_longest_cache():
    h = _evict()
    h.struct.budget = 524289
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_evict_workspace(h)
    assert e.value.status == UNS


def test_evict_refuses_overlap_and_small_scratch():
    h = _evict()
    assert fp2.fp2_evict_workspace(h) > 0
    for out, into in (("kv_len_out", "kv_len"), ("mass_out", "mass"), ("kept", "mass"), ("kept", "mass_out")):
        bad = _evict()
        setattr(bad.struct, out, getattr(bad.struct, into))
        with pytest.raises(fp2.FP2Error) as e:
            fp2.fp2_evict_workspace(bad)
        assert e.value.status == INV and "overlap" in str(e.value)
    h.struct.dst.k = h.struct.src.v
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_evict_workspace(h)
    assert e.value.status == INV and "overlap" in str(e.value)
    h = _evict(paged_out=True)
    raw = torch.zeros(4096, dtype=torch.uint8)
    off = -raw.data_ptr() % 256
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_evict(h, raw[off:off + 256], stream=0)
    assert e.value.status == SMALL


# ------------------------------------------------------------------ the 64-bit forms themselves

def test_reference_attention_is_softmax_attention():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 4, 16), (9, 2, 16), (9, 2, 16)))
    vis = R.visible(3, 9, None)
    out, lse, _, _ = R.attend(q.numpy(), k.numpy(), v.numpy(), 0.25, vis)
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    bias = torch.zeros(3, 9, dtype=torch.float64).masked_fill(~torch.from_numpy(vis), -float("inf"))
    s = torch.einsum("qhd,nhd->hqn", q, kk) * 0.25 + bias
    assert np.allclose(lse, torch.logsumexp(s, -1).numpy())
    assert np.allclose(out, torch.einsum("hqn,nhd->qhd", s.softmax(-1), vv).numpy())
    mass, _ = R.key_mass(q.numpy(), k.numpy(), 0.25, vis, lse)
    assert np.allclose(mass, s.softmax(-1).view(2, 2, 3, 9).sum((1, 2)).numpy())


def test_reference_rotation_is_a_complex_product():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((5, 2, 32), generator=g, dtype=torch.float64).numpy()
    pos, f = np.array([0, 1, 7, 1000, 131071]), fp2.rope_frequencies(16)[0]
    turn = np.exp(1j * pos[:, None, None] * f)
    y, _ = R.rotate(x, pos, f, True, 1.0)
    z = (x[..., 0:16:2] + 1j * x[..., 1:16:2]) * turn
    assert np.allclose(y[..., 0:16:2], z.real) and np.allclose(y[..., 1:16:2], z.imag) and (y[..., 16:] == x[..., 16:]).all()
    y, _ = R.rotate(x, pos, f, False, 1.0)
    z = (x[..., :8] + 1j * x[..., 8:16]) * turn
    assert np.allclose(y[..., :8], z.real) and np.allclose(y[..., 8:16], z.imag)


def test_reference_eviction():
    w = np.array([5.0, 1, 1, 7, 1, 0, 0, 9, 1, 2])
    assert list(R.evict(w, 10, 10, 0, 0)) == list(range(10))
    assert list(R.evict(w, 10, 4, 1, 1)) == [0, 3, 7, 9]
    assert list(R.evict(w, 10, 5, 0, 0)) == [0, 1, 3, 7, 9]
    assert list(R.evict(w, 10, 3, 2, 1)) == [0, 1, 9]


def test_the_late_tile_hook_validates_and_resets():
    for bad in (-2, fp2.FP2_MAX_CACHE_LEN + 1):
        with pytest.raises(fp2.FP2Error) as e:
            fp2.fp2_debug_set(fp2.FP2_DEBUG_LATE_V_TILE, bad)
        assert e.value.status == INV
    fp2.fp2_debug_set(fp2.FP2_DEBUG_LATE_V_TILE, 4)
    fp2.fp2_debug_set(fp2.FP2_DEBUG_LATE_V_TILE, -1)


def test_key_mass_refuses_overlap():
    """mass_in may be mass_out, not a shifted piece of it; other CTAs still read LSE and lengths."""
    h = _decode()
    scratch = fp2.alloc_scratch(fp2.fp2_decode_workspace(h) + 256, "cpu")
    scratch = scratch[-scratch.data_ptr() % 256:]
    raw = torch.zeros(1000)
    mass, lse = torch.zeros((2, 2, 100)), torch.zeros((4, 6))
    cases = [(dict(lse=lse, mass_in=raw[x:x + 400].view(2, 2, 100), mass_out=raw[100:500].view(2, 2, 100)))
             for x in (0, 1, 99, 101, 499)]
    cases.append(dict(lse=raw[:24].view(4, 6), mass_in=None, mass_out=raw[20:420].view(2, 2, 100)))
    cases.append(dict(lse=lse, mass_in=None, mass_out=mass, mass_len=mass.view(torch.int32).view(-1)[399 - 1:400]))
    for kw in cases:
        with pytest.raises(fp2.FP2Error) as e:
            fp2.fp2_key_mass(h, scratch=scratch, stream=0, **kw)
        assert e.value.status == INV and "overlap" in str(e.value)
    h.struct.kv_len = mass.data_ptr()
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_key_mass(h, lse, None, mass, scratch, stream=0)
    assert e.value.status == INV and "overlap" in str(e.value)


def test_tensors_of_the_host_are_refused():
    """Every other check passes: a kernel that got these pointers would fault the GPU."""
    h, e = _decode(), _evict(paged_out=True)
    scratch = fp2.alloc_scratch(max(fp2.fp2_decode_workspace(h), fp2.fp2_evict_workspace(e)) + 256, "cpu")
    scratch = scratch[-scratch.data_ptr() % 256:]
    none = fp2.make_decode(torch.zeros((0, 4, 128), dtype=torch.bfloat16),
                           fp2.make_cache(*(torch.zeros((1, 50, 2, 128), dtype=torch.bfloat16) for _ in "kv")), [0, 0],
                           torch.zeros(1, dtype=torch.int32), 50)
    out, lse, mass = torch.zeros((6, 4, 128), dtype=torch.bfloat16), torch.zeros((4, 6)), torch.zeros((2, 2, 100))
    for call in (lambda s: fp2.fp2_rotate(_rotation(), stream=s), lambda s: fp2.fp2_evict(e, scratch, stream=s),
                 lambda s: fp2.fp2_tree_attend(h, out, lse, scratch, stream=s),
                 lambda s: fp2.fp2_tree_attend(none, out[:0], lse[:, :0].contiguous(), scratch, stream=s),
                 lambda s: fp2.fp2_key_mass(h, lse, None, mass, scratch, stream=s)):
        for stream in (None, 0):
            with pytest.raises(fp2.FP2Error) as err:
                call(stream)
            assert err.value.status == INV and "GPU" in str(err.value)


def test_make_rotate_of_one_tensor_as_q_and_k():
    """K's output is checked although Q is the same tensor, and the rows are the smaller cache's, be it empty."""
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    x, rope, pos = z(4, 2, 64), fp2.make_rope(fp2.rope_frequencies(64)[0]), torch.zeros(4, dtype=torch.int32)
    h = fp2.make_rotate(x, x, x, pos, rope, z(4, 2, 64), z(9, 2, 64), z(7, 2, 64))
    assert h.struct.num_slots == 7 and h.struct.kv_out_stride_tok == 128
    h = fp2.make_rotate(x, x, z(4, 2, 64), pos, rope, z(4, 2, 64), z(5, 2, 64), z(7, 2, 64))
    assert h.struct.num_slots == 5
    for bad in (z(4, 3, 64), z(4, 2, 32), z(4, 4, 64)[:, ::2]):
        with pytest.raises(ValueError):
            fp2.make_rotate(x, x, z(4, 2, 64), pos, rope, z(4, 2, 64), bad, z(7, 2, 64))
    h = fp2.make_rotate(None, x, x, pos, rope, None, z(0, 2, 64), z(7, 2, 64), slots=torch.zeros(4, dtype=torch.int64))
    assert h.struct.num_slots == 0


def test_make_rotate_refuses_rows_that_overlap():
    """An expanded output has room for one row, whatever its shape says."""
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    for out in (z(1, 2, 64).expand(4, 2, 64), z(1, 16, 2, 64)[:, :1].expand(1, 16, 2, 64), z(1, 1, 2, 64).expand(4, 1, 2, 64)):
        with pytest.raises(ValueError):
            fp2.make_rotate(None, z(4, 2, 64), None, None, None, None, out, None)
    assert fp2.make_rotate(None, z(1, 2, 64), None, None, None, None, z(1, 2, 64).expand(1, 2, 64), None).struct.num_slots == 1


def test_rotate_in_place_needs_the_input_s_type_and_stride():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    pos, rope = z(4, t=torch.int32), fp2.make_rope(fp2.rope_frequencies(64)[0])
    q, k, v, slots = z(4, 4, 64), z(4, 2, 64), z(4, 2, 64), z(4, t=torch.int64)
    wide = z(4, 8, 64)
    good = dict(q=q, k=k, v=v, positions=pos, rope=rope, q_out=q, k_out=k, v_out=v)
    with pytest.raises(fp2.FP2Error) as e:       # all is well up to the buffers' being on the host
        fp2.fp2_rotate(fp2.make_rotate(**good))
    assert "GPU" in str(e.value)
    for bad in (dict(slots=slots), dict(slots=slots, v_out=z(4, 2, 64)), dict(q_out=wide.view(-1)[:4 * 256].view(4, 4, 64), q=wide[:, :4]),
                dict(k=wide[:, :2], k_out=wide.view(-1)[:4 * 128].view(4, 2, 64)),
                dict(v=wide[:, :2], v_out=wide.view(-1)[:4 * 128].view(4, 2, 64))):
        with pytest.raises(fp2.FP2Error) as e:
            fp2.fp2_rotate(fp2.make_rotate(**{**good, **bad}))
        assert e.value.status == INV and "in place" in str(e.value)
    one = _rotation(q=None)
    one.struct.q, one.struct.out_dtype = one.struct.q_out, fp2.FP2_E4M3
    with pytest.raises(fp2.FP2Error) as e:
        fp2.fp2_rotate(one)
    assert e.value.status == INV and "in place" in str(e.value)

"""CPU tests of the rotary-position and paged-cache entry points: struct layouts, validation
and refusals (nothing is launched), frequencies, workspace sizes."""
import ctypes
import math
import os
import subprocess
import tempfile

import pytest
import torch

import paged_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def spr():
    import __graft_entry__
    __graft_entry__.build()
    import free_block_sparse_rcp_b200 as m
    return m


def test_struct_layouts_match_the_header(spr):
    def fields(cls):
        return [n for n, _ in cls._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"sparsepr.h\"\nint main(void) {\n"
    for cls, c in ((spr.RopeParams, "sparsepr_rope_params"), (spr.CacheParams, "sparsepr_cache_params")):
        src += f'printf("{c}.size %zu\\n", sizeof({c}));\n'
        for f in fields(cls):
            src += f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));\n'
    src += 'printf("dt %d\\n", SPARSEPR_BF16 + 10 * SPARSEPR_FP16 + 100 * SPARSEPR_FP32);\nreturn 0; }\n'
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "t.c"), os.path.join(td, "t")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        out = dict(line.split() for line in subprocess.check_output([exe], text=True).splitlines())
    for cls, c in ((spr.RopeParams, "sparsepr_rope_params"), (spr.CacheParams, "sparsepr_cache_params")):
        assert int(out[f"{c}.size"]) == ctypes.sizeof(cls)
        for f in fields(cls):
            assert int(out[f"{c}.{f}"]) == getattr(cls, f).offset, f
    assert int(out["dt"]) == spr.BF16 + 10 * spr.FP16 + 100 * spr.FP32


def _rope(spr, **kw):
    base = dict(B=2, H=4, N=33, d=64)
    extra = {}
    for k in list(kw):
        if k in ("x_stride", "y_stride", "rot_raw", "axes_raw", "n_axes"):
            extra[k] = kw.pop(k)
    base.update(kw)
    p = spr.RopeParams.make(base.pop("B"), base.pop("H"), base.pop("N"), base.pop("d"), **base)
    for k in ("x_stride", "y_stride"):
        if k in extra:
            for i, v in enumerate(extra[k]):
                getattr(p, k)[i] = v
    if "n_axes" in extra:
        p.n_axes = extra["n_axes"]
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(N=0), 0), (dict(B=0), 1), (dict(H=0), 1), (dict(N=-1), 1), (dict(H2=-1), 1), (dict(H2=3), 0),
    (dict(d=1, rot_dim=2), 1), (dict(d=513, rot_dim=2), 1), (dict(d=512), 0), (dict(d=2), 0), (dict(d=65, rot_dim=64), 0),
    (dict(rot_dim=0), 1), (dict(rot_dim=31), 1), (dict(rot_dim=66), 1), (dict(rot_dim=22), 0),
    (dict(axis_dim=[24, 20, 20]), 0), (dict(axis_dim=[24, 20, 22]), 1), (dict(axis_dim=[23, 41]), 1),
    (dict(axis_dim=[64, 0]), 1), (dict(n_axes=4), 1), (dict(n_axes=0), 1),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(layout=2), 1), (dict(pos_batched=2), 1), (dict(scaling=4), 1),
    (dict(theta=0.0), 1), (dict(theta=float("inf")), 1), (dict(factor=0.0), 1), (dict(factor=float("nan")), 1),
    (dict(scaling="parts", factor=4.0, orig_len=4096), 0), (dict(scaling="parts", factor=4.0), 1),
    (dict(scaling="parts", factor=4.0, orig_len=4096, beta_fast=1.0, beta_slow=1.0), 1),
    (dict(scaling="parts", factor=4.0, orig_len=4096, theta=1.0), 1),
    (dict(magnitude=-1.0), 1), (dict(magnitude=float("nan")), 1),
    (dict(B=1 << 16, N=1 << 15), 2), (dict(H=65535, H2=1), 2),
    (dict(y_stride=[0, 64, 256]), 1), (dict(x_stride=[0, 64, 256]), 0), (dict(B=1, y_stride=[0, 64, 256]), 0),
])
def test_rope_validation(spr, kw, status):
    assert spr.sparsepr_rope_validate(_rope(spr, **dict(kw))) == status


@pytest.mark.parametrize("axes,scaling,factor,orig", [
    ([64], "none", 1.0, 0), ([44, 42, 42], "none", 1.0, 0), ([128], "linear", 4.0, 0), ([128], "base", 8.0, 0),
    ([2], "base", 8.0, 0), ([128], "parts", 8.0, 4096), ([64], "parts", 32.0, 8192), ([16, 48], "parts", 2.0, 1000),
])
def test_frequencies(spr, axes, scaling, factor, orig):
    p = spr.RopeParams.make(1, 1, 1, 128, rot_dim=sum(axes), axis_dim=axes, scaling=scaling, factor=factor, orig_len=orig)
    f, _, _ = R.rope_freqs(axes, scaling, factor, orig)
    got = spr.sparsepr_rope_frequencies(p) * (2 * math.pi)
    # a few roundings of 2^-53 in pow, the products and 2 pi
    assert torch.all((got - f).abs() <= 16 * 2.0 ** -53 * f + 1e-300)


def test_parts_with_a_long_axis_keeps_and_divides(spr):
    """Fast pairs keep their frequency, the slowest are divided by the factor."""
    kw = dict(rot_dim=128, axis_dim=[128])
    plain = spr.sparsepr_rope_frequencies(spr.RopeParams.make(1, 1, 1, 128, **kw))
    parts = spr.sparsepr_rope_frequencies(spr.RopeParams.make(1, 1, 1, 128, scaling="parts", factor=8.0, orig_len=4096, **kw))
    assert parts[0] == plain[0] and abs(parts[-1] * 8 / plain[-1] - 1) < 1e-12
    assert torch.all(parts <= plain) and torch.all(parts >= plain / 8 * (1 - 1e-12))


@pytest.mark.parametrize("dim,orig,factor,lo,hi", [
    # the pair that turns t times is dim ln(orig / (2 pi t)) / (2 ln 10000): 40.2 and 64.3, 45.0 and 69.1,
    # 13.8 and 22.1, and 26.7 and 50.7 of the pairs 0 .. 63 (0 .. 21)
    (128, 65536, 4.0, 40, 65), (128, 131072, 4.0, 45, 70), (44, 65536, 8.0, 13, 23), (128, 9216, 4.0, 26, 51),
])
def test_parts_ramp_may_end_behind_the_last_pair(spr, dim, orig, factor, lo, hi):
    """A long original length: the slowest pair turns more than beta_slow times, so none has its
    frequency divided by the whole factor."""
    kw = dict(rot_dim=dim, axis_dim=[dim])
    got = spr.sparsepr_rope_frequencies(spr.RopeParams.make(1, 1, 1, 128, scaling="parts", factor=factor, orig_len=orig, **kw))
    plain = spr.sparsepr_rope_frequencies(spr.RopeParams.make(1, 1, 1, 128, **kw))
    for j in range(dim // 2):
        share = min(max((j - lo) / (hi - lo), 0.0), 1.0)
        want = 1.0 - share + share / factor
        assert abs(got[j] / plain[j] - want) <= 16 * 2.0 ** -53, j      # a few roundings of 2^-53
        turns = orig / (2 * math.pi) * 10000.0 ** (-2.0 * j / dim)
        assert turns < 32 or share == 0.0
        assert (turns <= 1) == (share == 1.0)

def _cache(spr, **kw):
    base = dict(B=3, Hq=8, Hkv=2, d=64, page=32, n_pages=50, max_pages=10, T=40, max_chunk=20)
    st = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride")}
    base.update(kw)
    p = spr.CacheParams.make(base.pop("B"), base.pop("Hq"), base.pop("Hkv"), base.pop("d"), **base)
    for k, v in st.items():
        for i, x in enumerate(v):
            getattr(p, k)[i] = x
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(T=0), 0), (dict(B=0), 1), (dict(B=65537), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1),
    (dict(Hq=8192, Hkv=8192), 2), (dict(Hkv=8), 0), (dict(Hkv=1), 0),
    (dict(d=96), 2), (dict(d=128), 0), (dict(dtype=2), 2), (dict(dtype=1), 0), (dict(dtype=7), 2),
    (dict(page=8), 2), (dict(page=256), 2), (dict(page=48), 2), (dict(page=16), 0), (dict(page=128), 0),
    (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 26), 2), (dict(n_pages=1 << 26), 2),
    (dict(T=-1), 1), (dict(T=1 << 29), 1), (dict(max_chunk=0), 1), (dict(frame=-1), 1), (dict(frame=0), 0),
    (dict(frame=2 ** 31 - 1), 0), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(n_select=-1), 1), (dict(n_select=4), 1), (dict(n_select=4, q_block=1), 0),
    (dict(n_select=4, q_block=1, n_sink=3, n_recent=2), 1), (dict(n_select=4, q_block=1, n_sink=-1), 1),
    (dict(n_select=1 << 26, q_block=1), 2),
    (dict(q_stride=[512, 60]), 1), (dict(q_stride=[64, 40 * 64]), 0), (dict(o_stride=[0, 64]), 1),
    (dict(k_stride=[0, 64]), 0), (dict(v_stride=[4, 64]), 1),
])
def test_cache_validation(spr, kw, status):
    p = _cache(spr, **dict(kw))
    assert spr.sparsepr_cache_validate(p) == status
    assert (spr.sparsepr_paged_workspace_bytes(p) > 0) == (status == 0)


def test_select_units(spr):
    assert spr.sparsepr_select_units(_cache(spr, n_select=4, q_block=16)) == 40 // 16 + 3
    assert spr.sparsepr_select_units(_cache(spr, n_select=4, q_block=1)) == 40
    with pytest.raises(ValueError):
        spr.sparsepr_select_units(_cache(spr))


def test_workspace_holds_the_pieces(spr):
    """Partial results of single tokens are a fixed number of pieces, not one per sequence; larger
    chunks take the tile kernel's slots and plan, selections the scores of split lists."""
    one = spr.sparsepr_paged_workspace_bytes(_cache(spr, B=1, T=1, max_chunk=1, max_pages=1000, n_pages=1000))
    many = spr.sparsepr_paged_workspace_bytes(_cache(spr, B=4096, T=4096, max_chunk=1, max_pages=1000, n_pages=100000))
    assert 256 < one < many <= 5 * one
    chunk = _cache(spr, B=2, T=4000, max_chunk=2000, max_pages=1000, n_pages=2000)
    assert spr.sparsepr_paged_workspace_bytes(chunk) > 2 * 148 * 256 * 64 * 4
    plain = spr.sparsepr_paged_workspace_bytes(_cache(spr, B=1, T=1, max_chunk=1, max_pages=4000, n_pages=4000))
    sel = spr.sparsepr_paged_workspace_bytes(_cache(spr, B=1, T=1, max_chunk=1, max_pages=4000, n_pages=4000, n_select=8,
                                                    q_block=1))
    assert sel >= plain + 2 * 4000 * 4
    # scores of units that share their pages' means are stored, but not without bound
    chunk = dict(B=1, T=2048, max_chunk=2048, Hkv=8, n_select=64, max_pages=1024, n_pages=1024)
    assert spr.sparsepr_paged_workspace_bytes(_cache(spr, q_block=64, **chunk)) >= 32 * 8 * 1024 * 4
    chunk.update(T=32768, max_chunk=32768, max_pages=8192)
    assert spr.sparsepr_paged_workspace_bytes(_cache(spr, q_block=1, **chunk)) < 1 << 28


@pytest.mark.parametrize("T,q_block,Hkv,max_pages", [
    (32768, 1, 8, 8193), (32768, 1, 8, 16384), (32768, 64, 8, 16384), (4096, 1, 8, 16384), (32768, 1, 8, 1 << 20),
    (300, 1, 4096, 20000), (1, 1, 4096, 1 << 20), (16384, 4, 2, 8192),
])
def test_workspace_of_long_lists_is_bounded(spr, T, q_block, Hkv, max_pages):
    """Scores and 64-bit keys of lists beyond shared memory are kept for a batch of lists at a time: 256 MB
    each at most beside what the call has without a selection, whatever the number of lists."""
    kw = dict(B=1, T=T, max_chunk=T, Hq=Hkv, Hkv=Hkv, page=16, max_pages=max_pages, n_pages=100)
    plain = spr.sparsepr_paged_workspace_bytes(_cache(spr, **kw))
    sel = spr.sparsepr_paged_workspace_bytes(_cache(spr, n_select=64, q_block=q_block, **kw))
    units = -(-T // q_block)
    # 8 d + 16 bytes per list: mean queries, their sequences, error bounds
    assert 0 < plain <= sel <= plain + (2 << 28) + 2 * units * Hkv * (8 * 64 + 16) + 4096


@pytest.mark.parametrize("kw", [dict(), dict(n_select=4, q_block=40), dict(Hq=4096, Hkv=1, n_select=4, q_block=40)])
def test_limits_beyond_the_rows_of_the_call(spr, kw):
    """A max_chunk or q_block that no sequence can reach counts as T: same plan, same workspace."""
    big = dict(kw, max_chunk=2 ** 31 - 1)
    if "q_block" in kw:
        big["q_block"] = 2 ** 31 - 1
    same = dict(kw, max_chunk=40)
    for T in (1, 40):
        want = spr.sparsepr_paged_workspace_bytes(_cache(spr, **dict(same, T=T, B=1)))
        assert 0 < want == spr.sparsepr_paged_workspace_bytes(_cache(spr, **dict(big, T=T, B=1)))


def test_calls_refuse_before_cuda(spr):
    lib = spr._lib
    ok = ctypes.c_void_p(1 << 20)       # never dereferenced
    odd = ctypes.c_void_p((1 << 20) + 8)
    big = 1 << 40
    p = _cache(spr, n_select=4, q_block=16)
    P = ctypes.byref(p)
    r = _rope(spr)
    # rotary positions
    assert lib.sparsepr_rope(ctypes.byref(r), None, ok, ok, ok, None, None, None) == 1
    assert lib.sparsepr_rope(ctypes.byref(r), ok, None, ok, ok, None, None, None) == 1
    assert lib.sparsepr_rope(ctypes.byref(r), ok, ok, None, ok, None, None, None) == 1
    assert lib.sparsepr_rope(ctypes.byref(r), ctypes.c_void_p((1 << 20) + 1), ok, ok, ok, None, None, None) == 1
    r2 = _rope(spr, H2=2)
    assert lib.sparsepr_rope(ctypes.byref(r2), ok, ok, ok, ok, None, ok, None) == 1
    r3 = _rope(spr, x_stride=[8448, 2112, 64], y_stride=[8448, 64, 256])
    assert lib.sparsepr_rope(ctypes.byref(r3), ok, ok, ok, ok, None, None, None) == 1     # in place, other strides
    assert lib.sparsepr_rope(None, ok, ok, ok, ok, None, None, None) == 1
    assert lib.sparsepr_rope_frequencies(ctypes.byref(r), None) == 1
    # nothing to do is not an error
    assert lib.sparsepr_rope(ctypes.byref(_rope(spr, N=0)), None, None, None, None, None, None, None) == 0
    # append
    app = lambda q=P, K=ok, V=ok, qs=ok, ln=ok, tb=ok, kp=ok, vp=ok, km=ok, rp=None, pos=None, fr=None, ws=ok, n=big: \
        lib.sparsepr_cache_append(q, K, V, qs, ln, tb, kp, vp, km, rp, pos, fr, ws, n, None)
    for kw in (dict(K=None), dict(V=odd), dict(qs=None), dict(ln=None), dict(tb=None), dict(kp=odd), dict(vp=None),
               dict(km=odd), dict(rp=ctypes.byref(r)), dict(rp=ctypes.byref(r), pos=ok),
               dict(rp=ctypes.byref(_rope(spr, d=128)), pos=ok, fr=ok), dict(ws=None), dict(q=None)):
        assert app(**kw) == 1, kw
    assert app(ws=odd) == 3 and app(n=16) == 3
    zero = ctypes.byref(_cache(spr, T=0))
    assert app(q=zero, K=None, V=None) == 0
    # selection
    sel = lambda q=P, Q=ok, qs=ok, ln=ok, tb=ok, km=ok, s=ok, c=ok, ws=ok, n=big: \
        lib.sparsepr_page_select(q, Q, qs, ln, tb, km, s, c, ws, n, None)
    for kw in (dict(Q=odd), dict(qs=None), dict(ln=None), dict(tb=None), dict(km=None), dict(s=None), dict(c=None),
               dict(ws=None), dict(q=ctypes.byref(_cache(spr)))):
        assert sel(**kw) == 1, kw
    assert sel(n=0) == 3
    # attention
    att = lambda q=P, Q=ok, qs=ok, ln=ok, tb=ok, kp=ok, vp=ok, s=None, c=None, O=ok, z=None, ws=ok, n=big: \
        lib.sparsepr_paged_attention(q, Q, qs, ln, tb, kp, vp, s, c, O, z, ws, n, None)
    for kw in (dict(Q=None), dict(Q=odd), dict(qs=None), dict(ln=None), dict(tb=None), dict(kp=odd), dict(vp=odd),
               dict(O=odd), dict(s=ok), dict(c=ok), dict(q=ctypes.byref(_cache(spr)), s=ok, c=ok), dict(ws=None)):
        assert att(**kw) == 1, kw
    assert att(ws=odd) == 3 and att(n=0) == 3
    assert att(q=ctypes.byref(_cache(spr, d=96))) == 2
    assert att(q=zero, Q=None) == 0
    assert lib.sparsepr_paged_error(None, None) == -1
    assert lib.sparsepr_paged_clear_error(None, None) == 1


def test_binding_refuses_wrong_tensors(spr):
    """Shapes, types, devices and layouts that the library cannot see (CPU tensors: nothing runs)."""
    p = _cache(spr)
    bf = torch.bfloat16
    Q, O = torch.zeros(40, 8, 64, dtype=bf), torch.zeros(40, 8, 64, dtype=bf)
    qs, ln = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    tb = torch.zeros(3, 10, dtype=torch.int32)
    kp = torch.zeros(50, 2, 32, 64, dtype=bf)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    good = dict(Q=Q, q_start=qs, kv_len=ln, page_table=tb, k_pages=kp, v_pages=kp, O=O, lse=None, ws=ws)
    for bad in (dict(Q=Q[:39]), dict(Q=Q.half()), dict(q_start=qs[:3]), dict(kv_len=ln.long()), dict(page_table=tb[:, :9]),
                dict(k_pages=kp[:, :, :16]), dict(O=O.float()), dict(lse=torch.zeros(40, 8).double()),
                dict(Q=torch.zeros(40, 8, 128, dtype=bf)[..., ::2]), dict(sel=tb),
                dict(Q=torch.zeros(1, 1, 64, dtype=bf).expand(40, 8, 64))):
        with pytest.raises(ValueError):
            spr.sparsepr_paged_attention(p, **{**good, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        spr.sparsepr_paged_attention(p, **good)
    r = spr.RopeParams.make(1, 2, 3, 64)
    x, pos, f = torch.zeros(1, 2, 3, 64, dtype=bf), torch.zeros(1, 3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    for a in ((x[:, :, :2], pos, f, x), (x, pos.long(), f, x), (x, pos, f.float(), x), (x, pos, f, x.float()),
              (x, pos, f, x, x, x)):
        with pytest.raises(ValueError):
            spr.sparsepr_rope(r, *a)
    with pytest.raises(spr.SparsePRError):
        spr.sparsepr_rope(spr.RopeParams.make(1, 2, 3, 64, layout=5), x, pos, f, x)
    with pytest.raises(spr.SparsePRError):
        spr.paged_workspace(_cache(spr, page=8), "cpu")


class _FakeCuda:
    """Stands in for torch where a call picks its device and stream."""

    def __init__(self, current):
        self.current, self.entered = current, []
        self.cuda, self._C = self, self

    def current_device(self):
        return self.current

    def _cuda_getCurrentRawStream(self, dev):
        return 1000 + dev

    def device(self, dev):
        fake = self

        class Ctx:
            def __enter__(self):
                fake.entered.append(dev)

            def __exit__(self, *a):
                fake.entered.append(-1)
        return Ctx()


@pytest.mark.parametrize("current,dev", [(0, 0), (0, 1), (1, 0)])
def test_launches_go_to_the_tensors_device(spr, monkeypatch, current, dev):
    """A call on tensors of another device than the current one runs there, on that device's
    current stream, and leaves the current device as it was."""
    fake = _FakeCuda(current)
    monkeypatch.setattr(spr._torch(), "mod", fake)
    seen = []

    def fn(*args):
        seen.append((args, list(fake.entered)))
        return 0
    spr._launch(fn, lambda p: 0, "params", "name", dev, 7, 8)
    assert seen == [(("params", 7, 8, 1000 + dev), [] if dev == current else [dev])]
    assert fake.entered == ([] if dev == current else [dev, -1])
    with pytest.raises(spr.SparsePRError):
        spr._launch(lambda *a: 4, lambda p: 0, "params", "name", dev)

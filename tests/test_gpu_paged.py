"""GPU tests of rotary positions, cache append, page selection and attention over the paged cache
against plain fp64 forms.

Tolerances (u = half a step of the type: bf16 2^-8, fp16 2^-11, fp32 2^-24, e = 2^-24):
  rotation  u |y| for the rounding, and (|x_a| + |x_b|) m (4 e for the fp32 products, sum and
            magnitude, 2 e for sincospif, and for 16-bit types pi 2^-24 of the reduced angle's
            rounding, below 2^-22): 2^-21 (|x_a| + |x_b|) m, for fp32 rows 8 e (...)
  output    u |o| for the rounding; u A with A = sum_j w_j |v_j| for the probabilities' rounding;
            every probability is off by its logit's error: d + 3 fp32 steps of E = max_j s sum |q||k_j|
            (accumulation, which may truncate: 2 e each), 2 e times the exponent's size (below 2^7:
            smaller weights do not count) and ex2 (2 e); the sums over n keys add 2 e n, so
            A (2 e (d + 3) E + 2^-16 + 2 e n)
  lse       2 e (d + 3) E + 2^-16 + 2 e n + 4 e |lse|
  mean key  u |mean| + 128 e mean|k|
Lists, counts, copied values and untouched rows are compared exactly."""
import math

import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def spr():
    import free_block_sparse_rcp_b200 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------
def rope_tol(x, y, rot, layout, mag, dt):
    s = R.partner_sum(x, rot, layout) * mag
    return R.HALF_STEP[dt] * y.abs() + (8 * E24 if dt == F32 else 2.0 ** -21) * s + 1e-30


ROPE_CASES = [
    # B, H, H2, N, d, rot, layout, axes, dtype, scaling, factor, orig
    (1, 3, 0, 37, 64, 64, "half", [64], BF, "none", 1.0, 0),
    (2, 4, 1, 5, 128, 128, "interleaved", [44, 42, 42], BF, "none", 1.0, 0),
    (2, 5, 2, 70, 128, 128, "half", [44, 42, 42], FP, "none", 1.0, 0),
    (1, 2, 2, 19, 128, 64, "half", [64], F32, "parts", 8.0, 4096),
    (3, 1, 3, 1, 128, 96, "interleaved", [96], F32, "linear", 4.0, 0),
    (1, 9, 0, 33, 64, 22, "half", [22], FP, "base", 2.0, 0),          # pairs that 16 bytes do not hold
    (1, 7, 4, 33, 64, 22, "interleaved", [22], BF, "base", 2.0, 0),   # the rotation ends inside a chunk
    (2, 3, 1, 11, 40, 38, "half", [2, 36], BF, "none", 1.0, 0),
    (2, 19, 6, 23, 128, 22, "half", [10, 12], F32, "none", 1.0, 0),   # ... with chunks behind them
    (1, 5, 2, 9, 40, 18, "half", [18], BF, "none", 1.0, 0),
    (1, 2, 1, 6, 6, 4, "interleaved", [4], FP, "none", 1.0, 0),       # rows of 12 bytes
    (1, 2, 1, 6, 6, 4, "half", [4], FP, "none", 1.0, 0),
    (1, 2, 0, 6, 3, 2, "half", [2], F32, "none", 1.0, 0),
    (1, 1, 0, 2, 2, 2, "half", [2], BF, "none", 1.0, 0),
    (1, 3, 0, 9, 512, 512, "half", [512], FP, "none", 1.0, 0),
    (64, 40, 8, 1, 128, 128, "half", [128], BF, "none", 1.0, 0),      # one token of each sequence
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(str(x) for x in c[:8]))
@pytest.mark.parametrize("batched", [0, 1])
def test_rope(spr, gpu, case, batched):
    B, H, H2, N, d, rot, layout, axes, dt, scaling, factor, orig = case
    g = gen(1)
    x = torch.randn(B, H, N, d, generator=g).to(dt)
    x2 = torch.randn(B, H2, N, d, generator=g).to(dt) if H2 else None
    pos = torch.randint(0, 1 << 20, (len(axes), B, N) if batched else (len(axes), N), generator=g).to(torch.int32)
    p = spr.RopeParams.make(B, H, N, d, H2=H2, dtype=dt, rot_dim=rot, layout=layout, axis_dim=axes, pos_batched=batched,
                            scaling=scaling, factor=factor, orig_len=orig)
    f = spr.rope_frequencies(p, gpu)
    fr = R.rope_freqs(axes, scaling, factor, orig)
    for call, sign in ((spr.sparsepr_rope, 1.0), (spr.sparsepr_rope_backward, -1.0)):
        y = torch.empty_like(x, device=gpu)
        y2 = torch.empty_like(x2, device=gpu) if H2 else None
        call(p, x.to(gpu), pos.to(gpu), f, y, *([x2.to(gpu), y2] if H2 else []))
        for a, b in ((x, y), (x2, y2)):
            if a is None:
                continue
            want = R.rope(a.double(), pos, rot, layout, fr, sign)
            err = (b.cpu().double() - want).abs()
            assert torch.all(err <= rope_tol(a.double(), want, rot, layout, fr[2], dt)), err.max()
            assert torch.equal(b.cpu()[..., rot:], a[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_far_positions(spr, gpu, layout):
    """Positions up to 2^31 - 1 and negative ones keep the accuracy of small ones."""
    d = 128
    pos = torch.tensor([[0, 1, -5, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    x = torch.randn(1, 2, 7, d, generator=gen(2))
    p = spr.RopeParams.make(1, 2, 7, d, dtype=F32, layout=layout)
    y = torch.empty_like(x, device=gpu)
    spr.sparsepr_rope(p, x.to(gpu), pos.to(gpu), spr.rope_frequencies(p, gpu), y)
    fr = R.rope_freqs([d])
    want = R.rope(x.double(), pos, d, layout, fr)
    # the 64-bit product pos f is off by 2^-53 |pos f| turns: 2 pi 2^-22 at 2^31, in the reference too
    tol = rope_tol(x.double(), want, d, layout, 1.0, F32) + R.partner_sum(x.double(), d, layout) * (
        4 * math.pi * 2.0 ** -53 * pos.double().abs()[0][None, None, :, None])
    assert torch.all((y.cpu().double() - want).abs() <= tol)


def test_rope_strided_in_place_and_stream(spr, gpu):
    """Views of a fused [B, N, 3, H, d] projection, in place, on a stream of its own."""
    B, N, H, d = 2, 23, 4, 64
    qkv = torch.randn(B, N, 3, H, d, generator=gen(3)).to(BF)
    dev = qkv.to(gpu)
    q, k = dev[:, :, 0].transpose(1, 2), dev[:, :, 1].transpose(1, 2)
    pos = torch.arange(N, dtype=torch.int32)[None]
    p = spr.RopeParams.make(B, H, N, d, H2=H)
    f = spr.rope_frequencies(p, gpu)
    posd = pos.to(gpu)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        spr.sparsepr_rope(p, q, posd, f, q, k, k)
    st.synchronize()
    got = dev.cpu()
    fr = R.rope_freqs([d])
    for i in range(2):
        x = qkv[:, :, i].transpose(1, 2).double()
        want = R.rope(x, pos, d, "half", fr)
        assert torch.all((got[:, :, i].transpose(1, 2).double() - want).abs() <= rope_tol(x, want, d, "half", 1.0, BF))
    assert torch.equal(got[:, :, 2], qkv[:, :, 2])
    # a broadcast input (one head for all) into separate outputs; a misaligned view
    x = torch.randn(1, 1, N, d, generator=gen(4)).to(BF)
    y = torch.empty(1, H, N, d, dtype=BF, device=gpu)
    p1 = spr.RopeParams.make(1, H, N, d)
    spr.sparsepr_rope(p1, x.to(gpu).expand(1, H, N, d), posd, f, y)
    assert torch.equal(y, y[:, :1].expand_as(y))
    buf = torch.zeros(N * H * d + 1, dtype=BF, device=gpu)[1:].view(1, H, N, d)
    spr.sparsepr_rope(p1, x.to(gpu).expand(1, H, N, d), posd, f, buf)
    assert torch.equal(buf, y)
    spr.sparsepr_rope(spr.RopeParams.make(1, H, 0, d), x[:, :, :0].to(gpu).expand(1, H, 0, d), posd[:, :0], f, y[:, :, :0])


def test_rope_gradient(spr, gpu):
    """The gradient against the formula's (<w, R x> = <R^T w, x>) and against differences."""
    B, H, N, d, rot = 1, 2, 9, 64, 48
    p = spr.RopeParams.make(B, H, N, d, dtype=F32, rot_dim=rot, scaling="parts", factor=4.0, orig_len=2048)
    f = spr.rope_frequencies(p, gpu)
    pos = torch.randint(0, 5000, (1, N), generator=gen(5)).to(torch.int32).to(gpu)
    x, w = torch.randn(B, H, N, d, generator=gen(6)).to(gpu), torch.randn(B, H, N, d, generator=gen(7)).to(gpu)

    def fwd(t):
        y = torch.empty_like(t)
        spr.sparsepr_rope(p, t, pos, f, y)
        return (y.double() * w.double()).sum().item()
    g = torch.empty_like(x)
    spr.sparsepr_rope_backward(p, w, pos, f, g)
    xr = x.cpu().double().requires_grad_()
    (R.rope(xr, pos.cpu(), rot, "half", R.rope_freqs([rot], "parts", 4.0, 2048)) * w.cpu().double()).sum().backward()
    mag = 0.1 * math.log(4.0) + 1
    assert torch.all((g.cpu().double() - xr.grad).abs() <= rope_tol(w.cpu().double(), xr.grad, rot, "half", mag, F32))
    for i in (0, 17, 47, 48, 63):
        dx = torch.zeros_like(x)
        dx[0, 1, 3, i] = 0.5            # the map is linear: the difference is exact up to rounding
        diff = fwd(x + dx) - fwd(x - dx)
        # y changes by about 1 in two elements; each sum is off by 8 e of its terms
        scale = 8 * E24 * (x.abs().sum() + 1).item() * mag * 4
        assert abs(diff - g[0, 1, 3, i].item()) <= scale


@pytest.mark.parametrize("factor,want", [(8.0, 1.0 + 0.1 * math.log(8.0)), (1.0, 1.0), (0.5, 1.0), (1e-6, 1.0)])
def test_rope_default_magnitude_by_parts(spr, gpu, factor, want):
    """At position 0 a row is only multiplied: by 0.1 ln(factor) + 1, and by 1 for factors up to 1."""
    x = torch.ones(1, 1, 2, 64, device=gpu)
    p = spr.RopeParams.make(1, 1, 2, 64, dtype=F32, scaling="parts", factor=factor, orig_len=4096)
    y = torch.empty_like(x)
    spr.sparsepr_rope(p, x, torch.zeros(1, 2, dtype=torch.int32, device=gpu), spr.rope_frequencies(p, gpu), y)
    # the magnitude's rounding to 32 bits; the sine is 0 and the cosine 1
    assert torch.all((y.double() - want).abs() <= E24 * want)


# bit patterns that arithmetic would change: infinities, -0, quiet and signalling NaNs with payloads
ODD_BITS = {BF: (torch.int16, [0x7f80, -0x80, -0x8000, 0x7fc5, 0x7f85, -0x3a, 0x0001]),
            FP: (torch.int16, [0x7c00, -0x400, -0x8000, 0x7e05, 0x7c05, -0x1a, 0x0001]),
            F32: (torch.int32, [0x7f800000, -0x800000, -0x80000000, 0x7fc00005, 0x7f800005, -0x3ffffa, 0x00000001])}


def odd_tail(x, rot, seed):
    """x with such patterns in some of the elements from rot on."""
    it, bits = ODD_BITS[x.dtype]
    y = x.clone().view(it)
    pick = torch.randint(0, 2 * len(bits), y[..., rot:].shape, generator=gen(seed))
    vals = torch.tensor(bits, dtype=it)[pick % len(bits)]
    y[..., rot:] = torch.where(pick < len(bits), vals, y[..., rot:])
    return y.view(x.dtype), it


@pytest.mark.parametrize("dt", [BF, FP, F32])
@pytest.mark.parametrize("layout,d,rot", [("interleaved", 64, 22), ("interleaved", 64, 2), ("interleaved", 128, 126), ("half", 64, 22),
                                          ("half", 64, 32), ("interleaved", 6, 4)])
def test_rope_copies_what_is_behind_the_rotation(spr, gpu, layout, d, rot, dt):
    """Elements rot_dim .. d - 1 keep their bits, and what they hold does not reach the others."""
    H, N = 3, 37
    x = torch.randn(1, H, N, d, generator=gen(81)).to(dt)
    odd, it = odd_tail(x, rot, 82)
    p = spr.RopeParams.make(1, H, N, d, dtype=dt, rot_dim=rot, layout=layout)
    pos = torch.arange(5, 5 + N, dtype=torch.int32, device=gpu)[None]
    f = spr.rope_frequencies(p, gpu)
    for call in (spr.sparsepr_rope, spr.sparsepr_rope_backward):
        plain, got = torch.empty_like(x, device=gpu), torch.empty_like(x, device=gpu)
        call(p, x.to(gpu), pos, f, plain)
        call(p, odd.to(gpu), pos, f, got)
        assert torch.equal(got.view(it)[..., rot:].cpu(), odd.view(it)[..., rot:])
        assert torch.equal(got[..., :rot], plain[..., :rot])


# ---------------------------------------------------------------------------
# The cache
# ---------------------------------------------------------------------------
class Scene:
    """A cache of sequences of kv rows, of which new are new; pages in random order.  Slots past
    the rows in use hold NaN.  tiles: so many packed rows behind the last sequence that the call
    counts as a large one, whose chunks go to the tensor tiles."""

    def __init__(self, spr, gpu, new, kv, *, Hq, Hkv, d, page, dt, frame=1, q_block=0, n_select=0, n_sink=0, n_recent=0,
                 seed=0, tail_rows=0, max_pages=None, max_chunk=None, spare=2, bump=0.0, tiles=False):
        g = gen(seed)
        self.new, self.kv, self.gpu, self.spr = new, kv, gpu, spr
        B = len(new)
        pages = [-(-k // page) for k in kv]
        self.n_pages = sum(pages) + spare
        mp = max(max(pages), 1) if max_pages is None else max_pages
        self.T = sum(new) + tail_rows
        if tiles:
            self.T = max(self.T, 5_000_000 // (Hq * page * (min(mp, n_select) if n_select else mp)) + 1)
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((B, mp), 2 ** 31 - 1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        nan = float("nan")
        self.kp = torch.full((self.n_pages, Hkv, page, d), nan, dtype=dt)
        self.vp = torch.full((self.n_pages, Hkv, page, d), nan, dtype=dt)
        self.km = torch.full((self.n_pages, Hkv, d), nan, dtype=dt)
        for b in range(B):
            for j in range(pages[b]):
                r = min(page, kv[b] - j * page)
                pid = int(self.table[b, j])
                self.kp[pid, :, :r] = (torch.randn(Hkv, r, d, generator=g) + bump * torch.randn(Hkv, 1, d, generator=g)).to(dt)
                self.vp[pid, :, :r] = torch.randn(Hkv, r, d, generator=g).to(dt)
                self.km[pid] = self.kp[pid, :, :r].float().mean(1).to(dt)
        self.Q = torch.randn(self.T, Hq, d, generator=g).to(dt)
        qs = [0]
        for n in new:
            qs.append(qs[-1] + n)
        self.q_start = torch.tensor(qs, dtype=torch.int32)
        self.kv_len = torch.tensor(kv, dtype=torch.int32)
        self.p = spr.CacheParams.make(B, Hq, Hkv, d, dtype=dt, page=page, n_pages=self.n_pages, max_pages=mp, T=self.T,
                                      max_chunk=max(max(new), 1) if max_chunk is None else max_chunk, frame=frame,
                                      q_block=q_block, n_select=n_select, n_sink=n_sink, n_recent=n_recent)
        self.dev = {k: getattr(self, k).to(gpu) for k in ("table", "kp", "vp", "km", "Q", "q_start", "kv_len")}
        self.ws = spr.paged_workspace(self.p, gpu)
        self.frame, self.page, self.q_block, self.dt = frame, page, q_block, dt
        self.scale = 1 / math.sqrt(d)

    def seqs(self):
        return self.dev["q_start"], self.dev["kv_len"], self.dev["table"]

    def attend(self, sel=None, cnt=None, O=None, lse=True, Q=None):
        O = torch.full_like(self.dev["Q"], 7.0) if O is None else O
        z = torch.full(O.shape[:2], 7.0, dtype=torch.float32, device=self.gpu) if lse else None
        self.spr.sparsepr_paged_attention(self.p, self.dev["Q"] if Q is None else Q, *self.seqs(), self.dev["kp"],
                                          self.dev["vp"], O, z, self.ws, sel=sel, sel_count=cnt)
        return O, z

    def select(self):
        sel, cnt = self.spr.alloc_selection(self.p, self.gpu)
        sel.fill_(-9)
        cnt.fill_(-9)
        self.spr.sparsepr_page_select(self.p, self.dev["Q"], *self.seqs(), self.dev["km"], sel, cnt, self.ws)
        return sel, cnt

    def check(self, O, z, sel=None, cnt=None):
        n = sum(self.new)
        ref, L, A, E = R.attention(self.Q, self.new, self.kv, self.table, self.kp, self.vp, self.frame, self.scale,
                                   None if sel is None else sel.cpu(), None if cnt is None else cnt.cpu(), self.q_block)
        u, d = R.HALF_STEP[self.dt], self.Q.shape[2]
        rel = 2 * E24 * (d + 3) * E + 2.0 ** -16 + 2 * E24 * max(self.kv)
        got = O.cpu().double()[:n]
        tol = u * ref[:n].abs() + A[:n] * (u + rel[:n, :, None]) + 1e-30
        bad = (got - ref[:n]).abs() > tol
        assert not torch.isnan(got).any()
        assert not bad.any(), ((got - ref[:n]).abs() / tol).max()
        if z is not None:
            gz, L = z.cpu().double()[:n], L[:n]
            empty = L == -math.inf
            assert torch.equal(gz == -math.inf, empty)
            assert torch.all((gz - L).abs()[~empty] <= (rel[:n] + 4 * E24 * L.abs())[~empty])
        if O.shape[0] > n:      # rows behind the last sequence
            assert torch.all(O[n:] == 7.0) and (z is None or torch.all(z[n:] == 7.0))
        assert self.spr.sparsepr_paged_error(self.ws) == 0


ROWS = [   # new, kv, Hq, Hkv, d, page, dtype, frame
    ([1], [1], 1, 1, 64, 16, BF, 1),
    ([1], [4097], 8, 2, 128, 64, BF, 1),
    ([1, 1, 1, 1], [5, 129, 64, 700], 8, 2, 128, 16, FP, 1),
    ([1, 0, 1, 1], [0, 50, 33, 128], 4, 4, 64, 32, BF, 1),        # no keys; no new token
    ([3, 1, 4], [3, 300, 2], 6, 2, 64, 128, BF, 1),               # more new tokens than slots
    ([7, 2, 8], [260, 9, 513], 4, 1, 128, 128, FP, 4),            # 32 rows, frames of 4 tokens
    ([5, 5], [77, 1000], 3, 1, 64, 64, BF, 0),                    # group of 3, no mask
    ([16, 9], [100, 40], 2, 2, 128, 32, BF, 1),
    ([1] * 40, [17 * i % 900 for i in range(40)], 2, 1, 64, 16, BF, 1),
    ([1, 2], [700, 90], 40, 1, 128, 16, BF, 1),                   # a token's heads in two items
    ([19, 0, 3] * 120, [20 + 7 * i % 150 for i in range(360)], 2, 1, 64, 16, FP, 1),   # many sequences, some of two items
]
TILES = [
    ([40], [40], 1, 1, 64, 16, BF, 1),
    ([33], [1000], 4, 4, 128, 64, FP, 1),
    ([100, 3, 0, 57], [640, 3, 20, 200], 8, 2, 64, 32, BF, 1),
    ([130], [130], 3, 1, 128, 128, BF, 1),                        # parts begin inside a token's heads
    ([300], [900], 1, 1, 128, 16, FP, 100),                       # frames of 100 tokens
    ([50, 45], [1029, 300], 6, 2, 64, 128, BF, 0),
    ([64], [30], 2, 1, 64, 16, BF, 1),                            # more new tokens than slots
    ([257, 35], [257, 2000], 1, 1, 64, 64, FP, 1),
    ([40], [0], 2, 1, 64, 16, BF, 0),                             # nothing cached
]


@pytest.mark.parametrize("case,tiles", [(c, False) for c in ROWS + TILES] + [(c, True) for c in TILES],
                         ids=lambda c: "-".join(str(x) for x in c) if isinstance(c, tuple) else ("tiles" if c else "rows"))
def test_attention(spr, gpu, case, tiles):
    new, kv, Hq, Hkv, d, page, dt, frame = case
    s = Scene(spr, gpu, new, kv, Hq=Hq, Hkv=Hkv, d=d, page=page, dt=dt, frame=frame, tail_rows=3, seed=len(kv) + d,
              tiles=tiles)
    O, z = s.attend()
    s.check(O, z)
    O2, _ = s.attend(lse=False)
    assert torch.equal(O, O2)


@pytest.mark.parametrize("new,kv,Hq,Hkv,tiles", [([1], [3000], 4, 1, False), ([70], [2500], 2, 2, False),
                                                 ([70], [2500], 2, 2, True), ([1, 2], [1900, 10], 8, 4, False)])
def test_attention_logits_that_move(spr, gpu, new, kv, Hq, Hkv, tiles):
    """Large logits, growing along the keys: the running maximum moves and early chunks vanish."""
    s = Scene(spr, gpu, new, kv, Hq=Hq, Hkv=Hkv, d=64, page=32, dt=FP, frame=1, seed=9, tiles=tiles)
    for b, n in enumerate(kv):
        for j in range(-(-n // 32)):
            s.kp[int(s.table[b, j])] *= 0.2 + 4.0 * j * 32 / n
    s.Q *= 3
    s.dev["kp"], s.dev["Q"] = s.kp.to(gpu), s.Q.to(gpu)
    s.check(*s.attend())


@pytest.mark.parametrize("new,kv,tiles", [([1], [20000], False), ([40], [9000], False), ([40], [9000], True)])
def test_attention_many_small_weights_fp16(spr, gpu, new, kv, tiles):
    """One key far above thousands of equal others: their probabilities of 2^-18 still count."""
    s = Scene(spr, gpu, new, kv, Hq=1, Hkv=1, d=64, page=64, dt=FP, frame=0, seed=3, tiles=tiles)
    s.kp.zero_()
    s.Q.zero_()
    s.Q[:, :, 0] = 10.0
    pid = int(s.table[0, 0])
    s.kp[pid, 0, 5, 0] = 18 * math.log(2) * 8 / 10.0
    s.vp[:] = torch.nan_to_num(s.vp, nan=1.0).abs()
    s.dev["kp"], s.dev["vp"], s.dev["Q"] = s.kp.to(gpu), s.vp.to(gpu), s.Q.to(gpu)
    s.check(*s.attend())


@pytest.mark.parametrize("new,kv,tiles", [([1, 3], [900, 70], False), ([60], [300], False), ([60], [300], True)])
@pytest.mark.parametrize("scale", [0.03125, 0.375])
def test_attention_scale_of_the_caller(spr, gpu, new, kv, tiles, scale):
    s = Scene(spr, gpu, new, kv, Hq=4, Hkv=2, d=64, page=32, dt=BF, seed=101, tiles=tiles)
    s.p.scale = s.scale = scale
    s.check(*s.attend())


@pytest.mark.parametrize("tiles", [False, True])
def test_a_list_longer_than_the_cache_is_an_error(spr, gpu, tiles):
    """Every page once and the last one again, behind the chunks that the visible keys need."""
    s = Scene(spr, gpu, [40], [1280], Hq=2, Hkv=1, d=64, page=128, dt=BF, frame=0, q_block=40, n_select=12, seed=25,
              tiles=tiles)
    sel, cnt = spr.alloc_selection(s.p, gpu)
    sel[0, 0] = torch.tensor(list(range(10)) + [9, 9], dtype=torch.int32, device=gpu)
    cnt[0, 0] = 12
    O, _ = s.attend(sel, cnt)
    assert spr.sparsepr_paged_error(s.ws) == 1 and torch.isnan(O[:40]).all()


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("new,kv,d", [([2], [700], 64), ([50], [700], 64), ([50], [700], 128)])
def test_attention_large_values(spr, gpu, new, kv, d, tiles):
    """Values of 10^30 with a maximum that grows by thirty powers of two along the keys."""
    s = Scene(spr, gpu, new, kv, Hq=2, Hkv=1, d=d, page=32, dt=BF, frame=0, seed=35, tiles=tiles)
    s.Q.fill_(0)
    s.Q[:, :, 0] = 8.0
    for j in range(22):
        s.kp[int(s.table[0, j]), :, :, 0] = j * 30 * math.log(2) / 21 * math.sqrt(d) / 8
    s.vp *= 1e30
    s.dev["kp"], s.dev["vp"], s.dev["Q"] = s.kp.to(gpu), s.vp.to(gpu), s.Q.to(gpu)
    s.check(*s.attend())


@pytest.mark.parametrize("new,kv,tiles", [([1, 1], [300, 70], False), ([90], [400], False), ([90], [400], True)])
def test_attention_strided(spr, gpu, new, kv, tiles):
    """Q and O as views of head-major and fused tensors."""
    s = Scene(spr, gpu, new, kv, Hq=4, Hkv=2, d=64, page=32, dt=BF, seed=4, tiles=tiles)
    O, z = s.attend()
    s.check(O, z)
    qh = s.dev["Q"].transpose(0, 1).contiguous().transpose(0, 1)
    fused = torch.zeros(s.T, 3, 4, 64, dtype=BF, device=gpu)
    O2, z2 = s.attend(O=fused[:, 1], Q=qh)
    n = sum(new)
    assert torch.equal(O2[:n], O[:n]) and torch.equal(z2, z) and torch.all(O2[n:] == 0)
    assert torch.all(fused[:, 0] == 0) and torch.all(fused[:, 2] == 0)


@pytest.mark.parametrize("new,tiles", [([1, 1, 1], False), ([40, 50, 45], False), ([40, 50, 45], True)])
def test_attention_bad_inputs_are_errors(spr, gpu, new, tiles):
    """Bad page ids and lengths: error 1, NaN in the rows that depend on them, the others right."""
    kv = [200, 150, 90]
    for what in ("page", "negative", "len", "chunk"):
        s = Scene(spr, gpu, new, kv, Hq=2, Hkv=1, d=64, page=32, dt=BF, seed=5, tiles=tiles)
        t, ln = s.table.clone(), s.kv_len.clone()
        if what == "page":
            t[1, 2] = s.n_pages
        if what == "negative":
            t[1, 0] = -1
        if what == "len":
            ln[1] = t.shape[1] * 32 + 1
        if what == "chunk":
            s.p.max_chunk = max(1, new[1] - 1) if new[1] > 1 else 1
            if new[1] == 1:
                continue
        s.dev["table"], s.dev["kv_len"] = t.to(gpu), ln.to(gpu)
        if what == "len":
            s.dev["table"] = s.dev["table"].clamp(0, s.n_pages - 1)
        O, z = s.attend()
        assert spr.sparsepr_paged_error(s.ws) == 1
        spr.sparsepr_paged_clear_error(s.ws)
        assert spr.sparsepr_paged_error(s.ws) == 0
        a, b = new[0], new[0] + new[1]
        if what != "chunk":
            assert torch.isnan(O[a:b]).all() and torch.isnan(z[a:b]).all(), what
            ref, _, A, _ = R.attention(s.Q, new, kv, s.table, s.kp, s.vp, 1, s.scale)
            for r in (slice(0, a), slice(b, sum(new))):
                assert torch.all((O.cpu().double()[r] - ref[r]).abs() <= 2.0 ** -6 * A[r] + 1e-6)


def test_q_start_out_of_order_is_an_error(spr, gpu):
    s = Scene(spr, gpu, [2, 3, 1], [60, 70, 10], Hq=2, Hkv=1, d=64, page=32, dt=BF, seed=6)
    s.dev["q_start"] = torch.tensor([0, 4, 2, 50], dtype=torch.int32, device=gpu)
    s.attend()
    assert spr.sparsepr_paged_error(s.ws) == 1


def test_q_start_that_promises_more_than_there_is(spr, gpu):
    """Offsets that go back to 0 again and again count 2^32 units: an error, and every list that is
    written is one of the cache's."""
    B, T = 65536, 131072
    s = Scene(spr, gpu, [1], [64], Hq=1, Hkv=1, d=64, page=16, dt=BF, seed=16)
    p = spr.CacheParams.make(B, 1, 1, 64, page=16, n_pages=s.n_pages, max_pages=4, T=T, max_chunk=1, q_block=1, n_select=2)
    q_start = torch.tensor([0, T], dtype=torch.int32).repeat(B // 2 + 1)[:B + 1].to(gpu)
    kv_len = torch.full((B,), 64, dtype=torch.int32, device=gpu)
    table = s.dev["table"].expand(B, 4).contiguous()
    Q = s.dev["Q"].expand(T, 1, 64).contiguous()
    ws = spr.paged_workspace(p, gpu)
    sel, cnt = spr.alloc_selection(p, gpu)
    sel.fill_(-9)
    cnt.fill_(-9)
    spr.sparsepr_page_select(p, Q, q_start, kv_len, table, s.dev["km"], sel, cnt, ws)
    assert int(cnt.max()) <= 2 and int(sel.max()) <= 3
    spr.sparsepr_paged_clear_error(ws)
    O = torch.zeros_like(Q)
    spr.sparsepr_paged_attention(p, Q, q_start, kv_len, table, s.dev["kp"], s.dev["vp"], O, None, ws, sel=sel, sel_count=cnt)
    assert spr.sparsepr_paged_error(ws) == 1


def test_far_offsets(spr, gpu):
    """Pages past 2^31 elements of the pool, and queries past 2^31 elements of a strided buffer."""
    d, page, Hkv = 128, 128, 8
    n_pages = (1 << 31) // (d * page * Hkv) + 40
    s = Scene(spr, gpu, [1, 40], [300, 200], Hq=8, Hkv=8, d=d, page=page, dt=BF, seed=7, spare=0)
    kp = torch.empty(n_pages, Hkv, page, d, dtype=BF, device=gpu)
    vp = torch.empty_like(kp)
    km = torch.empty(n_pages, Hkv, d, dtype=BF, device=gpu)
    shift = n_pages - s.n_pages
    kp[shift:], vp[shift:], km[shift:] = s.dev["kp"], s.dev["vp"], s.dev["km"]
    table = s.table.clone()
    table[table < s.n_pages] += shift
    for mp in (table.shape[1], 150):       # 150: a large call, to the tensor tiles
        p = spr.CacheParams.from_buffer_copy(s.p)
        p.n_pages, p.max_pages = n_pages, mp
        O, z = torch.empty_like(s.dev["Q"]), torch.empty(41, 8, device=gpu)
        ws = spr.paged_workspace(p, gpu)
        t = torch.cat([table, table[:, :1].expand(2, mp - table.shape[1])], 1).to(gpu).contiguous()
        spr.sparsepr_paged_attention(p, s.dev["Q"], s.dev["q_start"], s.dev["kv_len"], t, kp, vp, O, z, ws)
        s.check(O, z)
    # append there too
    p = spr.CacheParams.from_buffer_copy(s.p)
    p.n_pages = n_pages
    K = torch.randn(41, Hkv, d, generator=gen(8)).to(BF).to(gpu)
    spr.sparsepr_cache_append(p, K, K, s.dev["q_start"], s.dev["kv_len"], table.to(gpu), kp, vp, km, ws)
    pid = int(table[0, 299 // 128])
    assert torch.equal(kp[pid, :, 299 % 128], K[0]) and torch.equal(vp[pid, :, 299 % 128], K[0])
    assert spr.sparsepr_paged_error(ws) == 0


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
APPEND = [  # new, kv, Hkv, d, page, dtype, rope (rot, layout, axes) or None
    ([1], [1], 1, 64, 16, BF, None),
    ([1, 1, 1], [17, 32, 200], 3, 128, 16, FP, (128, "half", [128])),
    ([40, 0, 3], [40, 10, 99], 2, 64, 32, BF, (64, "interleaved", [24, 20, 20])),
    ([130, 65], [300, 65], 4, 128, 64, BF, (96, "half", [96])),
    ([129], [140], 1, 64, 128, FP, (22, "half", [22])),
    ([70], [150], 2, 128, 128, BF, (22, "interleaved", [22])),
    ([70, 9], [150, 30], 5, 128, 64, BF, (22, "half", [10, 12])),
    ([50, 6], [20, 0], 2, 64, 16, BF, (64, "half", [64])),        # more new tokens than slots
    ([260], [260], 20, 64, 16, BF, (64, "half", [64])),           # several heads per block
]


def expect_append(s, K, V, pos, rope, freqs):
    """The cache after the append, and error scales of the new keys."""
    kp, vp, km = s.kp.double().clone(), s.vp.double().clone(), s.km.double().clone()
    K = K.double()
    tolK = torch.zeros_like(kp)
    scale = torch.zeros_like(K)
    if rope:
        scale = R.partner_sum(K.transpose(0, 1), rope[0], rope[1]).transpose(0, 1)
        K = R.rope(K.transpose(0, 1), pos, rope[0], rope[1], freqs).transpose(0, 1)
    touched = set()
    at = 0
    for b, (n, length) in enumerate(zip(s.new, s.kv)):
        for i in range(n):
            slot = length - n + i
            if slot < 0:
                continue
            pid, r = int(s.table[b, slot // s.page]), slot % s.page
            kp[pid, :, r], vp[pid, :, r] = K[at + i], V[at + i].double()
            tolK[pid, :, r] = scale[at + i]
            touched.add((pid, min(s.page, length - slot // s.page * s.page)))
        at += n
    return kp, vp, km, tolK, touched


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c))
def test_append(spr, gpu, case):
    new, kv, Hkv, d, page, dt, rope = case
    s = Scene(spr, gpu, new, kv, Hq=Hkv, Hkv=Hkv, d=d, page=page, dt=dt, seed=11, tail_rows=2)
    K = torch.randn(s.T, Hkv, d, generator=gen(12)).to(dt)
    V = torch.randn(s.T, Hkv, d, generator=gen(13)).to(dt)
    kw, freqs, pos = {}, None, None
    if rope:
        rp = spr.RopeParams.make(1, Hkv, s.T, d, dtype=dt, rot_dim=rope[0], layout=rope[1], axis_dim=rope[2])
        pos = torch.randint(0, 100000, (len(rope[2]), s.T), generator=gen(14)).to(torch.int32)
        freqs = R.rope_freqs(rope[2])
        kw = dict(rope=rp, pos=pos.to(gpu), freq=spr.rope_frequencies(rp, gpu))
    # strided inputs: K and V as halves of one fused tensor
    fused = torch.stack([K, V], 1).to(gpu)
    spr.sparsepr_cache_append(s.p, fused[:, 0], fused[:, 1], *s.seqs(), s.dev["kp"], s.dev["vp"], s.dev["km"], s.ws, **kw)
    kp, vp, km, scale, touched = expect_append(s, K, V, pos, rope, freqs)
    got = s.dev["kp"].cpu().double()
    nan = torch.isnan(kp)
    assert torch.equal(torch.isnan(got), nan)
    fresh = scale > 0
    u = R.HALF_STEP[dt]
    assert torch.all((got - kp).abs()[fresh] <= (u * kp.abs() + 2.0 ** -21 * scale)[fresh])
    old = ~fresh & ~nan
    assert torch.equal(got[old], kp[old])
    gv = s.dev["vp"].cpu().double()
    assert torch.equal(torch.nan_to_num(gv, nan=-99.0), torch.nan_to_num(vp, nan=-99.0))
    gm = s.dev["km"].cpu().double()
    for pid, r in touched:
        k = got[pid, :, :r]
        mean = k.mean(1)
        assert torch.all((gm[pid] - mean).abs() <= u * mean.abs() + 128 * E24 * k.abs().mean(1) + 1e-30)
    rest = [i for i in range(s.n_pages) if i not in {t[0] for t in touched}]
    assert torch.equal(torch.nan_to_num(gm[rest], nan=-99.0), torch.nan_to_num(km[rest], nan=-99.0))
    assert spr.sparsepr_paged_error(s.ws) == 0


def test_append_in_pieces_gives_the_same_cache(spr, gpu):
    """70 rows at once, in three calls, or row by row: the same pages and means bit for bit."""
    Hkv, d, page, n = 2, 128, 32, 70
    K = torch.randn(n, Hkv, d, generator=gen(15)).to(BF).to(gpu)
    V = torch.randn(n, Hkv, d, generator=gen(16)).to(BF).to(gpu)
    pos = torch.arange(100, 100 + n, dtype=torch.int32, device=gpu)[None]
    out = []
    for pieces in ([70], [1, 40, 29], [1] * 70):
        table = torch.tensor([[4, 0, 3]], dtype=torch.int32, device=gpu)
        p = spr.CacheParams.make(1, Hkv, Hkv, d, page=page, n_pages=5, max_pages=3, T=n, max_chunk=n)
        c = spr.alloc_cache(p, gpu)
        for t in c.values():
            t.zero_()
        done = 0
        for m in pieces:
            q = spr.CacheParams.make(1, Hkv, Hkv, d, page=page, n_pages=5, max_pages=3, T=m, max_chunk=m)
            rp = spr.RopeParams.make(1, Hkv, m, d)
            ws = spr.paged_workspace(q, gpu)
            spr.sparsepr_cache_append(q, K[done:done + m], V[done:done + m],
                                      torch.tensor([0, m], dtype=torch.int32, device=gpu),
                                      torch.tensor([done + m], dtype=torch.int32, device=gpu), table, c["k_pages"],
                                      c["v_pages"], c["k_mean"], ws, rope=rp, pos=pos[:, done:done + m].contiguous(),
                                      freq=spr.rope_frequencies(rp, gpu))
            done += m
        out.append(c)
    for c in out[1:]:
        for k in c:
            assert torch.equal(c[k], out[0][k]), k
    assert torch.all(out[0]["k_pages"][[1, 2]] == 0)


def test_append_bad_page(spr, gpu):
    s = Scene(spr, gpu, [40, 5], [60, 30], Hq=1, Hkv=1, d=64, page=16, dt=BF, seed=17)
    t = s.table.clone()
    t[0, 2] = s.n_pages + 3
    before = s.dev["kp"].clone()
    K = torch.ones(45, 1, 64, dtype=BF, device=gpu)
    spr.sparsepr_cache_append(s.p, K, K, s.dev["q_start"], s.dev["kv_len"], t.to(gpu), s.dev["kp"], s.dev["vp"],
                              s.dev["km"], s.ws)
    assert spr.sparsepr_paged_error(s.ws) == 1
    pid = int(s.table[0, 2])
    assert torch.equal(torch.nan_to_num(s.dev["kp"][pid]), torch.nan_to_num(before[pid]))
    assert torch.all(s.dev["kp"][int(s.table[1, 1]), 0, 9:14] == 1)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("layout,rot", [("interleaved", 22), ("interleaved", 126), ("half", 22), ("half", 32)])
def test_append_copies_what_is_behind_the_rotation(spr, gpu, layout, rot, dt):
    """Elements rot_dim .. d - 1 of the keys, and the values, keep their bits."""
    d, n = 128, 37
    s = Scene(spr, gpu, [n], [n + 20], Hq=3, Hkv=3, d=d, page=16, dt=dt, seed=83)
    K, it = odd_tail(torch.randn(n, 3, d, generator=gen(84)).to(dt), rot, 85)
    V, _ = odd_tail(torch.randn(n, 3, d, generator=gen(86)).to(dt), 0, 87)
    rp = spr.RopeParams.make(1, 3, n, d, dtype=dt, rot_dim=rot, layout=layout)
    pos = torch.arange(20, 20 + n, dtype=torch.int32, device=gpu)[None]
    spr.sparsepr_cache_append(s.p, K.to(gpu), V.to(gpu), *s.seqs(), s.dev["kp"], s.dev["vp"], s.dev["km"], s.ws, rope=rp, pos=pos,
                              freq=spr.rope_frequencies(rp, gpu))
    slot = torch.arange(20, 20 + n)
    pid = s.table[0][slot // 16].long()
    kp, vp = s.dev["kp"].cpu().view(it), s.dev["vp"].cpu().view(it)
    assert torch.equal(kp[pid, :, slot % 16][..., rot:], K.view(it)[..., rot:])
    assert torch.equal(vp[pid, :, slot % 16], V.view(it))


@pytest.mark.parametrize("what", ["full", "long", "negative", "chunk", "rows", "before"])
def test_append_of_a_sequence_with_bad_inputs_writes_nothing(spr, gpu, what):
    """A cache length beyond the table, more new tokens than max_chunk, offsets out of the rows: error 1,
    the sequence's pages and means stay as they were, the other sequence's rows arrive."""
    s = Scene(spr, gpu, [40, 21], [64, 100], Hq=2, Hkv=2, d=64, page=16, dt=BF, seed=88, max_pages=7, max_chunk=50)
    bad = 1 if what == "rows" else 0
    t = s.table.clone()
    t[0, 4:] = t[0, 0]                            # entries that a wrong length reaches: a page of the same sequence
    qs, ln = s.q_start.clone(), s.kv_len.clone()
    if what == "full":
        ln[bad] = 7 * 16 + 1
    if what == "long":
        ln[bad] = 2 ** 31 - 1
    if what == "negative":
        ln[bad] = -1
    if what == "chunk":
        s.p.max_chunk = 21
    if what == "rows":                            # the last sequence promises rows behind the call's
        qs[2] += 3
    if what == "before":                          # the first one rows before them
        qs[0] = -2
    before = {k: s.dev[k].cpu().view(torch.int16).clone() for k in ("kp", "vp", "km")}
    K = torch.randn(61, 2, 64, generator=gen(89)).to(BF)
    V = torch.randn(61, 2, 64, generator=gen(90)).to(BF)
    spr.sparsepr_cache_append(s.p, K.to(gpu), V.to(gpu), qs.to(gpu), ln.to(gpu), t.to(gpu), s.dev["kp"], s.dev["vp"], s.dev["km"], s.ws)
    assert spr.sparsepr_paged_error(s.ws) == 1
    mine = s.table[bad][:4 if bad == 0 else 7].long()
    for k, v in before.items():
        assert torch.equal(s.dev[k].cpu().view(torch.int16)[mine], v[mine]), k
    other = 1 - bad
    at, n, length = (40, 21, 100) if other else (0, 40, 64)
    slot = torch.arange(length - n, length)
    pid = s.table[other][slot // 16].long()
    assert torch.equal(s.dev["kp"].cpu()[pid, :, slot % 16], K[at:at + n])
    assert torch.equal(s.dev["vp"].cpu()[pid, :, slot % 16], V[at:at + n])


@pytest.mark.parametrize("dt,big", [(BF, 3e38), (FP, 5.9e4)])
def test_means_of_large_keys(spr, gpu, dt, big):
    """Keys near the end of the type's range: their sum leaves 32 bits, their mean does not."""
    n, d, page = 150, 64, 128
    s = Scene(spr, gpu, [n], [n], Hq=1, Hkv=1, d=d, page=page, dt=dt, seed=91)
    K = (big * (1 + 0.1 * torch.rand(n, 1, d, generator=gen(92)) * torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0))).to(dt)
    K[:, :, 1::4] = -K[:, :, 1::4]
    spr.sparsepr_cache_append(s.p, K.to(gpu), K.to(gpu), *s.seqs(), s.dev["kp"], s.dev["vp"], s.dev["km"], s.ws)
    for j, r in ((0, 128), (1, 22)):
        pid = int(s.table[0, j])
        k = s.dev["kp"][pid, :, :r].cpu().double()
        mean = k.mean(1)
        assert torch.all((s.dev["km"][pid].cpu().double() - mean).abs() <= R.HALF_STEP[dt] * mean.abs() + 128 * E24 * k.abs().mean(1))


def test_append_between_rows_of_no_sequence(spr, gpu):
    """Rows before the first sequence and behind the last one: the pages are those of the call without
    them, whatever they hold."""
    n, front, tail = [40, 1, 0, 9], 37, 300
    kw = dict(Hq=3, Hkv=3, d=64, page=16, dt=BF, seed=94)
    s, t = Scene(spr, gpu, n, [64, 100, 5, 30], **kw), Scene(spr, gpu, n, [64, 100, 5, 30], tail_rows=front + tail, **kw)
    nan = float("nan")
    K, V = (torch.randn(50, 3, 64, generator=gen(95 + i)).to(BF) for i in range(2))
    Kp, Vp = (torch.cat([x.new_full((front, 3, 64), nan), x, x.new_full((tail, 3, 64), nan)]) for x in (K, V))
    for rot in (64, 22):
        for c, k, v, q0 in ((s, K, V, 0), (t, Kp, Vp, front)):
            rp = spr.RopeParams.make(1, 3, c.T, 64, rot_dim=rot)
            pos = torch.full((1, c.T), -1, dtype=torch.int32)
            pos[0, q0:q0 + 50] = torch.arange(50)
            spr.sparsepr_cache_append(c.p, k.to(gpu), v.to(gpu), c.dev["q_start"] + q0, c.dev["kv_len"], c.dev["table"], c.dev["kp"],
                                      c.dev["vp"], c.dev["km"], c.ws, rope=rp, pos=pos.to(gpu), freq=spr.rope_frequencies(rp, gpu))
            assert spr.sparsepr_paged_error(c.ws) == 0
        for m in ("kp", "vp", "km"):
            assert torch.equal(s.dev[m].view(torch.int16), t.dev[m].view(torch.int16)), m


def test_append_offsets_out_of_order(spr, gpu):
    """A sequence that reaches behind the last offset is error 1 and is not written."""
    s = Scene(spr, gpu, [50, 11], [64, 100], Hq=2, Hkv=2, d=64, page=16, dt=BF, seed=96)
    before = {k: s.dev[k].cpu().view(torch.int16).clone() for k in ("kp", "vp", "km")}
    qs = torch.tensor([0, 50, 40], dtype=torch.int32, device=gpu)
    K = torch.randn(61, 2, 64, generator=gen(97)).to(BF).to(gpu)
    spr.sparsepr_cache_append(s.p, K, K, qs, s.dev["kv_len"], s.dev["table"], s.dev["kp"], s.dev["vp"], s.dev["km"], s.ws)
    assert spr.sparsepr_paged_error(s.ws) == 1
    for k, v in before.items():
        assert torch.equal(s.dev[k].cpu().view(torch.int16), v), k


# ---------------------------------------------------------------------------
# Selection, and attention over the lists
# ---------------------------------------------------------------------------
SELECT = [  # new, kv, Hq, Hkv, d, page, dtype, frame, q_block, n_select, n_sink, n_recent
    ([1], [1], 1, 1, 64, 16, BF, 1, 1, 1, 0, 1),
    ([1, 1, 1], [500, 16, 0], 8, 2, 128, 16, BF, 1, 1, 6, 1, 2),
    ([5, 0, 2], [300, 40, 900], 4, 2, 64, 32, FP, 1, 2, 4, 0, 1),
    ([1], [9000], 4, 1, 64, 16, BF, 1, 1, 20, 2, 3),              # several blocks per list
    ([70, 33], [700, 33], 8, 4, 128, 64, BF, 1, 16, 5, 1, 1),
    ([100], [1000], 2, 2, 64, 16, FP, 25, 64, 12, 0, 0),
    ([90], [400], 2, 1, 64, 128, BF, 0, 90, 2, 1, 0),
    ([20], [8], 1, 1, 64, 16, BF, 1, 4, 3, 1, 1),                 # units that see no page
    ([300], [600], 4, 1, 64, 32, BF, 1, 100, 9, 1, 2),            # units of several row parts
    ([3, 3], [90, 200], 16, 1, 64, 16, BF, 1, 2, 4, 1, 1),        # 32 rows per unit
    ([1, 3], [900, 64], 48, 1, 128, 16, FP, 1, 1, 6, 0, 1),       # a token's heads in two items
    ([200, 0, 130], [1500, 10, 900], 8, 4, 128, 64, BF, 1, 4, 6, 1, 1),     # units scored four at a time, across sequences
    ([150, 9, 70], [700, 9, 800], 32, 16, 64, 16, FP, 25, 7, 9, 0, 2),
]


@pytest.mark.parametrize("case,tiles", [(c, False) for c in SELECT] + [(c, True) for c in SELECT if min(c[8], max(c[0])) * c[2] > 32 * c[3]],
                         ids=lambda c: "-".join(str(x) for x in c) if isinstance(c, tuple) else ("tiles" if c else "rows"))
def test_select_and_attend(spr, gpu, case, tiles):
    new, kv, Hq, Hkv, d, page, dt, frame, qb, ns, sink, recent = case
    s = Scene(spr, gpu, new, kv, Hq=Hq, Hkv=Hkv, d=d, page=page, dt=dt, frame=frame, q_block=qb, n_select=ns, n_sink=sink,
              n_recent=recent, seed=21, bump=0.7, tail_rows=2, tiles=tiles)
    sel, cnt = s.select()
    want, wc = R.select(s.Q, new, kv, s.table, s.km, page, frame, qb, ns, sink, recent)
    n = want.shape[0]
    assert torch.equal(cnt.cpu()[:n], wc) and torch.equal(sel.cpu()[:n], want)
    assert torch.all(sel[n:] == -9) and torch.all(cnt[n:] == -9)
    O, z = s.attend(sel, cnt)
    s.check(O, z, sel, cnt)


def test_select_ties_and_nan(spr, gpu):
    """Equal scores go to the lowest pages, -0 equals 0, NaN is the lowest, infinities order."""
    page, d = 16, 64
    s = Scene(spr, gpu, [1], [16 * 400], Hq=1, Hkv=1, d=d, page=page, dt=BF, q_block=1, n_select=30, seed=23)
    s.km.zero_()
    s.Q.zero_()
    s.Q[0, 0, 0] = 1.0
    val = torch.zeros(400)
    val[:] = -1.0
    val[50:250:2] = 0.0
    val[51:250:2] = -0.0
    val[300:310] = 2.0
    val[7] = 3.0
    for j in range(400):
        s.km[int(s.table[0, j]), 0, 0] = val[j]
    s.km[int(s.table[0, 8]), 0, 0] = float("nan")
    s.dev["km"], s.dev["Q"] = s.km.to(gpu), s.Q.to(gpu)
    sel, cnt = s.select()
    assert cnt.item() == 30 and sel[0, 0].tolist() == [7] + list(range(50, 69)) + list(range(300, 310))
    s.p.n_select = 400
    s.ws = spr.paged_workspace(s.p, gpu)
    sel, cnt = s.select()
    assert sel[0, 0].tolist() == list(range(400))
    s.p.n_select = 399
    sel, cnt = s.select()
    assert 8 not in sel[0, 0].tolist() and cnt.item() == 399


@pytest.mark.parametrize("units", [1, 42])       # 42: scored four at a time
@pytest.mark.parametrize("n_pages", [300, 3000])
@pytest.mark.parametrize("kind", ["near", "tied", "tiny", "huge", "inf_query", "inf_mean"])
def test_select_scores_that_32_bits_cannot_order(spr, gpu, kind, n_pages, units):
    """Scores closer than the 32-bit sums are exact, hundreds of equal ones, values at the ends of
    the range, and infinities: the lists are still those of the 64-bit scores."""
    d, page = 64, 16
    g = gen(26)
    s = Scene(spr, gpu, [units], [16 * n_pages], Hq=2, Hkv=2, d=d, page=page, dt=BF, q_block=1, n_select=57, n_sink=1, n_recent=1, seed=27)
    base = torch.randn(2, d, generator=g)
    km = base.expand(s.n_pages, 2, d).clone()
    if kind == "near":        # one small element tells the pages apart
        km[:, :, 5] = 2.0 ** -12 * torch.rand(s.n_pages, 2, generator=g)
    if kind == "tiny":
        km = torch.randn(s.n_pages, 2, d, generator=g) * 1e-36
        s.Q *= 2.0 ** -110
    if kind == "huge":
        km = torch.randn(s.n_pages, 2, d, generator=g) * 1e37
        s.Q *= 50
    if kind in ("inf_query", "inf_mean"):
        km = torch.randn(s.n_pages, 2, d, generator=g)
    s.km = km.to(BF)
    if kind == "inf_query":
        s.Q[0, 1, 3] = float("inf")
    if kind == "inf_mean":
        s.km[torch.randperm(s.n_pages, generator=g)[:n_pages - 20], :, 7] = float("-inf")
    s.dev["km"], s.dev["Q"] = s.km.to(gpu), s.Q.to(gpu)
    sel, cnt = s.select()
    # a page or a query with an element that is not finite has no score: the lowest
    km, Q = s.km.clone(), s.Q.clone()
    km[~torch.isfinite(km).all(-1)] = float("nan")
    Q[~torch.isfinite(Q).all(-1)] = float("nan")
    want, wc = R.select(Q, s.new, s.kv, s.table, km, page, 1, 1, 57, 1, 1)
    assert torch.equal(cnt.cpu(), wc) and torch.equal(sel.cpu(), want)


@pytest.mark.parametrize("Hkv,T", [(1, 1), (160, 1), (16, 4)])
def test_select_many_pages(spr, gpu, Hkv, T):
    """More pages than shared memory holds (scores in the workspace), one block per list or several,
    and units scored together."""
    page, d, npg = 16, 64, 9000
    g = gen(24)
    km = torch.randn(64, Hkv, d, generator=g).to(BF)
    table = torch.randint(0, 64, (1, npg), generator=g).to(torch.int32)     # pages used many times: ties
    p = spr.CacheParams.make(1, Hkv, Hkv, d, page=page, n_pages=64, max_pages=npg, T=T, max_chunk=T, q_block=1,
                             n_select=700, n_sink=2, n_recent=5)
    Q = torch.randn(T, Hkv, d, generator=g).to(BF)
    ws = spr.paged_workspace(p, gpu)
    sel, cnt = spr.alloc_selection(p, gpu)
    spr.sparsepr_page_select(p, Q.to(gpu), torch.tensor([0, T], dtype=torch.int32, device=gpu),
                             torch.tensor([npg * page], dtype=torch.int32, device=gpu), table.to(gpu), km.to(gpu), sel, cnt, ws)
    for h in (0, Hkv - 1):
        want, _ = R.select(Q[:, h:h + 1], [T], [npg * page], table, km[:, h:h + 1], page, 1, 1, 700, 2, 5)
        assert torch.equal(sel[:, h].cpu(), want[:, 0])
    assert torch.all(cnt == 700)


@pytest.mark.parametrize("B,n,Hkv,npg", [
    (1, 240, 16, 9000),         # units scored together, their lists picked in two batches
    (100, 5, 16, 9000),         # batches of units, scores and picks
    (1, 2, 100, 400_000),       # batches of heads
])
def test_select_in_batches(spr, gpu, B, n, Hkv, npg):
    """More lists of more pages than the workspace holds scores and keys for at once, many pages
    with the same mean (ties by the hundred, decided in 64 bits)."""
    page, d, T, K, sink, recent = 16, 64, B * n, 300, 2, 5
    g = gen(98)
    km = torch.randn(64, Hkv, d, generator=g).to(BF)
    table = torch.randint(0, 64, (B, npg), generator=g).to(torch.int32)
    p = spr.CacheParams.make(B, Hkv, Hkv, d, page=page, n_pages=64, max_pages=npg, T=T, max_chunk=n, q_block=1, n_select=K,
                             n_sink=sink, n_recent=recent)
    Q = torch.randn(T, Hkv, d, generator=g).to(BF)
    kv = [npg * page - 700 * (b % 7) for b in range(B)]
    ws = spr.paged_workspace(p, gpu)
    sel, cnt = spr.alloc_selection(p, gpu)
    sel.fill_(-9)
    spr.sparsepr_page_select(p, Q.to(gpu), torch.arange(0, T + 1, n, dtype=torch.int32, device=gpu),
                             torch.tensor(kv, dtype=torch.int32, device=gpu), table.to(gpu), km.to(gpu), sel, cnt, ws)
    assert spr.sparsepr_paged_error(ws) == 0 and torch.all(cnt == K)
    score = torch.einsum("thd,phd->thp", Q.double(), km.double())          # the 64 scores there are
    sel = sel.cpu()
    for t in range(T):
        b, i = divmod(t, n)
        vis = -(-(kv[b] - n + i + 1) // page)
        s = score[t][:, table[b, :vis].long()]
        s[:, :sink] = s[:, vis - recent:] = math.inf
        want = torch.sort(s, dim=-1, descending=True, stable=True).indices[:, :K].sort(-1).values
        assert torch.equal(sel[t].long(), want), t


def test_bad_lists_are_errors(spr, gpu):
    for new, tiles in (([1, 1], False), ([40, 40], False), ([40, 40], True)):
        for what in ("order", "range", "count", "negative", "twice"):
            s = Scene(spr, gpu, new, [300, 300], Hq=2, Hkv=1, d=64, page=16, dt=BF, q_block=40, n_select=6, n_recent=1, seed=25,
                      tiles=tiles)
            sel, cnt = s.select()
            good, _ = s.attend(sel, cnt)
            if what == "order":
                sel[1, 0, 0], sel[1, 0, 1] = sel[1, 0, 1].item(), sel[1, 0, 0].item()
            if what == "range":
                sel[1, 0, 5] = 19
            if what == "negative":
                sel[1, 0, 0] = -1
            if what == "twice":
                sel[1, 0, 4] = sel[1, 0, 5].item()
            if what == "count":
                cnt[1, 0] = 7
            O, _ = s.attend(sel, cnt)
            assert spr.sparsepr_paged_error(s.ws) == 1, what
            assert torch.equal(O[:new[0]], good[:new[0]])
            assert torch.isnan(O[new[0]:sum(new)]).all(), what


@pytest.mark.parametrize("units", [1, 42])       # 42: scored four at a time
@pytest.mark.parametrize("pid", [-2, -1, -2 ** 31, -3, "n_pages"])
def test_select_bad_page_ids_are_errors(spr, gpu, pid, units):
    """Any id out of [0, n_pages) in a visible entry is error 1 and scores lowest."""
    s = Scene(spr, gpu, [units], [16 * 90], Hq=2, Hkv=2, d=64, page=16, dt=BF, q_block=1, n_select=87, seed=93)
    t, km = s.table.clone(), s.km.clone()
    sel, cnt = s.select()
    assert spr.sparsepr_paged_error(s.ws) == 0
    km[int(t[0, 33])] = float("nan")             # the lowest score of the definition
    t[0, 33] = s.n_pages if pid == "n_pages" else pid
    s.dev["table"] = t.to(gpu)
    sel, cnt = s.select()
    assert spr.sparsepr_paged_error(s.ws) == 1
    want, wc = R.select(s.Q, s.new, s.kv, s.table, km, 16, 1, 1, 87, 0, 0)
    assert torch.equal(cnt.cpu(), wc) and torch.equal(sel.cpu(), want)
    assert not torch.any(sel[-1] == 33)


@pytest.mark.parametrize("Hq", [2, 40])
def test_limits_beyond_the_rows_of_the_call(spr, gpu, Hq):
    """A max_chunk and a q_block that no sequence can reach count as T."""
    kw = dict(Hq=Hq, Hkv=1, d=64, page=16, dt=BF, n_select=6, n_recent=1, seed=27)
    s = Scene(spr, gpu, [30], [500], q_block=30, **kw)
    t = Scene(spr, gpu, [30], [500], q_block=2 ** 31 - 1, max_chunk=2 ** 31 - 1, **kw)
    O, z = s.attend()
    s.check(O, z)
    P, y = t.attend()
    assert torch.equal(O, P) and torch.equal(z, y)
    O, z = s.attend(*s.select())
    P, y = t.attend(*t.select())
    assert torch.equal(O, P) and torch.equal(z, y) and spr.sparsepr_paged_error(t.ws) == 0


# ---------------------------------------------------------------------------
# A run of them together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt,sparse,wide", [(BF, False, 0), (BF, False, 450), (FP, True, 0)])
def test_rollout(spr, gpu, dt, sparse, wide):
    """Three frames generated one after another, then single tokens: rotation, append, selection
    and attention through rollout_step, against attention over everything so far in 64 bits."""
    B, Hq, Hkv, d, page, F = 2, 4, 2, 64, 32, 48
    g = gen(31)
    total = 3 * F + 3
    q, k, v = (torch.randn(B, total, h, d, generator=g).to(dt) for h in (Hq, Hkv, Hkv))
    npg = -(-total // page)
    table = torch.randperm(B * npg + 1, generator=g)[:B * npg].reshape(B, npg).to(torch.int32)
    if wide:      # a page table for much longer sequences: the frames go to the tensor tiles
        table = torch.cat([table, torch.full((B, wide - npg), 2 ** 31 - 1, dtype=torch.int32)], 1)
    cache = None
    fr = R.rope_freqs([24, 20, 20])
    grid = torch.stack([torch.arange(total) // F, torch.arange(total) % F // 8, torch.arange(total) % 8]).to(torch.int32)
    at = 0
    for n in (F, F, F, 1, 1, 1):
        p = spr.CacheParams.make(B, Hq, Hkv, d, dtype=dt, page=page, n_pages=B * npg + 1, max_pages=wide or npg, T=B * n, max_chunk=n,
                                 frame=F, q_block=16 if sparse else 0, n_select=3 if sparse else 0, n_recent=1 if sparse else 0)
        if cache is None:
            cache = spr.alloc_cache(p, gpu)
        rq = spr.RopeParams.make(1, Hq, B * n, d, dtype=dt, layout="interleaved", axis_dim=[24, 20, 20])
        freq = spr.rope_frequencies(rq, gpu)
        new = slice(at, at + n)
        Q = q[:, new].reshape(B * n, Hq, d).to(gpu)
        K, V = (t[:, new].reshape(B * n, Hkv, d).to(gpu) for t in (k, v))
        pos = grid[:, new].repeat(1, B).contiguous().to(gpu)
        Qh = Q.transpose(0, 1).unsqueeze(0)                # [1, Hq, T, d] view
        spr.sparsepr_rope(rq, Qh, pos, freq, Qh)           # in place
        ws = spr.paged_workspace(p, gpu)
        O = torch.empty(B * n, Hq, d, dtype=dt, device=gpu)
        at += n
        seqs = (torch.arange(0, B * n + 1, n, dtype=torch.int32, device=gpu),
                torch.full((B,), at, dtype=torch.int32, device=gpu), table.to(gpu))
        selection = spr.alloc_selection(p, gpu) if sparse else None
        spr.rollout_step(p, cache, Q, K, V, *seqs, O, ws, rope=rq, pos=pos, freq=freq, selection=selection)
        assert spr.sparsepr_paged_error(ws) == 0
        # rotated queries and keys in 64 bits, rounded as stored
        qr = R.rope(q[:, new].double().transpose(1, 2), grid[:, new], d, "interleaved", fr).to(dt)
        kr = R.rope(k[:, :at].double().transpose(1, 2), grid[:, :at], d, "interleaved", fr).to(dt)
        for b in range(B):
            for h in range(Hq):
                for i in range(n):
                    x = kr[b, h // 2].double() @ qr[b, h, i].double() / math.sqrt(d)
                    pos_i = at - n + i
                    seen = torch.arange(at) < min(at, (pos_i // F + 1) * F)
                    if sparse:
                        u = b * -(-n // 16) + i // 16
                        lst = selection[0][u, h // 2].cpu()
                        seen &= torch.isin(torch.arange(at) // page, lst[lst >= 0])
                        assert (lst[lst >= 0] == (min(at, (pos_i // F + 1) * F) - 1) // page).any()
                    x[~seen] = -math.inf
                    w = torch.softmax(x, 0)
                    vv = v[b, :at, h // 2].double()
                    ref, A, E = w @ vv, w @ vv.abs(), (kr[b, h // 2].double().abs() @ qr[b, h, i].double().abs()).max() / 8
                    u_ = R.HALF_STEP[dt]
                    # the device's rotated rows may differ by one rounding step from the rounded 64-bit
                    # ones where the 32-bit result crosses a border: 2 u of a logit's terms, on few of them
                    tol = u_ * ref.abs() + A * (u_ + 2 * u_ * E * 0.25 + 2.0 ** -15)
                    assert torch.all((O[b * n + i, h].cpu().double() - ref).abs() <= tol)


@pytest.mark.parametrize("wide", [False, True])
def test_agrees_with_the_dense_frame_causal_call(spr, gpu, wide):
    """The last frame of a frame-causal dense call equals the chunk over the cache of all frames."""
    H, d, F, frames, page = 2, 64, 96, 3, 32
    N = F * frames
    g = gen(33)
    Q, K, V = (torch.randn(1, H, N, d, generator=g).to(BF).to(gpu) for _ in range(3))
    fid = (torch.arange(N, dtype=torch.int32) // F).to(gpu)
    dp = spr.Params.make(1, H, N, d, block=64, density=1.0, n_kgroups=4, n_qgroups=4, n_samples=64, n_probes=8, eig_rank=16,
                         sub_rank=8, kmeans_iters=1, frame_id=fid, n_frames=frames)
    O, lse = torch.empty_like(Q), torch.empty(H, N, device=gpu)
    spr.sparsepr_dense_attention(dp, Q, K, V, O, lse, torch.zeros(512, dtype=torch.uint8, device=gpu))
    mp = 900 if wide else N // page         # wide: to the tensor tiles
    p = spr.CacheParams.make(1, H, H, d, page=page, n_pages=N // page, max_pages=mp, T=F, max_chunk=F, frame=F)
    order = torch.randperm(N // page, generator=g).to(gpu)
    pages = {n: torch.empty(N // page, H, page, d, dtype=BF, device=gpu) for n in "kv"}
    for n, t in (("k", K), ("v", V)):
        pages[n][order] = t[0].reshape(H, N // page, page, d).transpose(0, 1)
    ws = spr.paged_workspace(p, gpu)
    table = torch.zeros(1, mp, dtype=torch.int32, device=gpu)
    table[0, :N // page] = order
    q = Q[0, :, N - F:].transpose(0, 1)
    o, z = torch.empty(F, H, d, dtype=BF, device=gpu), torch.empty(F, H, device=gpu)
    spr.sparsepr_paged_attention(p, q, torch.tensor([0, F], dtype=torch.int32, device=gpu),
                                 torch.tensor([N], dtype=torch.int32, device=gpu), table,
                                 pages["k"], pages["v"], o, z, ws)
    want = O[0, :, N - F:].transpose(0, 1).float()
    # each side within u |o| + u A of the exact value, A <= max |v| < 5
    assert torch.all((o.float() - want).abs() <= 2 * 2.0 ** -8 * (want.abs() + 1.2))
    assert torch.all((z - lse[:, N - F:].T).abs() <= 2.0 ** -12)


def test_graphs_and_streams(spr, gpu):
    """Captured steps replay on new inputs; graphs with a workspace each run at once."""
    scenes = [Scene(spr, gpu, [1, 1], [900, 400], Hq=4, Hkv=2, d=64, page=16, dt=BF, q_block=1, n_select=8, n_recent=2, seed=41),
              Scene(spr, gpu, [40], [700], Hq=2, Hkv=1, d=64, page=32, dt=BF, q_block=40, n_select=8, n_recent=2, seed=42),
              Scene(spr, gpu, [40], [700], Hq=2, Hkv=1, d=64, page=32, dt=BF, q_block=40, n_select=8, n_recent=2, seed=44,
                    tiles=True)]
    graphs = []
    for s in scenes:
        sel, cnt = spr.alloc_selection(s.p, gpu)
        O = torch.zeros_like(s.dev["Q"])
        z = torch.zeros(s.T, s.p.Hq, device=gpu)
        K = torch.randn(s.T, s.p.Hkv, 64, generator=gen(43)).to(BF).to(gpu)
        rp = spr.RopeParams.make(1, s.p.Hkv, s.T, 64)
        freq = spr.rope_frequencies(rp, gpu)
        pos = torch.zeros(1, s.T, dtype=torch.int32, device=gpu)
        cache = dict(k_pages=s.dev["kp"], v_pages=s.dev["vp"], k_mean=s.dev["km"])
        step = lambda s=s, c=cache, K=K, O=O, z=z, rp=rp, pos=pos, freq=freq, sel=sel, cnt=cnt: spr.rollout_step(
            s.p, c, s.dev["Q"], K, K, *s.seqs(), O, s.ws, rope=rp, pos=pos, freq=freq, selection=(sel, cnt), lse=z)
        step()
        torch.cuda.synchronize()
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            step()
        graphs.append((gph, step, O, z))
    for i in range(3):
        want = []
        for s, (gph, step, O, z) in zip(scenes, graphs):
            s.dev["Q"].copy_(torch.randn(s.Q.shape, generator=gen(50 + i)).to(BF))
            O.fill_(9.0)
            z.fill_(9.0)
            step()
            want.append((O.clone(), z.clone()))
            O.fill_(9.0)
            z.fill_(9.0)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(5):
            for st, (gph, *_r) in zip(streams, graphs):
                with torch.cuda.stream(st):
                    gph.replay()
        torch.cuda.synchronize()
        for (O, z), (_, _, go, gz) in zip(want, graphs):
            assert torch.equal(O, go) and torch.equal(z, gz)
    for s in scenes:
        assert spr.sparsepr_paged_error(s.ws) == 0


def test_repeat_is_bitwise_equal(spr, gpu):
    for new, kv, tiles in (([1], [9000], False), ([60], [3000], False), ([60], [3000], True)):
        s = Scene(spr, gpu, new, kv, Hq=4, Hkv=1, d=128, page=64, dt=BF, seed=61, tiles=tiles)
        O, z = s.attend()
        for _ in range(5):
            O2, z2 = s.attend()
            assert torch.equal(O, O2) and torch.equal(z, z2)

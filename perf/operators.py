"""Cases of the paged-cache operators: rotary positions, cache append, attention of a chunk over a
paged cache, and page selection with the attention restricted to the selected pages.

`own` chooses between the plain torch form of every operator and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _rope(name, op, B, H, H2, N, d, rot, layout, axes, dtype, scaling="none", factor=1.0, orig=0, grid=""):
    """axes: rotated widths of the position axes, "a+b+c"; grid: "t x h x w" of a video latent or
    "" for text-like positions."""
    return dict(name=name, op=op, B=B, H=H, H2=H2, N=N, d=d, rot=rot, layout=layout, axes=axes, dtype=dtype,
                scaling=scaling, factor=factor, orig=orig, grid=grid)


def _cache(name, op, B, Hq, Hkv, d, page, dtype, new_lo, new_hi, len_lo, len_hi, frame, q_block=0, n_select=0,
           n_sink=0, n_recent=0):
    """new_lo..new_hi: new tokens of each sequence; len_lo..len_hi: its cached tokens, the new ones
    included; frame: tokens per frame of the mask (1 = token-causal, 0 = everything visible)."""
    return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype, new_lo=new_lo, new_hi=new_hi,
                len_lo=len_lo, len_hi=len_hi, frame=frame, q_block=q_block, n_select=n_select, n_sink=n_sink,
                n_recent=n_recent)


def listed():
    return [
        # queries and keys of one layer of the 32,760-token, 40-head video call, rotated over (t, h, w)
        _rope("rope_video", "rope", 1, 40, 40, 32760, 128, 128, "interleaved", "44+42+42", "bf16", grid="21x30x52"),
        # gradient in a training step: part of the head, half layout, frequencies scaled by parts
        _rope("rope_grad", "rope_grad", 2, 32, 8, 5003, 128, 64, "half", "64", "fp32", "parts", 8.0, 4096),
        # one token of each of 64 sequences: the smallest call, latency only
        _rope("rope_tokens", "rope", 64, 32, 8, 1, 128, 128, "half", "128", "fp16", "linear", 4.0),
        # one new token of each sequence goes into its page, its key rotated on the way
        _cache("append_tokens", "append", 64, 8, 8, 128, 64, "bf16", 1, 1, 200, 3000, 1),
        # one frame of 32 x 32 tokens of four rollouts
        _cache("append_frame", "append", 4, 16, 16, 128, 128, "bf16", 1024, 1024, 4096, 16384, 1024),
        # one sequence, one token, a short cache: latency of a serving step
        _cache("token_one", "attend", 1, 32, 8, 128, 64, "bf16", 1, 1, 4097, 4097, 1),
        # a serving batch of ragged lengths
        _cache("tokens_ragged", "attend", 48, 32, 8, 128, 64, "bf16", 1, 1, 500, 32000, 1),
        # the last frame of four frame-causal rollouts of 16 frames of 1024 tokens
        _cache("chunk_frame", "attend", 4, 16, 16, 128, 128, "bf16", 1024, 1024, 16384, 16384, 1024),
        # ragged chunks of a mixed batch, some of them short; odd lengths
        _cache("chunk_ragged", "attend", 6, 16, 4, 64, 32, "fp16", 3, 2051, 2100, 9973, 1),
        # three new latent frames of the 40-head video call over the 21-frame cache
        _cache("chunk_video", "attend", 1, 40, 40, 128, 64, "bf16", 4680, 4680, 32760, 32760, 1560),
        # one token over long caches, 64 pages of up to 1000 read
        _cache("select_tokens", "sparse", 32, 32, 8, 128, 64, "bf16", 1, 1, 8000, 65536, 1, 1, 64, 1, 2),
        # a chunk over a long cache, 64 pages for each block of 64 tokens
        _cache("select_chunk", "sparse", 1, 32, 8, 128, 64, "bf16", 2048, 2048, 65536, 65536, 1, 64, 64, 1, 3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "append", "attend", "attend", "attend", "sparse", "sparse"])
    if kind == "rope":
        op = rng.choice(["rope", "rope_grad"])
        d = rng.choice([64, 128])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        B, H = rng.choice([1, 2, 4, 64]), rng.choice([8, 16, 24, 32, 40])
        H2 = rng.choice([0, H, max(1, H // 4)])
        N = 1 if B == 64 else _log(rng, 64, 8000)
        if rng.random() < 0.4 and N > 1:
            t, h = rng.randint(2, 16), rng.randint(3, 20)
            w = max(1, N // (t * h))
            axes = "44+42+42" if d == 128 else "24+20+20"
            return _rope(None, op, B, H, H2, t * h * w, d, d, rng.choice(["interleaved", "half"]), axes, dtype,
                         grid=f"{t}x{h}x{w}") | dict(name="drawn")
        rot = rng.choice([d, d // 2, d * 3 // 4, 22])
        sc = rng.choice(["none", "linear", "base", "parts"])
        return _rope("drawn", op, B, H, H2, N, d, rot, rng.choice(["interleaved", "half"]), str(rot), dtype, sc,
                     1.0 if sc == "none" else rng.choice([2.0, 4.0, 8.0]), 4096 if sc == "parts" else 0)
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv <= 8 else [1, 2])
    if kind == "append":
        B = rng.randint(1, 32)
        n = rng.choice([1, 1, _log(rng, 2, 1024)])
        return _cache("drawn", "append", B, Hkv, Hkv, d, page, dtype, max(1, n // 2), n, n + 1, n + _log(rng, 64, 6000), 1)
    if kind == "attend":
        if rng.random() < 0.5:      # serving: one or a few tokens of each sequence
            B, n = rng.randint(1, 40), rng.choice([1, 1, 1, rng.randint(2, 9)])
            hi = _log(rng, 300, 30000)
            return _cache("drawn", "attend", B, Hq, Hkv, d, page, dtype, 1, n, max(n, hi // 4), hi, rng.choice([0, 1, 1]))
        B = rng.randint(1, 4)
        n = _log(rng, 20, 3000)
        hi = n + _log(rng, 100, 16000)
        frame = rng.choice([0, 1, 1, rng.randint(16, 1600)])
        return _cache("drawn", "attend", B, Hq, Hkv, d, page, dtype, max(1, n // 3), n, n + (hi - n) // 2, hi, frame)
    n_sel = rng.choice([5, 16, 33, 64])
    hi = _log(rng, 4000, 50000)
    if rng.random() < 0.5:
        B = rng.randint(1, 24)
        return _cache("drawn", "sparse", B, Hq, Hkv, d, page, dtype, 1, 1, hi // 3, hi, 1, 1, n_sel, rng.randint(0, 2),
                      rng.randint(1, 3))
    q_block = rng.choice([16, 64, 128])
    n = _log(rng, 30, 2000)
    return _cache("drawn", "sparse", rng.randint(1, 2), Hq, Hkv, d, page, dtype, max(1, n // 2), n, n + hi // 2, n + hi,
                  rng.choice([1, 256]), q_block, n_sel, rng.randint(0, 2), rng.randint(1, 3))


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n sizes between lo and hi, the ends among them, in a fixed shuffled order."""
    if n == 1:
        return [hi]
    v = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    return [v[(i * 7 + 3) % n] for i in range(n)] if n % 7 else v


def _lengths(case):
    new = _spread(case["new_lo"], case["new_hi"], case["B"])
    kv = _spread(case["len_lo"], case["len_hi"], case["B"])[::-1]
    return new, [max(n, k) for n, k in zip(new, kv)]


def _positions(case, gen):
    """int32 [axes, B, N]: a video latent's (t, h, w), or running positions at an offset of each row."""
    B, N = case["B"], case["N"]
    if case["grid"]:
        t, h, w = (int(x) for x in case["grid"].split("x"))
        g = torch.stack(torch.meshgrid(torch.arange(t), torch.arange(h), torch.arange(w), indexing="ij"))
        return g.reshape(3, 1, N).expand(3, B, N).to(torch.int32).contiguous()
    off = torch.randint(0, 100000, (B, 1), generator=gen)
    return (off + torch.arange(N)).reshape(1, B, N).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dev = torch.device("cuda", torch.cuda.current_device())
    rnd = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    d = case["d"]
    if case["op"] in ("rope", "rope_grad"):
        B, N = case["B"], case["N"]
        heads = [case["H"]] + ([case["H2"]] if case["H2"] else [])
        s = dict(case=case, pos=_positions(case, gen).to(dev),
                 x=[torch.randn(B, h, N, d, generator=rnd, device=dev).to(dt) for h in heads])
        if own:
            import free_block_sparse_rcp_b200 as spr
            axes = [int(a) for a in case["axes"].split("+")]
            p = spr.RopeParams.make(B, case["H"], N, d, H2=case["H2"], dtype=dt, rot_dim=case["rot"],
                                    layout=case["layout"], axis_dim=axes, scaling=case["scaling"],
                                    factor=case["factor"], orig_len=case["orig"], pos_batched=1)
            s.update(p=p, freq=spr.rope_frequencies(p, dev), y=[torch.empty_like(x) for x in s["x"]])
        return s
    B, Hq, Hkv, page = case["B"], case["Hq"], case["Hkv"], case["page"]
    new, kv = _lengths(case)
    T = sum(new)
    pages = [-(-k // page) for k in kv]
    n_pages, max_pages = sum(pages) + 3, max(pages)
    order = torch.randperm(n_pages, generator=gen)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]].to(torch.int32)
        at += pages[b]
    # keys share a direction within a page (neighbouring tokens of a video look alike)
    k_pages = torch.randn(n_pages, Hkv, page, d, generator=rnd, device=dev).to(dt)
    k_pages += torch.randn(n_pages, Hkv, 1, d, generator=rnd, device=dev).to(dt)
    v_pages = torch.randn(n_pages, Hkv, page, d, generator=rnd, device=dev).to(dt)
    s = dict(case=case, new=new, kv=kv, T=T, table_host=table, table=table.to(dev),
             q_start=torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).to(dev),
             kv_len=torch.tensor(kv, dtype=torch.int32).to(dev), k_pages=k_pages, v_pages=v_pages)
    # mean key of every page (rows past a sequence's end are not counted)
    mean = k_pages.float().mean(2)
    for b in range(B):
        r = kv[b] % page
        if r:
            pg = int(table[b, pages[b] - 1])
            mean[pg] = k_pages[pg, :, :r].float().mean(1)
    s["k_mean"] = mean.to(dt)
    if case["op"] == "append":
        s["K"] = torch.randn(T, Hkv, d, generator=rnd, device=dev).to(dt)
        s["V"] = torch.randn(T, Hkv, d, generator=rnd, device=dev).to(dt)
        s["pos"] = torch.cat([torch.arange(k - n, k) for n, k in zip(new, kv)]).to(torch.int32).reshape(1, T).to(dev)
    else:
        s["Q"] = torch.randn(T, Hq, d, generator=rnd, device=dev).to(dt)
    if own:
        import free_block_sparse_rcp_b200 as spr
        p = spr.CacheParams.make(B, Hq, Hkv, d, dtype=dt, page=page, n_pages=n_pages, max_pages=max_pages, T=T,
                                 max_chunk=max(new), frame=case["frame"], q_block=case["q_block"],
                                 n_select=case["n_select"], n_sink=case["n_sink"], n_recent=case["n_recent"])
        s.update(p=p, ws=spr.paged_workspace(p, dev))
        if case["op"] == "append":
            rp = spr.RopeParams.make(1, Hkv, T, d, dtype=dt, rot_dim=d, layout="half", axis_dim=[d])
            s.update(rope=rp, freq=spr.rope_frequencies(rp, dev))
        else:
            s.update(O=torch.empty_like(s["Q"]), lse=torch.empty(T, Hq, dtype=torch.float32, device=dev))
        if case["op"] == "sparse":
            s["sel"], s["count"] = spr.alloc_selection(p, dev)
            s["units"] = sum(-(-n // case["q_block"]) for n in new)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _frequencies(case):
    """Angle per position of every pair, the pair's axis, and the magnitude, in 64 bits."""
    f, ax, mag = [], [], 1.0
    theta, factor = 10000.0, case["factor"]
    for a, dim in enumerate(int(x) for x in case["axes"].split("+")):
        for j in range(dim // 2):
            base = theta
            if case["scaling"] == "base":
                base = theta * factor ** (dim / (dim - 2.0))
            w = base ** (-2.0 * j / dim)
            if case["scaling"] == "linear":
                w /= factor
            elif case["scaling"] == "parts":
                # turns within the original length: 32 or more keep the frequency, 1 or fewer divide it
                def at(turns):
                    return dim * math.log(case["orig"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
                lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), dim // 2 - 1)
                ramp = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                w = w * (1.0 - ramp) + (w / factor) * ramp
                mag = 0.1 * math.log(factor) + 1.0
            f.append(w)
            ax.append(a)
    return f, ax, mag


def _rotate(x, pos, case, sign):
    """x [B, H, N, d], pos [axes, B, N]."""
    f, ax, mag = _frequencies(case)
    f = torch.tensor(f, dtype=torch.float64, device=x.device)
    ang = pos[torch.tensor(ax, device=x.device)].permute(1, 2, 0).double() * f        # [B, N, pairs]
    c = (torch.cos(ang) * mag).float().unsqueeze(1)
    s = (torch.sin(ang) * (mag * sign)).float().unsqueeze(1)
    rot = case["rot"]
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _gather(pages, ids):
    """Rows of the pages `ids` in order, fp32 [Hkv, rows, d]."""
    g = pages[ids.long()]
    return g.transpose(0, 1).reshape(g.shape[1], -1, g.shape[3]).float()


def _softmax_av(q, k, v, mask, scale):
    """q [n, h, d] on keys [m, d]: the rows' softmax over the keys where mask [n, m]."""
    s = torch.einsum("nhd,md->nhm", q, k) * scale
    s = s.masked_fill(~mask[:, None, :], -math.inf)
    mx = s.amax(-1, keepdim=True)
    mx = torch.where(mx == -math.inf, torch.zeros_like(mx), mx)
    e = torch.exp(s - mx)
    den = e.sum(-1, keepdim=True)
    o = torch.einsum("nhm,md->nhd", e, v) / torch.where(den > 0, den, torch.ones_like(den))
    return o, (mx + torch.log(den)).squeeze(-1)


def _visible_end(pos, frame, length):
    """Keys [0, end) that the query at `pos` sees."""
    if frame == 0:
        return torch.full_like(pos, length)
    return torch.clamp((torch.div(pos, frame, rounding_mode="floor") + 1) * frame, max=length)


def _attend_plain(s, sel=None, count=None):
    case = s["case"]
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(case["d"])
    Q = s["Q"]
    O = torch.empty_like(Q)
    lse = torch.empty(Q.shape[0], Hq, dtype=torch.float32, device=Q.device)
    at, unit = 0, 0
    for b, (n, length) in enumerate(zip(s["new"], s["kv"])):
        ids = s["table"][b, :-(-length // page)]
        pos = torch.arange(length - n, length, device=Q.device)
        end = _visible_end(pos, case["frame"], length)
        if sel is None:
            k, v = _gather(s["k_pages"], ids), _gather(s["v_pages"], ids)
            mask = torch.arange(k.shape[1], device=Q.device)[None, :] < end[:, None]
            for h in range(Hkv):
                o, l = _softmax_av(Q[at:at + n, h * G:(h + 1) * G].float(), k[h], v[h], mask, scale)
                O[at:at + n, h * G:(h + 1) * G] = o.to(Q.dtype)
                lse[at:at + n, h * G:(h + 1) * G] = l
        else:
            qb = case["q_block"]
            cols = torch.arange(page, device=Q.device)
            for u in range(-(-n // qb)):
                i0, i1 = u * qb, min((u + 1) * qb, n)
                rows = slice(at + i0, at + i1)
                for h in range(Hkv):
                    lst = sel[unit + u, h]
                    lst = torch.where(lst < 0, torch.zeros_like(lst), lst).long()
                    used = torch.arange(lst.numel(), device=Q.device) < count[unit + u, h]
                    pg = ids[lst].long()
                    k = s["k_pages"][pg, h].float().reshape(-1, case["d"])
                    v = s["v_pages"][pg, h].float().reshape(-1, case["d"])
                    kpos = (lst[:, None] * page + cols).reshape(-1)
                    mask = (kpos[None, :] < end[i0:i1, None]) & used.repeat_interleave(page)[None, :]
                    o, l = _softmax_av(Q[rows, h * G:(h + 1) * G].float(), k, v, mask, scale)
                    O[rows, h * G:(h + 1) * G] = o.to(Q.dtype)
                    lse[rows, h * G:(h + 1) * G] = l
            unit += -(-n // qb)
        at += n
    return O, lse


def _select_plain(s):
    """Pages of every (block of queries, key head): mean query times mean key of each page in 64 bits
    (whole numbers come out of a comparison), the first and last pages kept, ties to the lowest page."""
    case = s["case"]
    Hq, Hkv, page, K = case["Hq"], case["Hkv"], case["page"], case["n_select"]
    qb, d = case["q_block"], case["d"]
    sels, counts = [], []
    at = 0
    for b, (n, length) in enumerate(zip(s["new"], s["kv"])):
        npg = -(-length // page)
        means = s["k_mean"][s["table"][b, :npg].long()].double()              # [npg, Hkv, d]
        nu = -(-n // qb)
        # mean query of every block
        q = s["Q"][at:at + n].double().reshape(n, Hkv, Hq // Hkv, d).sum(2)
        q = torch.cat([q, q.new_zeros(nu * qb - n, Hkv, d)]).reshape(nu, qb, Hkv, d).sum(1)
        cnt = torch.full((nu,), float(qb), dtype=torch.float64, device=q.device)
        cnt[-1] = n - (nu - 1) * qb
        q = q / (cnt * (Hq // Hkv))[:, None, None]
        score = torch.einsum("uhd,phd->uhp", q, means)
        last = torch.clamp((torch.arange(nu, device=q.device) + 1) * qb, max=n) - 1 + (length - n)
        vis = torch.div(_visible_end(last, case["frame"], length) + page - 1, page, rounding_mode="floor")  # pages seen
        p = torch.arange(npg, device=q.device)
        seen = (p[None, :] < vis[:, None])[:, None, :]
        keep = ((p[None, :] < case["n_sink"]) | (p[None, :] >= vis[:, None] - case["n_recent"]))[:, None, :] & seen
        score = torch.where(keep, torch.full_like(score, math.inf), torch.where(seen, score, -math.inf))
        order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :K]
        c = torch.clamp(vis, max=K)[:, None].expand(nu, Hkv).to(torch.int32)
        if order.shape[-1] < K:
            order = torch.cat([order, order.new_full((nu, Hkv, K - order.shape[-1]), npg)], -1)
        order = torch.where(torch.arange(K, device=q.device) < c[..., None], order, torch.full_like(order, 1 << 40))
        order = torch.sort(order, dim=-1).values
        sels.append(torch.where(order >= (1 << 40), torch.full_like(order, -1), order).to(torch.int32))
        counts.append(c)
        at += n
    return torch.cat(sels), torch.cat(counts)


def _append_plain(s):
    case = s["case"]
    page, d = case["page"], case["d"]
    K = s["K"].permute(1, 0, 2).unsqueeze(0)
    rc = dict(rot=d, layout="half", axes=str(d), scaling="none", factor=1.0, orig=0)
    K = _rotate(K, s["pos"].unsqueeze(1), rc, 1.0)[0].permute(1, 0, 2)
    at = 0
    for b, (n, length) in enumerate(zip(s["new"], s["kv"])):
        slot = torch.arange(length - n, length, device=K.device)
        pg = s["table"][b][torch.div(slot, page, rounding_mode="floor")].long()
        s["k_pages"][pg, :, slot % page] = K[at:at + n]
        s["v_pages"][pg, :, slot % page] = s["V"][at:at + n]
        for j in range((length - n) // page, (length - 1) // page + 1):
            rows = min(page, length - j * page)
            p = int(s["table_host"][b, j])
            s["k_mean"][p] = s["k_pages"][p, :, :rows].float().mean(1).to(K.dtype)
        at += n
    return s["k_pages"], s["v_pages"], s["k_mean"]


# ---------------------------------------------------------------------------
def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import free_block_sparse_rcp_b200 as spr
        if op in ("rope", "rope_grad"):
            call = spr.sparsepr_rope if op == "rope" else spr.sparsepr_rope_backward
            call(s["p"], s["x"][0], s["pos"], s["freq"], s["y"][0], *([s["x"][1], s["y"][1]] if len(s["x"]) > 1 else []))
            return s["y"]
        if op == "append":
            spr.sparsepr_cache_append(s["p"], s["K"], s["V"], s["q_start"], s["kv_len"], s["table"], s["k_pages"],
                                      s["v_pages"], s["k_mean"], s["ws"], rope=s["rope"], pos=s["pos"], freq=s["freq"])
            return s["k_pages"], s["v_pages"], s["k_mean"]
        if op == "attend":
            spr.sparsepr_paged_attention(s["p"], s["Q"], s["q_start"], s["kv_len"], s["table"], s["k_pages"],
                                         s["v_pages"], s["O"], s["lse"], s["ws"])
            return s["O"], s["lse"]
        spr.sparsepr_page_select(s["p"], s["Q"], s["q_start"], s["kv_len"], s["table"], s["k_mean"], s["sel"],
                                 s["count"], s["ws"])
        spr.sparsepr_paged_attention(s["p"], s["Q"], s["q_start"], s["kv_len"], s["table"], s["k_pages"], s["v_pages"],
                                     s["O"], s["lse"], s["ws"], sel=s["sel"], sel_count=s["count"])
        return s["O"], s["lse"], s["sel"][:s["units"]], s["count"][:s["units"]]
    if op in ("rope", "rope_grad"):
        return [_rotate(x, s["pos"], case, 1.0 if op == "rope" else -1.0) for x in s["x"]]
    if op == "append":
        return _append_plain(s)
    if op == "attend":
        return _attend_plain(s)
    sel, count = _select_plain(s)
    O, lse = _attend_plain(s, sel, count)
    return O, lse, sel, count


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotate(x, pos, case, sign):
    """Every pair as a complex number times its unit (and the magnitude)."""
    f, ax, mag = _frequencies(case)
    half = case["rot"] // 2
    lo = np.arange(half) if case["layout"] == "half" else np.arange(half) * 2
    hi = lo + half if case["layout"] == "half" else lo + 1
    y = x.double()
    out = torch.empty_like(y)
    out[..., case["rot"]:] = y[..., case["rot"]:]
    for i in range(half):
        ang = (sign * f[i]) * pos[ax[i]].double().unsqueeze(1)
        u = torch.complex(torch.cos(ang), torch.sin(ang)) * mag
        z = torch.complex(y[..., int(lo[i])], y[..., int(hi[i])]) * u
        out[..., int(lo[i])] = z.real
        out[..., int(hi[i])] = z.imag
    return out


def _exact_select(s, b, at, n, length):
    """Lists of one sequence, block by block: the kept pages, then the best scores one after another."""
    case = s["case"]
    page, qb, G, want = case["page"], case["q_block"], case["Hq"] // case["Hkv"], case["n_select"]
    nu = -(-n // qb)
    sel = np.full((nu, case["Hkv"], want), -1, dtype=np.int32)
    cnt = np.zeros((nu, case["Hkv"]), dtype=np.int32)
    ids = s["table"][b, :-(-length // page)].long()
    means = s["k_mean"][ids].double()
    for u in range(nu):
        q = s["Q"][at + u * qb:at + min((u + 1) * qb, n)].double()
        last = length - n + min((u + 1) * qb, n) - 1
        end = length if case["frame"] == 0 else min(length, (last // case["frame"] + 1) * case["frame"])
        vis = -(-end // page)
        qm = q.reshape(q.shape[0], case["Hkv"], G, -1).mean((0, 2))
        score = (means[:vis] * qm).sum(-1).cpu().numpy()                       # [vis, Hkv]
        fixed = [j for j in range(vis) if j < case["n_sink"] or j >= vis - case["n_recent"]]
        free = np.array([j for j in range(vis) if not (j < case["n_sink"] or j >= vis - case["n_recent"])], dtype=int)
        for h in range(case["Hkv"]):
            best = free[np.lexsort((free, -score[free, h]))] if len(free) else free
            chosen = sorted((fixed + list(best))[:min(want, vis)])
            sel[u, h, :len(chosen)] = chosen
            cnt[u, h] = len(chosen)
    return sel, cnt


def _exact_attend(s, sels=None):
    """Row blocks of one head at a time, keys picked by position, log-sum-exp by its definition."""
    case = s["case"]
    page, G = case["page"], case["Hq"] // case["Hkv"]
    Q = s["Q"].double()
    O = torch.zeros_like(Q)
    L = torch.full(Q.shape[:2], -math.inf, dtype=torch.float64, device=Q.device)
    at = 0
    for b, (n, length) in enumerate(zip(s["new"], s["kv"])):
        j = torch.arange(length, device=Q.device)
        pg = s["table"][b].long()[j // page]
        step = 2048 if sels is None else case["q_block"]
        for h in range(case["Hkv"]):
            k_all = s["k_pages"][pg, h, j % page].double()
            v_all = s["v_pages"][pg, h, j % page].double()
            for i0 in range(0, n, step):
                i1 = min(i0 + step, n)
                key, k, v = j, k_all, v_all
                if sels is not None:
                    sel, cnt = sels[b]
                    u = i0 // step
                    lst = torch.from_numpy(sel[u, h, :cnt[u, h]].astype(np.int64)).to(Q.device)
                    key = (lst[:, None] * page + torch.arange(page, device=Q.device)).flatten()
                    key = key[key < length]
                    k, v = k_all[key], v_all[key]
                pos = torch.arange(length - n + i0, length - n + i1, device=Q.device)
                if case["frame"]:
                    hidden = (key[None, :] // case["frame"]) > (pos[:, None] // case["frame"])
                else:
                    hidden = torch.zeros(len(pos), len(key), dtype=torch.bool, device=Q.device)
                for g in range(G):
                    x = (Q[at + i0:at + i1, h * G + g] @ k.T) / math.sqrt(case["d"])
                    x[hidden] = -math.inf
                    z = torch.logsumexp(x, -1)
                    L[at + i0:at + i1, h * G + g] = z
                    w = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
                    O[at + i0:at + i1, h * G + g] = w @ v
        at += n
    return O, L


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "rope_grad"):
        return [_exact_rotate(x, s["pos"], case, 1.0 if op == "rope" else -1.0) for x in s["x"]]
    if op == "append":
        page = case["page"]
        rc = dict(rot=case["d"], layout="half", axes=str(case["d"]), scaling="none", factor=1.0, orig=0)
        K = _exact_rotate(s["K"].permute(1, 0, 2).unsqueeze(0), s["pos"].unsqueeze(1), rc, 1.0)[0].permute(1, 0, 2)
        kp, vp, km = s["k_pages"].double(), s["v_pages"].double(), s["k_mean"].double()
        at = 0
        for b, (n, length) in enumerate(zip(s["new"], s["kv"])):
            done = 0
            while done < n:
                slot = length - n + done
                p, r = int(s["table_host"][b, slot // page]), slot % page
                m = min(page - r, n - done)
                kp[p, :, r:r + m] = K[at + done:at + done + m].transpose(0, 1)
                vp[p, :, r:r + m] = s["V"][at + done:at + done + m].double().transpose(0, 1)
                # the mean is taken of the keys as the page holds them
                km[p] = kp[p, :, :r + m].to(s["k_pages"].dtype).double().sum(1) / (r + m)
                done += m
            at += n
        return kp, vp, km
    if op == "attend":
        return _exact_attend(s)
    new, kv = s["new"], s["kv"]
    starts = np.concatenate([[0], np.cumsum(new)])
    sels = [_exact_select(s, b, int(starts[b]), new[b], kv[b]) for b in range(len(new))]
    O, L = _exact_attend(s, sels)
    return (O, L, torch.from_numpy(np.concatenate([x[0] for x in sels])),
            torch.from_numpy(np.concatenate([x[1] for x in sels])))


# ---------------------------------------------------------------------------
def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    d = case["d"]
    if case["op"] in ("rope", "rope_grad"):
        rows = case["B"] * (case["H"] + case["H2"]) * case["N"]
        axes = len(case["axes"].split("+"))
        return {"bytes": 2 * rows * d * es + 4 * axes * case["B"] * case["N"], "flops": rows * case["rot"] * 3}
    new, kv = _lengths(case)
    page, Hq, Hkv, T = case["page"], case["Hq"], case["Hkv"], sum(new)
    row = Hkv * d * es
    table = 4 * sum(-(-k // page) for k in kv) + 4 * (2 * case["B"] + 1)
    if case["op"] == "append":
        touched = sum((k - 1) // page - (k - n) // page + 1 for n, k in zip(new, kv))
        old = sum((k - n) % page for n, k in zip(new, kv))        # keys that were in a touched page before
        return {"bytes": 4 * T * row + (old + touched) * row + 4 * T + 8 * touched, "flops": T * Hkv * d * 4}
    qo = T * Hq * (2 * d * es + 4)
    F = case["frame"]

    def end(pos, length):
        return length if F == 0 else min(length, (pos // F + 1) * F)

    if case["op"] == "attend":
        pairs = 0
        for n, k in zip(new, kv):
            pos = np.arange(k - n, k, dtype=np.int64)
            pairs += int(np.minimum(k, (pos // F + 1) * F).sum()) if F else n * k
        return {"bytes": qo + 2 * sum(kv) * row + table, "flops": 4 * d * Hq * pairs}
    # sparse: the means and the selected pages (each page of a sequence once), pairs on selected pages
    qb, want = case["q_block"], case["n_select"]
    read = means = lists = pairs = 0
    for n, k in zip(new, kv):
        npg, got = -(-k // page), 0
        for u in range(-(-n // qb)):
            i1 = min((u + 1) * qb, n)
            vis = -(-end(k - n + i1 - 1, k) // page)
            c = min(want, vis)
            got += c
            pairs += (i1 - u * qb) * min(c * page, k)
        read += min(got, npg) * page
        means += npg
        lists += -(-n // qb) * Hkv * 4 * (want + 1)
    return {"bytes": qo + 2 * read * row + means * row + lists + table,
            "flops": 4 * d * Hq * pairs + 2 * d * means * Hkv}

"""Plain fp64 forms of the rotary positions and the paged-cache operators (test infrastructure).

Everything is computed from the definitions on the CPU, in 64 bits, for the sizes of the tests.
"""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def rope_freqs(axes, scaling="none", factor=1.0, orig=0, theta=10000.0, fast=32.0, slow=1.0):
    """Angle per position of each pair, its axis, and the magnitude."""
    f, ax, mag = [], [], 1.0
    for a, dim in enumerate(axes):
        for j in range(dim // 2):
            base = theta * factor ** (dim / (dim - 2.0)) if scaling == "base" and dim > 2 else theta
            w = base ** (-2.0 * j / dim)
            if scaling == "linear":
                w /= factor
            if scaling == "parts":
                def pair(turns):
                    return dim * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))
                lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dim // 2 - 1)
                r = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                w = w * (1 - r) + w / factor * r
                mag = 0.1 * math.log(factor) + 1.0
            f.append(w)
            ax.append(a)
    return torch.tensor(f, dtype=torch.float64), torch.tensor(ax), mag


def rope(x, pos, rot, layout, freqs, sign=1.0):
    """x [..., N, d] fp64, pos [axes, N] (or [axes, B, N] with x [B, H, N, d])."""
    f, ax, mag = freqs
    ang = (pos.double()[ax] * f.reshape(-1, *([1] * (pos.dim() - 1)))).movedim(0, -1)
    if pos.dim() == 3:
        ang = ang.unsqueeze(1)
    c, s = torch.cos(ang) * mag, torch.sin(ang) * mag * sign
    a = x[..., :rot // 2] if layout == "half" else x[..., 0:rot:2]
    b = x[..., rot // 2:rot] if layout == "half" else x[..., 1:rot:2]
    ya, yb = a * c - b * s, a * s + b * c
    out = x.clone()
    if layout == "half":
        out[..., :rot // 2], out[..., rot // 2:rot] = ya, yb
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = ya, yb
    return out


def partner_sum(x, rot, layout):
    """|x_a| + |x_b| of each rotated element's pair (0 for the copied ones): scales its error."""
    out = torch.zeros_like(x)
    if layout == "half":
        s = x[..., :rot // 2].abs() + x[..., rot // 2:rot].abs()
        out[..., :rot // 2], out[..., rot // 2:rot] = s, s
    else:
        s = x[..., 0:rot:2].abs() + x[..., 1:rot:2].abs()
        out[..., 0:rot:2], out[..., 1:rot:2] = s, s
    return out


def visible_end(pos, frame, length):
    if frame == 0:
        return length
    return 0 if pos < 0 else min(length, (pos // frame + 1) * frame)


def attention(Q, new, kv, table, kp, vp, frame, scale, sel=None, cnt=None, q_block=0, q_start=None):
    """O, lse and the per-row error scales: A = sum_j w_j |v_j| and E = max_j scale sum |q||k_j|."""
    T, Hq, d = Q.shape
    Hkv, page = kp.shape[1], kp.shape[2]
    G = Hq // Hkv
    O, A = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    L = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    E = torch.zeros(T, Hq, dtype=torch.float64)
    at, unit = 0, 0
    for b, (n, length) in enumerate(zip(new, kv)):
        if q_start is not None:
            at = q_start[b]
        npg = -(-length // page)
        K = kp[table[b, :npg].long()].double().transpose(1, 2).reshape(-1, Hkv, d)
        V = vp[table[b, :npg].long()].double().transpose(1, 2).reshape(-1, Hkv, d)
        for i in range(n):
            end = visible_end(length - n + i, frame, length)
            for h in range(Hkv):
                if sel is None:
                    keys = torch.arange(end)
                else:
                    lst = sel[unit + i // q_block, h][:cnt[unit + i // q_block, h]].long()
                    keys = (lst[:, None] * page + torch.arange(page)).flatten()
                    keys = keys[keys < end]
                if keys.numel() == 0:
                    continue
                q = Q[at + i, h * G:(h + 1) * G].double()
                k, v = K[keys, h], V[keys, h]
                x = q @ k.T * scale
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z[:, None])
                O[at + i, h * G:(h + 1) * G] = w @ v
                A[at + i, h * G:(h + 1) * G] = w @ v.abs()
                L[at + i, h * G:(h + 1) * G] = z
                E[at + i, h * G:(h + 1) * G] = (q.abs() @ k.abs().T * scale).amax(-1)
        if sel is not None:
            unit += -(-n // q_block)
        at += n
    return O, L, A, E


def select(Q, new, kv, table, k_mean, page, frame, q_block, n_select, n_sink, n_recent):
    """Lists of every unit by the definition (Python comparisons of fp64 scores)."""
    Hq, Hkv = Q.shape[1], k_mean.shape[1]
    G = Hq // Hkv
    sel, cnt = [], []
    at = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        for u in range(-(-n // q_block)):
            i0, i1 = u * q_block, min((u + 1) * q_block, n)
            vis = -(-visible_end(length - n + i1 - 1, frame, length) // page)
            q = Q[at + i0:at + i1].double().reshape(i1 - i0, Hkv, G, -1).sum((0, 2)) / ((i1 - i0) * G)
            sc = (k_mean[table[b, :vis].long()].double() * q).sum(-1)      # [vis, Hkv]
            rows, counts = [], []
            for h in range(Hkv):
                kept = [j for j in range(vis) if j < n_sink or j >= vis - n_recent]
                free = [j for j in range(vis) if j not in set(kept)]
                key = {j: (float("-inf") if math.isnan(float(sc[j, h])) else float(sc[j, h])) for j in free}
                nan = {j: math.isnan(float(sc[j, h])) for j in free}
                free.sort(key=lambda j: (nan[j], -key[j], j))
                got = sorted((kept + free)[:min(n_select, vis)])
                rows.append(got + [-1] * (n_select - len(got)))
                counts.append(len(got))
            sel.append(rows)
            cnt.append(counts)
        at += n
    return torch.tensor(sel, dtype=torch.int32), torch.tensor(cnt, dtype=torch.int32)

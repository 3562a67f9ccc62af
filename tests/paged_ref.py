"""64-bit references of the norm + rotation, its gradient and the paged cache,
written from the definitions (numpy/torch float64 on the CPU; no code shared
with the package)."""
from __future__ import annotations

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}     # half a step among subnormals


def angles_table(max_pos, rot, base=10000.0):
    """[max_pos, rot] float32: rot/2 cosines, then rot/2 sines."""
    if rot == 0:
        return None
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(max_pos, dtype=np.float64)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32))


def pair_index(d, rot, interleaved):
    """(partner of each value, sign of the sine, index of its angle), numpy arrays of d entries; unrotated values
    are their own partners with sign 0."""
    partner, sign, which = np.arange(d), np.zeros(d), np.zeros(d, dtype=np.int64)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        partner[a], partner[b] = b, a
        sign[a], sign[b] = -1.0, 1.0
        which[a] = which[b] = i
    return partner, sign, which


def _turn(y, table_rows, rot, interleaved, back=False):
    """y [rows, heads, d] float64 turned by its row's angles; also the sum of magnitudes that enter each value."""
    d = y.shape[-1]
    if rot == 0:
        return y.clone(), y.abs()
    partner, sign, which = pair_index(d, rot, interleaved)
    t = table_rows.double()
    live = torch.from_numpy((sign != 0).astype(np.float64))
    c = t[:, :rot // 2][:, which] * live + (1 - live)
    s = t[:, rot // 2:][:, which] * torch.from_numpy(sign) * (-1.0 if back else 1.0)
    z = y[..., partner]
    z = torch.where(live.bool(), z, torch.zeros_like(z))
    return y * c[:, None] + z * s[:, None], y.abs() + z.abs()


def norm_rope(x, w, table_rows, rot, eps, interleaved):
    """(value, magnitude) of one tensor [rows, heads, d]."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    return _turn(y, table_rows, rot, interleaved)


def norm_rope_bwd(dy, x, w, table_rows, rot, eps, interleaved):
    """(dx, dx magnitude, dw, dw magnitude)."""
    x, w = x.double(), w.double()
    g, gm = _turn(dy.double(), table_rows, rot, interleaved, back=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h, hm = g * w, gm * w.abs()
    dx = r * h - x * r ** 3 * (h * x).mean(-1, keepdim=True)
    mag = r * hm + x.abs() * r ** 3 * (hm * x.abs()).mean(-1, keepdim=True)
    return dx, mag, (g * x * r).sum((0, 1)), (gm * x.abs() * r).sum((0, 1))


def token_places(cu, lens, page, table):
    """(row, page, slot, position, sequence) of every live token, numpy arrays."""
    out = []
    for b in range(len(lens)):
        q = int(cu[b + 1] - cu[b])
        for i in range(q):
            p = int(lens[b]) - q + i
            out.append((int(cu[b]) + i, int(table[b, p // page]), p % page, p, b))
    return np.array(out, dtype=np.int64).reshape(-1, 5).T


def make_pages(rng, lens, page, spare=3, cols=None):
    """(block table int32 with -1 behind each sequence's last page, number of pages): pages in random order."""
    need = [-(-int(n) // page) for n in lens]
    cols = max(need + [1]) if cols is None else cols
    ids = rng.permutation(sum(need) + spare)
    table, at = np.full((len(lens), cols), -1, dtype=np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, len(ids)


def paged_attention(q, kc, vc, table, lens, cu, page, order, causal, window, scale):
    """(O, LSE, sum p |v| / sum p, largest sum |q| |k| scale of a row), float64, of the packed rows; rows of no
    sequence are zero. kc, vc: CPU tensors in `order`."""
    q = q.double()
    rows, hq, _ = q.shape
    o, lse = torch.zeros(rows, hq, vc.shape[-1], dtype=torch.float64), torch.zeros(rows, hq, dtype=torch.float64)
    pv, mag = torch.zeros_like(o), torch.zeros_like(lse)
    if order == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    hkv = kc.shape[2]
    g = hq // hkv
    for b in range(len(lens)):
        lo, hi, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        if lo == hi:
            continue
        pos = np.arange(n)
        ids, slot = torch.from_numpy(table[b, pos // page].astype(np.int64)), torch.from_numpy(pos % page)
        k, v = kc[ids, slot].double(), vc[ids, slot].double()
        at = np.arange(n - (hi - lo), n)[:, None]
        seen = np.broadcast_to(pos[None, :] >= 0, (hi - lo, n))
        if causal:
            seen = seen & (pos[None, :] <= at)
            if window >= 0:
                seen = seen & (pos[None, :] >= at - window)
        hidden = torch.from_numpy(~seen)
        for h in range(hq):
            s = q[lo:hi, h] @ k[:, h // g].T * scale
            s[hidden] = -np.inf
            m = s.amax(-1, keepdim=True) if n else torch.full((hi - lo, 1), -np.inf, dtype=torch.float64)
            m0 = torch.where(m == -np.inf, torch.zeros_like(m), m)
            p = torch.exp(s - m0)
            t = p.sum(-1, keepdim=True)
            vv = v[:, h // g]
            # a key that no row of the batch's rows sees may hold anything
            vv = torch.where(torch.from_numpy(seen.any(0))[:, None], vv, torch.zeros_like(vv))
            t1 = torch.where(t == 0, torch.ones_like(t), t)
            o[lo:hi, h] = (p @ vv) / t1
            pv[lo:hi, h] = (p @ vv.abs()) / t1
            lse[lo:hi, h] = (m0 + torch.log(t))[:, 0]
            a = q[lo:hi, h].abs() @ k[:, h // g].abs().T * scale
            a[hidden] = 0
            mag[lo:hi, h] = a.amax(-1) if n else 0
    return o, lse, pv, mag

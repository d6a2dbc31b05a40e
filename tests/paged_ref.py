"""Plain references of the paged 8-bit cache in 64 bits (numpy on the host; no library code)."""
import math

import numpy as np
import torch


def decode_e4m3(codes):
    """uint8 E4M3 codes -> float64 values (0x7F / 0xFF: NaN), by the format's definition."""
    c = np.arange(256)
    sign = np.where(c & 128, -1.0, 1.0)
    e, man = (c >> 3) & 15, c & 7
    val = np.where(e == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (e.astype(np.float64) - 10))
    val = np.where((c & 127) == 127, np.nan, val) * sign
    return val[np.asarray(codes).astype(np.int64)]


def round_e4m3(x):
    """Nearest E4M3 value of float64 x (ties to even, saturating at 448, NaN stays)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    with np.errstate(invalid="ignore"):
        r = np.where(np.isinf(x), x, np.round(np.where(np.isinf(x), 0, x) / step) * step)
        return np.clip(r, -448.0, 448.0)


def pow2_scale(amax):
    """Least power of two s >= 2^-126 with amax / s <= 448."""
    s = 2.0 ** -126
    if amax > 0:
        man, e = math.frexp(amax / 448.0)
        s = max(s, math.ldexp(1.0, e - 1 if man == 0.5 else e))
    return s


def plan(keep, new, seq, table, free, n_free, page, T):
    """The plan by its definition on host lists; returns the updated state and the maps."""
    B, width = table.shape
    table, stack = table.copy(), list(free[:n_free])
    n_pages = len(free)
    up = lambda x: -(-x // page)  # noqa: E731
    status = 0
    seq_c = [min(max(s, 0), width * page) for s in seq]
    keep_c = [min(max(k, 0), s) for k, s in zip(keep, seq_c)]
    new_c = [max(n, 0) for n in new]
    if list(seq) != seq_c or list(keep) != keep_c or list(new) != new_c:
        status |= 16
    for b in reversed(range(B)):
        for j in reversed(range(up(keep_c[b]), up(seq_c[b]))):
            stack.append(int(table[b, j]))
            table[b, j] = -1
    assert len(stack) <= n_pages
    top, taken = len(stack), 0
    cu, pos, slot, seq_out = [0], [], [], []
    for b in range(B):
        fits = keep_c[b] + new_c[b] <= width * page
        need = up(keep_c[b] + new_c[b]) - up(keep_c[b]) if fits else 0
        ok = new_c[b] == 0 or (fits and cu[-1] + new_c[b] <= T and (need == 0 or taken + need <= top))
        taken += need
        if ok:
            for j in range(up(keep_c[b]), up(keep_c[b]) + need):
                table[b, j] = stack.pop()
        else:
            status |= 32
        for p in range(keep_c[b], keep_c[b] + new_c[b]):
            if len(pos) >= T:
                break
            pos.append(p)
            slot.append(int(table[b, p // page]) * page + p % page if ok else -1)
        seq_out.append(keep_c[b] + (new_c[b] if ok else 0))
        cu.append(cu[-1] + new_c[b])
    pad = [-1] * (T - len(pos))
    return dict(seq=seq_out, table=table, stack=stack, cu=[min(c, T) for c in cu], pos=pos + pad,
                slot=slot + pad, status=status)


def write(x, slot, codes, scale):
    """x float64 [T, Hkv, d] into copies of codes (uint8) / scale by the definition, page by page;
    returns (values the codes stand for / scale, i.e. code values, and scales)."""
    page = codes.shape[2]
    val, scale = decode_e4m3(codes), scale.astype(np.float64).copy()
    slot = np.asarray(slot)
    for pg in np.unique(slot[slot >= 0] // page):
        rows = np.nonzero((slot >= 0) & (slot // page == pg))[0]
        off = slot[rows] % page
        for g in range(x.shape[1]):
            a = np.abs(x[rows, g])
            a = a[np.isfinite(a)]
            s = pow2_scale(a.max() if a.size else 0.0)
            if off.min() > 0:
                s = max(s, scale[pg, g])
                val[pg, g, :off.min()] = round_e4m3(val[pg, g, :off.min()] * (scale[pg, g] / s))
            scale[pg, g] = s
            val[pg, g, off] = round_e4m3(x[rows, g] / s)
    return val, scale


def attn(q, cu, start, lens, table, k, ks, v, vs, page, m, W, scale, sink=None):
    """q float64 [T, H, d]; k, v uint8 codes [n_pages, Hkv, page, d].  Returns out, lse, and for
    the tolerance: mass = sum_j p_j |v_j| and zabs = max_j scale * sum |q_c k_jc| over the visible
    rows.  Rows of no request are NaN."""
    T, H, d = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    out, mass = np.full((T, H, d), np.nan), np.full((T, H, d), np.nan)
    lse, zabs = np.full((T, H), np.nan), np.full((T, H), 0.0)
    for b in range(len(lens)):
        for g in range(Hkv):
            n = min(max(int(lens[b]), 0), table.shape[1] * page)
            ids = table[b, :-(-n // page)]
            kk = (decode_e4m3(k[ids, g]) * ks[ids, g].astype(np.float64)[:, None, None]).reshape(-1, d)[:n]
            vv = kk if v is None else (
                decode_e4m3(v[ids, g]) * vs[ids, g].astype(np.float64)[:, None, None]).reshape(-1, d)[:n]
            for i in range(cu[b + 1] - cu[b]):
                p, t = int(start[b]) + i, cu[b] + i
                hi = min(n, (p + 1) // m) if p >= 0 else 0
                lo = min(hi, max(0, p - W + 1) if W else 0)
                for h in range(g * G, g * G + G):
                    z = kk[lo:hi] @ q[t, h] * scale
                    zz = z if sink is None else np.append(z, float(sink[h]))
                    if zz.size == 0:
                        out[t, h], mass[t, h], lse[t, h] = 0.0, 0.0, -np.inf
                        continue
                    top = zz.max()
                    l = top + math.log(np.exp(zz - top).sum()) if np.isfinite(top) else top
                    w = np.exp(z - l)
                    out[t, h], lse[t, h] = w @ vv[lo:hi], l
                    mass[t, h] = w @ np.abs(vv[lo:hi])
                    if hi > lo:
                        zabs[t, h] = (np.abs(kk[lo:hi]) @ np.abs(q[t, h])).max() * scale
    return out, lse, mass, zabs


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()

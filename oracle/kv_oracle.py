"""Float64 oracle of the quantised key/value cache: the tile layout, the quantiser, attention over
cached rows and the choice of blocks (include/gpt_ops.h, "Quantised key/value cache")."""
from __future__ import annotations

import numpy as np

BLOCK, REC = 64, 32


def geometry(bits: int, hd: int):
    """(bytes of a row's codes, scales of a row, bytes of a record)."""
    rowb = hd * bits // 8
    ng = hd // 64 if bits == 4 else 1
    return rowb, ng, 2 * REC * rowb + 4 * REC * ng


def key_byte(bits: int, hd: int, i: int, y: int) -> int:
    """Offset in its record of byte y (natural order) of key i."""
    R = hd * bits // 8
    w, x, P = y // 4, 4 * (y // 16) + y % 4, min(R // 4, 16)
    return (i // 16) * 16 * R + (x // P) * 64 * P + (i % 16) * 4 * P + (w % 4) * P + x % P


def value_byte(bits: int, hd: int, i: int, y: int) -> int:
    """Offset in its record of byte y of value i."""
    R = hd * bits // 8
    o, n = y // bits, i % 16
    z = (n % 2 + 2 * (n // 8)) * (R // 8) + (o // 8) * bits + y % bits
    return 32 * R + (i // 16) * 16 * R + (z // 16) * 512 + (4 * (o % 8) + n % 8 // 2) * 16 + z % 16


def _tables(bits, hd):
    R = hd * bits // 8
    return [np.array([[f(bits, hd, i, y) for y in range(R)] for i in range(REC)]) for f in (key_byte, value_byte)]


def bf16(x, how: str = "nearest"):
    """x (float64, finite or not) rounded to bfloat16: to nearest even, or "down" / "up"."""
    x = np.asarray(x, np.float64)
    f = x.astype(np.float32)
    b = f.view(np.uint32).astype(np.int64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    near = np.where(np.isfinite(x), (r & 0xFFFFFFFF).astype(np.uint32).view(np.float32).astype(np.float64), x)
    if how == "nearest":
        return near
    k = near.astype(np.float32).view(np.uint32).astype(np.int64)
    step = np.where((near > 0) == (how == "up"), 0x10000, -0x10000)
    out = (k + step).astype(np.uint32).view(np.float32).astype(np.float64)
    wrong = near > x if how == "down" else near < x
    return np.where(wrong & np.isfinite(x), out, near)


def quantise(x, bits: int):
    """Rows [..., hd] -> (codes, scales [..., ng], values).  A group with a non-finite value gets a NaN
    scale; one whose scale is below the normal range, zeros."""
    x = np.asarray(x, np.float64)
    hd = x.shape[-1]
    ng = geometry(bits, hd)[1]
    z = 1 << (bits - 1)
    g = x.reshape(*x.shape[:-1], ng, hd // ng)
    ok = np.isfinite(g).all(-1)
    s = bf16(np.abs(np.where(ok[..., None], g, 0.0)).max(-1) / (z - 1))
    s = np.where(s < 2.0 ** -126, 0.0, s)
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.where((s > 0)[..., None] & ok[..., None], np.rint(g / s[..., None]), 0.0)
    n = np.clip(n, -(z - 1), z - 1)
    s = np.where(ok, s, np.nan)
    return (n + z).reshape(x.shape).astype(np.uint8), s, (n * s[..., None]).reshape(x.shape)


def pack(kc, ks, vc, vs, bits: int):
    """Codes [..., 64, hd] and scales [..., 64, ng] of keys and values -> tile bytes [..., tile]."""
    hd = kc.shape[-1]
    R, ng, recb = geometry(bits, hd)
    lead = kc.shape[:-2]
    out = np.zeros((*lead, 2, recb), np.uint8)
    for which, (c, s, tab) in enumerate(zip((kc, vc), (ks, vs), _tables(bits, hd))):
        b = c if bits == 8 else (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)
        out[..., tab.reshape(-1)] = b.reshape(*lead, 2, REC * R)
        raw = (np.asarray(s, np.float32).view(np.uint32) >> 16).astype(np.uint16)
        raw = raw.reshape(*lead, 2, REC * ng, 1).view(np.uint8).reshape(*lead, 2, 2 * REC * ng)
        at = 2 * REC * R + which * 2 * REC * ng
        out[..., at:at + 2 * REC * ng] = raw
    return out.reshape(*lead, 2 * recb)


def unpack(tiles, bits: int, hd: int):
    """Tile bytes [..., tile] -> (k, v) values [..., 64, hd]."""
    R, ng, recb = geometry(bits, hd)
    lead = tiles.shape[:-1]
    rec = np.asarray(tiles).reshape(*lead, 2, recb)
    z = 1 << (bits - 1)
    out = []
    for which, tab in enumerate(_tables(bits, hd)):
        b = rec[..., tab.reshape(-1)].reshape(*lead, BLOCK, R)
        u = b if bits == 8 else np.stack((b & 15, b >> 4), -1).reshape(*lead, BLOCK, hd)
        at = 2 * REC * R + which * 2 * REC * ng
        raw = np.ascontiguousarray(rec[..., at:at + 2 * REC * ng]).view(np.uint16).astype(np.uint32) << 16
        s = raw.view(np.float32).astype(np.float64).reshape(*lead, BLOCK, ng, 1)
        out.append(((u.astype(np.float64) - z).reshape(*lead, BLOCK, ng, hd // ng) * s).reshape(*lead, BLOCK, hd))
    return out


def attend(q, k, v, weight):
    """q [H, hd], k and v [L, Hkv, hd], weight [Hkv, L] (how often each key counts, 0 = masked) ->
    (o [H, hd], lse [H], sum_j p_j |v_j| [H, hd])."""
    H, hd = q.shape
    G = H // k.shape[1]
    o, a, lse = np.zeros((H, hd)), np.zeros((H, hd)), np.full(H, -np.inf)
    for h in range(H):
        live = weight[h // G] > 0
        if not live.any():
            continue
        s = k[live, h // G] @ q[h] / np.sqrt(hd)
        m = s.max()
        p = np.exp(s - m) * weight[h // G][live]
        o[h] = p @ v[live, h // G] / p.sum()
        a[h] = p @ np.abs(v[live, h // G]) / p.sum()
        lse[h] = m + np.log(p.sum())
    return o, lse, a


def block_scores(q, bounds):
    """q [H, hd], bounds [nb, Hkv, 2, hd] -> scores [Hkv, nb]."""
    nb, Hkv, _, hd = bounds.shape
    qg = q.reshape(Hkv, -1, 1, hd)
    b = bounds.transpose(1, 2, 0, 3)[:, None]
    return np.maximum(qg * b[:, :, 0], qg * b[:, :, 1]).sum((1, 3))


def choose(scores, n: int, n_first: int, n_last: int):
    """scores [nb] -> ascending indices of the first n_first, last n_last and best others, n in all."""
    nb = len(scores)
    order = sorted(range(nb), key=lambda j: (not (j < n_first or j >= nb - n_last), -scores[j], j))
    return sorted(order[:n])

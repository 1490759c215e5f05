"""The quantised key/value cache on the GPU against the float64 oracle (oracle/kv_oracle.py).

Tolerances, from the roundings the kernels make:
  - q after RoPE and QK-norm: half a bf16 step, 2^-8 |q|, plus fp32 arithmetic: 16 operations of
    2^-24 on terms up to the row's largest raw value times its norm factor, 2^-20 of the row's largest.
  - cached values: half a step of the quantiser, half a bf16 step for the value read back, and the
    fp32 error above; and equal to the oracle's own value wherever the quotient is not within 2^-12
    of a border between two codes (the scale itself may sit on a border: those groups are let off).
  - attention: the probabilities times the value scale are fp16 operands, off by 2^-11 of themselves
    (and by 2^-25 / 64 of the largest value scale's power of two, absolutely), so a row by
    2^-11 sum_j p_j |v_j|; the scores are fp32 sums of exact products of q and codes, off by at most
    e_s = 2^-20 sum_d |q_d| 2 Z scale / sqrt(hd), which moves each p_j by 2 e_s of itself; the
    accumulated sums hold p scale (code - Z) as differences of terms up to p scale 2 Z, 2^-20 of
    those; and the output is bf16, 2^-8 |o|.  lse: e_s + 2^-21 (1 + |lse|).
  - block scores: fp64 sums rounded to fp32, 2^-24; chosen blocks: equal."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as O
import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _g():
    import decoder_only_gpt_tcgen05_b200 as g
    return g


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def normal(shape, seed):
    return synth.normal(shape, seed).astype(np.float64)


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().to(DEV)


def f64(t):
    return t.double().cpu().numpy()


class World:
    """A cache with random contents: sequences of the given lengths in shuffled blocks; every byte that
    holds no token (slots after a sequence's end, unused blocks) is 0xff, a NaN scale."""

    def __init__(self, bits, hd, Hkv, lens, seed, scale=1.0, spare=3):
        self.bits, self.hd, self.Hkv, self.lens = bits, hd, Hkv, list(lens)
        g = _g()
        need = [(n + 63) // 64 for n in lens]
        self.W = max(need + [1]) + 1
        self.n_blocks = sum(need) + spare
        perm = np.random.default_rng(seed).permutation(self.n_blocks)
        self.table = np.full((len(lens), self.W), -7)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        tile = 2 * O.kv.geometry(bits, hd)[2]
        tiles = np.full((self.n_blocks, Hkv, tile), 255, np.uint8)
        bounds = np.full((self.n_blocks, Hkv, 2, hd), np.nan)
        self.k, self.v = [], []
        R, ng, recb = O.kv.geometry(bits, hd)
        tabs = O.kv._tables(bits, hd)
        for b, n in enumerate(lens):
            x = normal((2, n, Hkv, hd), seed + 17 * b + 1) * scale
            parts = [O.kv.quantise(x[i], bits) for i in range(2)]
            self.k.append(parts[0][2])
            self.v.append(parts[1][2])
            for j in range(need[b]):
                m = min(64, n - 64 * j)
                for i in range(m):
                    rec, tok = divmod(i, 32)
                    dst = tiles[self.table[b, j], :, rec * recb:(rec + 1) * recb]
                    for which in range(2):
                        c, s = (p[64 * j + i] for p in parts[which][:2])
                        dst[:, tabs[which][tok]] = c if bits == 8 else c[:, 0::2] | (c[:, 1::2] << 4)
                        raw = (s.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).reshape(Hkv, ng, 1)
                        so = 2 * 32 * R + which * 64 * ng + tok * 2 * ng
                        dst[:, so:so + 2 * ng] = raw.view(np.uint8).reshape(Hkv, 2 * ng)
                kk = self.k[b][64 * j:64 * j + m]
                bounds[self.table[b, j]] = np.stack((O.kv.bf16(kk.min(0), "down"), O.kv.bf16(kk.max(0), "up")), 1)
        self.bounds = bounds
        self.cache = g.KVCache(self.n_blocks, Hkv, hd, bits=bits, tiles=torch.from_numpy(tiles).to(DEV), bounds=bf(bounds))

    def batch(self, new, max_new=None):
        cu = np.concatenate(([0], np.cumsum(new)))
        b = _g().KVBatch(i32(self.table), i32(self.lens), i32(cu), max_new=max(new) if max_new is None else max_new)
        return b, cu


def attend_bounds(w, b, q, o, lse, av, weight):
    """The tolerances of one token's row (module docstring): (of o [H, hd], of lse [H])."""
    G = q.shape[0] // w.Hkv
    Z = 1 << (w.bits - 1)
    to, tl = np.zeros_like(o), np.zeros(len(lse))
    for h in range(q.shape[0]):
        live = weight[h // G] > 0
        if not live.any():
            continue
        ksc = np.abs(w.k[b][live, h // G]).max() / (Z - 1) * 1.01
        vsc = np.abs(w.v[b][live, h // G]).max() / (Z - 1) * 1.01
        es = 2.0 ** -20 * np.abs(q[h]).sum() * 2 * Z * ksc / np.sqrt(w.hd)
        n = weight[h // G].sum()
        to[h] = 2.0 ** -8 * np.abs(o[h]) + (2.0 ** -11 + 2 * es) * av[h] + 2.0 ** -20 * 2 * Z * vsc + \
            n * 2.0 ** -31 * 2 * vsc * Z * np.exp(-min(0.0, lse[h]))
        tl[h] = es + 2.0 ** -21 * (1 + abs(lse[h]))
    return to, tl


def check_attend(w, new, q, o, lse, window=-1, sel=None, what=""):
    """Every row of o, lse against the oracle; sel: [M, Hkv, n] listed blocks."""
    cu = np.concatenate(([0], np.cumsum(new)))
    H = q.shape[1] // w.hd
    for b, n in enumerate(new):
        for i in range(n):
            m, p = cu[b] + i, w.lens[b] - n + i
            L = w.lens[b]
            j = np.arange(L)
            ok = (j <= p) & ((j >= p - window) if window >= 0 else True)
            wt = np.repeat(ok[None].astype(float), w.Hkv, 0)
            if sel is not None:
                nb = p // 64 + 1
                for h in range(w.Hkv):
                    cnt = np.zeros(w.W + 1)
                    for x in sel[m, h][:min(sel.shape[2], nb)]:
                        if 0 <= x < nb:
                            cnt[x] += 1
                    wt[h] *= cnt[j // 64]
            qr = q[m].reshape(H, w.hd)
            ro, rl, av = O.kv.attend(qr, w.k[b], w.v[b], wt)
            to, tl = attend_bounds(w, b, qr, ro, rl, av, wt)
            got = o[m].reshape(H, w.hd)
            assert np.all(np.isfinite(got)), (what, b, i)
            assert np.all(np.abs(got - ro) <= to), (what, b, i, (np.abs(got - ro) - to).max(), np.abs(ro).max())
            dead = ~np.isfinite(rl)
            assert np.all(lse[m][dead] == -np.inf) and np.all(got[dead] == 0), (what, b, i)
            assert np.all(np.abs(lse[m] - rl)[~dead] <= tl[~dead]), (what, b, i, np.abs(lse[m] - rl)[~dead].max())


# ---------------------------------------------------------------------------- append and read

APPEND = [
    # bits, hd, H, Hkv, rope, norm, lens, new tokens
    (8, 128, 2, 2, True, True, [1, 64, 65, 200], [1, 1, 1, 1]),
    (4, 128, 2, 2, True, True, [1, 64, 65, 200], [1, 1, 1, 1]),
    (4, 128, 4, 2, True, True, [130, 64, 5, 131], [130, 63, 0, 66]),
    (8, 64, 4, 1, True, True, [130, 64, 5, 131], [130, 63, 0, 66]),
    (4, 64, 3, 3, False, True, [7, 100], [3, 2]),
    (8, 128, 6, 3, True, False, [77, 129], [8, 9]),
    (8, 64, 12, 12, False, False, [300], [300]),
    (4, 128, 10, 10, True, True, [1000], [333]),
]


@pytest.mark.parametrize("case", APPEND)
def test_append_and_read_match_the_oracle(case):
    bits, hd, H, Hkv, rope, norm, lens, new = case
    w = World(bits, hd, Hkv, [n - m for n, m in zip(lens, new)], 100)
    # the sequences grow into spare blocks
    need = [(n + 63) // 64 for n in lens]
    had = [(n - m + 63) // 64 for n, m in zip(lens, new)]
    grow = sum(need) - sum(had)
    g = _g()
    cache = g.KVCache(w.n_blocks + grow, Hkv, hd, bits=bits, device=DEV)
    cache.tiles.fill_(255)
    cache.bounds.fill_(float("nan"))
    cache.tiles[:w.n_blocks] = w.cache.tiles
    cache.bounds[:w.n_blocks] = w.cache.bounds
    table = np.full((len(lens), max(need) + 2), -1)
    fresh = w.n_blocks
    for b in range(len(lens)):
        table[b, :had[b]] = w.table[b, :had[b]]
        for j in range(had[b], need[b]):
            table[b, j] = fresh
            fresh += 1
    before_t, before_b = cache.tiles.clone(), cache.bounds.clone()
    M, behind = sum(new), 3
    cu = np.concatenate(([0], np.cumsum(new)))
    raw = torch.from_numpy(synth.normal((M + behind, (H + 2 * Hkv) * hd), 5)).bfloat16()
    batch = g.KVBatch(i32(table), i32(lens), i32(cu), max_new=max(new))
    q = torch.full((M + behind, H * hd), 7.0, dtype=torch.bfloat16, device=DEV)
    cache.append(batch, raw.to(DEV), H, rope=rope, qk_norm=norm, q=q)
    k = torch.full((M + behind, Hkv, hd), 7.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    cache.read(batch, M + behind, k=k, v=v)
    g.model.sync_status(DEV)
    for t in (q, k, v):
        assert torch.all(t[M:] == 7.0)          # rows behind the last sequence
    q, k, v = f64(q), f64(k), f64(v)
    phi = O.rope_angles(max(lens), hd, 10000.0)
    used = {}
    for b, n in enumerate(new):
        if n == 0:
            continue
        x = raw[cu[b]:cu[b + 1]].double().numpy().reshape(n, H + 2 * Hkv, hd)
        pos = np.arange(lens[b] - n, lens[b])
        y = x[:, :H + Hkv]
        if rope:
            y = O.rope(y.transpose(1, 0, 2), phi[pos]).transpose(1, 0, 2)
        f = np.ones(y.shape[:2] + (1,))
        if norm:
            y, f = O.rmsnorm(y, 1e-5)
            f = f.reshape(*y.shape[:2], 1)
        top = np.abs(x[:, :H + Hkv]).max(-1, keepdims=True) * np.abs(f)
        eq = 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * top
        assert np.all(np.abs(q[cu[b]:cu[b + 1]].reshape(n, H, hd) - y[:, :H]) <= eq[:, :H])
        for got, ref, err in ((k[cu[b]:cu[b + 1]], y[:, H:], 2.0 ** -20 * top[:, H:]),
                              (v[cu[b]:cu[b + 1]], x[:, H + Hkv:], 0.0)):
            _, s, val = O.kv.quantise(ref, bits)
            step = np.repeat(s, hd // s.shape[-1], -1)
            assert np.all(np.abs(got - ref) <= 0.5 * step * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(got) + err)
            quo = ref / step
            clear = np.abs(quo - np.floor(quo) - 0.5) > 2.0 ** -12
            amax = np.abs(ref.reshape(n, Hkv, s.shape[-1], -1)).max(-1) / ((1 << (bits - 1)) - 1)
            edge = O.kv.bf16(amax * (1 - 2.0 ** -19)) != O.kv.bf16(amax * (1 + 2.0 ** -19))
            clear &= ~np.repeat(edge, hd // s.shape[-1], -1)
            assert np.all(np.abs(got - val)[clear] <= 2.0 ** -8 * np.abs(val)[clear]) and clear.mean() > 0.9
        for j in range((lens[b] - n) // 64, (lens[b] + 63) // 64):
            used[table[b, j]] = (b, j, max(lens[b] - n - 64 * j, 0), min(lens[b] - 64 * j, 64))
    # what was in the cache stays, but for the slots written; bounds hold every key of the block
    kk, vv = (O.kv.unpack(cache.tiles.cpu().numpy(), bits, hd))
    k0, v0 = O.kv.unpack(before_t.cpu().numpy(), bits, hd)
    bd, bd0 = f64(cache.bounds), f64(before_b)
    for ph in range(cache.n_blocks):
        keep = np.ones(64, bool)
        if ph in used:
            b, j, a, z = used[ph]
            keep[a:z] = False
            keys = kk[ph][:, :z]
            lo, hi = O.kv.bf16(keys.min(1), "down"), O.kv.bf16(keys.max(1), "up")
            assert np.array_equal(bd[ph][:, 0], lo) and np.array_equal(bd[ph][:, 1], hi), (ph, a, z)
        else:
            assert np.array_equal(bd[ph], bd0[ph], equal_nan=True)
        assert np.array_equal(kk[ph][:, keep], k0[ph][:, keep], equal_nan=True)
        assert np.array_equal(vv[ph][:, keep], v0[ph][:, keep], equal_nan=True)


def test_append_far_positions_and_default_rows():
    """Angles of positions far beyond 2^24 in fp32 steps; no cu_new: one row a sequence."""
    g = _g()
    H = Hkv = 1
    hd, W = 128, 1 << 16
    lens = [W * 64, W * 64 - 777]      # 4.2 million tokens
    table = np.zeros((2, W))
    table[0, (lens[0] - 1) // 64], table[1, (lens[1] - 1) // 64] = 1, 2
    cache = g.KVCache(3, Hkv, hd, bits=8, device=DEV)
    raw = torch.from_numpy(synth.normal((2, 3 * hd), 5)).bfloat16()
    q = cache.append(g.KVBatch(i32(table), i32(lens)), raw.to(DEV), H, qk_norm=False)
    g.model.sync_status(DEV)
    inv = 10000.0 ** (-2.0 * np.arange(hd // 2) / hd)
    for b in range(2):
        x = raw[b].double().numpy()[:hd]
        ref = O.rope(x[None], (lens[b] - 1) * inv[None])[0]
        assert np.all(np.abs(f64(q)[b] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.abs(x).max())


@pytest.mark.parametrize("bits", [4, 8])
def test_append_non_finite_zero_and_tiny_rows(bits):
    g = _g()
    hd, n = 128, 8
    raw = synth.normal((n, 3 * hd), 6)
    raw[1, hd + 3], raw[2, 2 * hd + 100], raw[3, hd:] = np.inf, np.nan, 0.0
    raw[4, hd:] = 1e-38
    raw[5, hd:] *= 1e30
    cache = g.KVCache(1, 1, hd, bits=bits, device=DEV)
    batch = g.KVBatch(i32([[0]]), i32([n]), i32([0, n]), max_new=n)
    rawb = torch.from_numpy(raw.astype(np.float32)).bfloat16()
    cache.append(batch, rawb.to(DEV), 1, rope=False, qk_norm=False)
    k, v = (f64(t)[:, 0] for t in cache.read(batch, n))
    g.model.sync_status(DEV)
    x = rawb.double().numpy()
    for got, ref in ((k, x[:, hd:2 * hd]), (v, x[:, 2 * hd:])):
        _, _, val = O.kv.quantise(ref, bits)
        assert np.array_equal(np.isnan(got), np.isnan(val))
        f = np.isfinite(val)
        assert np.all(np.abs(got - val)[f] <= 2.0 ** -8 * np.abs(val)[f])
    b = f64(cache.bounds)[0, 0]
    assert np.all(np.isnan(b[:, :64]))           # the infinite key's group
    assert np.all(np.isnan(b[:, 64:])) == (bits == 8)


def test_read_part_of_a_sequence():
    w = World(4, 128, 2, [200, 90], 3)
    b, cu = w.batch([37, 90])
    k, v = w.cache.read(b, 127)
    _g().model.sync_status(DEV)
    for got, ref in ((f64(k), w.k), (f64(v), w.v)):
        want = np.concatenate((ref[0][163:], ref[1]))
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want))


# ---------------------------------------------------------------------------- attention

ATTEND = [
    # bits, hd, H, Hkv, lens, new, window
    (8, 128, 2, 2, [1, 31, 32, 33, 64, 65, 700], [1] * 7, -1),
    (4, 128, 2, 2, [1, 31, 32, 33, 64, 65, 700], [1] * 7, -1),
    (4, 64, 3, 3, [1, 31, 32, 33, 64, 65, 700], [1] * 7, -1),
    (8, 64, 3, 3, [1, 31, 32, 33, 64, 65, 700], [1] * 7, -1),
    (8, 128, 4, 2, [5, 300, 64, 0, 129], [5, 3, 0, 0, 1], -1),      # no new tokens, no tokens
    (4, 128, 8, 1, [70, 1], [2, 1], -1),                            # 16 rows: two column tiles
    (8, 128, 20, 1, [130, 33], [1, 1], -1),                         # 20 query heads a kv head
    (4, 64, 9, 1, [200], [7], -1),                                  # 63 rows: several tiles
    (8, 64, 2, 2, [260], [260], -1),                                # a whole prompt
    (4, 128, 2, 2, [500, 40], [3, 2], 0),
    (8, 128, 2, 2, [500, 40], [3, 2], 31),
    (4, 64, 4, 2, [500, 40], [9, 2], 100),
    (8, 64, 4, 2, [500, 600], [40, 1], 64),
    (4, 128, 1, 1, [5000], [1], -1),                                # one head cut between many workers
    (8, 128, 13, 13, [900] * 3, [1] * 3, -1),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention_matches_the_oracle(case):
    bits, hd, H, Hkv, lens, new, window = case
    w = World(bits, hd, Hkv, lens, 40)
    batch, cu = w.batch(new)
    M = sum(new)
    q = bf(normal((M + 2, H * hd), 4))
    o = torch.full((M + 2, H * hd), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((M + 2, H), 7.0, device=DEV)
    w.cache.attend(batch, q, window=window, o=o, lse=lse)
    _g().model.sync_status(DEV)
    assert torch.all(o[M:] == 7.0) and torch.all(lse[M:] == 7.0)
    check_attend(w, new, f64(q), f64(o), f64(lse), window=window)
    again = w.cache.attend(batch, q, window=window)
    assert torch.equal(again[0][:M], o[:M]) and torch.equal(again[1][:M], lse[:M])


@pytest.mark.parametrize("qs,kvs", [(1e-20, 1.0), (1e12, 1e-12), (30.0, 1.0), (1.0, 1e20), (1.0, 1e-25), (0.0, 1.0)])
def test_attention_over_a_wide_range_of_magnitudes(qs, kvs):
    for bits in (4, 8):
        w = World(bits, 128, 1, [150], 50, scale=kvs)
        batch, _ = w.batch([2])
        q = bf(normal((2, 128), 4) * qs / (kvs if kvs > 1 else 1.0))
        o, lse = w.cache.attend(batch, q)
        _g().model.sync_status(DEV)
        check_attend(w, [2], f64(q), f64(o), f64(lse), what=(bits, qs, kvs))


def test_attention_with_growing_scores_and_scales():
    """Keys whose scores climb by hundreds and values whose scale climbs by powers of two: the running
    maximum and the values' unit move again and again, between warps' parts too."""
    for bits in (4, 8):
        w = World(bits, 128, 1, [640], 51)
        ramp = np.linspace(-3, 3, 640)[:, None, None]
        qv = normal((128,), 9)
        xk = w.k[0] * 0.05 + ramp * qv
        xv = w.v[0] * 2.0 ** np.floor(np.linspace(-20, 20, 640))[:, None, None]
        kc, ks, w.k[0] = O.kv.quantise(xk, bits)
        vc, vs, w.v[0] = O.kv.quantise(xv, bits)
        for j in range(10):
            sl = slice(64 * j, 64 * j + 64)
            tile = O.kv.pack(*(a[sl].transpose(1, 0, 2) for a in (kc, ks, vc, vs)), bits)
            w.cache.tiles[w.table[0, j]] = torch.from_numpy(tile).to(DEV)
        batch, _ = w.batch([1])
        q = bf(qv[None])
        o, lse = w.cache.attend(batch, q)
        _g().model.sync_status(DEV)
        check_attend(w, [1], f64(q), f64(o), f64(lse), what=bits)
        o, lse = w.cache.attend(batch, -q)
        check_attend(w, [1], -f64(q), f64(o), f64(lse), what=bits)


def test_non_finite_queries_keys_and_values_show_in_their_rows_only():
    w = World(8, 128, 2, [100, 100], 60)
    g = _g()
    R, ng, recb = O.kv.geometry(8, 128)
    batch, _ = w.batch([2, 2])
    q0 = normal((4, 256), 4)
    q = bf(q0)
    base = w.cache.attend(batch, q)[0].clone()
    q2 = q.clone()
    q2[1, 5], q2[2, 200] = float("nan"), float("inf")
    o, lse = w.cache.attend(batch, q2)
    bad = torch.zeros((4, 2), dtype=torch.bool, device=DEV)
    bad[1, 0] = bad[2, 1] = True
    assert torch.equal(torch.isnan(o.view(4, 2, 128)).all(-1), bad) and torch.equal(torch.isnan(lse), bad)
    assert torch.equal(o.view(4, 2, 128)[~bad], base.view(4, 2, 128)[~bad])
    # key 99 of sequence 0, head 1 is NaN: only the token at 99 sees it
    tile = w.cache.tiles[w.table[0, 1], 1]
    at = recb + 2 * 32 * R + 2 * (99 - 96)
    tile[at:at + 2] = 255
    o, _ = w.cache.attend(batch, q)
    bad[:] = False
    bad[1, 1] = True
    assert torch.equal(torch.isnan(o.view(4, 2, 128)).any(-1), bad)
    assert torch.equal(o.view(4, 2, 128)[~bad], base.view(4, 2, 128)[~bad])
    g.model.sync_status(DEV)


def test_bad_block_numbers_give_nan_rows_and_a_status():
    w = World(4, 64, 2, [200, 130, 64], 61)
    g = _g()
    good, _ = w.batch([1, 1, 1])
    q = bf(normal((3, 256), 4))
    o0, l0 = w.cache.attend(good, q)
    g.model.sync_status(DEV)
    for value in (w.n_blocks, -1, 2 ** 31 - 1, -2 ** 31):
        table = w.table.copy()
        table[1, 1] = value
        table[2, 1] = value      # not visible: never looked at
        batch = g.KVBatch(i32(table), i32(w.lens), i32([0, 1, 2, 3]))
        o, lse = w.cache.attend(batch, q)
        with pytest.raises(g.GptError) as e:
            g.model.sync_status(DEV)
        assert e.value.code == 1
        assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
        assert torch.equal(o[[0, 2]], o0[[0, 2]]) or torch.allclose(o[[0, 2]].float(), o0[[0, 2]].float(), rtol=2e-2)
        k, v = w.cache.read(g.KVBatch(i32(table), i32(w.lens), i32([0, 0, 130, 130]), max_new=130), 130)
        with pytest.raises(g.GptError):
            g.model.sync_status(DEV)
        nan = np.zeros(130, bool)
        nan[64:128] = True
        assert np.array_equal(np.isnan(f64(k)).all((1, 2)), nan) and np.array_equal(np.isnan(f64(v)).any((1, 2)), nan)
        before = w.cache.tiles.clone()
        raw = torch.zeros((1, 4 * 64 + 2 * 128), dtype=torch.bfloat16, device=DEV)
        t2 = i32([[value, value]])
        w.cache.append(g.KVBatch(t2, i32([65])), raw, 4)
        with pytest.raises(g.GptError):
            g.model.sync_status(DEV)
        assert torch.equal(w.cache.tiles, before)


@pytest.mark.parametrize("lens,cu,max_new", [
    ([200, 10 ** 6, 64], [0, 1, 2, 3], 1),        # longer than its block table
    ([200, -5, 64], [0, 1, 2, 3], 1),
    ([200, 130, 64], [0, 1, 9, 10], 1),           # more new tokens than max_new
    ([200, 2, 64], [0, 1, 5, 6], 4),              # more new tokens than tokens
    ([200, 130, 64], [0, 1, 0, 1], 1),            # rows that run backwards
    ([200, 130, 64], [0, 1, 2 ** 31 - 1, -2 ** 31], 1),
])
def test_sequences_out_of_range_are_left_out(lens, cu, max_new):
    """Sequence 1 of three is broken: it is reported, none of its rows is written, sequence 0 is right
    (unless another sequence claims its row as well: cu = 0, 1, 0, 1 gives row 0 to sequences 0 and 2,
    and it holds either's result)."""
    w = World(8, 64, 1, [200, 130, 64], 62)
    g = _g()
    q = bf(normal((12, 128), 4))
    batch = g.KVBatch(i32(w.table), i32(lens), i32(cu), max_new=max_new)
    o = torch.full_like(q, 7.0)
    lse = torch.full((12, 2), 7.0, device=DEV)
    w.cache.attend(batch, q, o=o, lse=lse)
    with pytest.raises(g.GptError) as e:
        g.model.sync_status(DEV)
    assert e.value.code == 1
    if cu[2:] != [0, 1]:
        check_attend(w, [1, 0, 0], f64(q), f64(o), f64(lse))
    assert torch.all(o[1] == 7.0)
    k, v = w.cache.read(batch, 12)
    with pytest.raises(g.GptError):
        g.model.sync_status(DEV)
    if cu[2:] != [0, 1]:
        assert np.all(np.abs(f64(k)[0] - w.k[0][199]) <= 2.0 ** -8 * np.abs(w.k[0][199]))
    before = w.cache.tiles.clone()
    w.cache.append(g.KVBatch(i32(w.table[1:2]), i32(lens[1:2]), i32(cu[1:3]), max_new=max_new),
                   torch.zeros((12, 4 * 64), dtype=torch.bfloat16, device=DEV), 2)
    with pytest.raises(g.GptError):
        g.model.sync_status(DEV)
    assert torch.equal(w.cache.tiles, before)
    blocks, _ = w.cache.select(batch, q, 3)
    with pytest.raises(g.GptError):
        g.model.sync_status(DEV)
    w.cache.attend(batch, q, blocks=torch.zeros((12, 1, 2), dtype=torch.int32, device=DEV))
    with pytest.raises(g.GptError):
        g.model.sync_status(DEV)
    if cu[2:] != [0, 1]:
        chosen = blocks[0, 0].tolist()
        assert chosen[0] == 0 and chosen[2] == 3 and chosen[1] in (1, 2)


def test_many_entries_use_the_scan_launch():
    """More than 512 sequences, and more than 512 tiles of a prompt."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    new = [min(1, n) for n in lens]
    w = World(4, 64, 1, lens, 63)
    batch, _ = w.batch(new, max_new=1)
    q = bf(normal((sum(new), 64), 4))
    o, lse = w.cache.attend(batch, q)
    _g().model.sync_status(DEV)
    check_attend(w, new, f64(q), f64(o), f64(lse))
    w = World(8, 64, 1, [1100], 64)
    batch, _ = w.batch([1040])
    q = bf(normal((1040, 512), 4))
    o, lse = w.cache.attend(batch, q, window=50)
    _g().model.sync_status(DEV)
    check_attend(w, [1040], f64(q), f64(o), f64(lse), window=50)


def test_blocks_beyond_four_gigabytes():
    """Tiles whose byte offsets pass 2^32."""
    g = _g()
    bits, hd, Hkv = 8, 128, 10
    small = World(bits, hd, Hkv, [300], 65)
    far = (1 << 32) // (Hkv * 2 * O.kv.geometry(bits, hd)[2]) + 11
    cache = g.KVCache(far + small.n_blocks, Hkv, hd, bits=bits,
                      tiles=torch.empty((far + small.n_blocks, Hkv, small.cache.tiles.shape[2]), dtype=torch.uint8,
                                        device=DEV), bounds=True)
    cache.tiles[far:] = small.cache.tiles
    cache.bounds[far:] = small.cache.bounds
    table = np.where(small.table >= 0, small.table + far, -1)
    batch = g.KVBatch(i32(table), i32([300]), i32([0, 2]), max_new=2)
    q = bf(normal((2, Hkv * hd), 4))
    o, lse = cache.attend(batch, q)
    b2, _ = small.batch([2])
    o2, lse2 = small.cache.attend(b2, q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    raw = bf(normal((2, 3 * Hkv * hd), 5))
    cache.append(batch, raw, Hkv)
    small.cache.append(b2, raw, Hkv)
    k, v = cache.read(batch, 2)
    k2, v2 = small.cache.read(b2, 2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert torch.equal(cache.bounds[far:].view(torch.int16), small.cache.bounds.view(torch.int16))
    assert torch.equal(cache.select(batch, q, 3)[0], small.cache.select(b2, q, 3)[0])
    g.model.sync_status(DEV)


# ---------------------------------------------------------------------------- selection

SELECT = [
    # bits, hd, H, Hkv, lens, new, n_select, n_first, n_last
    (4, 128, 2, 2, [1, 64, 65, 1000, 0], [1, 1, 1, 1, 0], 4, 1, 1),
    (8, 64, 4, 2, [700, 130], [3, 5], 5, 0, 0),
    (8, 128, 8, 1, [900, 64], [2, 1], 1, 0, 1),
    (4, 64, 3, 3, [1500], [1], 9, 2, 3),
    (8, 64, 32, 1, [300], [1], 3, 0, 0),
    (8, 64, 1, 1, [200], [1], 50, 1, 1),           # more than there are
]


@pytest.mark.parametrize("case", SELECT)
def test_selection_matches_the_oracle_and_feeds_attention(case):
    bits, hd, H, Hkv, lens, new, n, n_first, n_last = case
    w = World(bits, hd, Hkv, lens, 70)
    batch, cu = w.batch(new)
    M = sum(new)
    q = bf(normal((M + 1, H * hd), 4))
    blocks = torch.full((M + 1, Hkv, n), 77, dtype=torch.int32, device=DEV)
    scores = torch.full((M + 1, Hkv, w.W), 77.0, device=DEV)
    w.cache.select(batch, q, n, n_first=n_first, n_last=n_last, blocks=blocks, scores=scores)
    o, lse = w.cache.attend(batch, q, blocks=blocks)
    _g().model.sync_status(DEV)
    assert torch.all(blocks[M] == 77) and torch.all(scores[M] == 77.0)
    got, sc, qf = blocks.cpu().numpy(), f64(scores), f64(q)
    for b, m0 in enumerate(cu[:-1]):
        for i in range(new[b]):
            nb = (lens[b] - new[b] + i) // 64 + 1
            ref = O.kv.block_scores(qf[m0 + i].reshape(H, hd), w.bounds[w.table[b, :nb]])
            assert np.all(np.abs(sc[m0 + i, :, :nb] - ref) <= 2.0 ** -24 * np.abs(ref) + 1e-300)
            assert np.all(sc[m0 + i, :, nb:] == -np.inf)
            for h in range(Hkv):
                want = O.kv.choose(sc[m0 + i, h, :nb], n, n_first, n_last)
                assert got[m0 + i, h].tolist() == want + [-1] * (n - len(want))
    check_attend(w, new, qf, f64(o), f64(lse), sel=got)


def test_selection_ties_and_nan_scores():
    w = World(8, 64, 1, [64 * 600], 71)
    g = _g()
    batch, _ = w.batch([1])
    w.cache.bounds.zero_()
    q = bf(np.ones((1, 64)))
    top = [3, 77, 300, 301, 555]
    for j in top:
        w.cache.bounds[w.table[0, j]] = 1.0
    blocks, scores = w.cache.select(batch, q, 8, n_first=0, n_last=0)
    assert blocks[0, 0].tolist() == [0, 1, 2, 3, 77, 300, 301, 555]
    blocks, _ = w.cache.select(batch, q, 3, n_first=0, n_last=1)
    assert blocks[0, 0].tolist() == [3, 77, 599]
    w.cache.bounds[w.table[0, 400]] = float("nan")
    w.cache.bounds[w.table[0, 7]] = -1.0
    blocks, scores = w.cache.select(batch, q, 2, n_first=0, n_last=1)
    assert blocks[0, 0].tolist() == [400, 599] and torch.isnan(scores[0, 0, 400])
    blocks, _ = w.cache.select(batch, -q, 300, n_first=0, n_last=0)    # -1, 0 and 1 change places
    got = blocks[0, 0].tolist()
    assert 7 in got and 400 in got and not set(top) & set(got) and got == sorted(got)
    rest = [j for j in range(600) if j not in top and j not in (7, 400)][:298]
    assert got == sorted(rest + [7, 400])
    g.model.sync_status(DEV)


def test_attention_over_a_list_of_the_callers_own():
    """Entries that are negative or not visible are passed over; one listed twice counts twice."""
    w = World(4, 128, 2, [400, 130], 72)
    g = _g()
    batch, _ = w.batch([2, 1])
    q = bf(normal((3, 512), 4))
    sel = np.full((3, 2, 6), -1)
    sel[0, 0] = [2, -1, 2, 99, 0, 5]
    sel[0, 1] = [-5, -1, -1, -1, -1, -1]           # nothing: a row without keys
    sel[1, 0] = [6, 5, 4, 3, 2, 1]
    sel[1, 1] = [6, 7, -1, 6, 6, 0]
    sel[2, 0] = [2, 1, 0, 2, 2, 2]                 # three are visible: three entries are read
    sel[2, 1] = [1, 3, 2, 0, 0, 0]
    o, lse = w.cache.attend(batch, q, blocks=i32(sel))
    g.model.sync_status(DEV)
    check_attend(w, [2, 1], f64(q), f64(o), f64(lse), sel=sel)


@pytest.mark.parametrize("bits,hd,G,new", [(8, 128, 2, 12), (4, 64, 3, 7), (4, 128, 1, 3)])
def test_many_short_sequences(bits, hd, G, new):
    """More rows to join than a grid that scans the batch itself takes, fewer entries than need a scan of
    their own; sequences of very different lengths, the shortest without a key of an earlier call."""
    rng = np.random.default_rng(hd + G)
    lens = [int(x) for x in rng.integers(1, 400, 90)]
    lens[:3] = [0, 1, new]
    n = [min(new, x) for x in lens]
    w = World(bits, hd, 2, lens, 81)
    batch, cu = w.batch(n, max_new=new)
    q = bf(normal((cu[-1], 2 * G * hd), 5))
    o, lse = w.cache.attend(batch, q)
    _g().model.sync_status(DEV)
    check_attend(w, n, f64(q), f64(o), f64(lse))


def test_selection_of_many_rows_and_many_blocks():
    """More rows than a CTA scans by itself; more blocks than the choice keeps in shared memory.  Blocks
    may recur in a table: 5000 entries over five cache blocks, so that most scores are ties."""
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 200, 600)]
    new = [min(1 + b % 2, n) for b, n in enumerate(lens)]
    w = World(8, 64, 1, lens, 73)
    batch, cu = w.batch(new, max_new=2)
    M = sum(new)
    q = bf(normal((M, 128), 4))
    blocks, scores = w.cache.select(batch, q, 2, n_first=0, n_last=1)
    o, lse = w.cache.attend(batch, q, blocks=blocks)
    _g().model.sync_status(DEV)
    got, sc = blocks.cpu().numpy(), f64(scores)
    for b, m0 in enumerate(cu[:-1]):
        for i in range(new[b]):
            nb = (lens[b] - new[b] + i) // 64 + 1
            want = O.kv.choose(sc[m0 + i, 0, :nb], 2, 0, 1)
            assert got[m0 + i, 0].tolist() == want + [-1] * (2 - len(want))
    check_attend(w, new, f64(q), f64(o), f64(lse), sel=got)

    w = World(4, 64, 2, [64 * 5], 74)
    W = 5000
    at = rng.integers(0, 5, W)
    table = w.table[0, at][None]
    n = W * 64 - 20
    batch = _g().KVBatch(i32(table), i32([n]))
    q = bf(normal((1, 256), 5))
    blocks, scores = w.cache.select(batch, q, 300, n_first=2, n_last=3)
    sc = f64(scores)[0]
    for h in range(2):
        assert blocks[0, h].tolist() == O.kv.choose(sc[h], 300, 2, 3)
    o, lse = w.cache.attend(batch, q)
    _g().model.sync_status(DEV)
    # 320k keys, as 320 with the number of times that each occurs
    times = np.repeat(np.bincount(at, minlength=5), 64).astype(float)
    times[at[-1] * 64 + 44:at[-1] * 64 + 64] -= 1
    wt = np.repeat(times[None], 2, 0)
    ro, rl, av = O.kv.attend(f64(q)[0].reshape(4, 64), w.k[0], w.v[0], wt)
    to, tl = attend_bounds(w, 0, f64(q)[0].reshape(4, 64), ro, rl, av, wt)
    assert np.all(np.abs(f64(o)[0].reshape(4, 64) - ro) <= to) and np.all(np.abs(f64(lse)[0] - rl) <= tl)


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("bits,hd,H,Hkv", [(8, 128, 2, 2), (4, 64, 4, 2)])
def test_a_layer_answers_step_by_step(bits, hd, H, Hkv):
    """A prompt, then single tokens: each step appends, selects and attends, and must equal the
    oracle's attention over the values the cache holds; and with everything in view, the prompt's rows
    come near the framework's own attention over unquantised keys (8 bits: the quantiser's half step,
    1/254 of a row's largest, against scores of order one)."""
    g = _g()
    n0, steps = 150, 70
    total = n0 + steps
    raw = torch.from_numpy(synth.normal((total, (H + 2 * Hkv) * hd), 8)).bfloat16().to(DEV)
    cache = g.KVCache(8, Hkv, hd, bits=bits, device=DEV)
    table = i32([[5, 2, 7, 0]])
    lens, cu = i32([n0]), i32([0, n0])
    prompt = g.KVBatch(table, lens, cu, max_new=n0)
    q = cache.append(prompt, raw[:n0].contiguous(), H)
    o, lse = cache.attend(prompt, q)
    w = World.__new__(World)
    w.bits, w.hd, w.Hkv, w.W = bits, hd, Hkv, 4

    def held():
        k, v = O.kv.unpack(cache.tiles.cpu().numpy()[[5, 2, 7, 0]], bits, hd)
        w.lens = [int(lens.item())]
        w.k = [k.transpose(0, 2, 1, 3).reshape(-1, Hkv, hd)[:w.lens[0]]]
        w.v = [v.transpose(0, 2, 1, 3).reshape(-1, Hkv, hd)[:w.lens[0]]]

    held()
    check_attend(w, [n0], f64(q), f64(o), f64(lse))
    if bits == 8 and H == Hkv:
        f = g.ops.attention_fwd(raw[:n0].contiguous(), 1, n0, H, hd)
        d = (f["o"].float() - o.float())
        assert d.norm() <= 2e-2 * f["o"].float().norm()
    one = g.KVBatch(table, lens)
    for t in range(n0, total):
        lens.fill_(t + 1)
        q = cache.append(one, raw[t:t + 1].contiguous(), H)
        o, lse = cache.attend(one, q)
        blocks, _ = cache.select(one, q, 2, n_first=0, n_last=1)
        so, sl = cache.attend(one, q, blocks=blocks)
        if t % 23 == 0 or t == total - 1:
            held()
            check_attend(w, [1], f64(q), f64(o), f64(lse), what=t)
            check_attend(w, [1], f64(q), f64(so), f64(sl), sel=blocks.cpu().numpy(), what=t)
    g.model.sync_status(DEV)


def test_a_captured_step_replays_with_new_contents():
    g = _g()
    H = Hkv = 2
    hd = 128
    w = World(8, hd, Hkv, [190, 64, 300], 80)
    lens, table = i32(w.lens), i32(w.table)
    batch = g.KVBatch(table, lens)
    raw = bf(normal((3, 3 * H * hd), 5))

    def step():
        q = w.cache.append(batch, raw, H)
        blocks, scores = w.cache.select(batch, q, 3)
        return (q, blocks, scores, *w.cache.attend(batch, q), *w.cache.attend(batch, q, blocks=blocks))

    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(DEV).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    tiles = w.cache.tiles.clone()
    for seed, new_lens in ((6, [190, 64, 300]), (7, [100, 3, 257]), (8, [64, 1, 299])):
        raw.copy_(bf(normal((3, 3 * H * hd), seed)))
        lens.copy_(i32(new_lens))
        w.cache.tiles.copy_(tiles)
        w.cache.bounds.copy_(bf(w.bounds))
        graph.replay()
        got = [t.clone() for t in out]
        w.cache.tiles.copy_(tiles)
        w.cache.bounds.copy_(bf(w.bounds))
        ref = step()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    g.model.sync_status(DEV)


def test_calls_on_two_streams_at_once():
    g = _g()
    w = World(4, 128, 4, [3000, 2500, 1800], 81)
    batch, _ = w.batch([1, 1, 1])
    qs = [bf(normal((3, 4 * 128), s)) for s in (4, 5)]
    want = [[t.clone() for t in w.cache.attend(batch, q)] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(w.cache.attend(batch, qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_two_captured_graphs_replay_at_once():
    """Each capture has scratch of its own: two graphs on two streams do not disturb one another."""
    w = World(8, 128, 2, [1500, 900, 2000], 83)
    batch, _ = w.batch([1, 1, 1])
    qs = [bf(normal((3, 256), s)) for s in (4, 5)]
    want = [[t.clone() for t in w.cache.attend(batch, q)] for q in qs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(DEV) for _ in qs]
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w.cache.attend(batch, q))
        graphs.append(g)
    for _ in range(20):
        for o, lse in outs:
            o.zero_(), lse.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, lse), (ro, rl) in zip(outs, want):
            assert torch.equal(o, ro) and torch.equal(lse, rl)


def test_first_call_of_a_process_may_be_captured():
    code = ("import torch, decoder_only_gpt_tcgen05_b200 as g\n"
            "d = torch.device('cuda:0')\n"
            "c = g.KVCache(4, 2, 128, bits=4, device=d)\n"
            "b = g.KVBatch(torch.tensor([[1, 3]], dtype=torch.int32, device=d), torch.tensor([70], dtype=torch.int32, device=d))\n"
            "x = torch.randn(1, 6 * 128, device=d).bfloat16()\n"
            "torch.cuda.synchronize()\n"
            "h = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(h):\n"
            "    q = c.append(b, x, 2); s = c.select(b, q, 2); o = c.attend(b, q, blocks=s[0]); k = c.read(b, 1)\n"
            "h.replay(); torch.cuda.synchronize(); g.model.sync_status(d)\n"
            "q2 = c.append(b, x, 2); o2 = c.attend(b, q2, blocks=c.select(b, q2, 2)[0])\n"
            "assert torch.equal(o[0], o2[0]) and torch.equal(q, q2) and torch.isfinite(o[1]).all()\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]


def test_rows_before_the_first_sequence_and_sequences_without_new_tokens():
    w = World(4, 128, 2, [100, 50, 300], 84)
    batch = _g().KVBatch(i32(w.table), i32(w.lens), i32([4, 6, 6, 9]), max_new=7)
    q = bf(normal((12, 256), 4))
    for blocks in (None, torch.zeros((12, 2, 1), dtype=torch.int32, device=DEV)):
        o, lse = torch.full_like(q, 7.0), torch.full((12, 2), 7.0, device=DEV)
        w.cache.attend(batch, q, blocks=blocks, o=o, lse=lse)
        _g().model.sync_status(DEV)
        for t in (o, lse):
            assert torch.all(t[:4] == 7.0) and torch.all(t[9:] == 7.0)
        sel = None if blocks is None else np.zeros((5, 2, 1), int)
        check_attend(w, [2, 0, 3], f64(q)[4:9], f64(o)[4:9], f64(lse)[4:9], sel=sel)


def test_binding_refuses_wrong_tensors():
    g = _g()
    w = World(8, 64, 2, [100], 82)
    batch, _ = w.batch([1])
    q = bf(normal((1, 256), 4))
    for bad in (q.float(), q[:, :100].contiguous(), q.cpu(), bf(normal((1, 512), 4))[:, ::2]):
        with pytest.raises(AssertionError):
            w.cache.attend(batch, bad)
    with pytest.raises(AssertionError):
        w.cache.attend(batch, q, blocks=i32(np.zeros((1, 1, 3))))
    with pytest.raises(AssertionError):
        w.cache.append(batch, q, 4)
    with pytest.raises(AssertionError):
        g.KVBatch(batch.block_table, batch.lens.long())
    with pytest.raises(AssertionError):
        g.KVBatch(batch.block_table, batch.lens, max_new=3)
    with pytest.raises(g.GptError):
        w.cache.select(batch, q, 1, n_first=1, n_last=1)
    with pytest.raises(g.GptError):
        g.KVCache(4, 2, 64, bits=8, device=DEV, bounds=False).select(batch, q, 2)
    with pytest.raises(g.GptError):
        w.cache.attend(batch, q, scratch=torch.empty(256, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("max_new", [0, -3, 7])
def test_the_field_max_new_does_not_matter_without_cu_new(max_new):
    """Through the C calls (the binding always passes 1): append, read, selection and attention of one token
    a sequence do the same work whatever the field holds."""
    import ctypes as C

    from decoder_only_gpt_tcgen05_b200._lib import KVBatchParams
    g = _g()
    H, hd = 4, 64
    raw = bf(normal((3, (H + 4) * hd), 6))
    outs = []
    for field in (1, max_new):
        w = World(8, hd, 2, [200, 130, 64], 90)
        lens, table = i32(w.lens), i32(w.table)
        b = C.byref(KVBatchParams(table.data_ptr(), lens.data_ptr(), None, 3, w.W, field))
        c, st = w.cache._ref, torch.cuda.current_stream(DEV).cuda_stream
        q = torch.full((3, H * hd), 7.0, dtype=torch.bfloat16, device=DEV)
        k = torch.full((3, 2, hd), 7.0, dtype=torch.bfloat16, device=DEV)
        v, o = k.clone(), q.clone()
        blocks = torch.full((3, 2, 3), 77, dtype=torch.int32, device=DEV)
        scores, lse = torch.full((3, 2, w.W), 7.0, device=DEV), torch.full((3, H), 7.0, device=DEV)
        n = C.c_size_t()
        g._lib.call("gpt_op_kv_append", c, b, raw.data_ptr(), 3, H, 1, 1, 1e4, 1e-5, q.data_ptr(), st)
        g._lib.call("gpt_op_kv_read", c, b, 3, k.data_ptr(), v.data_ptr(), st)
        g._lib.call("gpt_op_kv_select", c, b, q.data_ptr(), 3, H, 3, 1, 1, blocks.data_ptr(), scores.data_ptr(), st)
        g._lib.call("gpt_op_attention_kv_scratch_size", c, b, 3, H, 0, C.byref(n))
        scratch = torch.empty(n.value, dtype=torch.uint8, device=DEV)
        g._lib.call("gpt_op_attention_kv", c, b, q.data_ptr(), 3, H, -1, None, 0, o.data_ptr(), lse.data_ptr(),
                    scratch.data_ptr(), n.value, st)
        g.model.sync_status(DEV)
        outs.append((q, k, v, o, blocks, scores, lse, w.cache.tiles))
        assert not any(torch.all(t == 7) or torch.all(t == 77) for t in outs[-1])
    for x, y in zip(*outs):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits,hd,H,Hkv,new,window", [
    (8, 128, 2, 2, 4, -1), (4, 128, 4, 2, 6, -1), (8, 64, 8, 1, 5, -1), (4, 64, 1, 1, 3, -1),   # tiles of 4, 8 and 16
    (8, 128, 2, 2, 4, 0), (8, 128, 4, 1, 4, 70), (4, 128, 2, 2, 40, 20), (4, 64, 2, 1, 66, 64), (8, 64, 6, 2, 70, 31)])
def test_a_bad_block_number_shows_in_the_rows_that_see_its_keys(bits, hd, H, Hkv, new, window):
    """New tokens before, in and behind a block whose number is bad: NaN exactly in the rows of which a key
    lies in it, by causality and by the window."""
    g = _g()
    for first in (64 - new // 2, 128 - new // 2, 128, 192 - new // 2, 150):     # position of the first new token
        w = World(bits, hd, Hkv, [first + new], 91)
        q = bf(normal((new, H * hd), 4))
        for j in range((first + new - 1) // 64 + 1):
            table = w.table.copy()
            table[0, j] = w.n_blocks + 5
            o, lse = w.cache.attend(g.KVBatch(i32(table), i32(w.lens), i32([0, new]), max_new=new), q, window=window)
            p = np.arange(first, first + new)
            sees = (p >= 64 * j) & ((p - window <= 64 * j + 63) if window >= 0 else True)
            if sees.any():
                with pytest.raises(g.GptError):
                    g.model.sync_status(DEV)
            else:
                g.model.sync_status(DEV)
            on, ln = np.isnan(f64(o)), np.isnan(f64(lse))
            assert np.array_equal(on.all(1), sees) and np.array_equal(on.any(1), sees), (first, j)
            assert np.array_equal(ln.all(1), sees) and np.array_equal(ln.any(1), sees), (first, j)
            if not sees.all():
                part = np.flatnonzero(~sees)
                ref = w.cache.attend(w.batch([new])[0], q, window=window)
                for m in part:
                    n = first + m + 1
                    ro, rl, av = O.kv.attend(f64(q)[m].reshape(H, hd), w.k[0][:n], w.v[0][:n],
                                             np.repeat((np.arange(n) >= n - 1 - window if window >= 0 else np.ones(n))
                                                       [None].astype(float), Hkv, 0))
                    wt = np.zeros((Hkv, first + new))
                    wt[:, :n] = 1.0
                    to, tl = attend_bounds(w, 0, f64(q)[m].reshape(H, hd), ro, rl, av, wt)
                    assert np.all(np.abs(f64(o)[m].reshape(H, hd) - ro) <= to) and np.all(np.abs(f64(lse)[m] - rl) <= tl)
                assert np.all(np.isfinite(f64(ref[0])))


def test_a_bad_block_number_in_a_list_shows_in_its_row_only():
    g = _g()
    w = World(8, 128, 2, [140, 70], 92)
    table = w.table.copy()
    table[0, 1] = -9
    batch = g.KVBatch(i32(table), i32(w.lens), i32([0, 14, 16]), max_new=14)
    q = bf(normal((16, 256), 4))
    sel = np.zeros((16, 2, 2), int)
    sel[:, :, 1] = -1
    sel[3, 0], sel[5, 1] = [0, 1], [1, 0]         # positions 129 and 131 see block 1
    sel[9, 0] = [2, 0]
    o, lse = w.cache.attend(batch, q, blocks=i32(sel))
    with pytest.raises(g.GptError):
        g.model.sync_status(DEV)
    bad = np.zeros((16, 2), bool)
    bad[3, 0] = bad[5, 1] = True
    assert np.array_equal(np.isnan(f64(o).reshape(16, 2, 128)).all(-1), bad) and np.array_equal(np.isnan(f64(lse)), bad)
    assert np.array_equal(np.isnan(f64(o).reshape(16, 2, 128)).any(-1), bad)


@pytest.mark.parametrize("lens,cu,max_new", [
    ([200, 10 ** 6, 64], [0, 1, 4, 5], 3),        # longer than its block table
    ([200, -5, 64], [0, 1, 2, 3], 1),
    ([200, 130, 64], [0, 1, 9, 10], 1),           # more new tokens than max_new
    ([200, 2, 64], [0, 1, 5, 6], 4),              # more new tokens than tokens
    ([200, 130, 64], [0, 1, 2 ** 31 - 1, -2 ** 31], 1),
    ([200, 0, 64], None, 1),                      # no cu_new: one new token, but no tokens
])
def test_selection_leaves_the_rows_of_a_broken_sequence_as_they_are(lens, cu, max_new):
    w = World(8, 64, 2, [200, 130, 64], 62)
    g = _g()
    q = bf(normal((12, 256), 4))
    blocks = torch.full((12, 2, 3), 77, dtype=torch.int32, device=DEV)
    scores = torch.full((12, 2, w.W), 77.0, device=DEV)
    batch = g.KVBatch(i32(w.table), i32(lens), None if cu is None else i32(cu), max_new=max_new)
    w.cache.select(batch, q, 3, blocks=blocks, scores=scores)
    with pytest.raises(g.GptError) as e:
        g.model.sync_status(DEV)
    assert e.value.code == 1
    cu = [0, 1, 2, 3] if cu is None else cu
    good = [0] + ([cu[2]] if 0 <= cu[2] < 12 and cu[3] == cu[2] + 1 else [])
    rest = [m for m in range(12) if m not in good]
    assert torch.all(blocks[rest] == 77) and torch.all(scores[rest] == 77.0)
    assert blocks[0, :, 0].tolist() == [0, 0] and blocks[0, :, 2].tolist() == [3, 3] and not torch.any(scores[0] == 77.0)
    for m in good[1:]:
        assert blocks[m].tolist() == [[0, -1, -1]] * 2 and torch.all(scores[m, :, 1:] == -float("inf"))


def test_a_window_beyond_32_bits_is_no_window():
    """Python numbers are longer than the call's: a window of 2^40 must not become one of 0."""
    w = World(8, 64, 2, [300, 70], 93)
    batch, _ = w.batch([3, 2])
    q = bf(normal((5, 256), 4))
    o, lse = w.cache.attend(batch, q)
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 3, 2 ** 40, 2 ** 63 - 1):
        o2, lse2 = w.cache.attend(batch, q, window=window)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), window
    for window in (-2, -2 ** 31, -2 ** 32, -2 ** 40):
        with pytest.raises(_g().GptError):
            w.cache.attend(batch, q, window=window)


@pytest.mark.parametrize("case", [
    (8, 128, 10, 10, True, True, [70, 130, 64, 7], [4, 5, 6, 7]),      # a token for each lane group of 128 dims
    (4, 128, 8, 2, True, True, [66, 131, 3, 260], [7, 6, 3, 7]),       # in both blocks, in one, in none
    (4, 64, 12, 12, True, False, [66, 131, 7], [7, 5, 4]),             # none of 64 dims
    (8, 64, 9, 3, False, True, [66, 131, 8], [8, 7, 8]),
])
def test_append_of_a_few_drafted_tokens(case):
    """New tokens about as many as a warp has lane groups, which decides how tokens and heads are dealt."""
    test_append_and_read_match_the_oracle(case)


@pytest.mark.parametrize("bits,hd,H,Hkv,new,window", [
    (8, 128, 2, 2, 4, -1), (4, 128, 2, 2, 2, -1), (8, 64, 12, 2, 1, 40),      # tiles of 4 and 8 rows
    (8, 128, 2, 1, 4, -1), (4, 128, 4, 2, 3, -1), (4, 64, 4, 1, 2, -1), (8, 64, 6, 2, 2, 31),
    (8, 128, 4, 1, 4, -1), (4, 128, 4, 1, 5, -1), (4, 64, 2, 2, 40, 20), (8, 64, 2, 1, 66, 64)])     # of 16
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 40, 1e30])
def test_large_values_of_keys_that_a_row_does_not_see_leave_it_alone(bits, hd, H, Hkv, new, window, size):
    """A value row of any finite size, in the place of a newer token's or of one that has left the window,
    changes the rows that see it and no other: those stay within the tolerance of their own keys."""
    L = 150 + new
    for at in (L - 1, L - 1 - new // 2, L - 1 - new // 2 - max(window, 0)):      # the large value's position
        w = World(bits, hd, Hkv, [L], 94)
        R, ng, recb = O.kv.geometry(bits, hd)
        rec, tok = divmod(at % 64, 32)
        so = rec * recb + 2 * 32 * R + 64 * ng + tok * 2 * ng
        dst = w.cache.tiles[w.table[0, at // 64]][:, so:so + 2 * ng].clone().view(torch.bfloat16)
        w.cache.tiles[w.table[0, at // 64], :, so:so + 2 * ng] = (dst.float() * size).bfloat16().view(torch.uint8)
        q = bf(normal((new, H * hd), 4))
        o, lse = w.cache.attend(w.batch([new])[0], q, window=window)
        _g().model.sync_status(DEV)
        blind = 0
        for m in range(new):
            p = L - new + m
            lo = max(0, p - window) if window >= 0 else 0
            if lo <= at <= p:
                continue
            blind += 1
            wt = np.zeros((Hkv, L))
            wt[:, lo:p + 1] = 1.0
            qr = f64(q)[m].reshape(H, hd)
            ro, rl, av = O.kv.attend(qr, w.k[0], w.v[0], wt)
            to, tl = attend_bounds(w, 0, qr, ro, rl, av, wt)
            assert np.all(np.abs(f64(o)[m].reshape(H, hd) - ro) <= to), (at, m)
            assert np.all(np.abs(f64(lse)[m] - rl) <= tl), (at, m)
        assert blind > 0 or new == 1 or at == L - new


@pytest.mark.parametrize("bits,hd,H,Hkv,new", [
    (8, 128, 2, 2, 1), (4, 128, 2, 2, 1), (4, 64, 3, 3, 1), (4, 128, 8, 1, 1), (8, 64, 4, 2, 3), (8, 128, 2, 2, 9),
    (4, 128, 4, 1, 5)])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e9, 1e13, 1e25, 1e35])
def test_scores_of_any_finite_size_choose_the_largest(bits, hd, H, Hkv, new, size):
    """Scores far apart: the softmax is the largest one's value row and the logsumexp that score.  Looked at are
    the rows where the first is ahead by 50 (e^-50 of the rest) and by 2^-6 of itself, which is above what the
    scores can be off: 2^-11 of the largest |q| times a key's scale for 16 dims each."""
    w = World(bits, hd, Hkv, [130 + new, 40], 95, scale=size ** 0.5)
    w.v = [v / size ** 0.5 for v in w.v]
    R, ng, recb = O.kv.geometry(bits, hd)
    for b, n in enumerate(w.lens):
        _, vs, w.v[b] = O.kv.quantise(w.v[b], bits)
        vc, vs, _ = O.kv.quantise(w.v[b], bits)
        for j in range((n + 63) // 64):
            m = min(64, n - 64 * j)
            part = [np.zeros((Hkv, 64, hd), np.uint8), np.full((Hkv, 64, ng), np.nan)]
            part[0][:, :m], part[1][:, :m] = vc[64 * j:64 * j + m].transpose(1, 0, 2), vs[64 * j:64 * j + m].transpose(1, 0, 2)
            new_t = O.kv.pack(np.zeros_like(part[0]), np.full_like(part[1], np.nan), *part, bits).reshape(Hkv, 2, recb)
            old = w.cache.tiles[w.table[b, j]].view(Hkv, 2, recb)
            t = torch.from_numpy(new_t).to(DEV)
            old[:, :, 32 * R:64 * R] = t[:, :, 32 * R:64 * R]
            old[:, :, 64 * R + 64 * ng:] = t[:, :, 64 * R + 64 * ng:]
    batch, cu = w.batch([new, 1])
    q = bf(normal((new + 1, H * hd), 4) * size ** 0.5)
    o, lse = (f64(t) for t in w.cache.attend(batch, q))
    _g().model.sync_status(DEV)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse))
    seen = 0
    for b, n in enumerate((new, 1)):
        for i in range(n):
            m, L = cu[b] + i, w.lens[b] - n + i + 1
            for h in range(H):
                s = w.k[b][:L, h // (H // Hkv)] @ f64(q)[m].reshape(H, hd)[h] / np.sqrt(hd)
                a = np.argsort(s)
                if s[a[-1]] - s[a[-2]] < max(50.0, 2.0 ** -6 * np.abs(s).max()):
                    continue
                seen += 1
                v = w.v[b][a[-1], h // (H // Hkv)]
                got = o[m].reshape(H, hd)[h]
                assert np.all(np.abs(got - v) <= 2.0 ** -8 * np.abs(v) + 2.0 ** -11 * np.abs(v).max()), (b, i, h)
                assert abs(lse[m, h] - s[a[-1]]) <= 2.0 ** -8 * np.abs(s).max(), (b, i, h)
    assert seen > 0 or size < 1e6


@pytest.mark.parametrize("bits,hd,H,Hkv,new", [(8, 128, 2, 2, 1), (4, 128, 2, 2, 1), (4, 64, 6, 2, 2), (8, 64, 4, 1, 4),
                                               (4, 128, 5, 1, 3)])
def test_small_values_beside_a_dominant_key(bits, hd, H, Hkv, new):
    """A key with most of the weight and nearly all of its value zero: what the others leave is small next to
    the terms that are summed.  A product of 16 cuts each term off below 2^-15 of its largest weight times a code
    step (a subnormal operand's exponent counts as 2^-14, its mantissa has 10 bits), so a row is off by up to
    16 x 2^-15 = 2^-11 of sum_j p_j scale_j beside the other roundings, and a score by as much of the largest |q|
    times the key's scale for each 16 dims."""
    L = 100 + new
    w = World(bits, hd, Hkv, [L], 96)
    xk, xv = w.k[0].copy(), normal((L, Hkv, hd), 97)
    qv = normal((new, Hkv, H // Hkv, hd), 98)
    for i in range(new):
        for h in range(Hkv):
            qm = qv[i, h].mean(0)
            xk[5 + 20 * i, h] = 8 * np.sqrt(hd) * qm / (qm @ qm)      # a score of 8 on average
            xv[5 + 20 * i, h, 1:] = 0.0
            xv[5 + 20 * i, h, 0] = 3.0
    kc, ks, w.k[0] = O.kv.quantise(xk, bits)
    vc, vs, w.v[0] = O.kv.quantise(xv, bits)
    for j in range((L + 63) // 64):
        part = []
        for a in (kc, ks, vc, vs):
            t = np.zeros((Hkv, 64, a.shape[-1]), a.dtype)
            m = min(64, L - 64 * j)
            t[:, :m] = a[64 * j:64 * j + m].transpose(1, 0, 2)
            part.append(t)
        w.cache.tiles[w.table[0, j]] = torch.from_numpy(O.kv.pack(*part, bits)).to(DEV)
    batch, _ = w.batch([new])
    q = bf(qv.reshape(new, H * hd))
    o, lse = (f64(t) for t in w.cache.attend(batch, q))
    _g().model.sync_status(DEV)
    G, Z = H // Hkv, 1 << (bits - 1)
    top = 0.0
    for i in range(new):
        n = L - new + i + 1
        qr = f64(q)[i].reshape(H, hd)
        ro, rl, av = O.kv.attend(qr, w.k[0][:n], w.v[0][:n], np.ones((Hkv, n)))
        for h in range(H):
            ksc, vsc = (np.abs(x[:n, h // G]).max(-1) / (Z - 1) * (1 + 2.0 ** -7) for x in (w.k[0], w.v[0]))
            p = np.exp(w.k[0][:n, h // G] @ qr[h] / np.sqrt(hd) - rl[h])
            top = max(top, p.max())
            es = (2.0 ** -20 * np.abs(qr[h]).sum() * 2 * Z + 2.0 ** -11 * hd / 16 * np.abs(qr[h]).max()) * ksc.max() / np.sqrt(hd)
            to = 2.0 ** -8 * np.abs(ro[h]) + (2.0 ** -11 + 2 * es) * av[h] + 2.0 ** -11 * (p * vsc).sum() + \
                2.0 ** -20 * 2 * Z * (p * vsc).sum()
            assert np.all(np.abs(o[i].reshape(H, hd)[h] - ro[h]) <= to * (1 + 2.0 ** -6)), (i, h)
            assert abs(lse[i, h] - rl[h]) <= es + 2.0 ** -21 * (1 + abs(rl[h])), (i, h)
    assert top > 0.9

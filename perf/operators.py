"""The cached-attention operators as measured: append to a quantised key/value cache, read it back,
attend over it, and attend over blocks selected by a cheap score.

``run`` gives the operators in plain 32-bit torch operations, or, with ``own`` set, through this
package's KVCache.  Both read and write the same bytes: the cache tile layout of include/gpt_ops.h,
restated by ``_perms`` below.
"""
import math

import torch

own = False

BLOCK, REC = 64, 32           # tokens of a cache block, and of one record of its tile
DEV = "cuda:0"


# ---------------------------------------------------------------------------- cases

def listed():
    d20 = dict(H=10, Hkv=10, hd=128, rope=True, norm=True)
    gpt2 = dict(H=12, Hkv=12, hd=64, rope=False, norm=False)
    d26 = dict(H=13, Hkv=13, hd=128, rope=True, norm=True)
    grouped = dict(H=16, Hkv=2, hd=128, rope=True, norm=True)
    return [
        # one decoding step of the d20 batch: one new token for each of 16 sequences
        dict(name="append_step_kv8", op="append", bits=8, B=16, lo=1, hi=2048, new=1, window=-1, select=0, **d20),
        # prompts of uneven lengths entering a 4-bit cache (the d20 training batch's 16 x 2048 at most)
        dict(name="append_prompts_kv4", op="append", bits=4, B=16, lo=301, hi=2048, new=2048, window=-1, select=0, **d20),
        # chunks of prompts on the GPT-2 shape (no RoPE, no QK-norm, heads of 64)
        dict(name="append_chunks_gpt2_kv8", op="append", bits=8, B=8, lo=129, hi=1024, new=129, window=-1, select=0, **gpt2),
        # reading one short sequence back
        dict(name="read_one_kv4", op="read", bits=4, B=1, lo=777, hi=777, new=777, window=-1, select=0, **d20),
        # reading a whole d26 batch back
        dict(name="read_batch_d26_kv8", op="read", bits=8, B=16, lo=1500, hi=2048, new=2048, window=-1, select=0, **d26),
        # latency of one sequence's decoding step
        dict(name="attend_one_kv4", op="attend", bits=4, B=1, lo=2047, hi=2047, new=1, window=-1, select=0, **d20),
        # an ordinary decoding step: 64 sequences of uneven lengths
        dict(name="attend_step_kv8", op="attend", bits=8, B=64, lo=65, hi=2048, new=1, window=-1, select=0, **d20),
        # several new tokens a sequence (drafted ones to be checked), grouped heads, a left window
        dict(name="attend_draft_window_kv8", op="attend", bits=8, B=24, lo=200, hi=8192, new=5, window=1023, select=0, **grouped),
        # long contexts held in 4 bits: the largest
        dict(name="attend_long_kv4", op="attend", bits=4, B=32, lo=16384, hi=32768, new=1, window=-1, select=0, **d20),
        # one sequence, a few selected blocks, heads of 64
        dict(name="sparse_one_gpt2_kv8", op="sparse", bits=8, B=1, lo=8100, hi=8100, new=1, window=-1, select=24, **gpt2),
        # a decoding step that attends to 64 of up to 512 blocks
        dict(name="sparse_step_kv4", op="sparse", bits=4, B=16, lo=4097, hi=32768, new=1, window=-1, select=64, **d20),
        # the same in 8 bits for grouped heads and two new tokens a sequence
        dict(name="sparse_draft_kv8", op="sparse", bits=8, B=32, lo=2000, hi=16384, new=2, window=-1, select=33, **grouped),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    op = rng.choice(["append", "read", "attend", "attend", "sparse"])
    H, Hkv, hd = rng.choice([(10, 10, 128), (13, 13, 128), (12, 12, 64), (16, 2, 128), (8, 4, 64), (12, 1, 128)])
    B = log(1, 64)
    # the cost of a case is about B x length x heads: keep it below the largest listed one
    cap = {"append": 32768, "read": 32768, "attend": 500000, "sparse": 260000}[op]
    hi = max(2, min(32768 if op in ("attend", "sparse") else 2048, cap * 10 // (B * Hkv), cap // B))
    hi = max(1, log(1, hi))
    lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
    if op in ("append", "read"):
        new = rng.choice([1, log(1, hi), hi])
    else:
        new = rng.choice([1, 1, log(1, min(8, hi))])
    window = rng.choice([-1, -1, log(1, 4096)]) if op == "attend" else -1
    select = log(2, 96) if op == "sparse" else 0
    if op == "sparse":
        new = min(new, 2)
    return dict(op=op, bits=rng.choice([4, 8]), B=B, lo=lo, hi=hi, new=new, window=window, select=select,
                H=H, Hkv=Hkv, hd=hd, rope=rng.random() < 0.8, norm=rng.random() < 0.8)


def _lengths(case):
    """Lengths of the sequences (new tokens included) and how many new tokens each has: plain numbers
    spread over [lo, hi], the same for every seed, so that a case has one size."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [hi if b == 0 else lo + (hi - lo) * ((b * 37 + 11) % B) // B for b in range(B)]
    return lens, [min(case["new"], n) for n in lens]


# ---------------------------------------------------------------------------- the tile layout

def _sizes(case):
    bits, hd = case["bits"], case["hd"]
    rowb = hd * bits // 8
    ng = hd // 64 if bits == 4 else 1
    return rowb, ng, 2 * REC * rowb + 4 * REC * ng


def _perms(case, dev):
    """Byte offsets within a record of key and value rows' bytes: two [REC, rowb] tables."""
    bits = case["bits"]
    rowb, ng, _ = _sizes(case)
    i = torch.arange(REC, device=dev)[:, None]
    lb = torch.arange(rowb, device=dev)[None, :]
    t, ii = i // 16, i % 16
    # keys: 32-bit word w of a row goes to lane w % 4 of the row's four
    kb = rowb // 4
    p = min(kb, 16)
    c, y = (lb // 4) % 4, (lb // 16) * 4 + lb % 4
    kperm = t * 16 * rowb + (y // p) * 64 * p + ii * 4 * p + c * p + y % p
    # values: octet o (8 dims) goes to lane row o % 8; the four keys of a lane are stored together
    ob = bits
    o = lb // ob
    r, y = o % 8, (o // 8) * ob + lb % ob
    c, s = (ii % 8) // 2, ii % 2 + 2 * (ii // 8)
    z = s * (rowb // 8) + y
    vperm = REC * rowb + t * 16 * rowb + (z // 16) * 512 + (4 * r + c) * 16 + z % 16
    return kperm, vperm


def _codes_to_values(b, scale, bits, hd, ng):
    """Natural-order code bytes [..., rowb] and scales [..., ng] to values [..., hd]."""
    if bits == 4:
        u = torch.stack((b & 15, b >> 4), -1).flatten(-2).float() - 8.0
    else:
        u = b.float() - 128.0
    return (u.unflatten(-1, (ng, hd // ng)) * scale.float()[..., None]).flatten(-2)


def _decode(case, tiles):
    """Tiles [..., tile bytes] to keys and values [..., BLOCK, hd], 32 bits."""
    bits, hd = case["bits"], case["hd"]
    rowb, ng, recb = _sizes(case)
    kperm, vperm = _perms(case, tiles.device)
    rec = tiles.unflatten(-1, (2, recb))
    sc = rec[..., 2 * REC * rowb:].contiguous().view(torch.bfloat16).unflatten(-1, (2, REC, ng))
    out = []
    for which, perm in ((0, kperm), (1, vperm)):
        b = rec[..., perm.flatten()].unflatten(-1, (REC, rowb))
        v = _codes_to_values(b, sc[..., which, :, :], bits, hd, ng)
        out.append(v.flatten(-3, -2))
    return out


def _quantise(x, bits, ng):
    """Rows [..., hd] (32 bits) to natural-order code bytes, scales (bf16) and the values they stand for."""
    top = 7 if bits == 4 else 127
    g = x.float().unflatten(-1, (ng, x.shape[-1] // ng))
    s = (g.abs().amax(-1) / top).bfloat16()
    sf = s.float()[..., None]
    n = torch.where(sf > 0, torch.round(g / sf), torch.zeros_like(g)).clamp(-top, top)
    u = (n + (top + 1)).flatten(-2).to(torch.uint8)
    b = u[..., 0::2] | (u[..., 1::2] << 4) if bits == 4 else u
    return b, s, (n * sf).flatten(-2)


def _bounds_of(k, live=None):
    """Elementwise bounds of the keys [..., tokens, hd] of a block as bf16 [..., 2, hd], rounded outward."""
    lo, hi = (k, k) if live is None else (torch.where(live, k, torch.inf), torch.where(live, k, -torch.inf))
    out = []
    for v, sign in ((lo.amin(-2), -1.0), (hi.amax(-2), 1.0)):
        r = v.bfloat16()
        off = (r.float() - v) * sign < 0          # rounded inward: one step further out
        bits = r.view(torch.int16).to(torch.int32)
        away = (v * sign) > 0                      # outward is away from zero
        bits = torch.where(off, torch.where(away, bits + 1, bits - 1), bits)
        out.append(bits.to(torch.int16).view(torch.bfloat16))
    return torch.stack(out, -2)


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device(DEV)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, H, Hkv, hd, bits = (case[k] for k in ("B", "H", "Hkv", "hd", "bits"))
    rowb, ng, recb = _sizes(case)
    lens, new = _lengths(case)
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    n_blocks, width = sum(need) + 3, max(need) + 1
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    perm = torch.randperm(n_blocks, generator=gen, device=dev).to(torch.int32)
    at = [0]
    for n in need:
        at.append(at[-1] + n)
    first = torch.tensor(at[:-1], device=dev)[:, None]
    j = torch.arange(width, device=dev)[None, :]
    used = j < torch.tensor(need, device=dev)[:, None]
    table = torch.where(used, perm[torch.clamp(first + j, max=n_blocks - 1)], -1).to(torch.int32).contiguous()
    state = dict(case=dict(case), table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                 cu=torch.tensor(cu, dtype=torch.int32, device=dev), rows=cu[-1], max_new=max(new))
    if case["op"] == "append":
        state["tiles"] = torch.zeros((n_blocks, Hkv, 2 * recb), dtype=torch.uint8, device=dev)
        state["bounds"] = torch.zeros((n_blocks, Hkv, 2, hd), dtype=torch.bfloat16, device=dev)
        state["qkv"] = torch.randn((cu[-1], (H + 2 * Hkv) * hd), generator=gen, device=dev).bfloat16()
        return state
    tiles = torch.empty((n_blocks, Hkv, 2 * recb), dtype=torch.uint8, device=dev)
    bounds = torch.empty((n_blocks, Hkv, 2, hd), dtype=torch.bfloat16, device=dev)
    kperm, vperm = _perms(case, dev)
    step = max(1, (1 << 25) // (Hkv * BLOCK * hd))
    for a in range(0, n_blocks, step):
        n = min(step, n_blocks - a)
        part = tiles[a:a + n].unflatten(-1, (2, recb))
        sc = []
        for which, perm in ((0, kperm), (1, vperm)):
            x = torch.randn((n, Hkv, 2, REC, hd), generator=gen, device=dev)
            if which == 0 and case["op"] == "sparse":
                # keys of a block lie near one another: what makes a block's score tell it apart
                x = 0.6 * x + 0.8 * torch.randn((n, Hkv, 1, 1, hd), generator=gen, device=dev)
            b, s, val = _quantise(x, bits, ng)
            part[..., perm.flatten()] = b.flatten(-2)
            sc.append(s)
            if which == 0:
                bounds[a:a + n] = _bounds_of(val.flatten(2, 3))
        part[..., 2 * REC * rowb:] = torch.stack(sc, 3).flatten(3).contiguous().view(torch.uint8)
    state["tiles"], state["bounds"] = tiles, bounds
    if case["op"] != "read":
        state["q"] = torch.randn((cu[-1], H * hd), generator=gen, device=dev).bfloat16()
    return state


# ---------------------------------------------------------------------------- plain forms

def _rows(state):
    """Sequence and position of every row, as index tensors."""
    cu = state["cu"].long()
    m = torch.arange(state["rows"], device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), m, right=True)
    i = m - cu[b]
    return b, i, state["lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _plain_append(state):
    case = state["case"]
    H, Hkv, hd, bits = (case[k] for k in ("H", "Hkv", "hd", "bits"))
    rowb, ng, recb = _sizes(case)
    b, _, pos = _rows(state)
    x = state["qkv"].float().unflatten(-1, (H + 2 * Hkv, hd))
    qk, v = x[:, :H + Hkv], x[:, H + Hkv:]
    if case["rope"]:
        f = 10000.0 ** (-torch.arange(hd // 2, device=x.device, dtype=torch.float64) * 2 / hd)
        phi = pos.double()[:, None] * f
        cos, sin = phi.cos().float()[:, None], phi.sin().float()[:, None]
        x1, x2 = qk[..., :hd // 2], qk[..., hd // 2:]
        qk = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
    if case["norm"]:
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + 1e-5)
    q, k = qk[:, :H], qk[:, H:]
    phys = state["table"].long()[b, pos // BLOCK]
    rec, tok = (pos % BLOCK) // REC, pos % REC
    tiles = state["tiles"].unflatten(-1, (2, recb))
    heads = torch.arange(Hkv, device=x.device)[None, :, None]
    for which, rows, perm in zip((0, 1), (k, v), _perms(case, x.device)):
        code, s, val = _quantise(rows, bits, ng)
        where = (phys[:, None, None], heads, rec[:, None, None])
        tiles[(*where, perm[tok][:, None, :])] = code
        so = 2 * REC * rowb + which * 2 * REC * ng + (tok[:, None] * ng * 2 + torch.arange(2 * ng, device=x.device))
        tiles[(*where, so[:, None, :])] = s.contiguous().view(torch.uint8)
        if which == 0:
            kval = val
    # bounds of the touched blocks: those of the new tokens, joined with what the block had before
    # unless its first token is among the new ones
    key = b * state["table"].shape[1] + pos // BLOCK
    nseg = state["table"].numel()
    idx = key[:, None, None].expand_as(kval)
    lo = torch.full((nseg, Hkv, hd), torch.inf, device=x.device).scatter_reduce(0, idx, kval, "amin")
    hi = torch.full((nseg, Hkv, hd), -torch.inf, device=x.device).scatter_reduce(0, idx, kval, "amax")
    fresh = torch.zeros(nseg, device=x.device).scatter_reduce(0, key, (pos % BLOCK == 0).float(), "amax") > 0
    new = _bounds_of(torch.stack((lo, hi), 2))
    old = state["bounds"][phys]
    fr = fresh[key][:, None, None]
    new = new[key]
    state["bounds"][phys] = torch.stack((torch.where(fr, new[:, :, 0], torch.minimum(new[:, :, 0], old[:, :, 0])),
                                         torch.where(fr, new[:, :, 1], torch.maximum(new[:, :, 1], old[:, :, 1]))), 2)
    return q.flatten(1).bfloat16()


def _plain_read(state):
    b, _, pos = _rows(state)
    k, v = _decode(state["case"], state["tiles"][state["table"].long().clamp(min=0)])
    return [x[b, pos // BLOCK, :, pos % BLOCK].bfloat16() for x in (k, v)]


def _softmax_av(s, live, v):
    """Masked softmax of s [..., rows, keys] times v [..., keys, hd], and the logsumexp."""
    s = torch.where(live, s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = torch.where(z > 0, (p @ v) / z, 0.0)
    return o, (m + torch.log(z))[..., 0]


def _plain_attend(state):
    case = state["case"]
    B, H, Hkv, hd, win = (case[k] for k in ("B", "H", "Hkv", "hd", "window"))
    G, n = H // Hkv, state["max_new"]
    b, i, pos = _rows(state)
    table = state["table"].long().clamp(min=0)
    k, v = _decode(case, state["tiles"][table])                       # [B, blocks, Hkv, BLOCK, hd]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))          # [B, Hkv, keys, hd]
    q = torch.zeros((B, n, Hkv, G, hd), device=k.device)
    q[b, i] = state["q"].float().view(-1, Hkv, G, hd)
    p = torch.full((B, n), -1, device=k.device)
    p[b, i] = pos
    j = torch.arange(k.shape[2], device=k.device)
    live = j <= p[..., None]
    if win >= 0:
        live = live & (j >= p[..., None] - win)
    s = (q.permute(0, 2, 1, 3, 4).flatten(2, 3) @ k.transpose(-1, -2)) / math.sqrt(hd)
    o, lse = _softmax_av(s, live[:, None, :, None].expand(-1, 1, -1, G, -1).flatten(2, 3), v)
    o = o.unflatten(2, (n, G)).permute(0, 2, 1, 3, 4)[b, i]
    lse = lse.unflatten(2, (n, G)).permute(0, 2, 1, 3)[b, i]
    return [o.flatten(1).bfloat16(), lse.flatten(1)]


N_FIRST, N_LAST = 1, 2


def _plain_sparse(state):
    case = state["case"]
    H, Hkv, hd, n = (case[k] for k in ("H", "Hkv", "hd", "select"))
    n = max(n, N_FIRST + N_LAST)
    G = H // Hkv
    b, _, pos = _rows(state)
    table = state["table"].long()[b].clamp(min=0)                      # [rows, blocks]
    W = table.shape[1]
    bd = state["bounds"][table].double()                               # [rows, W, Hkv, 2, hd]
    q = state["q"].view(-1, 1, Hkv, G, hd)
    qd = q.double()
    # next to the border between chosen and not, order counts: 64 bits, rounded once
    sc = torch.zeros(bd.shape[:3], dtype=torch.float64, device=q.device)
    sc = sc + torch.maximum(qd * bd[..., None, 0, :], qd * bd[..., None, 1, :]).sum((-1, -2))
    sc = sc.float().transpose(1, 2)                                    # [rows, Hkv, W]
    nb = (pos // BLOCK + 1)[:, None, None]
    jb = torch.arange(W, device=q.device)
    sc = torch.where(jb < nb, sc, -torch.inf)
    forced = ((jb < N_FIRST) | (jb >= nb - N_LAST)) & (jb < nb)
    key = torch.where(forced, torch.inf, sc)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :n]
    if n > W:
        order = torch.cat((order, torch.full((*order.shape[:2], n - W), W, device=q.device)), -1)
    pick = torch.where((torch.arange(n, device=q.device) < nb) & (order < W), order, W).sort(-1).values
    blocks = torch.where(pick < W, pick, -1)
    phys = table[torch.arange(len(b), device=q.device)[:, None, None], blocks.clamp(min=0)]
    k, v = _decode(case, state["tiles"][phys, torch.arange(Hkv, device=q.device)[None, :, None]])
    k, v = k.flatten(2, 3), v.flatten(2, 3)                            # [rows, Hkv, keys, hd]
    j = (blocks[..., None] * BLOCK + torch.arange(BLOCK, device=q.device)).flatten(2)
    live = (j >= 0) & (j <= pos[:, None, None]) & (blocks >= 0).repeat_interleave(BLOCK, -1)
    s = (q[:, 0].float() @ k.transpose(-1, -2)) / math.sqrt(hd)
    o, lse = _softmax_av(s, live[:, :, None], v)
    return [blocks.to(torch.int32), sc, o.flatten(1).bfloat16(), lse.flatten(1)]


# ---------------------------------------------------------------------------- one pass

def _handles(state):
    """The cache and batch objects that a program keeps between its calls."""
    if "cache" not in state:
        import decoder_only_gpt_tcgen05_b200 as g
        case = state["case"]
        state["cache"] = g.KVCache(state["tiles"].shape[0], case["Hkv"], case["hd"], bits=case["bits"],
                                   tiles=state["tiles"], bounds=state["bounds"])
        state["batch"] = g.KVBatch(state["table"], state["lens"], state["cu"], max_new=state["max_new"])
    return state["cache"], state["batch"]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        cache, batch = _handles(state)
        if op == "append":
            q = cache.append(batch, state["qkv"], case["H"], rope=case["rope"], qk_norm=case["norm"])
            k, v = cache.read(batch, state["rows"])
            return {"q": q, "k": k, "v": v, "bounds": state["bounds"]}
        if op == "read":
            k, v = cache.read(batch, state["rows"])
            return {"k": k, "v": v}
        if op == "attend":
            o, lse = cache.attend(batch, state["q"], window=case["window"])
            return {"o": o, "lse": lse}
        blocks, scores = cache.select(batch, state["q"], max(case["select"], N_FIRST + N_LAST), n_first=N_FIRST,
                                      n_last=N_LAST)
        o, lse = cache.attend(batch, state["q"], blocks=blocks)
        return {"blocks": blocks, "scores": scores, "o": o, "lse": lse}
    if op == "append":
        q = _plain_append(state)
        k, v = _plain_read(state)
        return {"q": q, "k": k, "v": v, "bounds": state["bounds"]}
    if op == "read":
        k, v = _plain_read(state)
        return {"k": k, "v": v}
    if op == "attend":
        o, lse = _plain_attend(state)
        return {"o": o, "lse": lse}
    blocks, scores, o, lse = _plain_sparse(state)
    return {"blocks": blocks, "scores": scores, "o": o, "lse": lse}


# ---------------------------------------------------------------------------- bytes and operations

def work(case):
    H, Hkv, hd, bits, win = (case[k] for k in ("H", "Hkv", "hd", "bits", "window"))
    rowb, ng, _ = _sizes(case)
    lens, new = _lengths(case)
    rows, row = sum(new), rowb + 2 * ng
    kv_out = 2 * 2 * Hkv * hd * rows                        # keys and values as bf16
    if case["op"] == "append":
        b = rows * (2 * (H + 2 * Hkv) * hd + 2 * H * hd + 2 * Hkv * row) + kv_out
        return {"bytes": b, "flops": 12.0 * rows * (H + 2 * Hkv) * hd}
    if case["op"] == "read":
        return {"bytes": rows * 2 * Hkv * row + kv_out, "flops": 2.0 * rows * 2 * Hkv * hd}
    q_o = rows * H * (4 * hd + 4)
    keys = pairs = sel = 0
    if case["op"] == "attend":
        for n, m in zip(lens, new):
            first = 0 if win < 0 else max(0, n - m - win)
            keys += n - first
            pairs += sum(min(p + 1, win + 1 if win >= 0 else p + 1) for p in range(n - m, n))
        return {"bytes": q_o + keys * 2 * Hkv * row, "flops": 4.0 * pairs * H * hd}
    k = max(case["select"], N_FIRST + N_LAST)
    for n, m in zip(lens, new):
        sel += 2 * 2 * hd * Hkv * ((n + BLOCK - 1) // BLOCK)
        for p in range(n - m, n):
            nb = p // BLOCK + 1
            pairs += min(k * BLOCK, p + 1)
            sel += Hkv * 4 * (k + nb)
    return {"bytes": q_o + sel + pairs * 2 * Hkv * row, "flops": 4.0 * pairs * H * hd}


# ---------------------------------------------------------------------------- 64 bits, from the definitions

def _values64(case, tiles, phys, tok, head):
    """Key and value rows of cache tokens (equal-shaped index tensors), element by element from the
    layout's definition."""
    bits, hd = case["bits"], case["hd"]
    rowb, ng, recb = _sizes(case)
    d = torch.arange(hd, device=tiles.device)
    rec, i = tok[..., None] // 32, tok[..., None] % 32
    half, key = i // 16, i % 16
    base = rec * recb + half * (16 * rowb)
    flat = tiles.reshape(-1, tiles.shape[-1])
    row = (phys * tiles.shape[1] + head)[..., None]
    per = 8 // bits                                         # codes in a byte
    byte = d // per
    shift = (d % per) * bits
    # key: the word that holds dim d belongs to lane (word mod 4)
    word = byte // 4
    lane_b = rowb // 4
    unit = min(lane_b, 16)
    pos_in_lane = (word // 4) * 4 + byte % 4
    koff = base + (pos_in_lane // unit) * (64 * unit) + key * (4 * unit) + (word % 4) * unit + pos_in_lane % unit
    # value: lane 4 ((d / 8) mod 8) + (key mod 8) / 2 holds 4 keys, those 2c, 2c+1, 2c+8, 2c+9
    lane = 4 * ((d // 8) % 8) + (key % 8) // 2
    slot = key % 2 + 2 * (key // 8)
    in_key = (d // 64) * bits + (d % 8) // per
    z = slot * (rowb // 8) + in_key
    voff = 32 * rowb + base + (z // 16) * 512 + lane * 16 + z % 16
    grp = (d // 64) if ng > 1 else torch.zeros_like(d)
    out = []
    for off, sbase in ((koff, 64 * rowb), (voff, 64 * rowb + 64 * ng)):
        code = (flat[row, off].int() >> shift) & ((1 << bits) - 1)
        so = rec * recb + sbase + 2 * (i * ng + grp)
        raw = flat[row, so].int() | (flat[row, so + 1].int() << 8)
        scale = (raw << 16).view(torch.float32).double()
        out.append((code - (1 << (bits - 1))).double() * scale)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op, H, Hkv, hd, bits = (case[k] for k in ("op", "H", "Hkv", "hd", "bits"))
    dev = st["tiles"].device
    lens, new = _lengths(case)
    table, heads = st["table"].long(), torch.arange(Hkv, device=dev)
    G, cu = H // Hkv, st["cu"].tolist()
    if op == "append":
        top, ng = (1 << (bits - 1)) - 1, _sizes(case)[1]
        qs, ks, vs = [], [], []
        bounds = st["bounds"].double()
        for s in range(case["B"]):
            x = st["qkv"][cu[s]:cu[s + 1]].double().reshape(-1, H + 2 * Hkv, hd)
            pos = torch.arange(lens[s] - new[s], lens[s], device=dev)
            qk, v = x[:, :H + Hkv], x[:, H + Hkv:]
            if case["rope"]:
                ang = pos.double()[:, None, None] * torch.exp(
                    -math.log(10000.0) * torch.arange(0, hd, 2, device=dev, dtype=torch.float64) / hd)
                z = torch.complex(qk[..., :hd // 2], qk[..., hd // 2:]) * torch.polar(torch.ones_like(ang), ang)
                qk = torch.cat((z.real, z.imag), -1)
            if case["norm"]:
                qk = qk / torch.sqrt((qk * qk).sum(-1, keepdim=True) / hd + 1e-5)
            qs.append(qk[:, :H].reshape(-1, H * hd))
            got = []
            for rows in (qk[:, H:], v):
                g = rows.reshape(len(rows), Hkv, ng, -1)
                sc = (g.abs().max(-1).values / top).bfloat16().double()[..., None]
                n = torch.where(sc > 0, torch.round(g / sc), 0.0).clamp(-top, top)
                got.append((n * sc).reshape(len(rows), Hkv, hd))
            ks.append(got[0])
            vs.append(got[1])
            for blk in range(int(pos[0]) // BLOCK, int(pos[-1]) // BLOCK + 1):
                part = got[0][max(0, blk * BLOCK - int(pos[0])):(blk + 1) * BLOCK - int(pos[0])]
                mn, mx = part.min(0).values, part.max(0).values
                if blk * BLOCK < int(pos[0]):           # joined with the bounds that were there: zeros
                    mn, mx = mn.clamp(max=0.0), mx.clamp(min=0.0)
                bounds[table[s, blk]] = torch.stack((mn, mx), 1)
        return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs), "bounds": bounds}
    if op == "read":
        ks, vs = [], []
        for s in range(case["B"]):
            pos = torch.arange(lens[s] - new[s], lens[s], device=dev)[:, None]
            ph = table[s][pos // BLOCK].expand(-1, Hkv)
            k, v = _values64(case, st["tiles"], ph, (pos % BLOCK).expand(-1, Hkv), heads[None].expand_as(ph))
            ks.append(k)
            vs.append(v)
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    if max(lens) * H * hd > 1 << 26:
        return None
    os_, ls, bl, scs = [], [], [], []
    W = table.shape[1]
    nsel = max(case["select"], N_FIRST + N_LAST)
    for s in range(case["B"]):
        pos = torch.arange(lens[s], device=dev)[:, None]
        ph = table[s][pos // BLOCK].expand(-1, Hkv)
        k, v = _values64(case, st["tiles"], ph, (pos % BLOCK).expand(-1, Hkv), heads[None].expand_as(ph))
        for r in range(new[s]):
            p = lens[s] - new[s] + r
            q = st["q"][cu[s] + r].double().reshape(Hkv, G, hd)
            z = torch.einsum("hgd,khd->hgk", q, k) / math.sqrt(hd)
            off = (pos[:, 0] > p)
            if case["window"] >= 0:
                off = off | (pos[:, 0] < p - case["window"])
            off = off[None].expand(Hkv, -1)
            if op == "sparse":
                bd = st["bounds"][table[s, :p // BLOCK + 1]].double()       # [nb, Hkv, 2, hd]
                sc = torch.where(q[None] > 0, q[None] * bd[:, :, None, 1], q[None] * bd[:, :, None, 0]).sum((2, 3)).T
                nb = sc.shape[1]
                key = sc.clone()
                key[:, :N_FIRST] = math.inf
                key[:, max(0, nb - N_LAST):] = math.inf
                pick = torch.argsort(key, dim=1, descending=True, stable=True)[:, :nsel].sort(1).values
                chosen = torch.zeros((Hkv, nb), dtype=torch.bool, device=dev).scatter(1, pick, True)
                off = off | ~chosen.repeat_interleave(BLOCK, 1)[:, :lens[s]] if nb * BLOCK >= lens[s] else \
                    off | ~torch.nn.functional.pad(chosen.repeat_interleave(BLOCK, 1), (0, lens[s] - nb * BLOCK))
                bl.append(torch.nn.functional.pad(pick, (0, nsel - pick.shape[1]), value=-1))
                scs.append(torch.nn.functional.pad(sc, (0, W - nb), value=-math.inf))
            z = z.masked_fill(off[:, None], -math.inf)
            l = torch.logsumexp(z, -1)
            os_.append(torch.einsum("hgk,khd->hgd", torch.exp(z - l[..., None]), v).reshape(H * hd))
            ls.append(l.reshape(H))
        del k, v
    out = {"o": torch.stack(os_), "lse": torch.stack(ls)}
    if op == "sparse":
        out = {"blocks": torch.stack(bl).to(torch.int32), "scores": torch.stack(scs), **out}
    return out

"""Pins of the key/value-cache oracle (CPU), and the host-side refusals of the cache calls."""
import ctypes as C

import numpy as np
import pytest

import oracle as O
import synth

GEOM = [(4, 64), (4, 128), (8, 64), (8, 128)]


@pytest.mark.parametrize("bits,hd", GEOM)
def test_layout_is_a_permutation_of_the_records_bytes(bits, hd):
    R, ng, recb = O.kv.geometry(bits, hd)
    at = [f(bits, hd, i, y) for f in (O.kv.key_byte, O.kv.value_byte) for i in range(32) for y in range(R)]
    assert sorted(at) == list(range(64 * R))
    assert recb == 64 * R + 128 * ng and recb % 64 == 0


@pytest.mark.parametrize("bits,hd", GEOM)
def test_tile_bytes_match_the_library(bits, hd):
    import decoder_only_gpt_tcgen05_b200 as g
    assert g.kv.tile_bytes(bits, hd) == 2 * O.kv.geometry(bits, hd)[2]


@pytest.mark.parametrize("bits,hd", GEOM)
def test_pack_unpack_round_trip(bits, hd):
    x = synth.normal((3, 2, 64, hd), 7)
    y = synth.normal((3, 2, 64, hd), 8)
    kc, ks, kv = O.kv.quantise(x, bits)
    vc, vs, vv = O.kv.quantise(y, bits)
    k, v = O.kv.unpack(O.kv.pack(kc, ks, vc, vs, bits), bits, hd)
    assert np.array_equal(k, kv) and np.array_equal(v, vv)


@pytest.mark.parametrize("bits,hd", GEOM)
def test_quantised_value_is_within_half_a_step(bits, hd):
    # scale = bf16(max / top) is off by at most 2^-8 of itself, so the largest code clips at most
    # top 2^-8 < 1/2 of a step
    x = synth.normal((50, hd), 9) * np.exp(synth.normal((50, 1), 10) * 4)
    _, s, val = O.kv.quantise(x, bits)
    step = np.repeat(s, hd // s.shape[-1], axis=-1)
    assert np.all(np.abs(val - x) <= 0.5 * step * (1 + 1e-12))


def test_quantise_edge_groups():
    for bits in (4, 8):
        x = np.zeros((4, 64))
        x[1, 3], x[2, 5], x[3, 0] = np.inf, np.nan, 1e-40
        c, s, val = O.kv.quantise(x, bits)
        assert np.all(val[0] == 0) and np.all(np.isnan(val[1])) and np.all(np.isnan(val[2])) and np.all(val[3] == 0)


def test_bf16_rounding_directions():
    x = np.array([1.0, 1.001, -1.001, 3.14159, -2.71828, 0.0, 1e-3, 65535.0])
    lo, hi, near = O.kv.bf16(x, "down"), O.kv.bf16(x, "up"), O.kv.bf16(x)
    assert np.all(lo <= x) and np.all(hi >= x) and np.all((near == lo) | (near == hi))
    assert np.all(hi - lo <= np.abs(x) * 2.0 ** -7)


def test_attend_matches_brute_force_and_block_scores_bound_the_keys():
    hd, L, H, Hkv = 64, 130, 4, 2
    q, k, v = (synth.normal(s, n).astype(np.float64) for n, s in ((1, (H, hd)), (2, (L, Hkv, hd)), (3, (L, Hkv, hd))))
    o, lse, _ = O.kv.attend(q, k, v, np.ones((Hkv, L)))
    for h in range(H):
        s = np.array([q[h] @ k[j, h // 2] for j in range(L)]) / 8.0
        p = np.exp(s) / np.exp(s).sum()
        assert np.allclose(o[h], sum(p[j] * v[j, h // 2] for j in range(L)), atol=1e-13)
        assert abs(lse[h] - np.log(np.exp(s).sum())) < 1e-12
    kb = np.stack([np.stack((k[a:a + 64].min(0), k[a:a + 64].max(0)), 1) for a in (0, 64, 128)])
    sc = O.kv.block_scores(q, kb)
    for b, a in enumerate((0, 64, 128)):
        for hk in range(Hkv):
            best = (q.reshape(Hkv, 2, hd)[hk].sum(0) @ k[a:a + 64, hk].T).max()
            assert sc[hk, b] >= best - 1e-12
    assert O.kv.choose(np.array([1.0, 5.0, 5.0, 0.0, 2.0, -1.0]), 4, 1, 1) == [0, 1, 2, 5]
    assert O.kv.choose(np.array([1.0, 1.0, 1.0, 1.0]), 2, 0, 0) == [0, 1]
    assert O.kv.choose(np.array([1.0, 2.0]), 5, 1, 1) == [0, 1]


# ---------------------------------------------------------------------------- refusals

P = 1 << 20  # an aligned address that is never dereferenced


def _args(cache={}, batch={}):
    from decoder_only_gpt_tcgen05_b200._lib import KVBatchParams, KVCacheParams
    c = dict(tiles=P, bounds=P, n_blocks=10, n_kv_head=2, head_dim=128, bits=8)
    b = dict(block_table=P, lens=P, cu_new=P, n_seq=3, max_blocks=4, max_new=5)
    return C.byref(KVCacheParams(**{**c, **cache})), C.byref(KVBatchParams(**{**b, **batch}))


BAD_BOTH = [
    (dict(bits=5), {}, 2), (dict(bits=16), {}, 2), (dict(head_dim=96), {}, 2), (dict(head_dim=256), {}, 2),
    (dict(n_blocks=0), {}, 1), (dict(n_kv_head=0), {}, 1), (dict(tiles=None), {}, 1), (dict(tiles=P + 8), {}, 1),
    (dict(bounds=P + 2), {}, 1), ({}, dict(n_seq=-1), 1), ({}, dict(max_blocks=0), 1), ({}, dict(max_new=-1), 1),
    ({}, dict(block_table=None), 1), ({}, dict(lens=None), 1), ({}, dict(lens=P + 1), 1),
    ({}, dict(cu_new=None, n_seq=9), 1), ({}, dict(max_blocks=(1 << 24) + 1), 2),
]


@pytest.mark.parametrize("cache,batch,code", BAD_BOTH)
def test_every_call_refuses_a_bad_cache_or_batch(cache, batch, code):
    import decoder_only_gpt_tcgen05_b200 as g
    L = g.lib()
    c, b = _args(cache, batch)
    n = C.c_size_t()
    assert L.gpt_op_kv_append(c, b, P, 8, 4, 1, 1, 1e4, 1e-5, P, None) == code
    assert L.gpt_op_kv_read(c, b, 8, P, P, None) == code
    assert L.gpt_op_kv_select(c, b, P, 8, 4, 4, 1, 1, P, P, None) == code
    assert L.gpt_op_attention_kv(c, b, P, 8, 4, -1, None, 0, P, P, P, 1 << 40, None) == code
    assert L.gpt_op_attention_kv_scratch_size(c, b, 8, 4, 0, C.byref(n)) == code


def test_call_arguments_are_refused_on_the_host():
    import decoder_only_gpt_tcgen05_b200 as g
    L = g.lib()
    c, b = _args()
    n = C.c_size_t()

    def append(M=8, H=4, rope=1, norm=1, base=1e4, eps=1e-5, qkv=P, q=P):
        return L.gpt_op_kv_append(c, b, qkv, M, H, rope, norm, base, eps, q, None)

    assert append(H=3) == 1 and append(H=0) == 1 and append(M=-1) == 1
    assert append(base=1.0) == 1 and append(base=float("nan")) == 1 and append(eps=0.0) == 1
    assert append(qkv=None) == 1 and append(q=None) == 1 and append(qkv=P + 8) == 1 and append(q=P + 2) == 1
    assert append(H=1 << 20) == 2
    assert L.gpt_op_kv_append(None, b, P, 8, 4, 1, 1, 1e4, 1e-5, P, None) == 1
    assert L.gpt_op_kv_append(c, None, P, 8, 4, 1, 1, 1e4, 1e-5, P, None) == 1

    assert L.gpt_op_kv_read(c, b, 8, None, P, None) == 1 and L.gpt_op_kv_read(c, b, 8, P, P + 4, None) == 1

    def select(H=4, n=4, first=1, last=1, q=P, blocks=P, scores=P, cache=c):
        return L.gpt_op_kv_select(cache, b, q, 8, H, n, first, last, blocks, scores, None)

    assert select(H=3) == 1 and select(n=0, first=0, last=0) == 1 and select(n=1) == 1 and select(first=-1) == 1
    assert select(first=2 ** 31 - 1, last=2 ** 31 - 1, n=2 ** 31 - 1) == 1
    assert select(H=2 * 33) == 2
    assert select(q=None) == 1 and select(blocks=None) == 1 and select(scores=None) == 1 and select(q=P + 4) == 1
    assert select(cache=_args(dict(bounds=None))[0]) == 1

    assert L.gpt_op_attention_kv_scratch_size(c, b, 8, 4, 0, C.byref(n)) == 0
    need = n.value

    def attend(H=4, window=-1, sel=None, n_sel=0, q=P, o=P, lse=P, scratch=P, size=need):
        return L.gpt_op_attention_kv(c, b, q, 8, H, window, sel, n_sel, o, lse, scratch, size, None)

    assert attend(H=5) == 1 and attend(window=-2) == 1 and attend(sel=P) == 1 and attend(n_sel=3) == 1
    assert attend(sel=P, n_sel=3, window=10, size=1 << 40) == 2
    assert attend(n_sel=-1) == 1
    assert attend(q=None) == 1 and attend(o=None) == 1 and attend(scratch=None) == 1 and attend(q=P + 8) == 1
    assert attend(scratch=P + 128) == 1 and attend(lse=P + 2) == 1 and attend(sel=P + 1, n_sel=2, size=1 << 40) == 1
    assert attend(size=need - 1) == 3 and b"scratch" in L.gpt_last_error()
    assert L.gpt_op_attention_kv_scratch_size(c, b, 8, 4, 0, None) == 1
    assert L.gpt_op_attention_kv_scratch_size(c, b, 8, 4, -1, C.byref(n)) == 1
    big = _args(batch=dict(n_seq=1 << 20, max_new=1 << 20))[1]
    assert L.gpt_op_attention_kv_scratch_size(c, big, 1 << 30, 4, 0, C.byref(n)) == 2
    assert L.gpt_kv_tile_bytes(8, 128, None) == 1 and L.gpt_kv_tile_bytes(2, 128, C.byref(n)) == 2


def test_nothing_to_do_is_no_error_and_launches_nothing():
    import decoder_only_gpt_tcgen05_b200 as g
    L = g.lib()
    before = g.ops.launch_count()
    for batch, M in ((dict(n_seq=0), 8), (dict(max_new=0), 8), ({}, 0)):
        c, b = _args(batch=batch)
        assert L.gpt_op_kv_append(c, b, P, M, 4, 1, 1, 1e4, 1e-5, P, None) == 0
        assert L.gpt_op_kv_read(c, b, M, P, P, None) == 0
        assert L.gpt_op_kv_select(c, b, P, M, 4, 4, 1, 1, P, P, None) == 0
        assert L.gpt_op_attention_kv(c, b, P, M, 4, -1, None, 0, P, P, P, 1 << 40, None) == 0
    assert g.ops.launch_count() == before


@pytest.mark.parametrize("max_new", [0, -3, 7])
def test_without_cu_new_the_field_max_new_is_ignored(max_new):
    """Every sequence has one new token then, so there is work and missing tensors are refused; the
    attention's scratch is that of one token each."""
    import decoder_only_gpt_tcgen05_b200 as g
    L = g.lib()
    c, b = _args(batch=dict(cu_new=None, max_new=max_new))
    assert L.gpt_op_kv_append(c, b, None, 8, 4, 1, 1, 1e4, 1e-5, P, None) == 1
    assert L.gpt_op_kv_read(c, b, 8, None, P, None) == 1
    assert L.gpt_op_kv_select(c, b, None, 8, 4, 4, 1, 1, P, P, None) == 1
    assert L.gpt_op_attention_kv(c, b, None, 8, 4, -1, None, 0, P, P, P, 1 << 40, None) == 1
    n, one = C.c_size_t(), C.c_size_t()
    assert L.gpt_op_attention_kv_scratch_size(c, b, 8, 4, 0, C.byref(n)) == 0
    assert L.gpt_op_attention_kv_scratch_size(c, _args(batch=dict(cu_new=None, max_new=1))[1], 8, 4, 0, C.byref(one)) == 0
    assert n.value == one.value


def test_the_attributes_that_the_calls_go_by_cannot_be_assigned_to():
    """A batch or cache whose tensor was replaced would go on using the old memory: that is refused, while the
    tensors' contents may change and every attribute reads as it was given."""
    import torch

    import decoder_only_gpt_tcgen05_b200 as g
    table, lens, cu = (torch.arange(n, dtype=torch.int32) for n in (6, 2, 3))
    b = g.KVBatch(table.view(2, 3), lens, cu, max_new=4)
    tiles = torch.zeros((5, 2, g.kv.tile_bytes(8, 64)), dtype=torch.uint8)
    c = g.KVCache(5, 2, 64, bits=8, tiles=tiles)
    want = {b: dict(lens=lens, cu_new=cu, max_new=4, n_seq=2, max_blocks=3, device=lens.device),
            c: dict(tiles=tiles, n_blocks=5, n_kv_head=2, head_dim=64, bits=8, device=tiles.device)}
    for x, attrs in want.items():
        for name, value in attrs.items():
            assert getattr(x, name) is value or getattr(x, name) == value
            with pytest.raises(AttributeError):
                setattr(x, name, value)
    for x, name in ((b, "block_table"), (c, "bounds")):
        assert torch.is_tensor(getattr(x, name))
        with pytest.raises(AttributeError):
            setattr(x, name, None)
    b.lens.add_(1)
    assert lens.tolist() == [1, 2]
    assert g.KVBatch(b.block_table, b.lens).cu_new is None and g.KVCache(5, 2, 64, tiles=tiles, bounds=False).bounds is None


def test_the_binding_refuses_numbers_that_32_bits_would_cut_off():
    """2^32 + 1 chosen blocks must not become one, nor 2^40 first ones none."""
    import torch

    import decoder_only_gpt_tcgen05_b200 as g
    table, lens, cu = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c = g.KVCache(1, 1, 64, bits=8, tiles=torch.zeros((1, 1, g.kv.tile_bytes(8, 64)), dtype=torch.uint8))
    b, q = g.KVBatch(table, lens), torch.zeros((1, 64), dtype=torch.bfloat16)
    out = torch.zeros((1, 1, 1), dtype=torch.int32), torch.zeros((1, 1, 1))
    for bad in (2 ** 31, 2 ** 32, 2 ** 40, 2 ** 63 - 1, -2 ** 40, float("inf")):
        for name in ("n_first", "n_last"):
            with pytest.raises(AssertionError, match="n_first"):
                c.select(b, q, 1, **{name: bad}, blocks=out[0], scores=out[1])
        with pytest.raises(AssertionError, match="max_new"):
            g.KVBatch(table, lens, cu, max_new=bad)
    with pytest.raises(AssertionError, match="n_select"):
        c.select(b, q, 2 ** 32 + 1)


@pytest.mark.parametrize("n_seq,max_new,H,Hkv,n_sel", [
    (2 ** 31 - 1, 2 ** 31 - 1, 64, 64, 0),        # products that pass 2^63, and come out below the limit
    (2 ** 31 - 1, 2 ** 31 - 16, 128, 128, 0), (2 ** 31 - 1, 5, 64, 64, 0), (3, 5, 2 ** 30, 2 ** 29, 9),
    (1, 2 ** 31 - 1, 2 ** 30, 1, 0)])
def test_a_batch_of_too_many_rows_is_refused_whatever_its_products_come_to(n_seq, max_new, H, Hkv, n_sel):
    import decoder_only_gpt_tcgen05_b200 as g
    L = g.lib()
    c, b = _args(dict(n_kv_head=Hkv), dict(n_seq=n_seq, max_new=max_new, max_blocks=1))
    n = C.c_size_t()
    M = 2 ** 31 - 1
    assert L.gpt_op_attention_kv_scratch_size(c, b, M, H, n_sel, C.byref(n)) == 2
    assert L.gpt_op_attention_kv(c, b, P, M, H, -1, P if n_sel else None, n_sel, P, P, P, 0, None) == 2

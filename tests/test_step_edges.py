"""Calls of a step's operators at the edges of what they take."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import step_ref as sref
from test_i4_cache import attn_setup, check, run
from test_paged_kv import DEV, gpu, i32, make_tables
from test_step_ops import ROPE, TD, angles, reserve


def _pkg():
    import speculative_decoding_verification_75_gb300 as sv
    from speculative_decoding_verification_75_gb300 import api, kv
    return sv, api, kv


# ---------------------------------------------- attention over 4 bits ----

def grow(s, lo, hi):
    """Scale bytes of k from lo at a request's first key to hi at its last one."""
    bs = s["c"][2].shape[2]
    for b, (L, n) in enumerate(zip(s["L"], s["n"])):
        for pos in range(L + n):
            s["c"][2][int(s["tables"][b, pos // bs]), :, pos % bs] = lo + (hi - lo) * pos // max(L + n - 1, 1)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("loud", [None, 0, 1, 2])
def test_references_rise_along_ranges_of_many_tiles(D, dt, loud):
    """Some 700 tiles of 128 keys in at most 152 ranges: most tiles are not a range's first.  Keys grow 512 times
    along a request, so that late tiles exceed a row's reference by 2^8 (2^15) again and again, the last ones by more than
    2^100; with `loud` only in that token's rows, which are one chunk of eight rows of one softmax group."""
    rng = np.random.default_rng(D + (loud or 0))
    L = [int(x) for x in rng.integers(2500, 3100, 4)]
    s = attn_setup(rng, 4, 3, 64, 8, D, 64, L, [3] * 4, dt, False)
    if loud is not None:
        quiet = [t for t in range(3) if t != loud]
        s["q"][:, quiet] *= 2.0 ** -10
    grow(s, 88, 160)
    out = check(s, dt)
    for _ in range(3):
        assert torch.equal(run(s), out)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rows_that_see_their_first_key_late(D, dt, monkeypatch):
    """Trees without committed tokens: nodes from 128 on see no key of the first tile, some none at all, and the
    first that they see is far above what a reference of nothing allows.

    Besides the other roundings: where a reference rises by more than 2^126, the factor of what was summed below it is
    a zero of fp32.  A probability is at most 2^8 of its reference then (fp16: 2^15, of 2^7 times it), and the largest one of
    the raised reference is at least 1 of l: of S keys S 2^(8 - 126) max |v| is lost at most.  (A bf16 result showed it
    where the likely key's value is 0 and the others' products are 2^-120.)"""
    plain = ref.attention

    def attention(q, cache, *args):
        w, wl, tol, *rest = plain(q, cache, *args)
        return w, wl, tol + q.shape[1] * 2.0 ** -118 * np.abs(cache.v).max(), *rest

    monkeypatch.setattr(ref, "attention", attention)
    rng = np.random.default_rng(D)
    B, T, H = 40, 300, 2
    n = [int(x) for x in rng.integers(260, T + 1, B)]
    s = attn_setup(rng, B, T, H, H, D, 16, [0] * B, n, dt, False)
    m = np.broadcast_to(np.eye(T, dtype=bool), (B, T, T)).copy()
    m |= rng.random((B, T, T)) < 0.02
    m[:, 128:, :128] &= rng.random((B, T - 128, 1)) < 0.3
    m[:, 200:, :256] &= rng.random((B, T - 200, 1)) < 0.3
    m[:, 150:160] = False
    s["mask"] = m
    s["c"][2][:] = torch.from_numpy(rng.integers(60, 150, tuple(s["c"][2].shape)).astype(np.uint8)).to(DEV)
    out = check(s, dt)
    assert (out[:, 150:160] == 0).all()


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,T", [("bf16", 4), ("fp16", 4), ("bf16", 11)])
@pytest.mark.parametrize("why", ["value", "key", "block"])
def test_marked_units_among_others_of_a_range(D, dt, T, why):
    """Units of a few tiles, several of them whole in a range; of some requests a new token's group is NaN for one
    head, or a block is missing.  What stands before and behind them in a range comes out as without them."""
    rng = np.random.default_rng(D + T)
    B, Hkv, G = 40, 8, 4
    L = [int(x) for x in rng.integers(0, 300, B)]
    n = [int(x) for x in rng.integers(1, T + 1, B)]
    s = attn_setup(rng, B, T, Hkv * G, Hkv, D, 16, L, n, dt, False)
    clean = run(s, torch.full_like(s["q"], 9.0))
    hit = np.zeros((B, Hkv), dtype=bool)
    for b in rng.choice(B, 14, replace=False):
        if why == "block":
            s["tables"][b, rng.integers(0, -(-(L[b] + n[b]) // 16))] = -1
            hit[b] = True
        else:
            h, pos = rng.integers(Hkv), L[b] + n[b] - 1
            s["c"][3 if why == "value" else 2][int(s["tables"][b, pos // 16]), h, pos % 16, rng.integers(D // 32)] = 255
            hit[b, h] = True
    out = check(s, dt)
    same = torch.from_numpy(~np.repeat(hit, G, 1)).to(DEV)[:, None].expand(B, T, Hkv * G)
    assert torch.equal(out[same], clean[same])


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [1e38, -2.3e38, 2.2e37])
def test_scores_of_zero_with_a_factor_near_the_largest(D, dt, scale):
    """A zero score is zero whatever it is multiplied by: the mean of the values."""
    s = attn_setup(np.random.default_rng(D), 2, 3, 8, 2, D, 16, [300, 20], [3, 2], dt, False)
    s["q"].zero_()
    check(s, dt, scale=scale)


@gpu
def test_blocks_past_32_bit_offsets():
    """Blocks of a cache of 4 bits 2^33 elements apart: written by both operators, attended to, moved, read back."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(1)
    H, bs, D = 2, 16, 64
    stride = (1 << 32) + 16 * 64                               # bytes
    sstride = (1 << 31) + 4096
    store = [torch.zeros(stride + H * bs * D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
    sstore = [torch.zeros(sstride + H * bs * D // 32, dtype=torch.uint8, device=DEV) for _ in range(2)]
    far = [x.as_strided((2, H, bs, D // 2), (stride, bs * D // 2, D // 2, 1)) for x in store]
    far += [x.as_strided((2, H, bs, D // 32), (sstride, bs * D // 32, D // 32, 1)) for x in sstore]
    near = [torch.zeros(x.shape, dtype=torch.uint8, device=DEV) for x in far]
    x = torch.from_numpy(rng.standard_normal((1, 20, 4 + 2 * H, D))).bfloat16().to(DEV)
    q, key, value = x.split([4, H, H], 2)
    t, L = i32([[0, 1]]), i32([5])
    cs, pos = torch.from_numpy(angles(40, D)).to(DEV), i32([list(range(5, 25))])
    got = []
    for k, v, ks, vs in (far, near):
        kw = dict(k_scale=ks, v_scale=vs)
        sv.kv_write(key, value, k, v, t, L, **kw)
        a = sv.kv_read(k, v, t, i32([20]), L, max_len=20, **kw)
        o, _ = sv.qk_norm_rope(q, key, cs, pos, value=value, k_cache=k, v_cache=v, slots=pos.long(), **kw)
        y = sv.tree_attention(o, k, v, t, L, **kw)
        sv.kv_compact(i32([[0, 12, 19]]), i32([3]), L, t, k, v, **kw)
        got.append((*a, o, y, k, v, ks, vs))
    for a, b in zip(*got):
        assert torch.equal(a, b) and a.any()


# ------------------------------------------------- rows at the ends of fp32 ----

def close_bf16(got, x, w, cs, pos, eps, pairs):
    """fp32's roundings as step_ref derives them, one rounding to bf16 (half a step, 2^-134 where it is subnormal)."""
    want, tol = sref.norm_rope(ref.to64(x), None if w is None else ref.to64(w), cs.astype(np.float64), pos, eps, pairs)
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134
    got = ref.to64(got)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


@gpu
@pytest.mark.parametrize("D,R,pairs", [(64, 64, False), (128, 64, True), (96, 32, False), (8, 0, False), (256, 256, False)])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
def test_norms_of_rows_near_the_ends_of_fp32(D, R, pairs, eps):
    """Rows whose squares fp32 does not hold, too large and too small; rows of one turn that are ordinary."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(D)
    e = np.array([0, 63, 64, 70, 100, 124, 0, -3, -20, -64, -70, -100, -122, 5, 50, -50])
    x = rng.standard_normal((2, 8, 12, D)).clip(-3.9, 3.9) * 2.0 ** rng.permutation(np.resize(e, (2 * 8 * 12)))\
        .reshape(2, 8, 12, 1)
    x = torch.from_numpy(x).bfloat16().to(DEV)
    x[0, 0, 0, :] = 3e38
    x[0, 1, 1, :2] = torch.tensor([-3.3e38, 1e-30], device=DEV).bfloat16()
    q, k = x.split([9, 3], 2)
    cs, pos = angles(50, R), rng.integers(0, 50, (2, 8))
    wq, wk = (torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).bfloat16().to(DEV) for _ in range(2))
    f = (torch.from_numpy(cs).to(DEV), i32(pos))
    out, ko = sv.qk_norm_rope(q, k, *f, wq, wk, eps=eps, interleaved=pairs)
    close_bf16(out, q, wq, cs, pos, eps, pairs)
    close_bf16(ko, k, wk, cs, pos, eps, pairs)
    # Only one of the two has a norm: the other is the same as without any.
    out, ko = sv.qk_norm_rope(q, k, *f, None, wk, eps=eps, interleaved=pairs)
    close_bf16(ko, k, wk, cs, pos, eps, pairs)
    assert torch.equal(out, sv.qk_norm_rope(q, k, *f, eps=eps, interleaved=pairs)[0])


@gpu
@pytest.mark.parametrize("big", [2.0 ** 70, 2.0 ** 100, 2.0 ** 120, 2.0 ** -70, 2.0 ** -100])
@pytest.mark.parametrize("D,R,pairs", [(64, 64, False), (80, 40, True)])
def test_norms_with_weights_near_the_ends_of_fp32(big, D, R, pairs):
    sv, _, _ = _pkg()
    rng = np.random.default_rng(D)
    x = rng.standard_normal((1, 6, 5, D)) * 2.0 ** rng.integers(-10, 34, (1, 6, 5, 1))
    x = torch.from_numpy(x).bfloat16().to(DEV)
    x[0, 0, 0] *= 2.0 ** 80
    q, k = x.split([3, 2], 2)
    cs, pos = angles(50, R), rng.integers(0, 50, (1, 6))
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(D)) * big).bfloat16().to(DEV)
    f = (torch.from_numpy(cs).to(DEV), i32(pos))
    out, ko = sv.qk_norm_rope(q, k, *f, w, w, eps=1e-6, interleaved=pairs)
    close_bf16(out, q, w, cs, pos, 1e-6, pairs)
    close_bf16(ko, k, w, cs, pos, 1e-6, pairs)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_norms_of_rows_that_are_not_finite(dt):
    """An infinity's row: x / inf is 0 for what is finite, and NaN for the infinity; a NaN's row is NaN; others stay."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((1, 2, 6, 64)) * 4).to(TD[dt]).to(DEV)
    clean = x.clone()
    x[0, 0, 1, 5] = float("inf")
    x[0, 1, 2, 40] = float("nan")
    big = 2.0 ** 100 if dt == "bf16" else 60000.0
    x[0, 0, 1, 6] = big
    w = torch.full((64,), big, dtype=TD[dt], device=DEV)
    cs = torch.zeros(1, 0, device=DEV)
    pos = i32([[0, 0]])
    q, k = x.split([4, 2], 2)
    out, _ = sv.qk_norm_rope(q, k, cs, pos, w, w)
    want, _ = sv.qk_norm_rope(*clean.split([4, 2], 2), cs, pos, w, w)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[0, 0, 1, 5] = True
    nan[0, 1, 2] = True
    assert torch.equal(out.isnan(), nan)
    zero = torch.zeros_like(nan)
    zero[0, 0, 1] = True
    assert (out[zero & ~nan] == 0).all() and torch.equal(out[~zero & ~nan], want[~zero & ~nan])


@gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i4"])
def test_rows_near_the_ends_of_fp32_into_the_cache(kind):
    """The cache gets what kv_write of the rounded rows puts there; rows of values, of any size, are not touched."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(7)
    B, T, H, D, bs = 2, 8, 3, 64, 16
    x = rng.standard_normal((B, T, 3 * H, D)) * 2.0 ** rng.choice([0, 1, 64, 100, -70, -110], (B, T, 3 * H, 1))
    q, k, v = torch.from_numpy(x).bfloat16().to(DEV).split([H, H, H], 2)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).bfloat16().to(DEV)
    cs, tab, L = torch.from_numpy(angles(20, D)).to(DEV), i32([[1], [0]]), i32([0, 3])
    pos = L[:, None] + torch.arange(T, dtype=torch.int32, device=DEV)
    slots = tab.long() * bs + pos
    dt, d = {"bf16": (torch.bfloat16, D), "e4m3": (torch.float8_e4m3fn, D), "i4": (torch.uint8, D // 2)}[kind]
    got, want = ([torch.zeros(2, H, bs, d, dtype=torch.bfloat16, device=DEV).to(dt) for _ in range(2)] for _ in range(2))
    sc = [[torch.zeros(2, H, bs, D // 32, dtype=torch.uint8, device=DEV) if kind != "bf16" else None for _ in range(2)]
          for _ in range(2)]
    for eps in (0.0, 1e-6):
        _, ko = sv.qk_norm_rope(q, k, cs, pos, w, w, eps=eps)
        assert ko.isfinite().all()
        sv.kv_write(ko, v, *want, tab, L, k_scale=sc[0][0], v_scale=sc[0][1])
        sv.qk_norm_rope(q, k, cs, pos, w, w, eps=eps, value=v, k_cache=got[0], v_cache=got[1], slots=slots,
                        k_scale=sc[1][0], v_scale=sc[1][1])
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert kind == "bf16" or all(torch.equal(a, b) for a, b in zip(*sc))


# ------------------------------------------- a rotation's arguments ----

def rope_words(p, **over):
    f = dict(k=0, v=0, ks=0, vs=0, layer=0, block=0, slayer=0, sblock=0, layers=0, blocks=0, heads=0, bs=0, D=0,
             cdtype=0, tables=0, max_blocks=0,
             q=p, key=p, val=0, qb=1024, qt=256, qh=64, kb=512, kt=128, kh=64, vb=0, vt=0, vh=0,
             out=p, kout=p, ob=1024, ot=256, oh=64, kob=512, kot=128, koh=64, qw=0, kw=0, cs=p, pos=p, slots=0,
             eps=1e-6, P=10, R=64, pairs=0, B=2, T=4, Hq=4, Hkv=2, hd=64, dtype=1, status=0)
    f.update(over)
    return ROPE.pack(ROPE.size, *f.values())


def test_results_of_a_rotation_in_one_place_are_refused():
    """Queries and keys that would be written over each other, or over what other threads still read."""
    _, api, _ = _pkg()
    lib = api.load_library()
    a, b, c, d, v = (i << 20 for i in range(1, 6))
    for over in (dict(out=a, kout=a), dict(out=b, kout=d), dict(out=c, kout=a), dict(out=a, ot=512, kout=d),
                 dict(out=a, oh=128, kout=d), dict(out=a, ob=2048, kout=d), dict(out=c, kout=b, koh=128)):
        words = rope_words(a, key=b, cs=a, pos=a, **over)
        assert lib.sv_qk_norm_rope(words, None) == api.SV_ERR_INVALID_ARG, over
    cache = dict(k=8 * a, v=9 * a, block=2048, layers=1, blocks=8, heads=2, bs=16, D=64, cdtype=1, slots=a, val=v, vb=512,
                 vt=128, vh=64)
    for over in (dict(out=v, kout=d), dict(out=c, kout=v), dict(out=c, kout=a)):
        words = rope_words(a, key=b, cs=a, pos=a, **{**cache, **over})
        assert lib.sv_qk_norm_rope(words, None) == api.SV_ERR_INVALID_ARG, over


@gpu
def test_a_rotation_without_a_cache_looks_at_neither_it_nor_values():
    sv, api, _ = _pkg()
    lib = api.load_library()
    x = torch.randn(2, 4, 6, 64, device=DEV).bfloat16()
    q, k = (t.contiguous() for t in x.split([4, 2], 2))
    cs, pos = torch.from_numpy(angles(10, 64)).to(DEV), i32(np.arange(8).reshape(2, 4))
    want = sv.qk_norm_rope(q, k, cs, pos)
    out, ko = torch.zeros_like(q), torch.zeros_like(k)
    p = dict(q=q.data_ptr(), key=k.data_ptr(), out=out.data_ptr(), kout=ko.data_ptr(), cs=cs.data_ptr(),
             pos=pos.data_ptr(), cdtype=77, bs=-3, tables=5, vb=-1)
    assert lib.sv_qk_norm_rope(rope_words(0, **p, val=3), torch.cuda.current_stream().cuda_stream) == api.SV_OK
    assert torch.equal(out, want[0]) and torch.equal(ko, want[1])
    # With a cache its block tables are not.
    kc, vc = (torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.arange(8, device=DEV).view(2, 4)
    p = dict(p, k=kc.data_ptr(), v=vc.data_ptr(), block=1024, layers=1, blocks=2, heads=2, bs=8, D=64, cdtype=1, tables=5,
             max_blocks=-2, slots=slots.data_ptr(), val=k.data_ptr(), vb=512, vt=128, vh=64)
    assert lib.sv_qk_norm_rope(rope_words(0, **p), torch.cuda.current_stream().cuda_stream) == api.SV_OK
    assert torch.equal(kc[0].transpose(0, 1).reshape(2, 4, 2, 64), want[1]) and torch.equal(
        vc[0].transpose(0, 1).reshape(2, 4, 2, 64), k)


# --------------------------------------------------------------- reserve ----

@gpu
@pytest.mark.parametrize("B,T", [(256, 64), (256, 65), (2100, 7), (1500, 4)])
def test_trees_of_many_requests(B, T):
    """More tokens than the kernel of the blocks places itself: a second one does, by the mask too."""
    rng = np.random.default_rng(T)
    bs = 16
    L, n = rng.integers(0, 100, B), rng.integers(0, T + 1, B)
    n[0] = T
    mask = np.broadcast_to(np.eye(T, dtype=bool), (B, T, T)).copy()
    par = (rng.random((B, T)) * np.maximum(np.arange(T), 1)).astype(int)
    for i in range(1, T):
        mask[:, i] |= mask[np.arange(B), par[:, i]]
    mask[:, :, T // 2:] |= rng.random((B, T, T - T // 2)) < 0.3     # columns past n among them: they do not count
    mask[0, 3] = False
    held = -(-L // bs)
    width = -(-(100 + T) // bs) + 1
    tables = make_tables(rng, held, int(held.sum()) + 1, width)
    want = int((-(-(L + n) // bs) - held).sum())
    free = 10 ** 6 + rng.permutation(want + 5)
    _, _, res, _, _, st = reserve(L, n, tables, bs, free, want, mask, T)
    assert st == 0 and np.array_equal(res, n)
    reserve(L, n, tables, bs, free, want, mask[1], T)               # one mask for all
    _, _, res, _, _, st = reserve(L, n, tables, bs, free, want // 2, mask, T)
    assert st == sref.NO_BLOCKS and 0 < (res > 0).sum() < B


@gpu
@pytest.mark.parametrize("B,T", [(9001, 1), (9001, 2), (32768, 1), (4097, 3)])
@pytest.mark.parametrize("short", [False, True])
def test_more_requests_than_threads(B, T, short):
    """Each thread block's prefix sums go on over several rounds of its threads."""
    rng = np.random.default_rng(B + T)
    bs = 2
    L, n = rng.integers(0, 9, B), rng.integers(0, T + 1, B)
    held = -(-L // bs) + rng.integers(0, 2, B)
    tables = make_tables(rng, held, int(held.sum()) + 1, 8)
    want = int(np.maximum(-(-(L + n) // bs) - held, 0).sum())
    free = 10 ** 6 + rng.permutation(want + 3)
    reserve(L, n, tables, bs, free, want * 2 // 3 if short else want, T=T)


@gpu
@pytest.mark.parametrize("B,T", [(5, 6), (700, 40)])
def test_counts_reserved_in_place(B, T):
    """`reserved` may be new_lens itself."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(B)
    L, n = rng.integers(0, 60, B), rng.integers(0, T + 1, B)
    held = -(-L // 16)
    tables = make_tables(rng, held, int(held.sum()) + 1, 8)
    want = int((-(-(L + n) // 16) - held).sum())
    free = i32(10 ** 6 + rng.permutation(want))
    a = (i32(L), i32(n), i32(tables), 16, free, i32([want // 2]))
    b = (i32(L), i32(n), i32(tables), 16, free, i32([want // 2]))
    x, y = sv.kv_reserve(*a, max_new=T), sv.kv_reserve(*b, max_new=T, reserved=b[1])
    assert y[2] is b[1]
    for u, v in zip((*x, a[2], a[5]), (*y, b[2], b[5])):
        assert torch.equal(u, v)


# ------------------------------------------------- a step without blocks ----

@gpu
def test_a_step_in_which_blocks_run_out():
    """Requests that get no blocks sit the step out: the calls that follow take `reserved` for their new tokens, and
    nothing of theirs changes."""
    sv, _, kv = _pkg()
    rng = np.random.default_rng(4)
    B, T, Hq, Hkv, D, bs = 4, 5, 8, 2, 64, 4
    L, n = np.array([3, 8, 6, 4]), np.array([5, 5, 2, 5])
    tables = np.full((B, 5), -1)
    for b, row in enumerate(([0], [1, 2], [3, 4], [5])):
        tables[b, :len(row)] = row
    pool = 9
    tab, seq, free, count = i32(tables), i32(L), i32([6, 7, 8, -1, -1, -1]), i32([2])
    cache = [torch.zeros(pool, Hkv, bs, d, dtype=torch.uint8, device=DEV) for d in (D // 2, D // 2, 2, 2)]
    kw = dict(k_scale=cache[2], v_scale=cache[3])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots, pos, new = sv.kv_reserve(seq, i32(n), tab, bs, free, count, max_new=T, status=status)
    assert new.tolist() == [5, 0, 2, 0] and status.item() == kv.SV_KV_NO_BLOCKS and count.item() == 1
    status.zero_()
    x = torch.from_numpy(rng.standard_normal((B, T, Hq + 2 * Hkv, D))).bfloat16().to(DEV)
    q, k, v = x.split([Hq, Hkv, Hkv], 2)
    before = q.clone()
    out, _ = sv.qk_norm_rope(q, k, torch.from_numpy(angles(20, D)).to(DEV), pos, out=q, value=v, k_cache=cache[0],
                             v_cache=cache[1], slots=slots, status=status, **kw)
    assert torch.equal(out[1], before[1]) and torch.equal(out[3], before[3])
    y = torch.full((B, T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    sv.tree_attention(out, cache[0], cache[1], tab, seq, None, new, out=y, status=status, **kw)
    assert (y[1] == 9).all() and (y[3] == 9).all() and y[0].isfinite().all()
    kept = torch.minimum(i32([3, 1, 2, 4]), new)            # what a verification of all would keep
    sv.kv_compact(i32([[0, 1, 2, 3]] * B), kept, seq, tab, cache[0], cache[1], status=status, **kw)
    sv.kv_rollback(kept, seq, tab, bs, free, count, new, gamma_max=T, status=status)
    assert status.item() == 0 and seq.tolist() == [6, 8, 8, 4]
    want = [[0, 7], [1, 2], [3, 4], [5]]
    assert [[b for b in row if b >= 0] for row in tab.tolist()] == want and count.item() == 1

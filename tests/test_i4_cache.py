"""A cache of 4 bits: writing, reading, compacting, and attention over it."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref
import step_ref as sref
from test_paged_kv import ATTN, COMPACT, DEV, PTR, READ, WRITE, dense_pair, gpu, i32, make_tables

TD = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def _pkg():
    import speculative_decoding_verification_75_gb300 as sv
    from speculative_decoding_verification_75_gb300 import api, kv
    return sv, api, kv


# ------------------------------------------------------------- reference ----

def test_reference_by_hand():
    assert sref.SCALE[0] == 2.0 ** -14 and sref.SCALE[112] == 1 and sref.SCALE[117] == 1.625
    assert sref.SCALE[215] == 7680 and np.isnan(sref.SCALE[216:]).all()
    x = np.zeros((1, 64))
    x[0, :5] = [7, -7, 2.5, 3.5, -0.5]
    x[0, 32:35] = [7.5, -1, 1e9]
    codes, scale = sref.quantise(x)
    assert scale.tolist() == [[112, 215]]
    assert sref.unpack(codes)[0, :5].tolist() == [15, 1, 10, 12, 8]         # ties to even
    assert sref.unpack(codes)[0, 34] == 15
    x[0, 40] = np.inf
    codes, scale = sref.quantise(x)
    assert scale.tolist() == [[112, 255]] and (sref.unpack(codes)[0, 32:] == 8).all()
    for s in range(sref.TOP + 1):        # exact in both 16-bit types
        v = torch.from_numpy(sref.SCALE[s] * (np.arange(16) - 8.0))
        assert torch.equal(v.bfloat16().double(), v) and torch.equal(v.half().double(), v)


# -------------------------------------------------------------- refusals ----

def _cache(**over):
    f = dict(k=PTR, v=PTR, ks=PTR, vs=PTR, layer=0, block=2048, slayer=0, sblock=64, layers=1,
             blocks=8, heads=2, bs=16, D=64, dtype=4, tables=PTR, max_blocks=4)
    f.update(over)
    return list(f.values())


def _calls(lib, cache):
    return [
        lib.sv_kv_write(WRITE.pack(WRITE.size, *cache, PTR, 0, PTR, PTR, 512, 128, 64, 512, 128, 64, 2, 4, 1, 0), None),
        lib.sv_kv_read(READ.pack(READ.size, *cache, 0, PTR, PTR, PTR, 512, 128, 64, 512, 128, 64, 2, 4, 1, 0), None),
        lib.sv_kv_compact(COMPACT.pack(COMPACT.size, *cache, PTR, PTR, PTR, 2, 4, 0), None),
        lib.sv_tree_attention(ATTN.pack(ATTN.size, *cache, PTR, 0, PTR, 1024, 256, 64, 0, 0, PTR, 0, 0.125, 2, 4, 4, 1,
                                        PTR, 1 << 30, 0), None)]


@pytest.mark.parametrize("over", [
    dict(ks=0), dict(vs=0), dict(ks=PTR + 8), dict(D=40), dict(D=16), dict(D=288), dict(block=2048 + 16), dict(block=2016),
    dict(sblock=63), dict(k=PTR + 8), dict(blocks=-1), dict(bs=0)], ids=str)
def test_a_bad_cache_is_refused(over):
    _, api, _ = _pkg()
    assert set(_calls(api.load_library(), _cache(**over))) == {api.SV_ERR_INVALID_ARG}


def test_other_types_are_refused():
    _, api, _ = _pkg()
    lib, cache = api.load_library(), _cache()
    for dtype in (0, 3, 4):                                   # of keys: fp32, codes
        args = WRITE.pack(WRITE.size, *cache, PTR, 0, PTR, PTR, 512, 128, 64, 512, 128, 64, 2, 4, dtype, 0)
        assert lib.sv_kv_write(args, None) == api.SV_ERR_UNSUPPORTED_DTYPE
    for dtype in (3, 4):
        args = READ.pack(READ.size, *cache, 0, PTR, PTR, PTR, 512, 128, 64, 512, 128, 64, 2, 4, dtype, 0)
        assert lib.sv_kv_read(args, None) == api.SV_ERR_UNSUPPORTED_DTYPE


# ------------------------------------------------------------------- GPU ----

def make_cache(rng, pool, H, bs, D, halves=False, lead=()):
    """k, v, k_scale, v_scale on the GPU: any code (0 among them), scales around 1 / 4."""
    shape = (*lead, pool, 2, H, bs)
    c = torch.from_numpy(rng.integers(0, 256, (*shape, D // 2)).astype(np.uint8)).to(DEV)
    s = torch.from_numpy(rng.integers(90, 104, (*shape, D // 32)).astype(np.uint8)).to(DEV)
    k, v, ks, vs = (x[..., i, :, :, :] for x in (c, s) for i in range(2))
    return (k, v, ks, vs) if halves else tuple(x.clone(memory_format=torch.contiguous_format) for x in (k, v, ks, vs))


WRITE_CASES = [
    # B, T, H, D, bs, L, n, dtype, layout
    (1, 1, 2, 64, 16, [0], None, "bf16", "dense"),
    (1, 1, 1, 32, 1, [7], None, "fp16", "dense"),
    (3, 6, 8, 128, 16, [1, 15, 100], [6, 0, 1], "bf16", "fused"),
    (2, 33, 7, 32, 5, [3, 4], [33, 17], "fp16", "odd"),
    (4, 9, 1, 256, 24, [0, 23, 24, 47], [9, 9, 8, 1], "bf16", "heads"),
    (2, 700, 32, 96, 48, [0, 31], [700, 655], "fp16", "dense"),
    (5, 17, 3, 64, 128, [0, 1, 127, 128, 129], None, "fp16", "halves"),
]


@gpu
@pytest.mark.parametrize("case", WRITE_CASES, ids=str)
def test_write_and_read(case):
    B, T, H, D, bs, L, n, dt, layout = case
    sv, _, _ = _pkg()
    rng = np.random.default_rng(D + T)
    n = [T] * B if n is None else n
    need = [-(-(a + m) // bs) for a, m in zip(L, n)]
    pool, width = sum(need) + 2, max(need) + 1
    tables = make_tables(rng, need, pool, width)
    c = make_cache(rng, pool, H, bs, D, halves=layout == "halves")
    key, value = dense_pair(rng, (B, T, H, D), TD[dt], layout)
    if T > 1:                # quotients that are a whole number and a half, and their neighbours
        key[0, 0, 0, :32] = torch.arange(-16, 16, device=DEV).to(TD[dt]) * 0.875 / 2
        key[0, 0, 0, 0] = 7 * 0.875
        value[0, 1, 0, :32] = torch.arange(0, 32, device=DEV).to(TD[dt]) * 3.25 / 4
        value[0, 1, 0, 31] = -7 * 3.25
    want = [x.cpu().numpy().copy() for x in c]
    for x, i in ((key, 0), (value, 1)):
        x = ref.to64(x)
        for b in range(B):
            for t in range(n[b]):
                blk, row = tables[b, (L[b] + t) // bs], (L[b] + t) % bs
                want[i][blk, :, row], want[i + 2][blk, :, row] = sref.quantise(x[b, t])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(k_scale=c[2], v_scale=c[3], status=status)
    lens = None if n == [T] * B else i32(n)
    sv.kv_write(key, value, c[0], c[1], i32(tables), i32(L), lens, **kw)
    for g, w in zip(c, want):             # every byte, the untouched rows among them
        assert np.array_equal(g.cpu().numpy(), w)
    for odt in TD:
        out = tuple(torch.full((B, T, H, D), 5.0, dtype=TD[odt], device=DEV) for _ in range(2))
        sv.kv_read(c[0], c[1], i32(tables), i32(n), i32(L), out=out, **kw)
        for o, i in ((out[0], 0), (out[1], 1)):
            o = ref.to64(o)
            for b in range(B):
                for t in range(n[b]):
                    blk, row = tables[b, (L[b] + t) // bs], (L[b] + t) % bs
                    assert np.array_equal(o[b, t], sref.values(want[i][blk, :, row], want[i + 2][blk, :, row]))
                assert (o[b, n[b]:] == 5).all()
    new = sv.kv_read(c[0], c[1], i32(tables), i32(n), i32(L), max_len=T, k_scale=c[2], v_scale=c[3])
    assert new[0].shape == (B, T, H, D) and new[0].dtype == torch.bfloat16
    assert status.item() == 0


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_write_what_is_not_finite_tiny_or_large(dt):
    sv, _, _ = _pkg()
    x = np.zeros((1, 8, 1, 96))
    x[0, 0, 0, :3] = [np.inf, 1, -2]
    x[0, 1, 0, 33:35] = [np.nan, 3]
    x[0, 2, 0, :3] = [2.0 ** -16, -(2.0 ** -15), 2.0 ** -24]           # half a step of the smallest scale
    x[0, 3, 0, :3] = [53760, 60000, -65504 if dt == "fp16" else -3e38]
    x[0, 4, 0, :] = -0.0
    x[0, 5, 0, :40] = 7 * 2.0 ** -14
    x[0, 6, 0, :2] = [7.03125, -7.03125]
    x[0, 7, 0, ::3] = -np.inf
    key = torch.from_numpy(x).to(TD[dt]).to(DEV)
    rng = np.random.default_rng(0)
    c = make_cache(rng, 1, 1, 8, 96)
    sv.kv_write(key, key.neg(), c[0], c[1], i32([[0]]), i32([0]), k_scale=c[2], v_scale=c[3])
    for i, s in ((0, 1.0), (1, -1.0)):
        codes, scale = sref.quantise(ref.to64(key)[0, :, 0] * s)
        assert np.array_equal(c[i].cpu().numpy()[0, 0], codes)
        assert np.array_equal(c[i + 2].cpu().numpy()[0, 0], scale)


@gpu
def test_write_every_16_bit_amplitude():
    """Scale bytes and codes of every finite bf16 and fp16 magnitude as the largest of its group."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(1)
    for dt in ("bf16", "fp16"):
        m = torch.arange(0x7C00 if dt == "fp16" else 0x7F80, dtype=torch.int32).to(torch.int16).view(TD[dt])
        n = m.numel()
        # The largest of a group and fractions of it near whole numbers and a half.
        f = torch.from_numpy((rng.integers(0, 15, (n, 31)) / 14 * (1 + rng.integers(-2, 3, (n, 31)) * 2.0 ** -9)))
        x = torch.cat([m.double()[:, None], (m.double()[:, None] * f).to(TD[dt]).double()], 1)
        x = torch.where(x.abs() > m.double()[:, None], m.double()[:, None], x)
        x[:, 1::2] *= -1
        key = x.to(TD[dt]).to(DEV).view(1, n, 1, 32)
        c = [torch.zeros(-(-n // 64), 1, 64, d, dtype=torch.uint8, device=DEV) for d in (16, 16, 1, 1)]
        sv.kv_write(key, key, c[0], c[1], torch.arange(c[0].shape[0], dtype=torch.int32, device=DEV)[None], i32([0]),
                    k_scale=c[2], v_scale=c[3])
        codes, scale = sref.quantise(ref.to64(key)[0, :, 0])
        assert np.array_equal(c[2].view(-1)[:n].cpu().numpy(), scale[:, 0])
        assert np.array_equal(c[0].view(-1, 16)[:n].cpu().numpy(), codes)


@gpu
def test_reading_scales_that_are_nan():
    sv, _, _ = _pkg()
    c = make_cache(np.random.default_rng(2), 2, 1, 8, 64)
    c[2][:] = torch.arange(256 - 32, 256, dtype=torch.uint8).to(DEV).view(2, 1, 8, 2)
    k, _ = sv.kv_read(c[0], c[1], i32([[0, 1]]), i32([16]), max_len=16, dtype=torch.float32, k_scale=c[2], v_scale=c[3])
    assert k.isnan().all()
    c[2][:] = 215
    k, _ = sv.kv_read(c[0], c[1], i32([[0, 1]]), i32([16]), max_len=16, dtype=torch.float16, k_scale=c[2], v_scale=c[3])
    assert k.isfinite().all() and k.abs().max() == 61440


@gpu
@pytest.mark.parametrize("layers,D", [(None, 64), (3, 32), (2, 160)])
def test_compact(layers, D):
    sv, _, _ = _pkg()
    rng = np.random.default_rng(D)
    B, P, H, bs = 4, 7, 3, 5
    L, k = [0, 4, 11, 3], [7, 1, 5, 0]
    path = np.stack([np.sort(rng.choice(20, P, replace=False)) for _ in range(B)]).astype(np.int32)
    path[0, :3] = [0, 1, 2]
    path[0, 3:] = np.sort(rng.choice(np.arange(4, 20), 4, replace=False))
    need = [-(-(x + 20) // bs) for x in L]
    tables = make_tables(rng, need, sum(need) + 1, max(need))
    c = make_cache(rng, sum(need) + 1, H, bs, D, lead=(layers,) if layers else ())
    want = [x.cpu().numpy().copy() for x in c]
    for w in want:
        src = w.copy()
        for b in range(B):
            for i in range(k[b]):
                f, t = L[b] + path[b, i], L[b] + i
                w[..., tables[b, t // bs], :, t % bs, :] = src[..., tables[b, f // bs], :, f % bs, :]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.kv_compact(i32(path), i32(k), i32(L), i32(tables), c[0], c[1], k_scale=c[2], v_scale=c[3], status=status)
    assert status.item() == 0
    for g, w in zip(c, want):
        assert np.array_equal(g.cpu().numpy(), w)


# ------------------------------------------------------------- attention ----

def attn_setup(rng, B, T, Hq, Hkv, D, bs, L, n, dt, tree, pad=0, halves=False):
    need = [max(-(-(a + m) // bs), 0) for a, m in zip(L, n)]
    pool, width = sum(need) + 3, max(max(need), 1) + pad
    s = dict(tables=make_tables(rng, need, pool, width), L=L, n=n)
    s["c"] = make_cache(rng, pool, Hkv, bs, D, halves=halves)
    s["q"] = torch.from_numpy(rng.standard_normal((B, T, Hq, D)) * 0.7).to(TD[dt]).to(DEV)
    s["mask"] = None
    if tree:
        m = np.broadcast_to(np.eye(T, dtype=bool), (B, T, T)).copy()
        for b in range(B):
            for i in range(1, T):
                m[b, i] |= m[b, rng.integers(0, i)]
        s["mask"] = m
    return s


def run(s, out=None, **kw):
    sv, _, _ = _pkg()
    c = s["c"]
    mask = None if s["mask"] is None else torch.from_numpy(s["mask"]).to(DEV)
    return sv.tree_attention(s["q"], c[0], c[1], i32(s["tables"]), i32(s["L"]), mask, i32(s["n"]), out=out,
                             k_scale=c[2], v_scale=c[3], **kw)


def check(s, dt, scale=None, want_status=0):
    q = s["q"]
    B, T, Hq, D = q.shape
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:3], 9.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    run(s, out, lse=lse, status=status, scale=scale)
    cache = sref.Cache(s["c"][0], s["c"][1], i32(s["tables"]), s["c"][2], s["c"][3])
    w, wl, tol, ltol, live, st = ref.attention(ref.to64(q), cache, s["L"], s["n"], s["mask"],
                                               D ** -0.5 if scale is None else scale, UNIT[dt])
    got, gl = ref.to64(out), ref.to64(lse)
    assert status.item() == want_status | st
    live4 = np.broadcast_to(live[:, :, None, None], got.shape)
    assert (got[~live4] == 9).all() and (gl[~live4[..., 0]] == 9).all()
    nan = np.isnan(w)
    assert np.array_equal(np.isnan(got) & live4, nan & live4)
    err = np.where(live4 & ~nan, np.abs(got - w), 0)
    assert (err <= tol)[live4 & ~nan].all(), float((err / (tol + 1e-300)).max())
    ok = live4[..., 0] & np.isfinite(wl)
    assert (np.abs(gl[ok] - wl[ok]) <= ltol[ok]).all()
    inf = live4[..., 0] & np.isneginf(wl)
    assert np.isneginf(gl[inf]).all()
    return out


ATTN_CASES = [
    # B, T, Hq, Hkv, D, bs, L, n, dtype, tree
    (1, 1, 14, 2, 64, 16, [500], [1], "bf16", False),
    (1, 1, 1, 1, 128, 8, [0], [1], "fp16", False),
    (3, 6, 16, 2, 128, 16, [0, 127, 1000], [6, 0, 5], "bf16", False),
    (3, 6, 16, 2, 64, 32, [1, 128, 700], [6, 3, 5], "fp16", False),
    (2, 9, 7, 7, 128, 64, [63, 300], [9, 4], "bf16", True),
    (2, 9, 7, 1, 64, 24, [129, 257], [9, 9], "fp16", True),
    (2, 33, 8, 2, 128, 16, [100, 0], [33, 20], "bf16", True),
    (2, 40, 28, 4, 64, 128, [130, 5], [37, 40], "fp16", True),
    (1, 150, 2, 1, 128, 16, [70], [150], "bf16", False),
    (1, 130, 3, 3, 64, 40, [0], [129], "fp16", True),
    (1, 2, 71, 1, 64, 16, [200], [2], "bf16", False),
    (40, 1, 8, 8, 128, 16, list(range(0, 400, 10)), [1] * 40, "fp16", False),
    # head dimensions and block sizes of the general kernel
    (2, 5, 6, 2, 32, 16, [0, 70], [5, 4], "bf16", True),
    (2, 3, 4, 2, 96, 7, [40, 9], [3, 3], "fp16", False),
    (1, 2, 2, 1, 256, 16, [33], [2], "bf16", False),
    (1, 4, 4, 2, 128, 5, [33], [4], "bf16", True),
]


@gpu
@pytest.mark.parametrize("case", ATTN_CASES, ids=str)
def test_attention(case):
    B, T, Hq, Hkv, D, bs, L, n, dt, tree = case
    s = attn_setup(np.random.default_rng(T * D + B), B, T, Hq, Hkv, D, bs, L, n, dt, tree)
    out = check(s, dt)
    if B > 1:
        check(s, dt, scale=-0.3)
    again = torch.full_like(out, 9.0)
    run(s, again)
    assert torch.equal(out, again)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rows_that_see_nothing_and_empty_requests(D, dt):
    s = attn_setup(np.random.default_rng(3), 4, 5, 8, 2, D, 16, [0, 0, 40, 128], [5, 0, 5, 1], dt, True)
    s["mask"][0, 2] = False
    s["mask"][0, 4] = [False, False, False, False, True]
    out = check(s, dt)
    assert (out[0, 2] == 0).all()


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_nan_groups(D, dt):
    """NaN among committed tokens reaches every row of its head, among new ones only those that see it; behind
    the last token it has no influence."""
    rng = np.random.default_rng(4)
    for where, side in (("old", 2), ("old", 3), ("new", 2), ("new", 3), ("behind", 2), ("behind", 3)):
        s = attn_setup(rng, 2, 6, 8, 2, D, 16, [130, 20], [6, 5], dt, True)
        pos = {"old": 3, "new": 132, "behind": 136}[where]
        s["mask"][0, 0, 1:] = False
        s["c"][side][int(s["tables"][0, pos // 16]), 1, pos % 16, D // 64] = 255
        out = check(s, dt)
        assert out[1].isfinite().all() and out[0, :, :4].isfinite().all()
        assert out[0, 0, 4:].isfinite().all() == (where != "old")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_large_and_small_scores(dt):
    """References that rise late, probabilities that vanish, scales at both ends."""
    for D in (64, 128):
        s = attn_setup(np.random.default_rng(5), 2, 4, 8, 2, D, 16, [700, 300], [4, 4], dt, False)
        s["c"][2][:] = torch.randint(60, 125, tuple(s["c"][2].shape), device=DEV).to(torch.uint8)
        check(s, dt)
        check(s, dt, scale=3.0)
        check(s, dt, scale=1e-30)
        s["c"][2][:] = torch.randint(0, 216, tuple(s["c"][2].shape), device=DEV).to(torch.uint8)
        s["c"][3][:] = torch.randint(0, 216, tuple(s["c"][3].shape), device=DEV).to(torch.uint8)
        check(s, dt)
        check(s, dt, scale=0.0)


@gpu
def test_missing_and_bad_blocks():
    for bad, bit in ((-1, ref.MISSING), (-7, ref.BLOCK), (1 << 20, ref.BLOCK)):
        for T, L in ((5, 300), (5, 1500), (1, 40)):
            s = attn_setup(np.random.default_rng(6), 2, T, 8, 2, 128, 16, [L, 90], [T, T], "bf16", False)
            s["tables"][0, 1] = bad
            s["tables"][1, 5] = bad
            check(s, "bf16", want_status=bit)
    # A table that is too short, and one without any block.
    s = attn_setup(np.random.default_rng(7), 2, 3, 8, 2, 64, 16, [100, 90], [3, 3], "fp16", False)
    s["tables"] = s["tables"][:, :4].copy()
    check(s, "fp16", want_status=ref.SHORT)
    s["tables"][:] = -1
    out = check(s, "fp16", want_status=ref.SHORT | ref.MISSING)
    assert (out == 0).all()


@gpu
def test_bad_lengths_and_halves_and_strides():
    s = attn_setup(np.random.default_rng(8), 3, 4, 8, 2, 128, 16, [100, 60, 30], [4, 4, 4], "bf16", False, halves=True)
    s["L"] = [100, -1, 30]
    s["n"] = [4, 4, 5]
    check(s, "bf16", want_status=ref.LENGTH)
    # Queries as a view of a projection, and heads outside tokens.
    s = attn_setup(np.random.default_rng(9), 3, 4, 8, 2, 128, 16, [100, 60, 30], [4, 4, 4], "bf16", True, pad=2)
    buf = torch.zeros(3, 4, 12, 128, dtype=torch.bfloat16, device=DEV)
    buf[:, :, 1:9] = s["q"]
    want = run(s)
    s["q"] = buf[:, :, 1:9]
    assert torch.equal(run(s), want)
    s["q"] = buf[:, :, 1:9].transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(run(s), want)
    odd = torch.zeros(3, 4, 8, 129, dtype=torch.bfloat16, device=DEV)
    odd[..., 1:] = buf[:, :, 1:9]
    s["q"] = odd[..., 1:]                     # rows on odd elements
    check(s, "bf16")


@gpu
@pytest.mark.parametrize("B,Hkv,D,G,T,L,dt", [(1, 2, 128, 8, 1, 50001, "fp16"), (1, 2, 64, 4, 3, 39997, "bf16"),
                                              (2, 8, 128, 8, 6, 33333, "bf16"), (3, 8, 64, 7, 2, 30000, "fp16"),
                                              (2, 8, 128, 2, 3, 45000, "fp16")])
def test_long_contexts(B, Hkv, D, G, T, L, dt):
    """Units cut into many ranges, and ranges of many tiles, against the dense form in 64 bits on the GPU."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(L)
    Ls = [L - 1111 * b for b in range(B)]
    s = attn_setup(rng, B, T, Hkv * G, Hkv, D, 64, Ls, [T] * B, dt, False)
    lse = torch.zeros(B, T, Hkv * G, device=DEV)
    out = run(s, lse=lse)
    S = max(Ls) + T
    K, V = sv.kv_read(s["c"][0], s["c"][1], i32(s["tables"]), i32([x + T for x in Ls]), max_len=S, dtype=torch.float32,
                      k_scale=s["c"][2], v_scale=s["c"][3])
    for b in range(B):
        k, v = K[b].double(), V[b].double()
        q = s["q"][b].double().view(T, Hkv, G, D)
        z = torch.einsum("thgd,shd->htgs", q, k) / math.sqrt(D)
        hide = torch.arange(S, device=DEV) > (Ls[b] + torch.arange(T, device=DEV))[:, None]
        z = z.masked_fill(hide[None, :, None], -math.inf)
        p = z.softmax(-1)

        def rows(x):
            return torch.einsum("htgs,shd->thgd", p, x).reshape(T, Hkv * G, D)

        w, a = rows(v), rows(v.abs())
        # Scores off by (D + 8) 2^-23 sum |q k|; probabilities and result rounded to the type, in fp16 those below its
        # normal range by 2^-25 of the largest, whose share of the sum is p.max(), and values are below 16; sums of S terms.
        ds = (D + 8) * 2.0 ** -23 * torch.einsum("thgd,shd->htgs", q.abs(), k.abs()).max() / math.sqrt(D)
        rel = 2 * ds + 2.0 ** -19 + 2 * S * 2.0 ** -24
        pm = p.amax(-1).permute(1, 0, 2).reshape(T, Hkv * G, 1)
        tol = (UNIT[dt] + rel) * a + UNIT[dt] * w.abs() + (S * 2.0 ** -25 * pm * 16 + 2.0 ** -25) * (dt == "fp16")
        assert ((out[b].double() - w).abs() <= tol).all()
        want = z.logsumexp(-1).permute(1, 0, 2).reshape(T, Hkv * G)
        assert (lse[b].double() - want).abs().max() < 1e-3


@gpu
@pytest.mark.parametrize("T,G,D,dt", [(3, 8, 64, "bf16"), (9, 8, 128, "fp16"), (7, 4, 64, "fp16"), (64, 1, 128, "bf16")])
def test_units_of_different_sizes_follow_each_other(T, G, D, dt):
    """A thread block's units of few and many rows in turn: nothing of one may reach the one before, however
    its warps are timed, so every run gives the same."""
    rng = np.random.default_rng(T)
    B, Hkv = 64, 8
    L = [int(x) for x in rng.integers(100, 200, B)]
    n = [int(x) for x in rng.integers(1, T + 1, B)]
    s = attn_setup(rng, B, T, Hkv * G, Hkv, D, 16, L, n, dt, False)
    want = check(s, dt)
    for _ in range(12):
        out = torch.full_like(want, 9.0)
        run(s, out)
        assert torch.equal(out, want)


@gpu
def test_graph_streams_and_shared_workspace():
    """Captured and replayed on new contents; on a side stream; one workspace for several sizes."""
    sv, _, kv = _pkg()
    rng = np.random.default_rng(11)
    a = attn_setup(rng, 2, 4, 8, 2, 128, 16, [700, 60], [4, 4], "bf16", False)
    b = attn_setup(rng, 3, 20, 8, 2, 64, 16, [100, 60, 900], [20, 4, 7], "bf16", True)
    wa, wb = run(a), run(b)
    ws = torch.empty(kv.tree_attention_workspace_bytes(3, 20, 8, 2, 128), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)
    dev = [dict(t=i32(s["tables"]), L=i32(s["L"]), n=i32(s["n"]),
                m=None if s["mask"] is None else torch.from_numpy(s["mask"]).to(DEV)) for s in (a, b)]
    outs = [torch.zeros_like(s["q"]) for s in (a, b)]

    def both():
        for s, d, o in zip((a, b), dev, outs):
            sv.tree_attention(s["q"], s["c"][0], s["c"][1], d["t"], d["L"], d["m"], d["n"], out=o, workspace=ws,
                              k_scale=s["c"][2], v_scale=s["c"][3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    live = torch.arange(20, device=DEV)[None] < dev[1]["n"][:, None]
    assert torch.equal(outs[0], wa) and torch.equal(outs[1][live], wb[live])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for s in (a, b):
        s["q"].mul_(0.5)
    want = [run(a), run(b)]
    for o in outs:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1][live], want[1][live])

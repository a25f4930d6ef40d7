"""Places for new tokens (kv_reserve), norm and rotation (qk_norm_rope), and a whole step through all operators."""
import struct

import numpy as np
import pytest
import torch

import paged_ref as ref
import step_ref as sref
from test_paged_kv import DEV, PTR, gpu, i32, make_tables

TD = {"bf16": torch.bfloat16, "fp16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def _pkg():
    import speculative_decoding_verification_75_gb300 as sv
    from speculative_decoding_verification_75_gb300 import api, kv
    return sv, api, kv


# -------------------------------------------------------------- refusals ----

RESERVE = struct.Struct("@17q")
ROPE = struct.Struct("@42qd10q")


def _reserve(lib, **over):
    f = dict(seq=PTR, new=0, tables=PTR, width=4, bs=16, list=PTR, count=PTR, cap=8, mask=0, msb=0, slots=PTR,
             pos=PTR, res=PTR, B=2, T=4, status=0)
    f.update(over)
    return lib.sv_kv_reserve(RESERVE.pack(RESERVE.size, *f.values()), None)


def test_bad_reservations_are_refused():
    _, api, _ = _pkg()
    lib = api.load_library()
    bad = api.SV_ERR_INVALID_ARG
    for over in (dict(seq=0), dict(seq=PTR + 2), dict(new=PTR + 1), dict(tables=0), dict(tables=PTR + 2), dict(width=-1),
                 dict(bs=0), dict(bs=-16), dict(bs=1 << 21), dict(width=1 << 28), dict(list=0), dict(list=PTR + 1),
                 dict(count=0), dict(count=PTR + 2), dict(cap=-1), dict(cap=1 << 31), dict(msb=-1), dict(slots=0),
                 dict(slots=PTR + 4), dict(pos=0), dict(pos=PTR + 2), dict(res=0), dict(B=-1), dict(T=-1),
                 dict(B=32769), dict(B=1 << 16, T=1 << 16)):
        assert _reserve(lib, **over) == bad, over
    assert _reserve(lib, B=0) == api.SV_OK
    assert lib.sv_kv_reserve(None, None) == bad
    assert lib.sv_kv_reserve((8).to_bytes(8, "little") + bytes(400), None) == bad


def _rope(lib, **over):
    f = dict(k=PTR, v=PTR, ks=0, vs=0, layer=0, block=2048, slayer=0, sblock=0, layers=1, blocks=8, heads=2, bs=16,
             D=64, cdtype=1, tables=0, max_blocks=0,
             q=PTR, key=PTR, val=PTR, qb=1024, qt=256, qh=64, kb=512, kt=128, kh=64, vb=512, vt=128, vh=64,
             out=PTR, kout=0, ob=1024, ot=256, oh=64, kob=0, kot=0, koh=0, qw=PTR, kw=0, cs=PTR, pos=PTR, slots=PTR,
             eps=1e-6, P=100, R=64, pairs=0, B=2, T=4, Hq=4, Hkv=2, hd=64, dtype=1, status=0)
    f.update(over)
    return lib.sv_qk_norm_rope(ROPE.pack(ROPE.size, *f.values()), None)


def test_bad_rotations_are_refused():
    _, api, _ = _pkg()
    lib = api.load_library()
    bad, dt = api.SV_ERR_INVALID_ARG, api.SV_ERR_UNSUPPORTED_DTYPE
    for over in (dict(k=0), dict(k=PTR + 8), dict(v=0), dict(block=100), dict(blocks=-1), dict(heads=3), dict(D=128),
                 dict(v=PTR, k=PTR), dict(q=0), dict(q=PTR + 1), dict(key=0), dict(val=0), dict(out=0), dict(out=PTR + 1),
                 dict(kout=PTR + 1), dict(qb=-8), dict(oh=-1), dict(vh=-64), dict(qw=PTR + 8), dict(kw=PTR + 2),
                 dict(cs=0), dict(cs=PTR + 4), dict(cs=PTR + 2, pairs=1), dict(pos=0), dict(pos=PTR + 2),
                 dict(slots=PTR + 4), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(P=-1),
                 dict(R=72), dict(R=66, hd=128), dict(R=8), dict(R=3, pairs=1), dict(R=-16), dict(hd=12, D=12),
                 dict(hd=264), dict(B=-1), dict(T=-1), dict(B=1 << 16, T=1 << 16), dict(Hq=-1), dict(Hkv=65537),
                 dict(slots=0)):                             # no cache and no key_out
        if "v" not in over:
            over = dict(over, v=2 * PTR)
        assert _rope(lib, **over) == bad, over
    assert _rope(lib, v=2 * PTR, dtype=0) == dt
    assert _rope(lib, v=2 * PTR, dtype=2) == dt              # fp16 into a bf16 cache
    assert _rope(lib, v=2 * PTR, cdtype=0) == dt
    assert _rope(lib, v=2 * PTR, B=0) == api.SV_OK
    assert _rope(lib, v=2 * PTR, Hq=0, Hkv=0, slots=0) == api.SV_OK
    assert lib.sv_qk_norm_rope(None, None) == bad
    assert lib.sv_qk_norm_rope((8).to_bytes(8, "little") + bytes(600), None) == bad


def test_cpu_tensors_are_refused():
    sv, _, _ = _pkg()
    x, t, n = torch.zeros(1, 3, 2, 64), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.kv_reserve(n, None, t, 16, n, n, max_new=3)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.qk_norm_rope(x.bfloat16(), x.bfloat16(), x[0, 0], t)
    with pytest.raises(TypeError):
        sv.qk_norm_rope(3, x, x, t)
    with pytest.raises(TypeError):
        sv.kv_reserve(n, None, [1], 16, n, n)


# --------------------------------------------------------------- reserve ----

def reserve(L, n, tables, bs, free, count, mask=None, T=None, **kw):
    """The call against the reference; every result compared."""
    sv, _, _ = _pkg()
    B = len(L)
    T = max(n) if T is None else T
    tab, cnt, status = i32(tables), i32([count]), torch.zeros(1, dtype=torch.int32, device=DEV)
    m = None if mask is None else torch.from_numpy(mask).to(DEV)
    got = sv.kv_reserve(i32(L), i32(n), tab, bs, i32(free), cnt, m, max_new=T, status=status, **kw)
    want = sref.reserve(L, n, tables, bs, np.asarray(free), count, mask if mask is None or mask.ndim == 3 else
                        np.broadcast_to(mask, (B, T, T)), T)
    for g, w in zip((*got, tab, cnt, status), (*want[:4], [want[4]], [want[5]])):
        assert np.array_equal(g.cpu().numpy(), w)
    return want


@gpu
@pytest.mark.parametrize("B,T,bs", [(1, 1, 16), (1, 1, 1), (8, 6, 16), (5, 64, 32), (3, 700, 16), (2, 5000, 8), (700, 6, 16),
                                    (300, 33, 4), (40, 4096, 128)])
@pytest.mark.parametrize("short", [False, True])
def test_reserve(B, T, bs, short):
    rng = np.random.default_rng(B + T)
    L, n = rng.integers(0, 300, B), rng.integers(0, T + 1, B)
    if B > 3:
        L[1], n[2], n[3] = 0, 0, T
    held = -(-L // bs) + rng.integers(0, 3, B)             # some have a block or two already
    width = int(max((-(-(L + n) // bs)).max(), held.max())) + 1
    tables = make_tables(rng, held, int(held.sum()) + 1, width)
    want = int(np.maximum(-(-(L + n) // bs) - held, 0).sum())
    free = 10 ** 6 + rng.permutation(want + 7)
    _, _, res, _, left, st = reserve(L, n, tables, bs, free, want // 2 if short else want, T=T)
    if not short:
        assert st == 0 and left == 0 and np.array_equal(res, n)


@gpu
@pytest.mark.parametrize("T", [1, 5, 8, 64, 97])
def test_reserve_tree(T):
    rng = np.random.default_rng(T)
    B, bs = 6, 16
    L, n = rng.integers(0, 100, B), rng.integers(0, T + 1, B)
    n[0] = T
    mask = np.broadcast_to(np.eye(T, dtype=bool), (B, T, T)).copy()
    for b in range(B):
        for i in range(1, T):
            mask[b, i] |= mask[b, rng.integers(0, i)]
    mask[:, :, T // 2:] |= rng.random((B, T, T - T // 2)) < 0.3     # columns past n among them: they do not count
    if T > 4:
        mask[0, 3] = False
    held = -(-L // bs)
    tables = make_tables(rng, held, int(held.sum()) + 1, 16)
    free = 1000 + rng.permutation(200)
    reserve(L, n, tables, bs, free, 200, mask, T)
    reserve(L, n, tables, bs, free, 200, mask[1], T)                # one mask for all
    reserve(L, n, tables, bs, free, 3, mask, T)


@gpu
def test_reserve_problems():
    bs, free = 16, 100 + np.arange(50)
    L = np.array([-1, 5, 20, 20, 40, 16, 2 ** 31 - 4, 33, 60, 0])
    n = np.array([3, -1, 9, 3, 3, 4, 5, 4, 5, 4])
    T = 8
    tables = np.full((10, 4), -1)
    tables[3, 0] = 5                                    # 20 tokens: the second block is missing
    tables[4, :3] = [1, 2, 3]
    tables[5, :2] = [4, -9]                             # an entry below -1 where a block is lacking
    tables[7, :3] = [6, 7, -5]                          # and where the last committed tokens are
    tables[8, :4] = [8, 9, 10, 11]                      # 65 tokens: the table is too short
    _, _, res, _, _, st = reserve(L, n, tables, bs, free, 50, T=T)
    assert st == ref.LENGTH | ref.SHORT | ref.MISSING | ref.BLOCK and res.tolist() == [0, 0, 0, 0, 3, 0, 0, 0, 0, 4]
    for count in (0, -3, 1, 50, 51, 2 ** 31 - 1):       # counts outside the list are its ends
        reserve([0, 0], [5, 5], np.full((2, 2), -1), bs, free, count)
    # A request that finds too few blocks, those behind it that lack none, and one that would fit.
    t = np.array([[-1, -1, -1], [7, -1, -1], [-1, -1, -1]])
    _, _, res, _, left, st = reserve([0, 3, 0], [40, 5, 10], t, bs, free, 2, T=40)
    assert res.tolist() == [0, 5, 0] and left == 2 and st == sref.NO_BLOCKS
    reserve([0, 0], [0, 0], np.full((2, 0), -1), bs, [], 0, T=0)
    reserve([0, 0], [0, 3], np.full((2, 0), -1), bs, [], 0, T=3)


@gpu
def test_reserve_given_results_and_refusals():
    sv, _, kv = _pkg()
    L, n, tab, free, cnt = i32([3, 20]), i32([4, 2]), i32([[0, -1], [1, 2]]), i32([9, 8]), i32([2])
    slots = torch.zeros(2, 4, dtype=torch.int64, device=DEV)
    pos, res = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    got = sv.kv_reserve(L, n, tab, 16, free, cnt, slots=slots, positions=pos, reserved=res)
    assert got[0] is slots and got[1] is pos and got[2] is res
    assert slots.tolist() == [[3, 4, 5, 6], [36, 37, -1, -1]] and cnt.item() == 2
    none = sv.kv_reserve(L, None, tab, 16, free, cnt, max_new=2)[2]
    assert none.tolist() == [2, 2]
    for call in (lambda: sv.kv_reserve(L, n, tab, 16, free, cnt),
                 lambda: sv.kv_reserve(L, n, tab.long(), 16, free, cnt, max_new=4),
                 lambda: sv.kv_reserve(L, n, tab.t(), 16, free, cnt, max_new=4),
                 lambda: sv.kv_reserve(L[:1], n, tab, 16, free, cnt, max_new=4),
                 lambda: sv.kv_reserve(L, n, tab, 16, free, free, max_new=4),
                 lambda: sv.kv_reserve(L, n, tab, 16, free, cnt, max_new=-1),
                 lambda: sv.kv_reserve(L, n, tab, 16, free, cnt, slots=slots.int()),
                 lambda: sv.kv_reserve(L, n, tab, 16, free, cnt, slots=slots[:, :3]),
                 lambda: sv.kv_reserve(L, n, tab, 16, free, cnt, slots=slots, positions=pos[:, ::2]),
                 lambda: sv.kv_reserve(L, n, tab, 16, free, cnt, slots.bool(), max_new=4),
                 lambda: sv.kv_reserve(L, n, tab, 0, free, cnt, max_new=4),
                 lambda: sv.kv_reserve(L, n, tab, "x", free, cnt, max_new=4)):
        with pytest.raises((TypeError, ValueError, kv.SpecVerifyError)):
            call()
    assert cnt.item() == 2


# ------------------------------------------------------------------ rope ----

def projection(rng, B, T, Hq, Hkv, D, dt, odd=False):
    x = rng.standard_normal((B, T, Hq + 2 * Hkv, D)) * 2.0 ** rng.integers(-6, 6, (B, T, Hq + 2 * Hkv, 1))
    x = torch.from_numpy(x).to(TD[dt]).to(DEV)
    if odd:
        buf = torch.zeros(B, T, Hq + 2 * Hkv, D + 1, dtype=TD[dt], device=DEV)
        buf[..., 1:] = x
        x = buf[..., 1:]
    return x.split([Hq, Hkv, Hkv], 2)


def angles(P, R):
    a = np.arange(P)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / max(R, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def close(got, x, w, cs, pos, eps, pairs, dt):
    want, tol = sref.norm_rope(ref.to64(x), None if w is None else ref.to64(w), cs.astype(np.float64), pos, eps, pairs)
    tol = tol + UNIT[dt] * (np.abs(want) + tol) + 2.0 ** -25     # fp16's subnormal numbers
    assert (np.abs(ref.to64(got) - want) <= tol).all()


ROPE_CASES = [
    # B, T, Hq, Hkv, D, R, dtype, pairs, odd rows
    (1, 1, 14, 2, 64, 64, "bf16", False, False),
    (2, 5, 8, 2, 128, 128, "bf16", False, False),
    (2, 5, 8, 2, 128, 64, "fp16", False, False),
    (3, 4, 5, 3, 96, 96, "bf16", False, False),
    (3, 4, 5, 3, 80, 32, "fp16", False, True),
    (1, 7, 1, 1, 8, 0, "bf16", False, False),
    (2, 3, 3, 1, 256, 256, "bf16", False, True),
    (2, 5, 8, 2, 128, 128, "fp16", True, False),
    (2, 5, 7, 1, 64, 42, "bf16", True, False),
    (1, 3, 2, 2, 40, 40, "fp16", True, True),
    (300, 9, 32, 8, 128, 128, "bf16", False, False),
    (2, 3, 0, 3, 64, 64, "bf16", False, False),
    (2, 3, 3, 0, 64, 64, "bf16", False, False),
]


@gpu
@pytest.mark.parametrize("case", ROPE_CASES, ids=str)
@pytest.mark.parametrize("norm", ["both", "q", "k", "none"])
def test_norm_rope(case, norm):
    B, T, Hq, Hkv, D, R, dt, pairs, odd = case
    if B > 100 and norm != "both":
        return
    sv, _, _ = _pkg()
    rng = np.random.default_rng(D + R)
    q, k, _ = projection(rng, B, T, Hq, Hkv, D, dt, odd)
    cs, pos = angles(500, R), rng.integers(0, 500, (B, T))
    wq, wk = (torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(TD[dt]).to(DEV) for _ in range(2))
    wq, wk = wq if norm in ("both", "q") else None, wk if norm in ("both", "k") else None
    c = torch.from_numpy(cs).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    eps = 1e-5
    out, ko = sv.qk_norm_rope(q, k, c, i32(pos), wq, wk, eps=eps, interleaved=pairs, status=status)
    close(out, q, wq, cs, pos, eps, pairs, dt)
    close(ko, k, wk, cs, pos, eps, pairs, dt)
    assert status.item() == 0
    # In place, as views of the projection.
    got = sv.qk_norm_rope(q, k, c, i32(pos), wq, wk, eps=eps, interleaved=pairs, out=q, key_out=k)
    assert got[0] is q and torch.equal(q, out) and torch.equal(k, ko)


@gpu
@pytest.mark.parametrize("cdt", ["same", "e4m3", "i4"])
@pytest.mark.parametrize("dt,D,R,pairs,odd", [("bf16", 128, 128, False, False), ("fp16", 64, 32, False, True),
                                             ("bf16", 96, 96, True, False), ("fp16", 32, 32, False, False),
                                             ("bf16", 256, 64, True, True)])
def test_into_the_cache(cdt, dt, D, R, pairs, odd):
    """The same bytes as norm and rotation into tensors and kv_write of these; what has no slot stays as it was."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(D)
    B, T, Hq, Hkv, bs = 3, 7, 5, 3, 8
    q, k, v = projection(rng, B, T, Hq, Hkv, D, dt, odd)
    k[0, 0, 0, 1] = float("inf")
    v[1, 0, 1, 0] = float("nan")
    L, n = [0, 13, 30], [7, 3, 0]
    need = [-(-(a + T) // bs) for a in L]
    tables = make_tables(rng, need, sum(need) + 2, max(need))
    pos = np.array(L)[:, None] + np.arange(T)
    slots = np.take_along_axis(tables, pos // bs, 1) * bs + pos % bs
    slots[np.arange(T) >= np.array(n)[:, None]] = -1
    c = torch.from_numpy(angles(64, R)).to(DEV)
    wq, wk = (torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(TD[dt]).to(DEV) for _ in range(2))
    shape = (sum(need) + 2, Hkv, bs)
    per, kind = {"same": (1, TD[dt]), "e4m3": (1, torch.float8_e4m3fn), "i4": (2, torch.uint8)}[cdt]
    cache = [torch.zeros(*shape, D // per, device=DEV, dtype=torch.float32 if cdt != "i4" else kind).to(kind) for _ in range(4)]
    sc = [torch.full((*shape, D // 32), 100, dtype=torch.uint8, device=DEV) if cdt != "same" else None for _ in range(4)]
    out, ko = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    res = sv.qk_norm_rope(q, k, c, i32(pos), wq, wk, interleaved=pairs, out=out, key_out=ko, value=v, k_cache=cache[0],
                          v_cache=cache[1], slots=torch.from_numpy(slots).to(DEV), k_scale=sc[0], v_scale=sc[1],
                          status=status)
    assert res[0] is out and res[1] is ko and status.item() == 0
    w_out, w_ko = sv.qk_norm_rope(q, k, c, i32(pos), wq, wk, interleaved=pairs)
    live = torch.from_numpy(slots >= 0).to(DEV)
    for g, w in ((out, w_out), (ko, w_ko)):
        assert torch.equal(g[live].nan_to_num(7), w[live].nan_to_num(7)) and (g[~live] == 3).all()
    sv.kv_write(w_ko, v, cache[2], cache[3], i32(tables), i32(L), i32(n), k_scale=sc[2], v_scale=sc[3])
    for a, b in ((0, 2), (1, 3)):
        assert torch.equal(cache[a].view(torch.uint8), cache[b].view(torch.uint8))
        assert cdt == "same" or torch.equal(sc[a], sc[b])
    none = sv.qk_norm_rope(q, k, c, i32(pos), wq, wk, interleaved=pairs, value=v, k_cache=cache[0], v_cache=cache[1],
                           slots=torch.from_numpy(slots).to(DEV), k_scale=sc[0], v_scale=sc[1])
    assert none[1] is None


@gpu
def test_bad_positions_and_slots():
    sv, _, _ = _pkg()
    rng = np.random.default_rng(1)
    q, k, v = projection(rng, 1, 6, 4, 2, 64, "bf16")
    c = torch.from_numpy(angles(10, 64)).to(DEV)
    cache = [torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    slots = torch.tensor([[0, 1, 2, 16, -5, 1 << 40]], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 3.0)
    sv.qk_norm_rope(q, k, c, i32([[0, -1, 10, 1, -9, 1]]), out=out, value=v, k_cache=cache[0], v_cache=cache[1],
                    slots=slots, status=status)
    assert status.item() == ref.LENGTH | ref.BLOCK
    assert (out[0, 1:] == 3).all() and (out[0, 0] == q[0, 0]).all()          # position 0 does not turn
    assert (cache[0][:, :, 1:] == 0).all() and (cache[0][0, :, 0] == k[0, 0]).all() and (cache[0][1] == 0).all()
    # An infinity that does not turn stays alone.
    q[0, 0, 0, 63] = float("inf")
    o, _ = sv.qk_norm_rope(q, k, c[:, :32].contiguous(), i32([[0] * 6]))
    assert o[0, 0, 0, :63].isfinite().all() and o[0, 0, 0, 63] == float("inf")


@gpu
def test_rope_refusals():
    sv, _, kv = _pkg()
    rng = np.random.default_rng(2)
    q, k, v = (x.contiguous() for x in projection(rng, 2, 3, 4, 2, 64, "bf16"))
    c, pos = torch.from_numpy(angles(10, 64)).to(DEV), i32(np.zeros((2, 3)))
    cache = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    other = torch.zeros_like(cache)
    slots = torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    f = sv.qk_norm_rope
    for call in (lambda: f(q.float(), k, c, pos), lambda: f(q, k.half(), c, pos), lambda: f(q, k[:1], c, pos),
                 lambda: f(q, k[..., :32], c, pos), lambda: f(q, k, c.half(), pos), lambda: f(q, k, c[:, ::2], pos),
                 lambda: f(q, k, c, pos.long()), lambda: f(q, k, c, pos[:1]), lambda: f(q, k, c, pos, w[:32]),
                 lambda: f(q, k, c, pos, w.float()), lambda: f(q, k, c, pos, eps=-1.0), lambda: f(q, k, c, pos, eps="x"),
                 lambda: f(q, k, c[:, :40].contiguous(), pos), lambda: f(q, k, c, pos, out=q[:, :1].expand_as(q)),
                 lambda: f(q, k, c, pos, out=k), lambda: f(q, k, c, pos, value=v), lambda: f(q, k, c, pos, slots=slots),
                 lambda: f(q, k, c, pos, k_cache=cache), lambda: f(q, k, c, pos, k_cache=cache, v_cache=other, slots=slots),
                 lambda: f(q, k, c, pos, value=v, k_cache=cache, v_cache=other),
                 lambda: f(q, k, c, pos, value=v, k_cache=cache, v_cache=cache, slots=slots),
                 lambda: f(q, k, c, pos, value=v, k_cache=cache, v_cache=other, slots=slots.int()),
                 lambda: f(q, k, c, pos, value=v, k_cache=cache.half(), v_cache=other.half(), slots=slots),
                 lambda: f(q, k, c, pos, value=v, k_cache=cache[:, :1], v_cache=other[:, :1], slots=slots)):
        with pytest.raises((TypeError, ValueError, kv.SpecVerifyError)):
            call()
    assert (cache == 0).all()
    empty = f(q[:0], k[:0], c, pos[:0])
    assert empty[0].shape == (0, 3, 4, 64) and empty[1].shape == (0, 3, 2, 64)


# ----------------------------------------------------------- a whole step ----

@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_two_steps_with_trees(D):
    """reserve, norm and rotation into a cache of 4 bits, attention, verify, compact, rollback, twice; the cache, the
    tables and the free list afterwards are those of the tokens kept, written one by one."""
    sv, _, kv = _pkg()
    rng = np.random.default_rng(D)
    B, T, Hq, Hkv, bs, V, P = 3, 6, 8, 2, 16, 50, 128
    tables, seq = torch.full((B, 6), -1, dtype=torch.int32, device=DEV), i32([0, 0, 0])
    pool = 14
    free, count = i32(rng.permutation(pool)), i32([pool])
    k_cache, v_cache = (torch.zeros(pool, Hkv, bs, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2))
    k_scale, v_scale = (torch.zeros(pool, Hkv, bs, D // 32, dtype=torch.uint8, device=DEV) for _ in range(2))
    kw = dict(k_scale=k_scale, v_scale=v_scale)
    cos_sin = torch.from_numpy(angles(P, D)).to(DEV)
    wq, wk = (torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).bfloat16().to(DEV) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def forward(n, mask, T):
        q, k, v = projection(rng, B, T, Hq, Hkv, D, "bf16")
        slots, pos, new = sv.kv_reserve(seq, i32(n), tables, bs, free, count, mask, max_new=T, status=status)
        q, ko = sv.qk_norm_rope(q, k, cos_sin, pos, wq, wk, key_out=k.clone(), value=v, k_cache=k_cache, v_cache=v_cache,
                                slots=slots, status=status, **kw)
        out = sv.tree_attention(q, k_cache, v_cache, tables, seq, mask, new, status=status, **kw)
        return q, ko, v, out, pos, new

    kept = [[] for _ in range(B)]                      # (rotated key, value) of each committed token
    q, k, v, _, _, new = forward([20, 33, 7], None, 33)    # prompts
    for b, m in enumerate(new.tolist()):
        kept[b] += [(k[b, i].clone(), v[b, i].clone()) for i in range(m)]
    seq += new
    path = [0, 1, 3, 4]                                # a branch of the tree below; 2 and 5 are others
    tree = np.eye(T, dtype=bool)
    for i, up in ((1, 0), (2, 0), (3, 1), (4, 3), (5, 2)):
        tree[i] |= tree[up]
    mask = torch.from_numpy(tree).to(DEV)
    for step in range(2):
        L = seq.tolist()
        q, k, v, out, pos, new = forward([T] * B, mask, T)
        assert status.item() == 0 and new.tolist() == [T] * B
        assert pos.tolist() == [[x + d for d in (0, 1, 1, 2, 3, 2)] for x in L]
        cache = sref.Cache(k_cache, v_cache, tables, k_scale, v_scale)
        w, _, tol, _, _, _ = ref.attention(ref.to64(q), cache, L, [T] * B, np.broadcast_to(tree, (B, T, T)), D ** -0.5,
                                           UNIT["bf16"])
        assert (np.abs(ref.to64(out) - w) <= tol).all()
        # The target accepts `step` drafts of the path in request 0, all in 1, none in 2.
        want = [1 + step, 3, 0]
        logits = torch.full((B, 4, V), -30.0, device=DEV)
        drafts = i32(rng.integers(0, V, (B, 3)))
        for b in range(B):
            for i in range(4):
                hit = i < want[b]
                logits[b, i, int(drafts[b, i]) if hit else (int(drafts[b, min(i, 2)]) + 1) % V] = 30.0
        half = torch.full((B, 3), 0.5, device=DEV)
        _, acc = sv.verify(logits, drafts, None, half, half[:, 0].contiguous(), torch.zeros(B, device=DEV))
        assert acc.tolist() == want
        keep = acc + 1
        sv.kv_compact(i32([path] * B), keep, seq, tables, k_cache, v_cache, status=status, **kw)
        sv.kv_rollback(keep, seq, tables, bs, free, count, new, gamma_max=T, status=status)
        for b in range(B):
            kept[b] += [(k[b, i].clone(), v[b, i].clone()) for i in path[:want[b] + 1]]
        assert seq.tolist() == [len(x) for x in kept] and status.item() == 0
        # Every block is in a table or free, once.
        held = [x for row in tables.tolist() for x in row if x >= 0]
        assert sorted(held + free[:count.item()].tolist()) == list(range(pool))
        assert len(held) == sum(-(-len(x) // bs) for x in kept)
    n = max(seq.tolist())
    got = sv.kv_read(k_cache, v_cache, tables, seq, max_len=n, dtype=torch.float32, **kw)
    for b in range(B):
        for side in range(2):
            x = np.stack([ref.to64(t[side]) for t in kept[b]])
            assert np.array_equal(ref.to64(got[side][b, :len(x)]), sref.values(*sref.quantise(x)))


@gpu
def test_step_in_a_graph_and_on_a_stream():
    sv, _, _ = _pkg()
    rng = np.random.default_rng(3)
    B, T, D, bs = 4, 5, 64, 16
    seq, n = i32([3, 20, 40, 0]), i32([5, 2, 5, 4])
    tab0 = i32(make_tables(rng, [1, 2, 3, 0], 6, 4))
    free, cnt0 = i32([20, 21, 22, 23, 24]), i32([5])
    tab, cnt = tab0.clone(), cnt0.clone()
    q, k, v = projection(rng, B, T, 4, 2, D, "fp16")
    c = torch.from_numpy(angles(64, D)).to(DEV)
    cache = [torch.zeros(25, 2, bs, D, dtype=torch.float16, device=DEV) for _ in range(2)]
    slots, pos = torch.zeros(B, T, dtype=torch.int64, device=DEV), torch.zeros(B, T, dtype=torch.int32, device=DEV)
    res, out = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros_like(q)

    def step(stream=None):
        sv.kv_reserve(seq, n, tab, bs, free, cnt, slots=slots, positions=pos, reserved=res, stream=stream)
        sv.qk_norm_rope(q, k, c, pos, out=out, value=v, k_cache=cache[0], v_cache=cache[1], slots=slots, stream=stream)

    step()
    want = [x.clone() for x in (tab, cnt, slots, pos, res, out, *cache)]
    side = torch.cuda.Stream()

    def again(how):
        for x, y in ((tab, tab0), (cnt, cnt0)):
            x.copy_(y)
        for x in (slots, pos, res, out, *cache):
            x.zero_()
        torch.cuda.synchronize()
        how()
        torch.cuda.synchronize()
        for x, w in zip((tab, cnt, slots, pos, res, out, *cache), want):
            assert torch.equal(x, w)

    again(lambda: step(side))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    again(g.replay)

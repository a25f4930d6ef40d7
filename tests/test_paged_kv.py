"""Writing to the paged cache, reading it back, moving an accepted path, and
what the operators refuse (the attention's own tests: test_tree_attention.py).
"""

import struct

import numpy as np
import pytest
import torch

import paged_ref as ref

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------- reference ----

def test_reference_e4m3_rounding_agrees_with_torch():
    x = torch.linspace(-448, 448, 20001, dtype=torch.float64)
    x = torch.cat([x, torch.tensor([0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 447.9])])
    want = x.float().to(F8).view(torch.uint8).numpy()
    assert np.array_equal(ref.round_e4m3(x.float().double().numpy()), want)
    assert np.array_equal(ref.E4M3[:127], torch.arange(127, dtype=torch.uint8).view(F8).double().numpy())


def test_reference_quantise_by_hand():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 2] = 448.0, -1.0, np.inf
    x[0, 32], x[0, 33] = 449.0, 448 * 2.0
    codes, scale = ref.quantise(x)
    assert scale.tolist() == [[127, 128]]
    assert ref.E4M3[codes[0, 0]] == 448 and ref.E4M3[codes[0, 1]] == -1 and codes[0, 2] == 0x7F
    assert ref.E4M3[codes[0, 32]] == 224 and ref.E4M3[codes[0, 33]] == 448
    assert ref.quantise(np.zeros((1, 32)))[1].tolist() == [[7]]


# -------------------------------------------------------------- refusals ----

def _pkg():
    import speculative_decoding_verification_75_gb300 as sv
    from speculative_decoding_verification_75_gb300 import api, kv
    return sv, api, kv


# The argument structs of include/sv_paged.h: struct_bytes, the cache, the rest.
WRITE = READ = struct.Struct("@31q")
COMPACT = struct.Struct("@23q")
ATTN = struct.Struct("@27qd7q")
PTR = 0x10000  # never dereferenced: the call returns before any launch


def _cache_words(**over):
    f = dict(k=PTR, v=PTR, ks=0, vs=0, layer=0, block=2048, slayer=0, sblock=0, layers=1,
             blocks=8, heads=2, bs=16, D=64, dtype=1, tables=PTR, max_blocks=4)
    f.update(over)
    return list(f.values())


def _write(lib, kv, cache=None, **over):
    f = dict(seq=PTR, new=0, key=PTR, value=PTR, kb=512, kt=128, kh=64, vb=512, vt=128, vh=64,
             B=2, T=4, dtype=1, status=0)
    f.update(over)
    return lib.sv_kv_write(WRITE.pack(WRITE.size, *(cache or _cache_words()), *f.values()), None)


def _read(lib, kv, cache=None, **over):
    f = dict(starts=0, lens=PTR, key=PTR, value=PTR, kb=512, kt=128, kh=64, vb=512, vt=128, vh=64,
             B=2, T=4, dtype=1, status=0)
    f.update(over)
    return lib.sv_kv_read(READ.pack(READ.size, *(cache or _cache_words()), *f.values()), None)


def _compact(lib, kv, cache=None, **over):
    f = dict(path=PTR, nacc=PTR, seq=PTR, B=2, P=4, status=0)
    f.update(over)
    return lib.sv_kv_compact(COMPACT.pack(COMPACT.size, *(cache or _cache_words()), *f.values()), None)


def _attn(lib, kv, cache=None, **over):
    f = dict(seq=PTR, new=0, q=PTR, qb=1024, qt=256, qh=64, mask=0, msb=0, out=PTR, lse=0,
             scale=0.125, B=2, T=4, H=4, dtype=1, ws=PTR, wsb=1 << 30, status=0)
    f.update(over)
    return lib.sv_tree_attention(ATTN.pack(ATTN.size, *(cache or _cache_words()), *f.values()), None)


CALLS = {"write": _write, "read": _read, "compact": _compact, "attn": _attn}


@pytest.mark.parametrize("op", sorted(CALLS))
@pytest.mark.parametrize("over", [
    dict(k=PTR + 8), dict(v=PTR + 4), dict(k=0), dict(v=0), dict(tables=0), dict(tables=PTR + 2),
    dict(block=2047), dict(block=2044), dict(block=-2048), dict(blocks=-1), dict(blocks=1 << 31),
    dict(heads=0), dict(bs=0), dict(D=0), dict(D=12), dict(D=264), dict(layers=0),
    dict(max_blocks=-1), dict(max_blocks=1 << 28), dict(heads=65536, bs=1024),
    dict(dtype=3), dict(dtype=3, ks=PTR, vs=PTR + 1, sblock=64),
    dict(dtype=3, ks=PTR, vs=PTR, sblock=63), dict(dtype=3, ks=PTR, vs=PTR, sblock=64, D=40),
    dict(layers=2, layer=2048 - 8)], ids=str)
def test_a_bad_cache_is_refused(op, over):
    _, api, kv = _pkg()
    lib = api.load_library()
    if "layers" in over and over["layers"] > 1 and op != "compact":
        over = dict(layers=2, layer=1 << 20)     # one layer only
    assert CALLS[op](lib, kv, _cache_words(**over)) == api.SV_ERR_INVALID_ARG


@pytest.mark.parametrize("op", sorted(CALLS))
def test_bad_arguments_are_refused(op):
    _, api, kv = _pkg()
    lib = api.load_library()
    call = CALLS[op]
    bad = api.SV_ERR_INVALID_ARG
    assert call(lib, kv, _cache_words(dtype=0)) == api.SV_ERR_UNSUPPORTED_DTYPE
    assert call(lib, kv, _cache_words(dtype=7)) == api.SV_ERR_UNSUPPORTED_DTYPE
    assert call(lib, kv, B=-1) == bad
    assert call(lib, kv, B=0) == api.SV_OK                       # nothing to do, nothing launched
    if op != "compact":
        assert call(lib, kv, T=-1) == bad
        assert call(lib, kv, T=0) == api.SV_OK
        assert call(lib, kv, B=1 << 20, T=1 << 20) == bad
        assert call(lib, kv, dtype=3) == api.SV_ERR_UNSUPPORTED_DTYPE
        assert call(lib, kv, dtype=9) == api.SV_ERR_UNSUPPORTED_DTYPE
    if op in ("write", "read"):
        for f in ("key", "value"):
            assert call(lib, kv, **{f: 0}) == bad
            assert call(lib, kv, **{f: PTR + 1}) == bad
        for f in ("kb", "kt", "kh", "vb", "vt", "vh"):
            assert call(lib, kv, **{f: -8}) == bad
    if op == "write":
        assert call(lib, kv, seq=0) == bad
        assert call(lib, kv, dtype=2) == api.SV_ERR_UNSUPPORTED_DTYPE   # fp16 into bf16
        assert call(lib, kv, dtype=0) == api.SV_ERR_UNSUPPORTED_DTYPE
    if op == "read":
        assert call(lib, kv, lens=0) == bad
    if op == "compact":
        assert call(lib, kv, P=-1) == bad
        for f in ("path", "nacc", "seq"):
            assert call(lib, kv, **{f: 0}) == bad
    if op == "attn":
        for f in ("seq", "q", "out", "ws"):
            assert call(lib, kv, **{f: 0}) == bad
        assert call(lib, kv, q=PTR + 1) == bad
        assert call(lib, kv, out=PTR + 8) == bad
        assert call(lib, kv, lse=PTR + 2) == bad
        assert call(lib, kv, ws=PTR + 16) == bad
        assert call(lib, kv, msb=-1) == bad
        assert call(lib, kv, H=3) == bad                         # not a multiple of 2
        assert call(lib, kv, H=0) == bad
        assert call(lib, kv, qh=-64) == bad
        assert call(lib, kv, scale=float("nan")) == bad
        assert call(lib, kv, scale=float("inf")) == bad
        assert call(lib, kv, scale=1e39) == bad
        assert call(lib, kv, wsb=0) == api.SV_ERR_WORKSPACE_TOO_SMALL
        assert call(lib, kv, dtype=2) == api.SV_ERR_UNSUPPORTED_DTYPE   # fp16 over bf16
    fn = {"write": lib.sv_kv_write, "read": lib.sv_kv_read, "compact": lib.sv_kv_compact,
          "attn": lib.sv_tree_attention}[op]
    assert fn(None, None) == bad
    assert fn((99).to_bytes(8, "little") + bytes(400), None) == bad     # another struct


def test_workspace_bytes_of_attention():
    _, api, kv = _pkg()
    n = kv.tree_attention_workspace_bytes
    assert n(8, 6, 64, 8, 128) > 0 and n(8, 6, 64, 8, 128) % 256 == 0
    assert n(8, 6, 64, 7, 128) == 0 and n(-1, 6, 64, 8, 128) == 0 and n(8, 6, 64, 8, 12) == 0


def test_cpu_tensors_are_refused():
    sv, _, _ = _pkg()
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    x = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: sv.kv_write(x, x, c, c, t, n), lambda: sv.kv_read(c, c, t, n, max_len=3),
                 lambda: sv.kv_compact(t, n, n, t, c, c), lambda: sv.tree_attention(x, c, c, t, n)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        sv.kv_write(3, x, c, c, t, n)


# ------------------------------------------------------------------- GPU ----

gpu = pytest.mark.gpu
DEV = "cuda:0"


def make_tables(rng, need, pool, width):
    t = np.full((len(need), width), -1, dtype=np.int32)
    ids = rng.permutation(pool)
    k = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[k:k + n]
        k += n
    return t


def make_cache(rng, pool, H, bs, D, dtype, layers=None, halves=False):
    """k, v, k_scale, v_scale on the GPU with N(0, 1) content."""
    lead = (layers,) if layers else ()
    shape = (*lead, pool, H, bs, D)
    if halves:   # k and v as the two halves of one buffer's blocks
        buf = torch.from_numpy(rng.standard_normal((*lead, pool, 2, H, bs, D)).astype(np.float32))
        buf = (buf.to(dtype) if dtype != F8 else buf.mul(100).clamp(-448, 448).to(F8)).to(DEV)
        k, v = (buf.view(torch.uint8)[..., i, :, :, :].view(F8) if dtype == F8 else buf[..., i, :, :, :]
                for i in range(2))
    else:
        k, v = (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) for _ in range(2))
        if dtype == F8:
            k, v = (x.mul(100).clamp(-448, 448).to(F8) for x in (k, v))
        k, v = k.to(dtype).to(DEV), v.to(dtype).to(DEV)
    if dtype != F8:
        return k, v, None, None
    s = [torch.from_numpy(rng.integers(118, 123, (*shape[:-1], D // 32)).astype(np.uint8)).to(DEV)
         for _ in range(2)]
    return k, v, s[0], s[1]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bits(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype != torch.uint8 else t.cpu().numpy()


WRITE_CASES = [
    # B, T, H, D, bs, L, n, dtype, cache dtype, layout
    (1, 1, 2, 64, 16, [0], None, "bf16", "bf16", "dense"),
    (1, 1, 2, 64, 16, [500], None, "bf16", "e4m3", "dense"),
    (3, 6, 8, 128, 16, [0, 13, 255], [6, 0, 5], "bf16", "bf16", "fused"),
    (3, 6, 8, 128, 16, [1, 15, 100], [6, 3, 1], "bf16", "e4m3", "fused"),
    (2, 33, 7, 32, 5, [3, 4], [33, 17], "fp16", "e4m3", "odd"),
    (2, 33, 7, 40, 1, [3, 0], [33, 17], "fp16", "fp16", "odd"),
    (4, 9, 1, 256, 24, [0, 23, 24, 47], [9, 9, 8, 1], "bf16", "e4m3", "heads"),
    (2, 700, 32, 96, 48, [0, 31], [700, 655], "bf16", "e4m3", "dense"),
    (5, 17, 32, 8, 128, [0, 1, 127, 128, 129], None, "bf16", "bf16", "halves"),
    (5, 17, 3, 64, 128, [0, 1, 127, 128, 129], None, "fp16", "e4m3", "halves"),
]
TD = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": F8, "fp32": torch.float32}


def dense_pair(rng, shape, dtype, layout, spread=True):
    """key, value with an awkward layout and a wide range of magnitudes."""
    B, T, H, D = shape
    x = rng.standard_normal((2, *shape))
    if spread:
        x *= 2.0 ** rng.integers(-12, 8, (2, B, T, H, 1))
        x[rng.random(x.shape) < 0.02] = 0
    x = torch.from_numpy(x).to(dtype)
    if layout == "fused":        # side by side behind a query of the same width
        buf = torch.zeros(B, T, 3, H, D, dtype=dtype, device=DEV)
        buf[:, :, 1], buf[:, :, 2] = x[0].to(DEV), x[1].to(DEV)
        return buf[:, :, 1], buf[:, :, 2]
    if layout == "odd":          # rows that start on odd elements
        buf = torch.zeros(2, B, T, H, D + 1, dtype=dtype, device=DEV)
        buf[..., 1:] = x.to(DEV)
        return buf[0][..., 1:], buf[1][..., 1:]
    if layout == "heads":        # [B, H, T, D] storage
        y = x.transpose(2, 3).contiguous().to(DEV)
        return y[0].transpose(1, 2), y[1].transpose(1, 2)
    y = x.to(DEV)
    return y[0], y[1]


@gpu
@pytest.mark.parametrize("case", WRITE_CASES, ids=str)
def test_write(case):
    B, T, H, D, bs, L, n, dt, cdt, layout = case
    sv, _, _ = _pkg()
    rng = np.random.default_rng(hash(case[:5]) % 1000)
    n = [T] * B if n is None else n
    need = [-(-(l + m) // bs) for l, m in zip(L, n)]
    pool, width = sum(need) + 2, max(need) + 1
    tables = make_tables(rng, need, pool, width)
    k, v, ks, vs = make_cache(rng, pool, H, bs, D, TD[cdt], halves=layout == "halves")
    key, value = dense_pair(rng, (B, T, H, D), TD[dt], layout)
    want = [bits(x).copy() for x in (k, v, ks, vs) if x is not None]
    for x, c, s in ((key, 0, 2), (value, 1, 3)):
        x = ref.to64(x)
        for b in range(B):
            for i in range(n[b]):
                blk, row = tables[b, (L[b] + i) // bs], (L[b] + i) % bs
                if ks is not None:
                    want[c][blk, :, row], want[s][blk, :, row] = ref.quantise(x[b, i])
                else:
                    raw = torch.from_numpy(x[b, i]).to(TD[dt]).view(torch.uint8).numpy()
                    want[c][blk, :, row] = raw.reshape(H, -1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.kv_write(key, value, k, v, i32(tables), i32(L), None if n == [T] * B else i32(n),
                k_scale=ks, v_scale=vs, status=status)
    got = [bits(x) for x in (k, v, ks, vs) if x is not None]
    assert status.item() == 0
    for g, w in zip(got, want):      # every byte, the untouched rows among them
        assert np.array_equal(g, w)


@gpu
def test_write_what_is_not_finite_and_what_is_tiny():
    sv, _, _ = _pkg()
    x = np.zeros((1, 5, 1, 64))
    x[0, 0, 0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    x[0, 1, 0, :] = np.nan
    x[0, 2, 0, :3] = [2.0 ** -130, -(2.0 ** -126), 2.0 ** -133]       # bf16 subnormals
    x[0, 3, 0, :4] = [3.3e38, -3.3e38, 1e38, 1.0]
    x[0, 4, 0, :3] = [448.0, 450.0, -0.0]
    key = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    k, v, ks, vs = make_cache(np.random.default_rng(0), 1, 1, 8, 64, F8)
    sv.kv_write(key, key, k, v, i32([[0]]), i32([0]), k_scale=ks, v_scale=vs)
    codes, scale = ref.quantise(ref.to64(key)[0, :, 0])
    assert np.array_equal(bits(ks)[0, 0, :5], scale)
    got, want = ref.E4M3[bits(k)[0, 0, :5]], ref.E4M3[codes]
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(bits(k), bits(v)) or np.array_equal(bits(k)[0, 0, :5], bits(v)[0, 0, :5])


@gpu
def test_write_reports_bad_data_and_leaves_the_rest():
    sv, api, kv = _pkg()
    rng = np.random.default_rng(3)
    B, T, H, D, bs = 7, 4, 2, 64, 4
    k, v, _, _ = make_cache(rng, 12, H, bs, D, torch.bfloat16)
    before = bits(k).copy()
    key, value = dense_pair(rng, (B, T, H, D), torch.bfloat16, "dense")
    tables = np.array([[0, 1], [2, -1], [3, 12], [4, -5], [5, 6], [7, 8], [9, 10]])
    L = [0, 2, 2, 2, 6, -1, 2]
    n = [4, 4, 4, 4, 4, 4, 5]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.kv_write(key, value, k, v, i32(tables), i32(L), i32(n), status=status)
    assert status.item() == (api.SV_KV_MISSING_BLOCK | kv.SV_KV_BAD_BLOCK | api.SV_KV_TABLE_SHORT
                             | api.SV_KV_BAD_LENGTH)
    want = before.copy()
    raw = bits(key)
    want[0] = raw[0].transpose(1, 0, 2)
    for b, blk in ((1, 2), (2, 3), (3, 4)):      # the second half has no block
        want[blk, :, 2:] = raw[b, :2].transpose(1, 0, 2)
    want[6, :, 2:] = raw[4, :2].transpose(1, 0, 2)  # positions 8, 9 are behind the table
    assert np.array_equal(bits(k), want)


READ_CASES = [
    # B, T, H, D, bs, starts, lens, cache dtype, out dtype, layout
    (1, 1, 2, 64, 16, None, [1], "bf16", "bf16", "dense"),
    (3, 40, 8, 128, 16, [0, 5, 100], [40, 0, 33], "bf16", "bf16", "dense"),
    (3, 40, 8, 128, 16, [0, 5, 100], [40, 1, 33], "e4m3", "bf16", "dense"),
    (2, 33, 7, 32, 5, None, [33, 17], "e4m3", "fp16", "odd"),
    (2, 33, 3, 40, 7, [1, 2], [33, 17], "fp16", "fp32", "odd"),
    (2, 300, 1, 256, 24, None, [300, 299], "e4m3", "fp32", "heads"),
    (2, 9, 32, 96, 128, [120, 0], [9, 9], "bf16", "fp16", "fused"),
    (4, 17, 5, 64, 1, None, [17, 16, 0, 3], "bf16", "bf16", "halves"),
]


@gpu
@pytest.mark.parametrize("case", READ_CASES, ids=str)
def test_read(case):
    B, T, H, D, bs, starts, lens, cdt, odt, layout = case
    sv, _, _ = _pkg()
    rng = np.random.default_rng(hash(case[:5]) % 1000)
    st = [0] * B if starts is None else starts
    need = [-(-(a + m) // bs) for a, m in zip(st, lens)]
    pool, width = sum(need) + 2, max(need) + 1
    tables = make_tables(rng, need, pool, width)
    k, v, ks, vs = make_cache(rng, pool, H, bs, D, TD[cdt], halves=layout == "halves")
    out = dense_pair(rng, (B, T, H, D), TD[odt], layout)
    want = [ref.to64(x).copy() for x in out]
    cache = ref.Cache(k, v, torch.from_numpy(tables), ks, vs)
    for w, c in ((want[0], cache.k), (want[1], cache.v)):
        for b in range(B):
            for i in range(lens[b]):
                blk, row, _ = cache.place(b, st[b] + i)
                w[b, i] = torch.from_numpy(c[blk, :, row]).to(TD[odt]).double().numpy()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.kv_read(k, v, i32(tables), i32(lens), None if starts is None else i32(starts),
                     out=out, k_scale=ks, v_scale=vs, status=status)
    assert got[0] is out[0] and status.item() == 0
    for g, w in zip(got, want):
        assert np.array_equal(ref.to64(g), w)


@gpu
def test_read_allocates_zeroed_rows_and_reports_bad_data():
    sv, api, kv = _pkg()
    k, v, _, _ = make_cache(np.random.default_rng(5), 4, 2, 4, 64, torch.float16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, b = sv.kv_read(k, v, i32([[0, -1], [9, 1], [2, 3], [2, 3]]), i32([8, 8, 9, 3]), i32([0, 0, 0, 7]),
                      max_len=8, dtype=torch.float32, status=status)
    assert a.dtype == torch.float32 and a.shape == (4, 8, 2, 64)
    assert status.item() == (api.SV_KV_MISSING_BLOCK | kv.SV_KV_BAD_BLOCK | api.SV_KV_BAD_LENGTH
                             | api.SV_KV_TABLE_SHORT)
    assert torch.equal(a[0, :4], k[0].transpose(0, 1).float()) and not a[0, 4:].any()
    assert torch.equal(b[1, 4:], v[1].transpose(0, 1).float()) and not a[1, :4].any()
    assert not a[2].any()                                   # a length past T
    assert torch.equal(a[3, 0], k[3, :, 3].float()) and not a[3, 1:].any()


@gpu
@pytest.mark.parametrize("dt,cdt", [("bf16", "e4m3"), ("fp16", "e4m3"), ("bf16", "bf16")])
def test_write_then_read_loses_half_a_step_at_most(dt, cdt):
    """A dense cache gives back what went in; e4m3 is off by at most 2^-4 of
    the value or, among its subnormals, 2^(e - 10)."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(11)
    B, T, H, D, bs = 2, 50, 4, 128, 16
    key, value = dense_pair(rng, (B, T, H, D), TD[dt], "fused")
    k, v, ks, vs = make_cache(rng, 10, H, bs, D, TD[cdt])
    tables, L = i32(make_tables(rng, [5, 5], 10, 5)), i32([3, 17])
    sv.kv_write(key, value, k, v, tables, L, k_scale=ks, v_scale=vs)
    got = sv.kv_read(k, v, tables, i32([T, T]), L, max_len=T, dtype=torch.float32, k_scale=ks, v_scale=vs)
    for g, x in zip(got, (key, value)):
        if cdt != "e4m3":
            assert torch.equal(g, x.float())
            continue
        x, g = ref.to64(x), ref.to64(g)
        _, s = ref.quantise(x)
        step = np.repeat(2.0 ** (s.astype(float) - 127 - 10), 32, -1)
        assert (np.abs(g - x) <= np.maximum(2.0 ** -4 * np.abs(x), step)).all()


def compact_reference(arrays, tables, bs, path, k, L):
    out = [a.copy() for a in arrays]
    for b in range(len(k)):
        for i in range(max(k[b], 0)):
            s, d = L[b] + path[b][i], L[b] + i
            for o, a in zip(out, arrays):
                o[:, tables[b][d // bs], :, d % bs] = a[:, tables[b][s // bs], :, s % bs]
    return out


@gpu
@pytest.mark.parametrize("layers,B,H,D,bs,P,cdt", [
    (None, 1, 2, 64, 16, 1, "bf16"), (1, 3, 8, 128, 16, 6, "bf16"), (3, 4, 8, 128, 16, 9, "e4m3"),
    (2, 5, 1, 32, 5, 7, "e4m3"), (2, 2, 33, 256, 1, 20, "fp16"), (1, 2, 3, 8, 64, 150, "bf16"),
    # More layers than run at once: several to a thread block, one left over.
    (21, 40, 2, 32, 8, 5, "e4m3"), (71, 10, 1, 8, 4, 70, "bf16")])
def test_compact(layers, B, H, D, bs, P, cdt):
    sv, _, _ = _pkg()
    rng = np.random.default_rng(P)
    N = 2 * P + 3
    L = rng.integers(0, 3 * bs + 5, B)
    k = [int(rng.integers(-1, P + 1)) for _ in range(B)]
    k[0] = P
    path = np.stack([np.sort(rng.permutation(N)[:P]) for _ in range(B)])
    path[-1] = np.arange(P)                      # already in place
    if B > 2:
        path[1, :2] = [0, 1]                     # a prefix in place
    need = [-(-(int(l) + N) // bs) for l in L]
    pool = sum(need) + 1
    tables = make_tables(rng, need, pool, max(need))
    k_c, v_c, ks, vs = make_cache(rng, pool, H, bs, D, TD[cdt], layers=layers)
    all_ = [x for x in (k_c, v_c, ks, vs) if x is not None]
    flat = [bits(x).copy() if layers else bits(x).copy()[None] for x in all_]
    want = compact_reference(flat, tables, bs, path, k, L)
    full = np.where(np.arange(P) < np.array(k)[:, None], path, -9)   # what is behind k is not read
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.kv_compact(i32(full), i32(k), i32(L), i32(tables), k_c, v_c, k_scale=ks, v_scale=vs, status=status)
    assert status.item() == 0
    for g, w in zip(all_, want):
        assert np.array_equal(bits(g) if layers else bits(g)[None], w)


@gpu
def test_compact_leaves_bad_requests_unchanged():
    sv, api, kv = _pkg()
    rng = np.random.default_rng(2)
    k_c, v_c, _, _ = make_cache(rng, 16, 2, 4, 64, torch.bfloat16)
    before = bits(k_c).copy()
    tables = [[0, 1], [2, 3], [4, 5], [6, -1], [8, 16], [10, 11], [12, 13], [14, 15]]
    path = [[0, 2, 5], [0, 2, 2], [-1, 2, 3], [0, 2, 5], [0, 2, 5], [0, 2, 9], [0, 2, 5], [0, 2, 5]]
    nacc = [3, 3, 3, 3, 3, 3, 4, 3]
    L = [0, 0, 0, 0, 0, 0, 0, -1]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.kv_compact(i32(path), i32(nacc), i32(L), i32(tables), k_c, v_c, status=status)
    assert status.item() == (kv.SV_KV_BAD_PATH | api.SV_KV_MISSING_BLOCK | kv.SV_KV_BAD_BLOCK
                             | api.SV_KV_TABLE_SHORT | api.SV_KV_BAD_LENGTH)
    want = before.copy()
    want[0, :, 1], want[0, :, 2] = before[0, :, 2], before[1, :, 1]
    assert np.array_equal(bits(k_c), want)


@gpu
def test_python_refuses_what_does_not_belong_together():
    sv, _, _ = _pkg()
    rng = np.random.default_rng(0)
    bf = torch.bfloat16
    k, v, _, _ = make_cache(rng, 4, 2, 16, 64, bf)
    k8, v8, ks, vs = make_cache(rng, 4, 2, 16, 64, F8)
    x = torch.zeros(1, 3, 2, 64, dtype=bf, device=DEV)
    t, n = i32([[0, 1]]), i32([0])
    w = lambda *a, **kw: sv.kv_write(*a, **kw)  # noqa: E731
    for err, call in [
        (TypeError, lambda: w(x.half(), x.half(), k, v, t, n)),
        (TypeError, lambda: w(x, x.half(), k, v, t, n)),
        (TypeError, lambda: w(x.float(), x.float(), k, v, t, n)),
        (TypeError, lambda: w(x, x, k, v, t.long(), n)),
        (TypeError, lambda: w(x, x, k, v, t, n.long())),
        (TypeError, lambda: w(x, x, k.float(), v.float(), t, n)),
        (ValueError, lambda: w(x, x, k, v, t, i32([0, 0]))),
        (ValueError, lambda: w(x, x, k, v, i32([[0], [1]]), n)),
        (ValueError, lambda: w(x, x[:, :2], k, v, t, n)),
        (ValueError, lambda: w(x[..., :32], x[..., :32], k, v, t, n)),
        (ValueError, lambda: w(x, x, k, v[:3], t, n)),
        (ValueError, lambda: w(x, x, k, v.transpose(1, 2).contiguous().transpose(1, 2), t, n)),
        (ValueError, lambda: w(x, x, k8, v8, t, n)),
        (ValueError, lambda: w(x, x, k8, v8, t, n, k_scale=ks, v_scale=vs[..., :1])),
        (ValueError, lambda: w(x, x, k, v, t, n, k_scale=ks, v_scale=vs)),
        (ValueError, lambda: w(x, x, k, v, t.t().contiguous().t() if False else i32([[0, 9, 1]])[:, ::2], n)),
        (ValueError, lambda: w(x, x, k, v, t, n, status=i32([0, 0]))),
        (ValueError, lambda: w(x.transpose(-1, -2).contiguous().transpose(-1, -2), x, k, v, t, n)),
        (ValueError, lambda: w(x[0], x[0], k, v, t, n)),
        (ValueError, lambda: sv.kv_read(k, v, t, n)),
        (TypeError, lambda: sv.kv_read(k, v, t, n, out=(x.double(), x.double()))),
        (ValueError, lambda: sv.kv_read(k, v, t, n, out=(x[:, :1].expand(1, 3, 2, 64), x))),
        (ValueError, lambda: sv.kv_compact(n, n, n, t, k, v)),
        (ValueError, lambda: sv.tree_attention(x[:, :, :1], k, v, t, n)),
        (TypeError, lambda: sv.tree_attention(x.half(), k, v, t, n)),
        (TypeError, lambda: sv.tree_attention(x, k, v, t, n, torch.ones(3, 3, device=DEV))),
        (ValueError, lambda: sv.tree_attention(x, k, v, t, n, torch.ones(2, 2, device=DEV).bool())),
        (ValueError, lambda: sv.tree_attention(x, k, v, t, n, torch.ones(3, 3).bool())),
        (ValueError, lambda: sv.tree_attention(x, k, v, t, n, out=x.transpose(1, 2))),
        (TypeError, lambda: sv.tree_attention(x, k, v, t, n, out=x.half())),
        (TypeError, lambda: sv.tree_attention(x, k, v, t, n, lse=torch.zeros(1, 3, 2, device=DEV).half())),
        (sv.SpecVerifyError, lambda: sv.tree_attention(
            x, k, v, t, n, workspace=torch.zeros(0, dtype=torch.uint8, device=DEV))),
    ]:
        with pytest.raises(err):
            call()


@gpu
@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
def test_blocks_past_32_bit_offsets(cdt):
    """Blocks more than 2^31 elements apart: written, moved and read back."""
    sv, _, _ = _pkg()
    rng = np.random.default_rng(1)
    H, bs, D = 2, 16, 64
    esz = 1 if cdt == "e4m3" else 2
    stride = (1 << 31) + 16 * 64
    store = [torch.zeros((stride + H * bs * D) * esz, dtype=torch.uint8, device=DEV) for _ in range(2)]
    k, v = (s.view(TD[cdt]).as_strided((2, H, bs, D), (stride, bs * D, D, 1)) for s in store)
    ks = vs = None
    if cdt == "e4m3":
        ks, vs = (torch.zeros(2, H, bs, D // 32, dtype=torch.uint8, device=DEV) for _ in range(2))
    key, value = dense_pair(rng, (1, 20, H, D), torch.bfloat16, "dense")
    t = i32([[0, 1]])
    sv.kv_write(key, value, k, v, t, i32([5]), k_scale=ks, v_scale=vs)
    a = sv.kv_read(k, v, t, i32([20]), i32([5]), max_len=20, dtype=torch.float32, k_scale=ks, v_scale=vs)
    if cdt == "bf16":
        assert torch.equal(a[0], key.float()) and torch.equal(a[1], value.float())
    sv.kv_compact(i32([[0, 12, 19]]), i32([3]), i32([5]), t, k, v, k_scale=ks, v_scale=vs)
    c = sv.kv_read(k, v, t, i32([3]), i32([5]), max_len=3, dtype=torch.float32, k_scale=ks, v_scale=vs)
    for x, y in zip(a, c):
        assert torch.equal(y, x[:, [0, 12, 19]])


@gpu
def test_calls_on_another_stream_and_in_a_graph():
    sv, _, _ = _pkg()
    rng = np.random.default_rng(8)
    B, T, H, D, bs = 3, 6, 4, 64, 16
    k, v, _, _ = make_cache(rng, 9, H, bs, D, torch.bfloat16)
    tables, L = i32(make_tables(rng, [3, 3, 3], 9, 3)), i32([0, 9, 20])
    key, value = dense_pair(rng, (B, T, H, D), torch.bfloat16, "dense")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sv.kv_write(key, value, k, v, tables, L, stream=side)
    a, b = sv.kv_read(k, v, tables, i32([T] * B), L, max_len=T, stream=side)
    side.synchronize()
    assert torch.equal(a, key) and torch.equal(b, value)
    lens, out = i32([T] * B), (torch.zeros_like(key), torch.zeros_like(value))
    path, nacc = i32([[0, 3], [1, 2], [0, 5]]), i32([2, 2, 2])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sv.kv_write(key, value, k, v, tables, L)
        sv.kv_compact(path, nacc, L, tables, k, v)
        sv.kv_read(k, v, tables, lens, L, out=out)
    for seed in range(2):
        x, y = dense_pair(np.random.default_rng(seed), (B, T, H, D), torch.bfloat16, "dense")
        key.copy_(x)
        value.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for o, z in ((out[0], x), (out[1], y)):
            want = z.clone()
            for r, p in enumerate(path.tolist()):
                want[r, :2] = z[r, p]
            assert torch.equal(o, want)

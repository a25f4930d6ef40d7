"""Attention of drafted tokens over the paged cache against a 64-bit
restatement, at the sizes, masks and contents where it can go wrong."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from test_paged_kv import DEV, F8, TD, i32, make_cache, make_tables

pytestmark = pytest.mark.gpu
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def tree(rng, B, T, kind):
    """Visibility of new tokens: None (chain), a random tree, one shared by
    the batch, or anything at all with empty rows."""
    if kind == "chain":
        return None
    if kind == "any":
        m = rng.random((B, T, T)) < 0.3
        m[:, ::3] = False
        return m
    m = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for i in range(T):
            if i:
                m[b, i] = m[b, rng.integers(0, i)]
            m[b, i, i] = True
    if kind == "shared":
        m[:] = m[:1]
    return m


def build(rng, B, T, Hq, Hkv, D, bs, L, n, kind, dt, cdt, halves=False, spare=0):
    n = [T] * B if n is None else n
    need = [-(-(l + m) // bs) for l, m in zip(L, n)]
    pool, width = sum(need) + 2, max(need) + 1 + spare
    tables = make_tables(rng, need, pool, width)
    k, v, ks, vs = make_cache(rng, pool, Hkv, bs, D, TD[cdt], halves=halves)
    q = torch.from_numpy(2 * rng.standard_normal((B, T, Hq, D))).to(TD[dt]).to(DEV)
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, tables=tables, L=L, n=n, mask=tree(rng, B, T, kind),
                kind=kind, dt=dt)


def operands(s):
    """The call's small operands on the GPU: tables, L, mask, n."""
    B, T = s["q"].shape[:2]
    mask = s["mask"]
    if mask is not None:
        mask = torch.from_numpy(mask[0] if s["kind"] == "shared" else mask).to(DEV)
    return i32(s["tables"]), i32(s["L"]), mask, None if s["n"] == [T] * B else i32(s["n"])


def call(s, ops=None, **kw):
    import speculative_decoding_verification_75_gb300 as sv
    return sv.tree_attention(s["q"], s["k"], s["v"], *(ops or operands(s)),
                             k_scale=s["ks"], v_scale=s["vs"], **kw)


def check(s, scale=None, want_status=0, **kw):
    B, T, Hq, D = s["q"].shape
    out = torch.full_like(s["q"], -7.0).contiguous()
    lse = torch.full((B, T, Hq), -7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = call(s, out=out, lse=lse, status=status, scale=scale, **kw)
    assert got is out
    assert status.item() == want_status
    cache = ref.Cache(s["k"], s["v"], torch.from_numpy(s["tables"]), s["ks"], s["vs"])
    o, l, tol, ltol, live, st = ref.attention(ref.to64(s["q"]), cache, s["L"], s["n"], s["mask"],
                                              D ** -0.5 if scale is None else scale, UNIT[s["dt"]])
    assert st == want_status
    out, lse = ref.to64(out), ref.to64(lse)
    assert (out[~live] == -7).all() and (lse[~live] == -7).all()     # rows behind a request's last
    out, o, tol = out[live], o[live], tol[live]
    assert np.array_equal(np.isnan(out), np.isnan(o))
    fine = np.isfinite(o)
    with np.errstate(invalid="ignore"):
        assert (np.abs(out[fine] - o[fine]) <= tol[fine]).all(), (
            np.abs(out[fine] - o[fine]) / np.maximum(tol[fine], 1e-30)).max()
    lse, l, ltol = lse[live], l[live], ltol[live]
    assert np.array_equal(lse == -np.inf, l == -np.inf) and np.array_equal(np.isnan(lse), np.isnan(l))
    f = np.isfinite(l)
    assert (np.abs(lse[f] - l[f]) <= ltol[f]).all()
    return out


CASES = [
    # B, T, Hq, Hkv, D, bs, L, n, mask, dtype, cache dtype
    (1, 1, 1, 1, 64, 16, [0], None, "chain", "bf16", "bf16"),            # sees itself alone
    (1, 1, 14, 2, 64, 16, [500], None, "chain", "bf16", "bf16"),
    (2, 1, 64, 8, 128, 16, [127, 128], None, "chain", "bf16", "e4m3"),
    (3, 6, 64, 8, 128, 16, [0, 129, 777], [6, 6, 3], "chain", "bf16", "bf16"),
    (3, 6, 64, 8, 128, 32, [5, 129, 777], [1, 6, 3], "tree", "bf16", "e4m3"),
    (4, 9, 8, 8, 128, 16, [1, 100, 250, 0], [9, 0, 2, 9], "shared", "fp16", "fp16"),
    (2, 33, 7, 1, 64, 48, [95, 31], [33, 30], "tree", "fp16", "fp16"),   # 231 rows of one head
    (2, 64, 32, 8, 128, 64, [300, 64], [64, 50], "tree", "bf16", "bf16"),  # 256 rows
    (1, 65, 8, 2, 128, 128, [200], None, "tree", "bf16", "e4m3"),        # 260 rows
    (1, 130, 4, 2, 64, 8, [120], None, "any", "bf16", "bf16"),
    (2, 200, 4, 2, 128, 16, [0, 70], [200, 137], "chain", "bf16", "bf16"),  # prompts
    (3, 5, 16, 2, 64, 24, [0, 0, 50], [5, 4, 5], "any", "bf16", "e4m3"),
    (2, 5, 6, 3, 80, 16, [10, 40], None, "tree", "bf16", "bf16"),        # other head dimensions
    (2, 5, 6, 3, 256, 16, [10, 40], None, "tree", "bf16", "e4m3"),
    (2, 5, 6, 3, 8, 16, [10, 40], None, "chain", "fp16", "fp16"),
    (2, 5, 8, 2, 128, 5, [10, 43], None, "tree", "bf16", "bf16"),        # other block sizes
    (2, 5, 8, 2, 64, 1, [10, 43], [5, 1], "tree", "fp16", "fp16"),
    (2, 5, 8, 2, 128, 12, [10, 43], None, "any", "fp16", "e4m3"),
    (1, 2, 8, 1, 128, 256, [700], None, "chain", "fp16", "fp16"),
    (1, 3, 8, 1, 64, 160, [700], None, "chain", "bf16", "e4m3"),
    (40, 2, 2, 1, 64, 8, list(range(40)), None, "chain", "bf16", "bf16"),
    (3, 6, 64, 8, 128, 16, [5, 129, 777], [1, 6, 3], "tree", "fp16", "e4m3"),
    (1, 65, 8, 2, 64, 32, [200], None, "chain", "fp16", "e4m3"),
    (2, 513, 4, 2, 64, 32, [0, 300], [513, 400], "chain", "fp16", "e4m3"),   # long prompts
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(case):
    rng = np.random.default_rng(sum(case[:6]))
    check(build(rng, *case))


def test_scales_of_an_e4m3_cache_that_differ_widely():
    """Groups whose scales lie far apart, within a tile and from tile to tile,
    a row that nobody sees with an enormous one, zeros at the smallest scale."""
    rng = np.random.default_rng(31)
    for D, T, kind in ((128, 6, "chain"), (64, 40, "tree"), (128, 3, "tree")):
        for spread in ((100, 140), (60, 130), (120, 122)):
            s = build(rng, 2, T, 8, 2, D, 16, [700, 300], None, kind, "bf16", "e4m3")
            for x in (s["ks"], s["vs"]):
                x[:] = torch.from_numpy(rng.integers(*spread, tuple(x.shape)).astype(np.uint8)).to(DEV)
                # Whole pages at one scale, others at random ones.
                x[::2] = torch.from_numpy(rng.integers(*spread, (x.shape[0] + 1) // 2).astype(np.uint8)).to(DEV)[:, None, None, None]
            s["q"] *= 2.0 ** (118 - spread[1])       # scores of a few units
            for c in (s["k"], s["v"]):               # a page of zeros
                c.view(torch.uint8)[int(s["tables"][0, 2])] = 0
            s["ks"][int(s["tables"][0, 2])] = 7
            s["vs"][int(s["tables"][0, 2])] = 7
            check(s)
            for i in range(8):                       # a first tile of zeros
                for c, x in ((s["k"], s["ks"]), (s["v"], s["vs"])):
                    c.view(torch.uint8)[int(s["tables"][1, i])] = 0
                    x[int(s["tables"][1, i])] = 7
            check(s)
            if s["mask"] is not None:
                s["mask"][0, :, T - 1] = False       # hidden from all
                blk, row = int(s["tables"][0, (700 + T - 1) // 16]), (700 + T - 1) % 16
                s["ks"][blk, :, row] = 250
                s["vs"][blk, :, row] = 250
                check(s)


@pytest.mark.parametrize("D,T,bs,H", [(128, 3, 16, 24), (64, 2, 32, 32), (128, 40, 64, 12), (64, 70, 16, 12)])
def test_values_of_an_e4m3_cache_that_begin_with_zeros(D, T, bs, H):
    """Sequences whose first tokens' values are zeros at the smallest scale: the
    scale that a range's values refer to is found in a later tile, its first,
    its last or none, in ranges of many tiles."""
    rng = np.random.default_rng(D + T)
    zeros = [0, 30, 64, 100, 128, 200, 449, 2000, 320, 640]
    L = [700, 400, 900, 130, 700, 1300, 1000, 800, 321, 641]
    s = build(rng, len(L), T, 4 * H, H, D, bs, L, None, "chain", "bf16", "e4m3")
    for b, m in enumerate(zeros):
        for pos in range(min(m, L[b] + T)):
            blk = int(s["tables"][b, pos // bs])
            s["v"].view(torch.uint8)[blk, :, pos % bs] = 0
            s["vs"][blk, :, pos % bs] = 7
    check(s)


@pytest.mark.parametrize("D,T", [(128, 3), (64, 70)])
def test_the_smallest_scales_of_an_e4m3_cache(D, T):
    """Values of 2^-112 and less: at the smallest scale, alone and beside zeros."""
    s = build(np.random.default_rng(35), 2, T, 8, 2, D, 16, [300, 70], None, "chain", "bf16", "e4m3")
    s["vs"][:] = 7
    check(s)
    assert ref.to64(call(s)).any()
    s["vs"][int(s["tables"][0, 3])] = 90
    check(s)


def test_the_largest_scales_of_an_e4m3_cache():
    rng = np.random.default_rng(34)
    for nan in (False, True):
        s = build(rng, 2, 3, 8, 2, 128, 16, [900, 70], None, "chain", "bf16", "e4m3")
        s["vs"][:] = 248
        s["v"].view(torch.uint8)[:] &= 0x8F          # codes of 2^-5 at most
        if nan:
            s["vs"][int(s["tables"][0, 3]), 1, 5, 1] = 255
        out = check(s)
        assert np.isnan(out).any() == nan


@pytest.mark.parametrize("where", ["ks", "vs", "k", "v"])
def test_not_a_number_among_the_committed_tokens_of_an_e4m3_cache(where):
    for T, D in ((3, 128), (70, 64)):
        s = build(np.random.default_rng(33), 2, T, 4, 2, D, 16, [300, 40], None, "tree", "bf16", "e4m3")
        x = s[where].view(torch.uint8)
        x[int(s["tables"][0, 9]), 1, 5, 1] = 0xFF      # one group, or one code, of request 0's head 1
        out = check(s)
        assert np.isnan(out).any() and np.isfinite(out).any()


@pytest.mark.parametrize("big", [-130, -40, 0, 100])
def test_queries_of_any_magnitude(big):
    """Query rows that are huge, tiny, zero or of one element, against keys
    that bring the scores back to a few units."""
    rng = np.random.default_rng(32)
    for cdt in ("bf16", "e4m3"):
        s = build(rng, 1, 5, 8, 2, 64, 16, [200], None, "chain", "bf16", cdt)
        q = s["q"].double()
        q *= 2.0 ** big
        q[0, 1, :, 1:] = 0
        q[0, 2] = 0
        q[0, 3] *= torch.from_numpy(2.0 ** rng.integers(-30, 1, (8, 64))).to(DEV)
        s["q"] = q.to(torch.bfloat16)
        check(s, scale=2.0 ** -3 * 2.0 ** -big if abs(big) < 120 else 1.0)


@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,T,L", [(1, 1, [20011]), (2, 7, [4999, 9001]), (1, 40, [6007])])
def test_long_contexts_are_split_and_joined(B, T, L, cdt):
    rng = np.random.default_rng(B + T)
    check(build(rng, B, T, 8, 1, 128, 16, L, None, "tree", "bf16", cdt))


MANY = [
    # Ranges of many tiles: the rings of stages go round several times, units
    # begin and end within a range, and short ones lie between.
    (6, 2, 8, 8, 128, 16, [3000, 2500, 40, 3100, 0, 2222], None, "chain", "bf16", "bf16"),
    (6, 3, 16, 16, 128, 64, [1500, 2500, 40, 1100, 129, 2222], [3, 1, 0, 2, 3, 3], "tree", "bf16", "e4m3"),
    (5, 1, 32, 32, 64, 32, [2000, 1000, 1, 127, 1800], None, "chain", "fp16", "fp16"),
    (5, 2, 32, 32, 64, 8, [2000, 1000, 1, 127, 1500], None, "any", "bf16", "e4m3"),
    (4, 40, 16, 4, 128, 16, [9000, 20, 5000, 7000], [40, 40, 31, 33], "tree", "bf16", "bf16"),
    (4, 40, 16, 4, 128, 128, [9000, 20, 5000, 7000], [40, 7, 40, 36], "chain", "bf16", "e4m3"),
    (4, 70, 8, 4, 64, 32, [6000, 120, 4000, 5000], None, "any", "fp16", "fp16"),
    (4, 70, 8, 4, 64, 64, [6000, 120, 4000, 5000], None, "tree", "bf16", "e4m3"),
    (5, 2, 32, 32, 128, 16, [2000, 1000, 1, 127, 1500], None, "any", "fp16", "e4m3"),
    (4, 70, 8, 4, 128, 64, [6000, 120, 4000, 5000], None, "tree", "fp16", "e4m3"),
]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_ranges_of_many_tiles(case):
    check(build(np.random.default_rng(len(case[6]) + case[4]), *case))


@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
def test_many_short_and_one_long(cdt):
    rng = np.random.default_rng(0)
    L = [int(x) for x in rng.integers(0, 60, 300)]
    L[137] = 15000
    n = [int(x) for x in rng.integers(0, 4, 300)]
    check(build(rng, 300, 3, 4, 2, 64, 16, L, n, "chain", "bf16", cdt))


@pytest.mark.parametrize("dt,cdt,D", [("bf16", "bf16", 128), ("bf16", "e4m3", 128), ("fp16", "fp16", 64),
                                      ("fp16", "e4m3", 128), ("bf16", "bf16", 40)])
def test_what_is_not_visible_has_no_influence(dt, cdt, D):
    """NaN, infinities and the type's lowest values behind a request's last
    token, in blocks of nobody and in drafts that a row does not see."""
    rng = np.random.default_rng(9)
    B, T, bs = 3, 12, 16
    s = build(rng, B, T, 8, 2, D, bs, [30, 100, 3], [12, 5, 12], "tree", dt, cdt)
    raw_k, raw_v = (x.view(torch.uint8) if cdt == "e4m3" else x for x in (s["k"], s["v"]))
    junk = [0x7F, 0xFF, 0x7E] if cdt == "e4m3" else [float("nan"), float("inf"), -float("inf"),
                                                     torch.finfo(TD[cdt]).min]
    used = np.zeros((s["k"].shape[0], bs), dtype=bool)
    for b in range(B):
        for j in range(s["L"][b] + s["n"][b]):
            used[s["tables"][b, j // bs], j % bs] = True
    for x in (raw_k, raw_v):
        for c, (blk, row) in enumerate(zip(*np.nonzero(~used))):
            x[blk, :, row] = junk[c % len(junk)]
    # Draft 4 of request 0 is hidden from all but itself, draft 7 from everyone.
    s["mask"][0, :, 4] = False
    s["mask"][0, 4, 4] = True
    s["mask"][0, :, 7] = False
    for c, (j, x) in enumerate([(34, raw_v), (37, raw_k), (37, raw_v)]):
        x[int(s["tables"][0, j // bs]), :, j % bs] = junk[0]
    out = check(s)
    assert np.isnan(out).any()          # draft 4's own row


@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
def test_a_later_token_of_a_prompt_that_is_not_finite(cdt):
    rng = np.random.default_rng(4)
    s = build(rng, 1, 150, 2, 1, 64, 16, [37], None, "chain", "bf16", cdt)
    x = s["v"].view(torch.uint8) if cdt == "e4m3" else s["v"]
    x[int(s["tables"][0, 100 // 16]), :, 100 % 16] = 0x7F if cdt == "e4m3" else float("inf")
    out = check(s)                      # rows before position 100 are finite
    assert np.isfinite(out[:63]).all() and not np.isfinite(out[63:]).any()


@pytest.mark.parametrize("dt,cdt", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
def test_scores_that_jump_and_a_scale_of_one(dt, cdt):
    """Maxima that rise from tile to tile by far more than the exponent of a
    16-bit type, and a last key that outweighs all."""
    rng = np.random.default_rng(5)
    s = build(rng, 2, 3, 8, 2, 64, 16, [600, 1000], None, "chain", dt, cdt)
    if cdt == "e4m3":
        s["ks"][:] = torch.from_numpy(rng.integers(112, 126, tuple(s["ks"].shape)).astype(np.uint8)).to(DEV)
    else:
        s["k"] *= torch.from_numpy(2.0 ** rng.integers(-3, 4, (s["k"].shape[0], 1, 1, 1))).to(DEV)
    check(s, scale=1.0)
    check(s, scale=-0.5)
    check(s, scale=0.0)


def test_strided_queries_and_caches_in_one_buffer():
    rng = np.random.default_rng(6)
    for dt, cdt, off in (("bf16", "bf16", 0), ("bf16", "e4m3", 0), ("fp16", "fp16", 1), ("bf16", "bf16", 3)):
        s = build(rng, 2, 6, 8, 2, 128, 16, [50, 333], [6, 4], "tree", dt, cdt, halves=True)
        B, T, H, D = s["q"].shape
        wide = torch.zeros(B, T, H + 4, D + off, dtype=s["q"].dtype, device=DEV)
        wide[:, :, :H, off:] = s["q"]
        s["q"] = wide[:, :, :H, off:]
        check(s)
        turned = s["q"].transpose(1, 2).contiguous().transpose(1, 2)   # [B, H, T, D] storage
        s["q"] = turned
        check(s)


def test_bad_data_is_reported_and_the_rest_is_right():
    import speculative_decoding_verification_75_gb300 as sv
    from speculative_decoding_verification_75_gb300 import api, kv
    for D, bs in ((128, 16), (40, 16)):
        rng = np.random.default_rng(7)
        s = build(rng, 5, 4, 8, 2, D, bs, [40, 200, 100, 33, 70], None, "chain", "bf16", "bf16")
        s["tables"] = s["tables"][:, :12].copy()          # request 1 needs 13 blocks
        s["tables"][2, 3] = -1
        s["tables"][3, 0] = s["k"].shape[0]
        s["L"][4] = -3
        check(s, want_status=api.SV_KV_TABLE_SHORT | api.SV_KV_MISSING_BLOCK | kv.SV_KV_BAD_BLOCK
              | api.SV_KV_BAD_LENGTH)
        s["tables"][:] = -1                                # nothing left to see
        s["L"][4] = 0
        out = check(s, want_status=api.SV_KV_TABLE_SHORT | api.SV_KV_MISSING_BLOCK)
        assert not out.any()
        # An empty pool and an empty table.
        e = torch.empty(0, 2, bs, D, dtype=torch.bfloat16, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = sv.tree_attention(s["q"], e, e, i32(np.zeros((5, 3))), i32([0] * 5), status=st)
        assert not o.any() and st.item() == kv.SV_KV_BAD_BLOCK
        st.zero_()
        o = sv.tree_attention(s["q"], s["k"], s["v"], i32(np.zeros((5, 0))), i32([0] * 5), status=st)
        assert not o.any() and st.item() == api.SV_KV_TABLE_SHORT


def test_nothing_to_do():
    rng = np.random.default_rng(0)
    s = build(rng, 2, 3, 4, 2, 64, 16, [5, 6], [0, 0], "chain", "bf16", "bf16")
    check(s)
    import speculative_decoding_verification_75_gb300 as sv
    q = s["q"]
    assert sv.tree_attention(q[:0], s["k"], s["v"], i32(np.zeros((0, 2))), i32([])).shape == (0, 3, 4, 64)
    assert sv.tree_attention(q[:, :0], s["k"], s["v"], i32(s["tables"]), i32(s["L"])).shape == (2, 0, 4, 64)


@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
def test_results_repeat_and_streams_do_not_share(cdt):
    """The same call twice, on two streams at once with other inputs in
    between, and in a captured graph replayed on changed inputs."""
    rng = np.random.default_rng(12)
    s = build(rng, 4, 6, 16, 2, 128, 16, [3000, 10, 999, 0], None, "tree", "bf16", cdt)
    t = build(rng, 4, 6, 16, 2, 128, 16, [100, 2000, 0, 77], None, "tree", "bf16", cdt)
    a, b = call(s), call(t)
    s_ops, t_ops = operands(s), operands(t)      # in place before the streams read them
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((call(s, s_ops, stream=s1), call(t, t_ops, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, a) and torch.equal(y, b)

    import speculative_decoding_verification_75_gb300 as sv
    tab, L, mask, _ = s_ops
    out = [torch.zeros_like(s["q"]) for _ in range(2)]
    graphs = []
    for o in out:                       # two graphs of the same call
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.tree_attention(s["q"], s["k"], s["v"], tab, L, mask, k_scale=s["ks"], v_scale=s["vs"], out=o)
        graphs.append(g)
    for new_L in ([3000, 10, 999, 0], [17, 10, 1000, 5]):
        L.copy_(i32(new_L))
        s["L"] = new_L
        want = call(s)
        torch.cuda.synchronize()
        for g, st in zip(graphs, (s1, s2)):          # both at once
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want)


def test_workspace_of_the_caller_holds_anything():
    from speculative_decoding_verification_75_gb300 import kv
    rng = np.random.default_rng(13)
    s = build(rng, 2, 6, 16, 2, 128, 16, [3000, 10], None, "chain", "bf16", "bf16")
    want = call(s)
    ws = torch.empty(kv.tree_attention_workspace_bytes(2, 6, 16, 2, 128), dtype=torch.uint8, device=DEV)
    for fill in (0, 0xA5, 0xFF):
        ws.fill_(fill)
        assert torch.equal(call(s, workspace=ws), want)


@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
def test_blocks_past_32_bit_offsets(cdt):
    rng = np.random.default_rng(1)
    H, bs, D = 2, 16, 64
    stride = (1 << 31) + 16 * 64
    s = build(rng, 1, 6, 8, H, D, bs, [20], None, "tree", "bf16", cdt)
    far = []
    for x in (s["k"], s["v"]):
        esz = x.element_size()
        raw = torch.zeros((3 * stride + H * bs * D) * esz, dtype=torch.uint8, device=DEV)
        y = raw.view(x.dtype).as_strided((4, H, bs, D), (stride, bs * D, D, 1))
        y.view(torch.uint8).copy_(x.view(torch.uint8)) if cdt == "e4m3" else y.copy_(x)
        far.append(y)
    near = call(s)
    s["k"], s["v"] = far
    assert torch.equal(call(s), near)


def test_a_speculative_step_with_a_tree():
    """A step as a server runs it, greedy: write the tree's keys and values,
    attend, verify every root-to-leaf path, move the best path together, cut
    the rest, and decode the next token from the same cache; against the same
    model on dense float64 tensors without a cache."""
    import speculative_decoding_verification_75_gb300 as sv
    rng = np.random.default_rng(21)
    V, Hq, Hkv, D, bs, n_prompt = 97, 8, 2, 64, 16, 45
    E, Wq, Wk, Wv, Wo = (rng.standard_normal(s) * f for s, f in (
        ((V, 64), 1.0), ((64, Hq * D), 0.25), ((64, Hkv * D), 0.25), ((64, Hkv * D), 1.0),
        ((Hq * D, V), 1.0)))
    E, Wq, Wk, Wv, Wo = (torch.from_numpy(x).to(DEV).float() for x in (E, Wq, Wk, Wv, Wo))
    bf = torch.bfloat16

    def proj(tok, W, H):
        return (E[tok] @ W).view(1, -1, H, D).to(bf)

    def dense_logits(tokens):
        """Logits behind a plain sequence, from dense attention in 64 bits."""
        t = torch.tensor(tokens, device=DEV)
        q, k, v = proj(t, Wq, Hq).double(), proj(t, Wk, Hkv).double(), proj(t, Wv, Hkv).double()
        s = torch.einsum("hd,shd->hs", q[0, -1], k[0].repeat_interleave(Hq // Hkv, 1)) * D ** -0.5
        o = torch.einsum("hs,shd->hd", s.softmax(-1), v[0].repeat_interleave(Hq // Hkv, 1))
        return o.flatten() @ Wo.double()

    prompt = rng.integers(0, V, n_prompt).tolist()
    greedy = list(prompt)
    for _ in range(6):
        greedy.append(int(dense_logits(greedy).argmax()))
    root, cont = greedy[n_prompt], greedy[n_prompt + 1:]

    # The tree: the emitted token, then a wrong and a right child per level.
    parent, token = [-1, 0, 0, 2, 2, 3], [root, (cont[0] + 1) % V, cont[0], cont[1], (cont[1] + 5) % V,
                                         (cont[2] + 9) % V]
    N = len(token)
    mask = torch.zeros(N, N, dtype=torch.bool)
    for i in range(N):
        j = i
        while j >= 0:
            mask[i, j] = True
            j = parent[j]
    k, v, _, _ = make_cache(rng, 8, Hkv, bs, D, bf)
    tables = i32(make_tables(rng, [5], 8, 6))
    L = i32([0])
    pt = torch.tensor(prompt, device=DEV)
    sv.kv_write(proj(pt, Wk, Hkv), proj(pt, Wv, Hkv), k, v, tables, L)
    L.fill_(n_prompt)
    tt = torch.tensor(token, device=DEV)
    sv.kv_write(proj(tt, Wk, Hkv), proj(tt, Wv, Hkv), k, v, tables, L)
    out = sv.tree_attention(proj(tt, Wq, Hq), k, v, tables, L, mask.to(DEV))
    logits = out[0].flatten(1).float() @ Wo                     # [N, V]
    # Every root-to-leaf path is one request of the verification.
    paths = [[0, 1], [0, 2, 3, 5], [0, 2, 4]]
    g = max(len(p) for p in paths) - 1
    rows = torch.zeros(len(paths), g + 1, V, device=DEV)
    ids = torch.zeros(len(paths), g, dtype=torch.int32, device=DEV)
    for r, p in enumerate(paths):
        rows[r, :len(p)] = logits[p]
        ids[r, :len(p) - 1] = tt[p[1:]].int()
    zeros = torch.zeros(len(paths), device=DEV)
    toks, nacc = sv.verify(rows, ids, None, torch.zeros(len(paths), g, device=DEV), zeros, zeros,
                           i32([len(p) - 1 for p in paths]))
    best = int(nacc.argmax())
    kept = int(nacc[best])
    assert best in (1, 2) and kept >= 1
    assert toks[best, :kept + 1].tolist() == cont[:kept + 1]
    assert (paths[best][:3] == [0, 2, 3]) == (kept >= 2)
    # Keep the root and the accepted drafts, cut the rest.
    path = i32([paths[best][:kept + 1] + [-1] * (N - kept - 1)])
    count = i32([kept + 1])
    free, nfree = i32([-1] * 8), i32([0])
    sv.kv_compact(path, count, L, tables, k, v)
    sv.kv_rollback(count, L, tables, bs, free, nfree, i32([N]), gamma_max=N)
    assert L.item() == n_prompt + kept + 1
    # The next token from the cache equals the one of the plain sequence.
    seq = greedy[:n_prompt + 1 + kept] + [int(toks[best, kept])]
    nt = torch.tensor(seq[-1:], device=DEV)
    if int(tables[0, L.item() // bs]) < 0:
        tables[0, L.item() // bs] = free[0]
    sv.kv_write(proj(nt, Wk, Hkv), proj(nt, Wv, Hkv), k, v, tables, L)
    o = sv.tree_attention(proj(nt, Wq, Hq), k, v, tables, L)
    got = o[0].flatten().double() @ Wo.double()
    want = dense_logits(seq)
    # Each output element is off by at most 2 * 2^-8 of sum p |v| + |o| (see
    # paged_ref); |v| <= max|v| bounds it for the logits' sum of products.
    vmax = proj(torch.arange(V, device=DEV), Wv, Hkv).abs().max().double()
    bound = 3 * 2.0 ** -8 * vmax * Wo.double().abs().sum(0)
    assert ((got - want).abs() <= bound).all()

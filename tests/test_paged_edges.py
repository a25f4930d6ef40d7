"""Calls of the paged-cache operators at the edges of what they take: marked
units with other requests behind them, rows without a finite score, powers of
two at the ends of their range, lengths far behind the table, and one workspace
for all sizes."""
import math
from pathlib import Path

import numpy as np
import pytest
import torch

import paged_ref as ref
from test_paged_kv import (DEV, F8, TD, PTR, _attn, _cache_words, _compact, _read, _write, bits,
                           compact_reference, i32, make_cache, make_tables)
from test_tree_attention import UNIT, build, call, check

gpu = pytest.mark.gpu


def raw(t):
    return t.view(torch.uint8) if t.dtype == F8 else t


# ---------------------------------------------------------- marked units ----

MARKED = [
    (330, 2, 2, 2, 64, "bf16", "bf16"), (330, 2, 2, 2, 128, "bf16", "e4m3"),
    # 136 rows of a KV head: two row tiles.
    (80, 17, 32, 4, 64, "fp16", "fp16"), (80, 17, 32, 4, 128, "bf16", "e4m3")]


@gpu
@pytest.mark.parametrize("B,T,Hq,Hkv,D,dt,cdt,why", [
    (*c, why) for c in MARKED for why in ("value", "block", "scale") if why != "scale" or c[-1] == "e4m3"])
def test_marked_units_among_others_of_a_range(B, T, Hq, Hkv, D, dt, cdt, why):
    """Units of one or two tiles, several to a range, some of them to be
    recomputed: a new token's value that is not finite, a missing block, scales
    too far apart for the products."""
    rng = np.random.default_rng(B + T)
    L = [int(x) for x in rng.integers(0, 60, B)]
    s = build(rng, B, T, Hq, Hkv, D, 16, L, None, "chain", dt, cdt)
    status = 0
    for b in (0, 3, 4, 5, 40, B - 1):
        if why == "value":
            j = L[b] + T - 1
            raw(s["v"])[int(s["tables"][b, j // 16]), :, j % 16] = 0x7F if cdt == "e4m3" else float("inf")
        elif why == "block":
            s["tables"][b, 0] = -1
            status = ref.MISSING
        else:
            s["vs"][int(s["tables"][b, 0]), :, :, 0] = 90
    check(s, want_status=status)


@gpu
def test_more_units_in_a_range_than_marks_are_kept_for():
    """Over a thousand units of one tile in each range; some requests' only
    block is missing, and their rows are 0."""
    import speculative_decoding_verification_75_gb300 as sv
    B, H, D, bs, L = 10400, 32, 64, 16, 9
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn(64, H, bs, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(B, 1, H, D, generator=g, device=DEV).bfloat16()
    tab = torch.randint(64, (B, 1), generator=g, device=DEV).int()
    gone = torch.randperm(B, generator=g, device=DEV)[:40]
    tab[gone] = -1
    out = torch.full_like(q, -7.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.tree_attention(q, k, v, tab, i32([L] * B), out=out, status=status)
    assert status.item() == ref.MISSING
    assert not out[gone].any()
    live = torch.ones(B, dtype=torch.bool, device=DEV)
    live[gone] = False
    at = tab[live, 0].long()
    for i in range(0, at.numel(), 2000):
        kk, vv = (x[at[i:i + 2000], :, :L + 1].double() for x in (k, v))
        p = torch.einsum("bhd,bhsd->bhs", q[live][i:i + 2000, 0].double(), kk).mul(D ** -0.5).softmax(-1)
        o, a = (torch.einsum("bhs,bhsd->bhd", p, x) for x in (vv, vv.abs()))
        # Probabilities and results rounded to bf16; fp32 scores and sums are
        # off by far less than the tenth of that allowed for them.
        assert ((out[live][i:i + 2000, 0].double() - o).abs() <= UNIT["bf16"] * (1.1 * a + o.abs())).all()


@gpu
def test_a_marked_unit_of_a_long_context_holds_up_nobody():
    """Two requests over 98304 keys with a value that is not finite at their
    last token, and healthy ones behind them in the same ranges.  (One warp
    recomputes a row at about 1 us a key; 32 rows to a warp took 3.2 s, longer
    than the kernel's other warps wait.)

    Every request has the same 64 blocks over and over, so that a softmax over
    its keys is one over 8192 keys, each counted 12 times, and its new tokens."""
    import speculative_decoding_verification_75_gb300 as sv
    B, T, G, D, bs, pool, times = 640, 16, 8, 128, 128, 64, 12
    L = pool * bs * times
    g = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.randn(pool + B, 1, bs, D, generator=g, device=DEV).mul(100).clamp(-448, 448).to(F8)
            for _ in range(2))
    ks, vs = (torch.full((pool + B, 1, bs, D // 32), 120, dtype=torch.uint8, device=DEV) for _ in range(2))
    tab = torch.empty(B, pool * times + 1, dtype=torch.int32, device=DEV)
    tab[:, :-1] = (torch.arange(pool * times, device=DEV) % pool).int()
    tab[:, -1] = torch.arange(B, device=DEV).int() + pool
    q = torch.randn(B, T, G, D, generator=g, device=DEV).bfloat16()
    # Range i of 304 begins with unit 640 i / 304: 99 and 300 lie within one,
    # with others behind them.
    for b in (99, 300):
        raw(v)[pool + b, 0, T - 1] = 0x7F
    out = torch.full_like(q, -7.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.tree_attention(q, k, v, tab, i32([L] * B), k_scale=ks, v_scale=vs, out=out, status=status)
    assert status.item() == 0
    K, V = ((x.double() / 128).squeeze(1) for x in (k, v))
    K0, V0 = K[:pool].flatten(0, 1), V[:pool].flatten(0, 1)
    see = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
    for b in (98, 99, 100, 101, 300, 301):
        x0 = torch.einsum("tgd,sd->tgs", q[b].double(), K0) * D ** -0.5
        x1 = torch.einsum("tgd,sd->tgs", q[b].double(), K[pool + b, :T]) * D ** -0.5
        x1 = x1.masked_fill(~see[:, None], -math.inf)
        m = torch.maximum(x0.amax(-1), x1.amax(-1))[..., None]
        p0, p1 = times * (x0 - m).exp(), (x1 - m).exp()
        l = (p0.sum(-1) + p1.sum(-1))[..., None]
        o = torch.einsum("tgs,sd->tgd", p0 / l, V0)
        a = torch.einsum("tgs,sd->tgd", p0 / l, V0.abs()) + torch.einsum("tgs,sd->tgd", p1 / l, V[pool + b, :T].nan_to_num().abs())
        for t in range(T):                    # a row's own values only: 0 * NaN
            o[t] += torch.einsum("gs,sd->gd", p1[t, :, :t + 1] / l[t], V[pool + b, :t + 1])
        assert bool(o.isnan().any()) == (b in (99, 300))
        assert torch.equal(out[b].isnan(), o.isnan())
        # Tolerance: probabilities to fp16 (2^-11, below its normal numbers
        # 2^-32 of the largest), the result to bf16, scores and exponentials as
        # in paged_ref, fp32 sums: a chain of 1536 tiles of 4 products each,
        # doubled where additions truncate, and of 1536 tiles and 64 terms for
        # the denominator; a recomputed row's is one term per key.
        S = L + T
        ds = (D + 8) * 2.0 ** -23 * D ** -0.5 * max(
            torch.einsum("tgd,sd->tgs", q[b].double().abs(), x.abs()).max().item() for x in (K0, K[pool + b, :T]))
        chain = 2 * (S + 8) if b in (99, 300) else 2 * 1536 * 4 + 1536 + 64
        t = (2.0 ** -11 + 2 * ds + 2.0 ** -19 + chain * 2.0 ** -24) * a + 2.0 ** -8 * o.abs()
        t = 1.01 * (t + S * 2.0 ** -32 * V0.abs().max() / l)
        fine = ~o.isnan()
        assert ((out[b].double() - o).abs()[fine] <= t[fine]).all()


@gpu
@pytest.mark.parametrize("T", [2, 20])
@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
def test_a_missing_block_at_any_place_of_a_tile(T, cdt):
    """Eight blocks to a tile, each looked up by another lane: the mark of one
    that is missing reaches the warps that store the rows."""
    for j in range((140 + T + 7) // 8):
        s = build(np.random.default_rng(j), 1, T, 8, 1, 64, 8, [140], None, "chain", "bf16", cdt)
        s["tables"][0, j] = -1
        check(s, want_status=ref.MISSING)


# ---------------------------------------------------------------- scales ----

def lse_within_fp32(s, scale):
    """The log-sum-exp against 64 bits, to what fp32 scores and sums lose: each
    score's error counts by its probability (the log's derivative), so that a
    key without weight allows none."""
    B, T, Hq, D = s["q"].shape
    lse = torch.zeros(B, T, Hq, device=DEV)
    call(s, lse=lse, scale=scale)
    cache = ref.Cache(s["k"], s["v"], torch.from_numpy(s["tables"]), s["ks"], s["vs"])
    q, lse = ref.to64(s["q"]), ref.to64(lse)
    for b in range(B):
        L, n = s["L"][b], s["n"][b]
        at = [cache.place(b, j)[:2] for j in range(L + n)]
        K = np.stack([cache.k[blk, :, row] for blk, row in at])
        for i in range(n):
            see = np.ones(L + n, dtype=bool)
            see[L:] = np.arange(n) <= i if s["mask"] is None else s["mask"][b, i, :n]
            for h in range(Hq):
                k = K[see, h // (Hq // K.shape[1])]
                x = k @ q[b, i, h] * scale
                # Products of two 16-bit values are exact in fp32, one rounding
                # per addition, doubled where an addition truncates.
                dx = (D + 8) * 2.0 ** -23 * (np.abs(k) @ np.abs(q[b, i, h])) * scale
                p = np.exp(x - x.max())
                want = x.max() + np.log(p.sum())
                p /= p.sum()
                tol = (p @ dx) * 1.01 + abs(x.max()) * 2.0 ** -22 + (len(x) + 8) * 2.0 ** -24 + 2.0 ** -19
                assert abs(lse[b, i, h] - want) <= tol, (b, i, h, lse[b, i, h] - want, tol)


@gpu
@pytest.mark.parametrize("above", [15, 16, 18, 20, 22, 24, 25, 40])
@pytest.mark.parametrize("T", [4, 20])
def test_a_large_key_without_weight_does_not_round_the_others(above, T):
    """A draft that no row sees, and a committed key whose scores are far below
    the rest, 2^above times as large as the other keys."""
    rng = np.random.default_rng(above)
    s = build(rng, 1, T, 8, 1, 128, 16, [12], None, "tree", "bf16", "e4m3")
    sign = torch.from_numpy(np.where(rng.random(128) < 0.5, -1.0, 1.0)).to(DEV)
    s["q"] = (s["q"].abs() * sign).to(torch.bfloat16)
    s["ks"][:] = 120
    place = lambda j: (int(s["tables"][0, j // 16]), j % 16)  # noqa: E731
    plain = s["k"].view(torch.uint8).clone()
    for what in ("hidden", "unlikely"):
        s["k"].view(torch.uint8).copy_(plain)
        s["ks"][:] = 120
        if what == "hidden":
            s["mask"][0, :, T - 2] = False
            blk, row = place(12 + T - 2)
        else:
            blk, row = place(5)
            s["k"][blk, 0, row] = (-448 * sign).to(F8)
        s["ks"][blk, :, row] = 120 + above
        check(s)
        lse_within_fp32(s, 128 ** -0.5)


# --------------------------------------------------------- rows and keys ----

@gpu
@pytest.mark.parametrize("D,dt,cdt", [(128, "bf16", "bf16"), (64, "fp16", "fp16"), (128, "bf16", "e4m3"),
                                      (40, "bf16", "bf16"), (32, "bf16", "e4m3")])
@pytest.mark.parametrize("T,L", [(2, [9, 0]), (2, [5000, 700]), (20, [3000, 33])])
def test_a_row_with_no_score_above_minus_infinity_is_zero(D, dt, cdt, T, L):
    """Whatever its values hold, infinities and NaN among them, in a unit of
    one range and in one that ranges cut."""
    s = build(np.random.default_rng(T), 2, T, 8, 1, D, 16, L, None, "chain", dt, cdt)
    if cdt == "e4m3":
        s["k"].view(torch.uint8).bitwise_and_(0x7F).bitwise_or_(0x08).clamp_(max=0x7E)
        s["q"][:] = -math.inf
    else:
        s["q"] = s["q"].abs() + 0.5
        s["k"][:] = -math.inf
    for b in range(2):
        for j in range(3, L[b], 5):         # committed tokens' values
            raw(s["v"])[int(s["tables"][b, j // 16]), :, j % 16] = (
                0x7F if cdt == "e4m3" else math.inf if j % 2 else math.nan)
    lse = torch.zeros(2, T, 8, device=DEV)
    out = call(s, lse=lse)
    assert (out == 0).all()
    assert (lse == -math.inf).all()


@gpu
@pytest.mark.parametrize("q_exp,k_byte", [(-120, 240), (-126, 246), (-112, 232), (100, 20), (-60, 60)])
def test_powers_of_queries_and_keys_that_cancel(q_exp, k_byte):
    """Tiny queries over keys with enormous scales, and the reverse: scores of
    a few units."""
    for T in (3, 20):
        rng = np.random.default_rng(T)
        s = build(rng, 2, T, 8, 1, 64, 16, [100, 7], None, "chain", "bf16", "e4m3")
        s["q"] = (s["q"].double() * 2.0 ** q_exp).to(torch.bfloat16)
        s["ks"][:] = torch.from_numpy(rng.integers(k_byte - 1, k_byte + 2, tuple(s["ks"].shape)).astype(np.uint8)).to(DEV)
        check(s)


@gpu
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -140, -(2.0 ** -140)])
def test_a_scale_that_leaves_nothing_of_large_products(scale):
    """q . k of 2^120 and more, and a scale that makes every score next to 0."""
    s = build(np.random.default_rng(2), 2, 3, 8, 1, 64, 16, [100, 7], None, "chain", "bf16", "bf16")
    s["q"] *= 2.0 ** 58
    s["k"] *= 2.0 ** 58
    check(s, scale=scale)


@gpu
@pytest.mark.parametrize("D", [40, 128])
def test_problems_of_hidden_positions_are_reported_too(D):
    """Drafts that no row sees, in a missing block, one behind the pool or
    behind the table: the status word is the same for every head dimension."""
    from speculative_decoding_verification_75_gb300 import api, kv
    for entry, want in ((-1, api.SV_KV_MISSING_BLOCK), (99, kv.SV_KV_BAD_BLOCK), (None, api.SV_KV_TABLE_SHORT)):
        s = build(np.random.default_rng(D), 1, 20, 4, 2, D, 16, [16], None, "tree", "bf16", "bf16")
        s["mask"][0, :, 16:] = False            # drafts 16 .. 19: positions 32 .. 35
        if entry is None:
            s["tables"] = s["tables"][:, :2].copy()
        else:
            s["tables"][0, 2] = entry
        check(s, want_status=want)


@gpu
@pytest.mark.parametrize("D,hole", [(40, False), (40, True), (128, False), (128, True)])
def test_a_length_far_behind_the_table(D, hole):
    """Every row sees what the table holds; nothing walks the 2^31 positions
    behind it, which would take seconds (a hole has rows recomputed)."""
    from speculative_decoding_verification_75_gb300 import api
    s = build(np.random.default_rng(D), 2, 3, 8, 2, D, 16, [61, 61], None, "chain", "bf16", "bf16")
    s["tables"] = s["tables"][:, :4].copy()
    want = api.SV_KV_TABLE_SHORT
    if hole:
        s["tables"][0, 1] = -1
        want |= api.SV_KV_MISSING_BLOCK
    s["L"] = [64, 64]
    check(s, want_status=want)
    near = call(s)
    s["L"] = [2 ** 31 - 100, 2 ** 31 - 4]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    far = call(s, status=status)
    end.record()
    assert torch.equal(far, near) and status.item() == want
    assert begin.elapsed_time(end) < 100


# ------------------------------------------------------------- workspace ----

def test_a_workspace_serves_every_smaller_batch():
    from speculative_decoding_verification_75_gb300 import kv
    n = kv.tree_attention_workspace_bytes
    for Hkv in (1, 2, 7, 8):
        for G in (1, 2, 3, 4, 7, 8, 16, 100, 128, 130):
            for D in (8, 64, 128, 256):
                by_T = [n(4, T, G * Hkv, Hkv, D) for T in (*range(1, 140), 1000)]
                assert by_T == sorted(by_T)
    for T in (1, 2, 3, 16, 17, 64, 65, 128, 129):
        by_heads = [n(4, T, 8 * G, 8, 128) for G in range(1, 140)]
        assert by_heads == sorted(by_heads)
        by_kv_heads = [n(4, T, 64, Hkv, 128) for Hkv in (64, 32, 16, 8, 4, 2, 1)]
        assert by_kv_heads == sorted(by_kv_heads)
        by_D = [n(4, T, 32, 8, D) for D in range(8, 257, 8)]
        assert by_D == sorted(by_D)
        assert len({n(B, T, 32, 8, 128) for B in (1, 2, 100, 5000)}) == 1


@gpu
@pytest.mark.parametrize("cdt", ["bf16", "e4m3"])
def test_one_workspace_for_steps_of_all_sizes(cdt):
    from speculative_decoding_verification_75_gb300 import kv
    ws = torch.empty(kv.tree_attention_workspace_bytes(2, 64, 16, 2, 128), dtype=torch.uint8, device=DEV)
    for T in (64, 16, 17, 15, 1, 33):            # 16 tokens are one tile, 17 a pair
        ws.fill_(0xA5)
        check(build(np.random.default_rng(T), 2, T, 16, 2, 128, 16, [3000, 10], None, "chain", "bf16", cdt),
              workspace=ws)


# -------------------------------------------------------------- refusals ----

def test_a_table_of_2_31_positions_is_refused_by_attention():
    """Within the last tile below 2^31 the kernel's positions would overflow."""
    from speculative_decoding_verification_75_gb300 import api, kv
    lib = api.load_library()
    for bs, blocks in ((65528, 32772), (1 << 20, 2047), (1, 2 ** 31 - 1), (1, 2 ** 31 - 4095)):
        cache = _cache_words(bs=bs, max_blocks=blocks, block=2 * bs * 64)
        assert (bs * blocks > 0x7ffff000) == (bs != 1 << 20)
        # Nothing is launched for an empty batch; its sizes are checked.
        want = api.SV_ERR_INVALID_ARG if bs * blocks > 0x7ffff000 else api.SV_OK
        assert _attn(lib, kv, cache, B=0) == want
        assert _write(lib, kv, cache, B=0) == api.SV_OK


def test_two_results_in_one_place_are_refused():
    from speculative_decoding_verification_75_gb300 import api, kv
    lib, bad = api.load_library(), api.SV_ERR_INVALID_ARG
    assert _read(lib, kv, _cache_words(v=2 * PTR)) == bad               # key and value in one tensor
    assert _write(lib, kv, _cache_words(), value=2 * PTR) == bad        # k and v in one cache
    assert _write(lib, kv, _cache_words(), vt=256) == bad
    f8 = dict(dtype=3, block=2048, sblock=64)
    for call in (_write, _compact):
        assert call(lib, kv, _cache_words(v=2 * PTR, ks=PTR, vs=PTR, **f8)) == bad
        assert call(lib, kv, _cache_words(ks=PTR, vs=2 * PTR, **f8)) == bad


@gpu
@pytest.mark.parametrize("B,H,D,bs,P,cdt", [(3, 8, 128, 16, 9, "bf16"), (2, 33, 256, 4, 70, "e4m3"), (1, 1, 32, 5, 200, "e4m3")])
def test_compact_where_keys_and_values_are_one_array(B, H, D, bs, P, cdt):
    import speculative_decoding_verification_75_gb300 as sv
    rng = np.random.default_rng(P)
    L = rng.integers(0, 3 * bs, B)
    path = np.stack([np.sort(rng.permutation(2 * P)[:P]) for _ in range(B)])
    need = [-(-(int(x) + 2 * P) // bs) for x in L]
    tables = make_tables(rng, need, sum(need) + 1, max(need))
    c, _, s, _ = make_cache(rng, sum(need) + 1, H, bs, D, TD[cdt], layers=2)
    want = compact_reference([bits(x).copy() for x in (c, s) if x is not None], tables, bs, path, [P] * B, L)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.kv_compact(i32(path), i32([P] * B), i32(L), i32(tables), c, c, k_scale=s, v_scale=s, status=status)
    assert status.item() == 0
    for x, w in zip((c, s), want):
        assert np.array_equal(bits(x), w)


# --------------------------------------------------------------- a step ----

@gpu
def test_the_step_of_the_readme_keeps_every_token():
    """The step as README.md spells it out, on ragged batches: the sequences
    read back are the committed tokens, the emitted one and the accepted drafts."""
    readme = (Path(__file__).resolve().parents[1] / "README.md").read_text()
    code = next(b for b in readme.split("```python")[1:] if "kv_compact" in b).split("```")[0]
    rng = np.random.default_rng(17)
    B, T, H, D, block_size, n = 4, 6, 2, 64, 4, 30
    L, new, accepted = [0, 7, 20, 3], [6, 1, 4, 6], [3, 0, -1, 5]
    nodes = [[0, 2, 3, 5, -1, -1], [0, -1, -1, -1, -1, -1], [-1] * 6, [0, 1, 2, 3, 4, 5]]
    k, v = (torch.from_numpy(rng.standard_normal((B, 30, H, D))).bfloat16().to(DEV) for _ in range(2))
    k_cache, v_cache = (torch.zeros(40, H, block_size, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tables = make_tables(rng, [-(-(a + b) // block_size) for a, b in zip(L, new)], 40, 8)
    space = dict(k_cache=k_cache, v_cache=v_cache, block_tables=i32(tables), seq_lens=i32(L), new_lens=i32(new),
                 block_size=block_size, T=T, n=n, tree_mask=None, path=i32(nodes), num_accepted=i32(accepted),
                 query=torch.zeros(B, T, 2 * H, D, dtype=torch.bfloat16, device=DEV),
                 free_list=i32([-1] * 40), free_count=i32([0]))
    import speculative_decoding_verification_75_gb300 as sv
    sv.kv_write(k, v, k_cache, v_cache, space["block_tables"], i32([0] * B), i32(L))   # committed tokens
    space["key"], space["value"] = (torch.stack([x[b, l:l + T] for b, l in enumerate(L)]) for x in (k, v))
    exec(code, space)
    kept = [a + 1 for a in accepted]
    assert space["seq_lens"].tolist() == [l + m for l, m in zip(L, kept)]
    for got, x in ((space["keys"], k), (space["values"], v)):
        for b, l in enumerate(L):
            want = torch.cat([x[b, :l], x[b, [l + j for j in nodes[b][:kept[b]]]]])
            assert torch.equal(got[b, :l + kept[b]], want) and not got[b, l + kept[b]:].any()

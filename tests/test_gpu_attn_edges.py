"""The attention half of a decoder layer where it meets its surroundings and
its ranges' ends: handles used at once on other streams, shared prefixes of
every kind of end, tables as wide as they may be, values that are not finite in
one part of a cut row."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as A
from tests.test_gpu_attn import S, bf, check, f64, i32, make_cache, make_table  # noqa: F401  (S: the device fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,rot,layout", [(128, 128, "half"), (64, 32, "interleaved")])
def test_rotation_is_ready_on_any_stream(S, D, rot, layout):
    """A new rotation serves the next call at once, also on a stream that does
    not wait for the default one."""
    rng = np.random.default_rng(101)
    T, Hq, Hkv, page = 40, 2, 1, 16
    table, n_pages = make_table(rng, [T], page)
    q, k, v = (bf(rng.normal(size=(T, h * D))).cuda() for h in (Hq, Hkv, Hkv))
    cu, kv, tab = i32([0, T]), i32([T]), i32(table)
    cache = S.KVCache(n_pages, page, Hkv, D)
    torch.cuda.synchronize()
    for i in range(24):
        side = torch.cuda.Stream()
        theta = 2000.0 * (i + 2)
        rope = S.Rope(D, rot_dim=rot, layout=layout, theta=theta)
        out = S.rope_append(rope, cache, q, k, v, cu, kv, tab, stream=side)
        side.synchronize()
        y, mag = A.rotate(f64(q).reshape(T, Hq, D), np.arange(T), A.frequencies(rot, theta), layout)
        check(out, y, A.rotate_bound(y, mag, False), np.ones(T, bool), Hq, D)
        keys = f64(cache.K)[table[0]].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:T]
        y, mag = A.rotate(f64(k).reshape(T, Hkv, D), np.arange(T), A.frequencies(rot, theta), layout)
        assert np.all(np.abs(keys - y) <= A.rotate_bound(y, mag, False))
    assert S.device_error() == 0


def test_calls_behind_a_long_one(S):
    """A call whose blocks start beside a kernel that lasts longer than the
    bounded waits' second: its waits do not count that kernel's time."""
    rng = np.random.default_rng(102)
    D, page, far = 128, 256, 1 << 27
    # one row over 2^27 keys, the same page again and again, on one SM (a hint of one key: no shares)
    K = bf(rng.normal(size=(1, 1, page, D))).cuda()
    one = S.KVCache(K=K, V=K.clone())
    table = torch.zeros((1, far // page), dtype=torch.int32, device="cuda")
    q1 = bf(rng.normal(size=(1, D))).cuda()
    kv, Hq, Hkv = [900, 70], 8, 2
    tab, n_pages = make_table(rng, kv, 64)
    cache, k, v = make_cache(S, rng, kv, tab, n_pages, Hkv, 64, D)
    q = bf(rng.normal(size=(2, Hq * D)))
    qd, lens, tabd, cu = q.cuda(), i32(kv), i32(tab), i32([0, 1, 2])
    ref, tol, written = A.attention(f64(q).reshape(2, Hq, D), k, v, [0, 1, 2], kv, tab)
    far_len, far_cu = i32([far]), i32([0, 1])
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    e0.record()
    S.attn_prefill(one, q1, far_cu, far_len, table, max_kv=1)
    o = S.attn_prefill(cache, qd, cu, lens, tabd)
    p = S.attn_decode(cache, qd, lens, tabd)
    e1.record()
    torch.cuda.synchronize()
    assert e0.elapsed_time(e1) > 1050.0, "the first kernel ended within the waits' limit: nothing is tested"
    assert S.device_error() == 0
    check(o, ref, tol, written, Hq, D)
    check(p, ref, tol, written, Hq, D)


def prefix_case(rng, kv, prefix, page, Hkv, D):
    """Table whose row 0 names every page of the prefix that any sequence uses."""
    table, n_pages = make_table(rng, kv, page, shared=prefix // page)
    far = int(np.argmax(kv))
    n = min(prefix // page, -(-kv[far] // page))
    table[0, :n] = table[far, :n]
    return table, n_pages


def has_own_pass(S, cache, B, Hq, cols, prefix):
    ws = [S._ws_bytes(cache, S.lib.serq_attn_decode_ws_bytes, B, Hq, cols, p, 0) for p in (0, prefix)]
    return ws[0] != ws[1]


# ----------------------------------------------------- what is not finite, and large
def cliff_cache(rng, kv, page, D, edge, nan_at):
    """One kv head: keys of score 0 up to `edge`, of 500 from there on (for a
    query of e_0 and a scale of 1), and a NaN key far in front."""
    table, n_pages = make_table(rng, [kv], page)
    k = np.zeros((n_pages, 1, page, D), np.float32)
    v = rng.normal(size=k.shape).astype(np.float32)
    for j in range(edge, kv):
        k[table[0, j // page], 0, j % page, 0] = 500.0
    for j in nan_at:
        k[table[0, j // page], 0, j % page, 3] = np.nan
    return table, k, v


@pytest.mark.parametrize("D,Hq,kv,rows", [(128, 1, 4000, 1), (64, 4, 2000, 20), (128, 1, 900, 300)])
def test_prefill_shows_nan_beside_much_larger_scores(S, D, Hq, kv, rows):
    """A NaN key whose part of the row, or whose step, weighs nothing beside a
    later one still shows, wherever in a step it lies."""
    page = 64
    for at in (0, 1, 2, 7, 8, 9, 64, 127, 130):
        rng = np.random.default_rng(106)
        table, k, v = cliff_cache(rng, kv, page, D, kv - rows - 60, [at])
        cache = S.KVCache(K=bf(k).cuda(), V=bf(v).cuda())
        q = np.zeros((rows, Hq, D), np.float32)
        q[:, :, 0] = 1.0
        for hint in (0, 1):  # cut into shares where few items are long, and whole
            o = S.attn_prefill(cache, bf(q.reshape(rows, -1)).cuda(), i32([0, rows]), i32([kv]), i32(table), scale=1.0,
                               max_kv=hint)
            assert not torch.isfinite(o.float()).any(), (at, hint)


def test_decode_shows_nan_beside_much_larger_scores(S):
    B, prefix, Hq, Hkv, D, page = 70, 8192, 2, 1, 128, 64
    for at in (0, 1, 5, 8192 - 16, 8192 - 1):
        rng = np.random.default_rng(107)
        kv = prefix + 100
        table, k, v = cliff_cache(rng, kv, page, D, prefix + 10, [at])
        full = np.repeat(table, B, 0)
        full[:, prefix // page:] = table[0, prefix // page:]
        cache = S.KVCache(K=bf(k).cuda(), V=bf(v).cuda())
        assert has_own_pass(S, cache, B, Hq, full.shape[1], prefix)
        q = np.zeros((B, Hq, D), np.float32)
        q[:, :, 0] = 1.0
        lens = i32([kv] * B)
        for p in (0, prefix):
            o = S.attn_decode(cache, bf(q.reshape(B, -1)).cuda(), lens, i32(full), prefix_len=p, scale=1.0)
            assert not torch.isfinite(o.float()).any(), (at, p)


@pytest.mark.parametrize("B,prefix,Hq,Hkv,D,own", [
    (2, 8192, 32, 32, 128, False),    # 52 us with the pass, 35 without
    (2, 4096, 32, 32, 128, False),    # 31, 20
    (4, 8192, 32, 8, 128, False),     # 23, 19
    (16, 8192, 32, 8, 128, True),     # 26, 53
    (32, 8192, 14, 2, 64, True),      # 18, 22
    (64, 8192, 32, 8, 128, True),     # 41, 188
])
def test_when_a_prefix_has_its_own_pass(S, B, prefix, Hq, Hkv, D, own):
    """Batches for which one way is faster by far: repeated reading, counted in
    bytes alone, does not tell them apart."""
    cache = S.KVCache(4, 64, Hkv, D)
    assert has_own_pass(S, cache, B, Hq, prefix // 64 + 8, prefix) == own


PREFIX_ENDS = [
    # batch, prefix, longest past it (negative: inside it), Hq, Hkv, D, page
    (40, 4112, 100, 8, 4, 128, 16),     # 16 keys in the last step of 128
    (33, 4000, 70, 6, 6, 64, 32),       # 32
    (20, 8256, 200, 14, 2, 128, 64),    # 64
    (6, 2160, 40, 60, 60, 64, 16),      # 112, and shares that begin and end inside them
    (24, 8192, -1191, 8, 2, 128, 64),   # the longest sequence ends inside the prefix, and inside a page
    (70, 2048, -1, 4, 4, 64, 256),
    (3, 33040, 1, 7, 7, 128, 16),
]


@pytest.mark.parametrize("B,prefix,past,Hq,Hkv,D,page", PREFIX_ENDS)
def test_prefix_pass_ends(S, B, prefix, past, Hq, Hkv, D, page):
    """Prefixes that end inside a step, lengths that end inside the prefix; NaN
    behind every sequence's last key."""
    rng = np.random.default_rng(prefix + B)
    top = prefix + past
    kv = [top - int(n) for n in rng.integers(0, max(1, abs(past)) + 300, size=B)]
    kv[B // 2] = top
    kv[0] = 5
    if B > 3:
        kv[1] = 0
    table, n_pages = prefix_case(rng, kv, prefix, page, Hkv, D)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    if table.shape[1] * page < prefix:  # the table holds the whole prefix, whatever the lengths
        wide = np.full((B, prefix // page), -7, np.int64)
        wide[:, :table.shape[1]] = table
        table = wide
    assert has_own_pass(S, cache, B, Hq, table.shape[1], prefix)
    q = bf(rng.normal(size=(B, Hq * D)) * 1.5)
    full = table.copy()
    full[:, :prefix // page] = table[0, :prefix // page]
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), kv, full)
    used = table.copy()
    used[1:, :prefix // page] = -5
    ws = S.attn_decode_ws(cache, B, Hq, table.shape[1], prefix)
    for fill in (float("nan"), 1e30):
        ws.view(torch.float32).fill_(fill)
        check(S.attn_decode(cache, q.cuda(), i32(kv), i32(used), prefix_len=prefix, ws=ws), ref, tol, written, Hq, D)
    assert S.device_error() == 0


@pytest.mark.parametrize("prefix", [0, 4096 + 48])
@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-0.2, 1.0), (1.0, 4.0), (-1.0, 4.0), (1e-3, 1.0)])
def test_decode_scales(S, scale, spread, prefix):
    """No scale, negative ones and logits of several hundred, with the prefix's
    own pass and without."""
    rng = np.random.default_rng(103)
    Hq, Hkv, D, page, B = 16, 4, 128, 16, 20
    kv = [prefix + int(n) for n in rng.integers(1, 300, size=B)]
    table, n_pages = prefix_case(rng, kv, prefix, page, Hkv, D)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D, spread=spread)
    assert has_own_pass(S, cache, B, Hq, table.shape[1], prefix) == (prefix > 0)
    q = bf(rng.normal(size=(B, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), kv, table, scale=scale)
    check(S.attn_decode(cache, q.cuda(), i32(kv), i32(table), prefix_len=prefix, scale=scale), ref, tol, written, Hq, D)


def test_sequences_longer_than_a_table_of_prefix_only(S):
    """A table that holds the prefix and nothing else: what it holds is attended
    to, and lengths beyond it are reported."""
    rng = np.random.default_rng(104)
    B, prefix, Hq, Hkv, D, page = 20, 8192, 8, 2, 128, 64
    kv = [prefix] * B
    table, n_pages = prefix_case(rng, kv, prefix, page, Hkv, D)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    assert has_own_pass(S, cache, B, Hq, table.shape[1], prefix)
    q = bf(rng.normal(size=(B, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), kv, table)
    for lens, code in ((kv, 0), ([prefix + 1] + kv[1:], 5), (kv[1:] + [prefix + 700], 5)):
        o = S.attn_decode(cache, q.cuda(), i32(lens), i32(table), prefix_len=prefix)
        assert S.device_error() == code
        check(o, ref, tol, written, Hq, D)


def test_tables_of_more_positions_than_32_bits_round(S):
    """2^31 - 16 positions: the last blocks of keys would end behind 2^31."""
    D, page = 128, 16
    cache, rope = S.KVCache(8, page, 2, D), S.Rope(D)
    q = torch.zeros((1, 4 * D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    cu, kv, tab = i32([0, 1]), i32([1]), i32([[0]])
    L, p, cols = S.lib, S._ptr, (1 << 27) - 1
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    assert L.serq_rope_append(rope.handle, cache.handle, p(q), 4 * D, p(q), 4 * D, p(q), 4 * D, 1, 4, None, None, 0.0, 1,
                              p(cu), p(kv), p(tab), cols, cols, p(out), 4 * D, None) == S.ERR_INVALID_ARG
    assert L.serq_attn_prefill(cache.handle, p(q), 4 * D, 1, 4, 1.0, 1, p(cu), p(kv), p(tab), cols, cols, 0, p(ws),
                               ws.numel(), p(out), 4 * D, None) == S.ERR_INVALID_ARG
    assert L.serq_attn_decode(cache.handle, p(q), 4 * D, 4, 1.0, 1, p(kv), p(tab), cols, cols, 0, 0, p(ws), ws.numel(),
                              p(out), 4 * D, None) == S.ERR_INVALID_ARG
    assert b"max_pages" in L.serq_last_error_string()
    torch.cuda.synchronize()
    assert bool((out == 5.0).all())


# ------------------------------------------------------------------ wide tables
@pytest.mark.parametrize("q_lens,past,Hq,Hkv,D,page", [
    ([33], [0], 8, 2, 128, 64),
    ([512], [0], 8, 2, 64, 16),
    ([700, 1, 90], [0, 2500, 33], 4, 4, 128, 128),
])
def test_tables_wider_than_the_sequences(S, q_lens, past, Hq, Hkv, D, page):
    """Tables as wide as a context limit, their unused entries invalid: the
    split differs, results do not."""
    rng = np.random.default_rng(105)
    kv = [a + b for a, b in zip(q_lens, past)]
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    T, B = int(cu[-1]), len(kv)
    table, n_pages = make_table(rng, kv, page)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    q, qd = bf(rng.normal(size=(T, Hq * D))), bf(rng.normal(size=(B, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(T, Hq, D), k, v, cu, kv, table)
    dref, dtol, dwritten = A.attention(f64(qd).reshape(B, Hq, D), k, v, range(B + 1), kv, table)
    for limit in (4096, 32768, 131072):
        wide = np.full((B, limit // page), -9, np.int64)
        wide[:, :table.shape[1]] = table
        for hint in (0, max(kv)):
            o = S.attn_prefill(cache, q.cuda(), i32(cu), i32(kv), i32(wide), max_kv=hint)
            check(o, ref, tol, written, Hq, D)
            o = S.attn_decode(cache, qd.cuda(), i32(kv), i32(wide), max_kv=hint)
            check(o, dref, dtol, dwritten, Hq, D)
    assert S.device_error() == 0


def test_one_sequence_a_little_above_one_item_per_sm(S):
    """One chunk whose tile pairs are a few more than the SMs, over a long
    context: their number is exact, and a second round for a few is not taken."""
    rng = np.random.default_rng(109)
    T, kv, Hq, Hkv, D, page = 301, 2600, 128, 1, 64, 64   # 151 pairs of two tokens
    table, n_pages = make_table(rng, [kv], page)
    cache, k, v = make_cache(S, rng, [kv], table, n_pages, Hkv, page, D)
    ws = S.attn_prefill_ws(cache, T, Hq, 1, table.shape[1])
    assert ws is not None
    ws.view(torch.float32).fill_(float("nan"))
    q = bf(rng.normal(size=(T, Hq * D)))
    o = S.attn_prefill(cache, q.cuda(), i32([0, T]), i32([kv]), i32(table), ws=ws)
    ref, tol, written = A.attention(f64(q).reshape(T, Hq, D), k, v, [0, T], [kv], table)
    check(o, ref, tol, written, Hq, D)
    assert S.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_large_values(S, D):
    """Values up to 2^63, with scores that rise so that weights are large while
    a row is summed."""
    rng = np.random.default_rng(108)
    page, kv, rows = 64, 3000, 140
    table, n_pages = make_table(rng, [kv], page)
    cache, k, v = make_cache(S, rng, [kv], table, n_pages, 1, page, D)
    for j in range(kv):
        k[table[0, j // page], 0, j % page] = 0.0
        k[table[0, j // page], 0, j % page, 0] = 22.0 * (j >= 128) + rng.uniform(0, 0.1)
    kt, vt = bf(k), bf(np.nan_to_num(v) * 2.0 ** 60)
    cache.K.copy_(kt), cache.V.copy_(vt)
    q = np.zeros((rows, 1, D), np.float32)
    q[:, :, 0] = 1.0
    ref, tol, written = A.attention(q.astype(np.float64), f64(kt), f64(vt), [0, rows], [kv], table, scale=1.0)
    for hint in (0, 1):
        o = S.attn_prefill(cache, bf(q.reshape(rows, -1)).cuda(), i32([0, rows]), i32([kv]), i32(table), scale=1.0,
                           max_kv=hint)
        check(o, ref, tol, written, 1, D)
    o = S.attn_decode(cache, bf(q[-1]).cuda(), i32([kv]), i32(table), scale=1.0)
    check(o, ref[-1:], tol[-1:], written[-1:], 1, D)


def test_a_cache_has_pages(S):
    with pytest.raises(ValueError, match="at least one page"):
        S.KVCache(0, 64, 2, 128)
    K = torch.empty((1, 65536, 16, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(S.SerqError):
        S.KVCache(K=K, V=K)


def test_workspace_shared_by_two_graphs_replayed_in_turn(S):
    """Two captured calls with one workspace, replayed in turn on one stream,
    with work that is cut and joined in both; the results are those of eager
    calls with workspaces of their own."""
    rng = np.random.default_rng(110)
    Hq, Hkv, D, page = 8, 2, 128, 64
    jobs = []
    for kv in ([3000, 400], [900, 2048]):
        table, n_pages = make_table(rng, kv, page)
        cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
        q = bf(rng.normal(size=(2, Hq * D))).cuda()
        jobs.append([cache, q, i32(kv), i32(table), i32([0, 1, 2])])

    def needs(j):
        cols = j[3].shape[1]
        return (S._ws_bytes(j[0], S.lib.serq_attn_prefill_ws_bytes, 2, Hq, 2, cols, 0),
                S._ws_bytes(j[0], S.lib.serq_attn_decode_ws_bytes, 2, Hq, cols, 0, 0))

    n = max(max(needs(j)) for j in jobs)
    assert min(min(needs(j)) for j in jobs) > 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN as floats
    want, graphs, outs = [], [], []
    for cache, q, lens, tab, cu in jobs:
        want.append((S.attn_prefill(cache, q, cu, lens, tab), S.attn_decode(cache, q, lens, tab)))
        o = [torch.empty_like(q) for _ in range(2)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.attn_prefill(cache, q, cu, lens, tab, O=o[0], ws=ws)
            S.attn_decode(cache, q, lens, tab, O=o[1], ws=ws)
        graphs.append(g)
        outs.append(o)
    for _ in range(10):
        for o in outs:
            o[0].fill_(7.0), o[1].fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (a, b), o in zip(want, outs):
            assert torch.equal(a, o[0]) and torch.equal(b, o[1])
    assert S.device_error() == 0


def test_items_longer_than_a_second(S):
    """A tile whose next item waits for the other tile's, which lasts longer
    than the waits' second."""
    rng = np.random.default_rng(111)
    D, page, far, H, n = 128, 256, 3 << 25, 150, 200   # two rounds of items; the first of one row, a tile's
    K, V = (bf(rng.normal(size=(2, H, page, D))).cuda() for _ in range(2))
    cache = S.KVCache(K=K, V=V)
    table = torch.zeros((2, far // page), dtype=torch.int32, device="cuda")
    table[1] = 1
    q = bf(rng.normal(size=(1 + n, H * D)))
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    e0.record()
    o = S.attn_prefill(cache, q.cuda(), i32([0, 1, 1 + n]), i32([far, n]), table, max_kv=1)
    e1.record()
    torch.cuda.synchronize()
    assert e0.elapsed_time(e1) > 2200.0, "two items last less than the waits' limit: nothing is tested"
    assert S.device_error() == 0
    ref, tol, written = A.attention(f64(q[1:]).reshape(n, H, D), f64(K), f64(V), [0, n], [n], np.array([[1]]))
    check(o[1:], ref, tol, written, H, D)

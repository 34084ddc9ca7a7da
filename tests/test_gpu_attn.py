"""GPU parity of the attention half of a decoder layer (rotation and append,
prompt attention, decode attention) against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from w4a4_rank_gemm_b200 import serq
    torch.cuda.set_device(0)
    serq.device_error()
    return serq


def bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def padded_rows(x, pad):
    """CUDA rows with a row stride `pad` elements above their length."""
    T, n = x.shape
    buf = torch.full((T, n + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, :n] = x.cuda()
    return buf[:, :n]


def make_table(rng, kv_lens, page, extra=1, shared=0):
    counts = [-(-n // page) for n in kv_lens]
    n_pages = shared + sum(max(0, c - shared) for c in counts) + extra
    perm = rng.permutation(n_pages)
    t = np.full((len(kv_lens), max([1] + counts)), -7, np.int64)
    at = shared
    for b, c in enumerate(counts):
        m = min(c, shared)
        t[b, :m] = perm[:m]
        t[b, m:c] = perm[at:at + c - m]
        at += c - m
    return t, n_pages


def make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D, spread=1.0, stride_pad=0):
    """Cache with random contents at the sequences' positions and NaN
    everywhere else."""
    k = np.full((n_pages, Hkv, page, D), np.nan, np.float32)
    v = k.copy()
    for b, n in enumerate(kv_lens):
        for j in range(0, n, page):
            m = min(page, n - j)
            pg = table[b, j // page]
            k[pg, :, :m] = spread * rng.normal(size=(Hkv, m, D))
            v[pg, :, :m] = rng.normal(size=(Hkv, m, D)) + 0.3
    tk, tv = bf(k), bf(v)
    if stride_pad:
        both = torch.full((n_pages, Hkv * page * D + stride_pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        vb = both.clone()
        K = both[:, :Hkv * page * D].view(n_pages, Hkv, page, D)
        V = vb[:, :Hkv * page * D].view(n_pages, Hkv, page, D)
        K.copy_(tk), V.copy_(tv)
    else:
        K, V = tk.cuda(), tv.cuda()
    return S.KVCache(K=K, V=V), f64(tk), f64(tv)


def check(o, ref, tol, written, Hq, D, fill=None):
    T = ref.shape[0]
    got = f64(o).reshape(T, Hq, D)
    err = np.abs(got - ref)
    bad = ~(err <= tol) & written[:, None, None]
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{bad.sum()} of {bad.size} outside the bound; first at {i}: {got[i]} for {ref[i]}, "
                             f"bound {tol[i]}")
    if fill is not None:
        assert np.all(got[~written] == fill)


# ------------------------------------------------------------- rotation, append
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot,page,Hq,Hkv,pad,scaling", [
    (128, 128, 64, 4, 4, 0, "none"),
    (128, 64, 16, 14, 2, 8, "by_parts"),
    (64, 64, 256, 3, 3, 64, "linear"),
    (64, 16, 32, 16, 1, 0, "by_parts"),
    (128, 112, 128, 8, 2, 0, "none"),
])
def test_rope_append(S, layout, norm, D, rot, page, Hq, Hkv, pad, scaling):
    rng = np.random.default_rng(D + rot + page)
    q_lens = [1, 0, 37, 5, 0, 130, 3]
    kv = [120001, 4, 37, 2, 0, 300, 3]  # the fourth sequence's first three rows lie before position 0
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    T = int(cu[-1]) + 2  # two rows behind the last sequence
    table, n_pages = make_table(rng, [min(n, 4 * page) for n in kv], page)
    wide = np.full((len(kv), 120001 // page + 1), -7, np.int64)
    wide[:, :table.shape[1]] = table
    wide[0, 120000 // page] = table[0, 0]
    q, k, v = (bf(rng.normal(size=(T, h * D)) * 2) for h in (Hq, Hkv, Hkv))
    qw, kw = bf(1 + 0.2 * rng.normal(size=D)), bf(1 + 0.2 * rng.normal(size=D))
    cK = torch.full((n_pages, Hkv, page, D), 77.0, dtype=torch.bfloat16, device="cuda")
    cV = torch.full_like(cK, 78.0)
    cache = S.KVCache(K=cK, V=cV)
    factor = 1.0 if scaling == "none" else 8.0
    amp = 1.2 if scaling == "by_parts" else 1.0
    rope = S.Rope(D, rot_dim=rot, layout=layout, theta=500000.0, scaling=scaling, factor=factor, amplitude=amp)
    qd, kd, vd = padded_rows(q, pad), padded_rows(k, pad), padded_rows(v, pad)
    out = torch.full((T, Hq * D + pad), 5.0, dtype=torch.bfloat16, device="cuda")[:, :Hq * D]
    kws = dict(q_weight=qw.cuda(), k_weight=kw.cuda(), eps=1e-5) if norm else {}
    S.rope_append(rope, cache, qd, kd, vd, i32(cu), i32(kv), i32(wide), Qout=out, **kws)
    torch.cuda.synchronize()
    code = S.device_error()

    freq = A.frequencies(rot, 500000.0, scaling, factor)
    held = A.rows(cu, kv)
    pos = np.zeros(T)
    for t, _, p in held:
        pos[t] = p

    def expect(x, H, w):
        x = f64(x).reshape(T, H, D)
        if norm:
            x = A.rms_norm(x, f64(w), 1e-5)
        y, mag = A.rotate(x, pos, freq, layout, amp)
        return y, A.rotate_bound(y, mag, norm)

    yq, tq = expect(q, Hq, qw)
    yk, tk = expect(k, Hkv, kw)
    written = np.zeros(T, bool)
    written[[t for t, _, _ in held]] = True
    check(out, yq, tq, written, Hq, D, fill=5.0)
    eK, eV = np.full(cK.shape, 77.0), np.full(cK.shape, 78.0)
    bound = np.zeros(cK.shape)
    stored = A.append(eK, eV, yk, f64(v).reshape(T, Hkv, D), cu, kv, wide)
    A.append(bound, bound.copy(), tk, tk, cu, kv, wide)
    assert np.all(np.abs(f64(cK) - eK) <= bound)
    assert np.array_equal(f64(cV), eV)
    # small pages: the table ends before the sixth sequence does, and the call says so
    assert code == (5 if len(stored) < len(held) else 0) and (code == 0) == (page >= 128)
    # in place
    S.rope_append(rope, cache, qd, kd, vd, i32(cu), i32(kv), i32(wide), Qout=qd, **kws)
    assert torch.equal(qd[torch.from_numpy(written).cuda()], out[torch.from_numpy(written).cuda()])
    assert torch.equal(qd[~torch.from_numpy(written).cuda()].cpu(), q[~torch.from_numpy(written)])
    S.device_error()


def test_rope_append_large_and_single(S):
    """Several tokens per block, and one."""
    rng = np.random.default_rng(3)
    D, Hq, Hkv, page = 128, 8, 2, 64
    for T, past in ((2503, 9), (1, 0)):
        cu, kv = [0, T], [T + past]
        table, n_pages = make_table(rng, kv, page)
        q, k, v = (bf(rng.normal(size=(T, h * D))) for h in (Hq, Hkv, Hkv))
        cache = S.KVCache(n_pages, page, Hkv, D)
        cache.K.zero_(), cache.V.zero_()
        out = S.rope_append(S.Rope(D), cache, q.cuda(), k.cuda(), v.cuda(), i32(cu), i32(kv), i32(table))
        pos = past + np.arange(T)
        y, mag = A.rotate(f64(q).reshape(T, Hq, D), pos, A.frequencies(D))
        check(out, y, A.rotate_bound(y, mag, False), np.ones(T, bool), Hq, D)
        y, mag = A.rotate(f64(k).reshape(T, Hkv, D), pos, A.frequencies(D))
        eK, eV, bound = (np.zeros(tuple(cache.K.shape)) for _ in range(3))
        A.append(eK, eV, y, f64(v).reshape(T, Hkv, D), cu, kv, table)
        A.append(bound, bound.copy(), A.rotate_bound(y, mag, False), y, cu, kv, table)
        assert np.all(np.abs(f64(cache.K) - eK) <= bound) and np.array_equal(f64(cache.V), eV)


# ------------------------------------------------------------------- prefill
PREFILL = [
    # q_lens, kv_lens, Hq, Hkv, D, page
    ([1], [1], 4, 4, 128, 64),
    ([33], [33], 8, 2, 128, 64),
    ([128], [128], 2, 2, 128, 16),
    ([129, 0, 1, 300, 17], [129, 5, 700, 300, 17], 8, 2, 128, 16),
    ([257, 64], [640, 64], 4, 4, 64, 128),
    ([5, 7, 3], [4, 0, 3], 6, 2, 128, 32),        # rows before position 0: empty rows
    ([200, 31], [333, 31], 14, 2, 64, 256),       # 7 query heads per key head
    ([70, 1], [700, 513], 16, 1, 128, 64),        # 16 per key head
    ([40], [1111], 3, 1, 128, 128),               # few rows over a long context
    ([9], [50], 128, 1, 64, 16),                  # the largest group
    ([2], [3], 129, 1 * 3, 128, 16),              # 43 per key head
    ([600], [600], 2, 1, 128, 64),
]


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page", PREFILL)
def test_prefill(S, q_lens, kv_lens, Hq, Hkv, D, page):
    rng = np.random.default_rng(sum(q_lens) + Hq + D)
    cu = np.concatenate([[0], np.cumsum(q_lens)]) + 1  # a row in front of the first sequence
    T = int(cu[-1]) + 3                                # and rows behind the last
    table, n_pages = make_table(rng, kv_lens, page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D, stride_pad=64 if page == 16 else 0)
    q = bf(rng.normal(size=(T, Hq * D)) * 1.5)
    qd = padded_rows(q, 24)
    out = torch.full((T, Hq * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")[:, :Hq * D]
    S.attn_prefill(cache, qd, i32(cu), i32(kv_lens), i32(table), O=out)
    torch.cuda.synchronize()
    assert S.device_error() == 0
    ref, tol, written = A.attention(f64(q).reshape(T, Hq, D), k, v, cu, kv_lens, table)
    check(out, ref, tol, written, Hq, D, fill=5.0)


@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-0.2, 1.0), (1.0, 4.0), (1e-3, 1.0)])
def test_prefill_scales(S, scale, spread):
    """No scale, a negative one, and logits of several hundred."""
    rng = np.random.default_rng(7)
    Hq, Hkv, D, page, n = 4, 2, 128, 64, 290
    table, n_pages = make_table(rng, [n], page)
    cache, k, v = make_cache(S, rng, [n], table, n_pages, Hkv, page, D, spread=spread)
    q = bf(rng.normal(size=(n, Hq * D)))
    out = S.attn_prefill(cache, q.cuda(), i32([0, n]), i32([n]), i32(table), scale=scale)
    ref, tol, written = A.attention(f64(q).reshape(n, Hq, D), k, v, [0, n], [n], table, scale=scale)
    check(out, ref, tol, written, Hq, D)


def test_prefill_growing_scores(S):
    """Every block of keys raises the running maximum by a lot, then by a little."""
    rng = np.random.default_rng(8)
    D, page, n = 128, 64, 640
    table, n_pages = make_table(rng, [n], page)
    cache, k, v = make_cache(S, rng, [n], table, n_pages, 1, page, D)
    grow = np.concatenate([np.linspace(-200, 200, n // 2), np.linspace(200, 206, n - n // 2)])
    for j in range(n):
        k[table[0, j // page], 0, j % page] = 0.0
        k[table[0, j // page], 0, j % page, 0] = grow[j]
    kt = bf(k)
    cache.K.copy_(kt)
    k = f64(kt)
    q = np.zeros((n, D), np.float32)
    q[:, 0] = 1.0
    out = S.attn_prefill(cache, bf(q).cuda(), i32([0, n]), i32([n]), i32(table), scale=1.0)
    ref, tol, written = A.attention(q.reshape(n, 1, D).astype(np.float64), k, v, [0, n], [n], table, scale=1.0)
    check(out, ref, tol, written, 1, D)


# -------------------------------------------------------------------- decode
DECODE = [
    # kv_lens, prefix, Hq, Hkv, D, page
    ([1], 0, 4, 4, 128, 64),
    ([5, 0, 64, 65, 1], 0, 8, 2, 128, 16),
    ([1000, 17, 333], 0, 8, 8, 128, 64),
    ([4097], 0, 8, 1, 64, 128),
    ([3001], 0, 4, 2, 128, 32),
    ([300, 299], 0, 14, 2, 64, 256),
    ([130, 7], 0, 48, 1, 128, 16),                 # 48 query heads per key head
    ([700, 513, 640, 512, 100, 0], 512, 8, 2, 128, 64),   # one ends at the prefix, one inside it, one is empty
    ([256 + 3, 256 + 90, 257], 256, 2, 2, 64, 16),
    ([2048 + i for i in range(33)], 2048, 8, 1, 128, 128),  # more rows than a tile
    ([512] * 3, 512, 4, 1, 128, 256),              # nothing but the prefix
]


@pytest.mark.parametrize("kv_lens,prefix,Hq,Hkv,D,page", DECODE)
def test_decode(S, kv_lens, prefix, Hq, Hkv, D, page):
    rng = np.random.default_rng(sum(kv_lens) + Hq + D)
    B = len(kv_lens)
    table, n_pages = make_table(rng, kv_lens, page, shared=prefix // page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D, stride_pad=64 if page == 16 else 0)
    q = bf(rng.normal(size=(B, Hq * D)) * 1.5)
    qd = padded_rows(q, 24)
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, np.arange(B + 1), kv_lens, table)
    used = table.copy()
    used[1:, :prefix // page] = -5  # only row 0 names the prefix's pages
    out = torch.full((B, Hq * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")[:, :Hq * D]
    S.attn_decode(cache, qd, i32(kv_lens), i32(used), prefix_len=prefix, O=out)
    torch.cuda.synchronize()
    assert S.device_error() == 0
    check(out, ref, tol, written, Hq, D)
    if prefix:  # and as if nothing were shared
        out2 = S.attn_decode(cache, qd, i32(kv_lens), i32(table))
        check(out2, ref, tol, written, Hq, D)


def test_results_repeat_and_follow_the_hint(S):
    """The same call gives the same bits; a hint that is too small or too
    large changes the split, not what is computed."""
    rng = np.random.default_rng(21)
    kv, Hq, Hkv, D, page = [2500, 40], 8, 2, 128, 64
    table, n_pages = make_table(rng, kv, page)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(2, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(2, Hq, D), k, v, [0, 1, 2], kv, table)
    for hint in (0, 1, 64, 100000):
        for f in (lambda: S.attn_decode(cache, q.cuda(), i32(kv), i32(table), max_kv=hint),
                  lambda: S.attn_prefill(cache, q.cuda(), i32([0, 1, 2]), i32(kv), i32(table), max_kv=hint)):
            o = f()
            check(o, ref, tol, written, Hq, D)
            assert torch.equal(o, f())


def test_invalid_pages_count_as_zeros_and_are_reported(S):
    rng = np.random.default_rng(22)
    kv, Hq, Hkv, D, page = [200, 150], 4, 2, 128, 16
    table, n_pages = make_table(rng, kv, page)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    bad = table.copy()
    bad[0, 3], bad[0, 12], bad[1, 9] = -1, n_pages, 2 ** 31 - 1
    q = bf(rng.normal(size=(2, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(2, Hq, D), k, v, [0, 1, 2], kv, bad)
    for f in (lambda: S.attn_decode(cache, q.cuda(), i32(kv), i32(bad)),
              lambda: S.attn_prefill(cache, q.cuda(), i32([0, 1, 2]), i32(kv), i32(bad))):
        o = f()
        assert S.device_error() == 5 and S.device_error() == 0
        check(o, ref, tol, written, Hq, D)
    # a sequence longer than its table: what the table holds is attended to
    ref, tol, written = A.attention(f64(q).reshape(2, Hq, D), k, v, [0, 1, 2], [200 + 500, 150], table[:, :9])
    long = i32([700, 144])
    ref2, tol2, _ = A.attention(f64(q).reshape(2, Hq, D), k, v, [0, 1, 2], [700, 144], table[:, :9])
    for f in (lambda: S.attn_decode(cache, q.cuda(), long, i32(table)[:, :9]),
              lambda: S.attn_prefill(cache, q.cuda(), i32([0, 1, 2]), long, i32(table)[:, :9])):
        o = f()
        assert S.device_error() == 5
        check(o, ref2, tol2, written, Hq, D)
    # the append leaves the cache alone where the page is invalid
    before = cache.K.clone()
    k2 = bf(rng.normal(size=(2, Hkv * D))).cuda()
    S.rope_append(S.Rope(D), cache, q.cuda(), k2, k2, i32([0, 1, 2]), i32([200, 2000]), i32(bad))
    assert S.device_error() == 5
    assert torch.equal(cache.K.view(torch.int16), before.view(torch.int16))


def test_prefix_pages_invalid(S):
    rng = np.random.default_rng(23)
    kv, Hq, Hkv, D, page = [300, 280, 257], 4, 2, 64, 64
    table, n_pages = make_table(rng, kv, page, shared=4)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    bad = table.copy()
    bad[:, 2] = n_pages + 3
    q = bf(rng.normal(size=(3, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(3, Hq, D), k, v, range(4), kv, bad)
    o = S.attn_decode(cache, q.cuda(), i32(kv), i32(bad), prefix_len=256)
    assert S.device_error() == 5
    check(o, ref, tol, written, Hq, D)


# ------------------------------------------------------- streams, graphs, a run
def test_graph_follows_changed_lengths(S):
    """A captured append and attention, replayed with other lengths, tables and rows."""
    rng = np.random.default_rng(31)
    Hq, Hkv, D, page, B = 8, 2, 128, 16, 3
    first, then = [200, 17, 90], [33, 260, 1]
    table, n_pages = make_table(rng, [max(a, b) for a, b in zip(first, then)], page)
    cache, k, v = make_cache(S, rng, first, table, n_pages, Hkv, page, D)
    rope = S.Rope(D)
    q, kn, vn = (bf(rng.normal(size=(B, h * D))).cuda() for h in (Hq, Hkv, Hkv))
    cu, kv_len, tab = i32([0, 1, 2, 3]), i32(first), i32(table)
    qr, o1, o2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    w1 = S.attn_prefill_ws(cache, B, Hq, B, tab.shape[1])
    w2 = S.attn_decode_ws(cache, B, Hq, tab.shape[1])

    def step():
        S.rope_append(rope, cache, q, kn, vn, cu, kv_len, tab, Qout=qr)
        S.attn_prefill(cache, qr, cu, kv_len, tab, O=o1, ws=w1)
        S.attn_decode(cache, qr, kv_len, tab, O=o2, ws=w2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in (first, then):
        cache2, k, v = make_cache(S, rng, lens, table, n_pages, Hkv, page, D)
        cache.K.copy_(cache2.K), cache.V.copy_(cache2.V)
        kv_len.copy_(i32(lens))
        q.copy_(bf(rng.normal(size=(B, Hq * D))))
        g.replay()
        torch.cuda.synchronize()
        ref, tol, written = A.attention(f64(qr).reshape(B, Hq, D), f64(cache.K), f64(cache.V), range(B + 1), lens,
                                        table)
        check(o1, ref, tol, written, Hq, D)
        check(o2, ref, tol, written, Hq, D)
    assert S.device_error() == 0


def test_other_stream(S):
    rng = np.random.default_rng(32)
    kv, Hq, Hkv, D, page = [1200, 7], 8, 2, 128, 64
    table, n_pages = make_table(rng, kv, page)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(2, Hq * D))).cuda()
    lens, tab = i32(kv), i32(table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = S.attn_decode(cache, q, lens, tab, stream=side)
    with torch.cuda.stream(side):
        p = S.attn_decode(cache, q, lens, tab)
    side.synchronize()
    ref, tol, written = A.attention(f64(q).reshape(2, Hq, D), k, v, range(3), kv, table)
    check(o, ref, tol, written, Hq, D)
    assert torch.equal(o, p)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2)])
def test_attention_half_of_a_layer(S, Hq, Hkv):
    """q/k/v linears -> rotation and append -> prompt attention -> o_proj's
    quantizer and linear, then one decode step; against the oracle at every
    stage, and the decode step against the prompt pass over all tokens."""
    rng = np.random.default_rng(41)
    D, page, r, n = 64, 16, 32, 75
    K, Nq, Nk = 256, Hq * D, Hkv * D
    W = [torch.from_numpy(rng.normal(0, 0.08, (K, m)).astype(np.float32)).cuda() for m in (Nq, Nk, Nk)]
    Xc = torch.from_numpy(rng.normal(0, 1, (64, K)).astype(np.float32)).cuda()
    qkv = S.prepare_group(W, Xc, r)
    Wo = torch.from_numpy(rng.normal(0, 0.08, (Nq, K)).astype(np.float32)).cuda()
    oproj = S.prepare(Wo, torch.from_numpy(rng.normal(0, 1, (64, Nq)).astype(np.float32)).cuda(), r)
    x = bf(rng.normal(size=(n, K))).cuda()
    rope = S.Rope(D)
    table, n_pages = make_table(rng, [n], page)
    tab = i32(table)

    def project(rows):
        xq, sx = S.quantize_act(S.flatten_permute(qkv[0], rows))
        return S.linear_group(qkv, xq, sx)

    def run(split):
        """Tokens [0, split) as a prompt, the rest one at a time."""
        cache = S.KVCache(n_pages, page, Hkv, D)
        cache.K.fill_(float("nan")), cache.V.fill_(float("nan"))
        q, k, v = project(x[:split])
        q = S.rope_append(rope, cache, q, k, v, i32([0, split]), i32([split]), tab)
        outs, qs = [S.attn_prefill(cache, q, i32([0, split]), i32([split]), tab)], [q]
        for t in range(split, n):
            q, k, v = project(x[t:t + 1])
            q = S.rope_append(rope, cache, q, k, v, i32([0, 1]), i32([t + 1]), tab)
            outs.append(S.attn_decode(cache, q, i32([t + 1]), tab))
            qs.append(q)
        o = torch.cat(outs)
        xq, sx = S.quantize_act(S.flatten_permute(oproj, o))
        return cache, torch.cat(qs), o, S.linear(oproj, xq, sx)

    for split in (n, n - 3):
        cache, q, o, y = run(split)
        ref, tol, written = A.attention(f64(q).reshape(n, Hq, D), np.nan_to_num(f64(cache.K)),
                                        np.nan_to_num(f64(cache.V)), [0, n], [n], table)
        check(o, ref, tol, written, Hq, D)
        assert torch.isfinite(y.float()).all()
        # the queries are the rotated projections
        raw = torch.cat([project(x[:split])[0]] + [project(x[t:t + 1])[0] for t in range(split, n)])
        yq, mag = A.rotate(f64(raw).reshape(n, Hq, D), np.arange(n), A.frequencies(D))
        check(q, yq, A.rotate_bound(yq, mag, False), np.ones(n, bool), Hq, D)
    assert S.device_error() == 0


# ---------------------------------------------------------------- refusals
def test_refusals(S):
    """Refused calls launch nothing and leave outputs untouched."""
    D, page = 128, 16
    cache = S.KVCache(8, page, 2, D)
    rope = S.Rope(D)
    q = torch.zeros((3, 4 * D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((3, 2 * D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    cu, kv, tab = i32([0, 3]), i32([3]), i32([[0, 1]])
    L, p = S.lib, S._ptr
    st = None

    def append(r=rope, c=cache, q=q, ldq=4 * D, k=k, ldk=2 * D, v=k, ldv=2 * D, T=3, H=4, qw=None, kw=None, eps=0.0, B=1,
               cu=cu, kv=kv, tab=tab, cols=2, ldt=2, o=out, ldo=4 * D):
        return L.serq_rope_append(r.handle, c.handle, p(q), ldq, p(k), ldk, p(v), ldv, T, H, p(qw), p(kw), eps, B, p(cu),
                                  p(kv), p(tab), cols, ldt, p(o), ldo, st)

    def prefill(q=q, ldq=4 * D, T=3, H=4, scale=1.0, B=1, cu=cu, kv=kv, tab=tab, cols=2, ldt=2, mk=0, o=out, ldo=4 * D):
        return L.serq_attn_prefill(cache.handle, p(q), ldq, T, H, scale, B, p(cu), p(kv), p(tab), cols, ldt, mk, None, 0,
                                   p(o), ldo, st)

    def decode(q=q, ldq=4 * D, H=4, scale=1.0, B=1, kv=kv, tab=tab, cols=2, ldt=2, prefix=0, mk=0, ws=None, wb=0, o=out,
               ldo=4 * D):
        return L.serq_attn_decode(cache.handle, p(q), ldq, H, scale, B, p(kv), p(tab), cols, ldt, prefix, mk, p(ws), wb,
                                  p(o), ldo, st)

    bad, shape = S.ERR_INVALID_ARG, S.ERR_UNSUPPORTED_SHAPE
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    for f in (append, prefill, decode):
        for kw, want in ((dict(H=3), shape), (dict(H=0), shape), (dict(H=258), shape), (dict(ldq=4 * D - 8), bad),
                         (dict(ldq=4 * D + 4), bad), (dict(ldo=4 * D - 8), bad), (dict(q=None), bad), (dict(o=None), bad),
                         (dict(B=0), bad), (dict(kv=None), bad), (dict(tab=None), bad), (dict(cols=0), bad),
                         (dict(ldt=1), bad), (dict(cols=1 << 28, ldt=1 << 28), bad)):
            assert f(**kw) == want, (f, kw)
    for kw in (dict(T=0), dict(cu=None), dict(k=None), dict(v=None), dict(ldk=2 * D - 8), dict(ldv=2 * D + 1),
               dict(qw=w), dict(kw=w), dict(qw=w, kw=w, eps=-1.0), dict(qw=w, kw=w, eps=float("nan"))):
        assert append(**kw) == bad, kw
    assert append(r=S.Rope(64)) == shape
    for kw in (dict(T=0), dict(cu=None), dict(scale=float("inf")), dict(scale=float("nan")), dict(mk=-1)):
        assert prefill(**kw) == bad, kw
    for kw in (dict(scale=float("nan")), dict(prefix=-16), dict(prefix=8), dict(prefix=48), dict(mk=-1)):
        assert decode(**kw) == bad, kw
    torch.cuda.synchronize()
    assert bool((out == 5.0).all())
    # the binding's own checks
    for f in (lambda: S.attn_decode(cache, q.float(), i32([1, 1, 1]), i32([[0]] * 3)),
              lambda: S.attn_decode(cache, q, kv, tab),
              lambda: S.attn_decode(cache, q[:1, :100], kv, tab),
              lambda: S.attn_prefill(cache, q, cu, kv.long(), tab),
              lambda: S.attn_prefill(cache, q, cu[:1], kv, tab),
              lambda: S.attn_prefill(cache, q, cu, kv, tab, O=out[:2]),
              lambda: S.rope_append(rope, cache, q, k[:, :D], k, cu, kv, tab),
              lambda: S.rope_append(rope, cache, q, k[:2], k, cu, kv, tab),
              lambda: S.rope_append(rope, cache, q, k, k, cu, kv, tab, q_weight=w.float(), k_weight=w),
              lambda: S.KVCache(K=k, V=k),
              lambda: S.KVCache(K=cache.K)):
        with pytest.raises(ValueError):
            f()


# ------------------------------------------------------------ harder batches
def test_many_sequences(S):
    """More sequences than a warp has lanes, some empty; every kind of split."""
    rng = np.random.default_rng(51)
    Hq, Hkv, D, page = 4, 2, 64, 16
    q_lens = [int(n) for n in rng.choice([0, 1, 2, 40, 70], size=71)]
    kv_lens = [n + int(rng.integers(0, 90)) if n or rng.random() < 0.5 else 0 for n in q_lens]
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    T = int(cu[-1])
    table, n_pages = make_table(rng, kv_lens, page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(T, Hq * D)))
    o = S.attn_prefill(cache, q.cuda(), i32(cu), i32(kv_lens), i32(table))
    ref, tol, written = A.attention(f64(q).reshape(T, Hq, D), k, v, cu, kv_lens, table)
    check(o, ref, tol, written, Hq, D)
    B = len(kv_lens)
    q = bf(rng.normal(size=(B, Hq * D)))
    o = S.attn_decode(cache, q.cuda(), i32(kv_lens), i32(table))
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), kv_lens, table)
    check(o, ref, tol, written, Hq, D)
    assert S.device_error() == 0


@pytest.mark.parametrize("q_lens,past,Hq,Hkv,D,page", [
    ([300, 5, 0, 90], [2000, 1500, 9, 0], 2, 1, 128, 64),   # few tile pairs: shares that cut items, one head
    ([100], [3000], 8, 2, 64, 128),
    ([17, 33], [4000, 10], 14, 2, 128, 16),
    ([130], [1000], 2, 2, 128, 256),
])
def test_prefill_shares(S, q_lens, past, Hq, Hkv, D, page):
    """Work cut into equal shares; the workspace holds NaN before the call."""
    rng = np.random.default_rng(sum(q_lens) + D)
    kv_lens = [a + b for a, b in zip(q_lens, past)]
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    T = int(cu[-1])
    table, n_pages = make_table(rng, kv_lens, page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(T, Hq * D)) * 1.5)
    ws = S.attn_prefill_ws(cache, T, Hq, len(kv_lens), table.shape[1])
    assert ws is not None
    ws.view(torch.float32).fill_(float("nan"))
    o = S.attn_prefill(cache, q.cuda(), i32(cu), i32(kv_lens), i32(table), ws=ws)
    ref, tol, written = A.attention(f64(q).reshape(T, Hq, D), k, v, cu, kv_lens, table)
    check(o, ref, tol, written, Hq, D)
    with pytest.raises(S.SerqError) as e:
        S.attn_prefill(cache, q.cuda(), i32(cu), i32(kv_lens), i32(table), ws=ws[:-16])
    assert e.value.status == S.ERR_INVALID_ARG and "workspace" in str(e.value)
    assert S.device_error() == 0


def test_decode_workspace_is_written_before_it_is_read(S):
    rng = np.random.default_rng(53)
    kv_lens, prefix, Hq, Hkv, D, page = [1024 + n for n in (0, 1, 700, 64, 5)], 1024, 8, 2, 128, 64
    table, n_pages = make_table(rng, kv_lens, page, shared=prefix // page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(5, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(5, Hq, D), k, v, range(6), kv_lens, table)
    for p in (0, prefix):
        ws = S.attn_decode_ws(cache, 5, Hq, table.shape[1], p)
        for fill in (float("nan"), 1e30):
            ws.view(torch.float32).fill_(fill)
            o = S.attn_decode(cache, q.cuda(), i32(kv_lens), i32(table), prefix_len=p, ws=ws)
            check(o, ref, tol, written, Hq, D)


def test_two_streams_with_a_workspace_each(S):
    rng = np.random.default_rng(54)
    Hq, Hkv, D, page = 8, 2, 128, 64
    jobs = []
    for kv in ([3000, 10], [77, 2048]):
        table, n_pages = make_table(rng, kv, page)
        cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
        q = bf(rng.normal(size=(2, Hq * D)))
        ref = A.attention(f64(q).reshape(2, Hq, D), k, v, range(3), kv, table)
        jobs.append((cache, q.cuda(), i32(kv), i32(table), S.attn_decode_ws(cache, 2, Hq, table.shape[1]), ref,
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (cache, q, kv, tab, ws, ref, st) in enumerate(jobs):
            with torch.cuda.stream(st):
                outs[i].append(S.attn_decode(cache, q, kv, tab, ws=ws))
                outs[i].append(S.attn_prefill(cache, q, i32([0, 1, 2]), kv, tab))
    torch.cuda.synchronize()
    for (cache, q, kv, tab, ws, (r, tol, written), st), os_ in zip(jobs, outs):
        for o in os_:
            check(o, r, tol, written, Hq, D)


def test_offsets_beyond_32_bits(S):
    """Pages far apart: element offsets of the cache pass 2^31."""
    rng = np.random.default_rng(55)
    Hq, Hkv, D, page, stride, n_pages = 4, 2, 128, 64, 1 << 29, 6
    raw = [torch.empty((n_pages - 1) * stride + Hkv * page * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    K, V = (t.as_strided((n_pages, Hkv, page, D), (stride, page * D, D, 1)) for t in raw)
    K.fill_(float("nan")), V.fill_(float("nan"))
    cache = S.KVCache(K=K, V=V)
    kv, table = [6 * page - 3], np.array([[5, 0, 4, 2, 3, 1]])
    T = kv[0]
    q, k, v = (bf(rng.normal(size=(T, h * D))) for h in (Hq, Hkv, Hkv))
    out = S.rope_append(S.Rope(D), cache, q.cuda(), k.cuda(), v.cuda(), i32([0, T]), i32(kv), i32(table))
    o = S.attn_prefill(cache, out, i32([0, T]), i32(kv), i32(table))
    od = S.attn_decode(cache, out[-1:], i32(kv), i32(table))
    yk, mag = A.rotate(f64(k).reshape(T, Hkv, D), np.arange(T), A.frequencies(D))
    ck, cv = f64(cache.K), f64(cache.V)
    for t in range(T):
        assert np.all(np.abs(ck[table[0, t // page], :, t % page] - yk[t]) <= A.rotate_bound(yk[t], mag[t], False))
    ref, tol, written = A.attention(f64(out).reshape(T, Hq, D), np.nan_to_num(ck), np.nan_to_num(cv), [0, T], kv, table)
    check(o, ref, tol, written, Hq, D)
    check(od, ref[-1:], tol[-1:], written[-1:], Hq, D)
    assert S.device_error() == 0


def test_infinite_and_nan_outside_the_batch(S):
    """Rows of Q outside the batch and cache slots behind the sequences hold
    NaN and infinities; results do not see them."""
    rng = np.random.default_rng(56)
    Hq, Hkv, D, page = 4, 4, 128, 32
    q_lens, kv_lens = [50, 3], [170, 35]
    cu = np.concatenate([[0], np.cumsum(q_lens)]) + 2
    T = int(cu[-1]) + 80
    table, n_pages = make_table(rng, kv_lens, page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D)
    cache.V[torch.isnan(cache.V)] = float("inf")
    cache.K[torch.isnan(cache.K)] = float("-inf")
    q = bf(rng.normal(size=(T, Hq * D)))
    qd = q.cuda()
    qd[:2], qd[int(cu[-1]):] = float("nan"), float("inf")
    o = torch.full_like(qd, 5.0)
    S.attn_prefill(cache, qd, i32(cu), i32(kv_lens), i32(table), O=o)
    ref, tol, written = A.attention(f64(q).reshape(T, Hq, D), k, v, cu, kv_lens, table)
    check(o, ref, tol, written, Hq, D, fill=5.0)


@pytest.mark.parametrize("shape", ["rising", "falling", "jumps", "flat_then_cliff"])
@pytest.mark.parametrize("D,Hq", [(128, 1), (64, 2)])
def test_long_contexts_whose_scores_move(S, shape, D, Hq):
    """More than 2048 keys, where most steps do without a look at the maximum:
    scores that rise and fall by far more than the weights' range allows."""
    rng = np.random.default_rng(61)
    page, n, kv = 64, 150, 2700
    table, n_pages = make_table(rng, [kv], page)
    cache, k, v = make_cache(S, rng, [kv], table, n_pages, 1, page, D)
    at = np.arange(kv)
    grow = {"rising": -300 + 0.23 * at, "falling": 300 - 0.23 * at,
            "jumps": 45.0 * (at // 300) + rng.normal(size=kv), "flat_then_cliff": np.where(at < 2400, 0.0, 500.0)}[shape]
    for j in range(kv):
        k[table[0, j // page], 0, j % page] = 0.0
        k[table[0, j // page], 0, j % page, 0] = grow[j]
    kt = bf(k)
    cache.K.copy_(kt)
    k = f64(kt)
    q = np.zeros((n, Hq, D), np.float32)
    q[:, :, 0] = 1.0
    q[1::3, :, 0] = -1.0  # some rows see the mirror image
    q[2::3, :, 0] = 0.125
    cu = [0, n]
    out = S.attn_prefill(cache, bf(q.reshape(n, -1)).cuda(), i32(cu), i32([kv]), i32(table), scale=1.0)
    ref, tol, written = A.attention(q.astype(np.float64), k, v, cu, [kv], table, scale=1.0)
    check(out, ref, tol, written, Hq, D)


LONG_PREFIX = [
    # batch, prefix, Hq, Hkv, D, page: repeated reads far above what makes the prefix's own pass pay
    (40, 4096, 8, 4, 128, 64),
    (70, 8192, 16, 2, 64, 256),    # 560 rows per key head: three tile pairs
    (3, 32768, 14, 7, 128, 16),
    (36, 4096, 96, 4, 128, 128),   # 24 query heads per key head
]


def long_prefix_case(S, B, prefix, Hq, Hkv, D, page, seed):
    rng = np.random.default_rng(seed)
    kv = [prefix + int(n) for n in rng.integers(0, 3 * page, size=B)]
    kv[1 % B], kv[2 % B] = prefix, prefix + 1     # nothing of its own; one key
    if B > 5:
        kv[3], kv[4] = prefix - 100, 0            # ends inside the prefix; empty
    table, n_pages = make_table(rng, kv, page, shared=prefix // page)
    cache, k, v = make_cache(S, rng, kv, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(B, Hq * D)) * 1.5)
    return rng, kv, table, n_pages, cache, k, v, q


@pytest.mark.parametrize("B,prefix,Hq,Hkv,D,page", LONG_PREFIX)
def test_decode_long_prefix(S, B, prefix, Hq, Hkv, D, page):
    rng, kv, table, n_pages, cache, k, v, q = long_prefix_case(S, B, prefix, Hq, Hkv, D, page, B + D)
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), kv, table)
    used = table.copy()
    used[1:, :prefix // page] = -5  # only row 0 names the prefix's pages
    ws = S.attn_decode_ws(cache, B, Hq, table.shape[1], prefix)
    outs = []
    for fill in (float("nan"), 1e30):
        ws.view(torch.float32).fill_(fill)
        outs.append(S.attn_decode(cache, q.cuda(), i32(kv), i32(used), prefix_len=prefix, ws=ws))
        check(outs[-1], ref, tol, written, Hq, D)
    assert torch.equal(*outs)
    assert S.device_error() == 0
    check(S.attn_decode(cache, q.cuda(), i32(kv), i32(table)), ref, tol, written, Hq, D)


def test_decode_long_prefix_graph_and_invalid_pages(S):
    B, prefix, Hq, Hkv, D, page = 40, 4096, 8, 4, 128, 64
    rng, kv, table, n_pages, cache, k, v, q = long_prefix_case(S, B, prefix, Hq, Hkv, D, page, 71)
    qd, lens, tab = q.cuda(), i32(kv), i32(table)
    ws = S.attn_decode_ws(cache, B, Hq, table.shape[1], prefix)
    out = torch.empty_like(qd)
    S.attn_decode(cache, qd, lens, tab, prefix_len=prefix, O=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.attn_decode(cache, qd, lens, tab, prefix_len=prefix, O=out, ws=ws)
    shorter = [max(0, n - int(rng.integers(0, 80))) for n in kv]
    for lengths in (kv, shorter, [0] * B, kv):
        lens.copy_(i32(lengths))
        out.fill_(7.0)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), lengths, table)
        check(out, ref, tol, written, Hq, D)
    assert S.device_error() == 0
    bad = table.copy()
    bad[:, 7] = n_pages + 3
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), kv, bad)
    o = S.attn_decode(cache, qd, i32(kv), i32(bad), prefix_len=prefix)
    assert S.device_error() == 5
    check(o, ref, tol, written, Hq, D)


NONFINITE = [  # q_lens, tokens before, Hq, Hkv, D, page
    ([40, 300], [0, 0], 4, 4, 128, 32),      # whole items
    ([64, 3], [4000, 900], 8, 2, 128, 16),   # cut ones, past 2048 keys
    ([200, 5], [2300, 0], 2, 2, 64, 64),
]


@pytest.mark.parametrize("where", ["query", "key", "value"])
@pytest.mark.parametrize("q_lens,past,Hq,Hkv,D,page", NONFINITE)
def test_prefill_shows_nan(S, where, q_lens, past, Hq, Hkv, D, page):
    """A NaN in a query, or in a key or value that a row sees, is in its result,
    and nowhere in the other sequence's."""
    rng = np.random.default_rng(81)
    kv_lens = [a + b for a, b in zip(q_lens, past)]
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    T = int(cu[-1])
    table, n_pages = make_table(rng, kv_lens, page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(T, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(T, Hq, D), k, v, cu, kv_lens, table)
    qd, group = q.cuda(), Hq // Hkv
    for key in (past[0], past[0] + 1, past[0] + 6):
        hit = np.zeros((T, Hq), bool)      # rows that have to show it
        free = np.ones((T, Hq), bool)      # rows that may not
        t = key - past[0]
        if where == "query":
            old = qd[t, D:2 * D].clone()
            qd[t, D:2 * D] = float("nan")
            hit[t, 1] = True
            free = ~hit
        else:
            at = (cache.K if where == "key" else cache.V)[table[0, key // page], 0, key % page]
            old = at.clone()
            at[3] = float("nan")
            hit[t:q_lens[0], :group] = True
            free[(0 if where == "value" else t):q_lens[0], :group] = False
        got = f64(S.attn_prefill(cache, qd, i32(cu), i32(kv_lens), i32(table))).reshape(T, Hq, D)
        bad = ~np.isfinite(got)
        assert np.all(bad[hit][:, 3] if where == "value" else bad[hit])
        assert np.all(np.abs(got - ref)[free] <= tol[free])
        if where == "query":
            qd[t, D:2 * D] = old
        else:
            at.copy_(old)


@pytest.mark.parametrize("where", ["query", "key", "value"])
@pytest.mark.parametrize("kv_lens,prefix,Hq,Hkv,D,page", [
    ([40, 64, 7000], 0, 4, 4, 128, 32),
    ([300 + 11 * i for i in range(40)], 0, 8, 2, 64, 16),
    ([4096 + 37 * i for i in range(40)], 4096, 8, 4, 128, 64),
])
def test_decode_shows_nan(S, where, kv_lens, prefix, Hq, Hkv, D, page):
    rng = np.random.default_rng(82)
    B = len(kv_lens)
    table, n_pages = make_table(rng, kv_lens, page, shared=prefix // page)
    cache, k, v = make_cache(S, rng, kv_lens, table, n_pages, Hkv, page, D)
    q = bf(rng.normal(size=(B, Hq * D)))
    ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), kv_lens, table)
    qd, group = q.cuda(), Hq // Hkv
    for b in (1, B - 1):
        for key in {prefix, kv_lens[b] - 1} - {kv_lens[b]}:
            hit = np.zeros((B, Hq), bool)
            if where == "query":
                old = qd[b, D:2 * D].clone()
                qd[b, D:2 * D] = float("nan")
                hit[b, 1] = True
            else:
                at = (cache.K if where == "key" else cache.V)[table[b, key // page], 0, key % page]
                old = at.clone()
                at[3] = float("nan")
                hit[b, :group] = True
            o = S.attn_decode(cache, qd, i32(kv_lens), i32(table), prefix_len=prefix)
            got = f64(o).reshape(B, Hq, D)
            bad = ~np.isfinite(got)
            assert np.all(bad[hit][:, 3] if where == "value" else bad[hit])
            assert np.all(np.abs(got - ref)[~hit] <= tol[~hit])
            if where == "query":
                qd[b, D:2 * D] = old
            else:
                at.copy_(old)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 4, 128, 64), (40, 2, 64, 16)])
def test_decode_cuts_at_every_block(S, Hq, Hkv, D, page):
    """Lengths of 0 to a few blocks beside long ones: shares begin inside a
    pair, at its first block and behind its last one."""
    rng = np.random.default_rng(91)
    for lens in ([1] * 200, list(range(60, 70)) * 9, [0, 64, 0, 128, 1] * 12 + [4000],
                 [int(n) for n in rng.integers(0, 400, size=77)], [20000, 1, 1], [193]):
        table, n_pages = make_table(rng, lens, page)
        cache, k, v = make_cache(S, rng, lens, table, n_pages, Hkv, page, D)
        B = len(lens)
        q = bf(rng.normal(size=(B, Hq * D)))
        ref, tol, written = A.attention(f64(q).reshape(B, Hq, D), k, v, range(B + 1), lens, table)
        ws = S.attn_decode_ws(cache, B, Hq, table.shape[1])
        ws.view(torch.float32).fill_(float("nan"))
        check(S.attn_decode(cache, q.cuda(), i32(lens), i32(table), ws=ws), ref, tol, written, Hq, D)
    assert S.device_error() == 0

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

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

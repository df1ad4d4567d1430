"""Infinities in the open block's V rows, which are attended over in bf16 as they came: an infinity
with a weight above zero makes its column infinite, two of opposite signs NaN, and the other columns
stay as they are.  (In a completed block an infinity is held as NaN.)"""

import numpy as np
import pytest
import torch

from parity import f64
from test_gpu_kv8 import close, dev, filled, rnd

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("D,G,n", [(128, 1, 20), (128, 4, 150), (64, 2, 100), (64, 8, 63), (128, 8, 700), (64, 1, 1)])
def test_infinite_values_in_the_open_block(kvc, D, G, n):
    H = 3
    cache, orc = filled(kvc, 1, 1, H, D, 1024, torch.full((1, 1, H), n, dtype=torch.int32), 5)
    t = n % 64 - 1
    cache.v_tail[0, 0, 0, t, 2] = INF
    cache.v_tail[0, 0, 0, 0, 5] = -INF
    cache.v_tail[0, 0, 2, t, 7] = INF
    kn, vn = rnd((1, 1, H, D), 6, boost=False), rnd((1, 1, H, D), 7, boost=False)
    vn[0, 0, 1, D - 1] = -INF
    vn[0, 0, 2, 7] = -INF
    q = rnd((1, 1, H * G, D), 8, boost=False)
    # without the new row, then with it
    for new in (False, True):
        kw = dict(k_new=kn.cuda(), v_new=vn.cuda()) if new else {}
        out = f64(kvc.kv8_decode_attn(q.cuda(), cache, **kw))[0, 0].reshape(H, G, D)
        want = {0: {2: INF, 5: -INF}, 1: {}, 2: {7: INF}}
        if new:
            want[1][D - 1] = -INF
            want[2][7] = float("nan")
        for h in range(H):
            for c, x in want[h].items():
                assert np.array_equal(out[h, :, c], np.full(G, x), equal_nan=True), (new, h, c)
            rest = [c for c in range(D) if c not in want[h]]
            rk, rv = (u.read().copy() for u in orc[(0, 0, h)])
            if new:
                rk, rv = np.concatenate([rk, f64(kn[0, 0, h])[None]]), np.concatenate([rv, f64(vn[0, 0, h])[None]])
            rv[:, [c for c in range(D) if c in want[h]]] = 0
            x = out[h].copy()
            x[:, [c for c in range(D) if c in want[h]]] = 0
            assert np.isfinite(out[h][:, rest]).all()
            close(x, f64(q)[0, 0, h * G:h * G + G], rk, rv)
    assert kvc.kvc_device_status() == 0

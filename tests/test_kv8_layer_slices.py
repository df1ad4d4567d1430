"""One layer's slice of a stacked 8-bit cache is a cache: its scales begin at any multiple of 4 bytes."""

import pytest
import torch

from test_gpu_kv8 import BF, dev, rnd
from test_kv8_refusals import A, ALIGN, EVERY, UNSUPPORTED, cache

NAMES = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "n_valid", "pos", "k_last", "v_last", "blocks")


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: host checks only")
@pytest.mark.parametrize("call", EVERY)
def test_scales_need_four_bytes(call):
    for off in (4, 8, 12, 24):
        assert call(c=cache(k_scale=A + off, v_scale=A + 16 + off)) == UNSUPPORTED
    for off in (1, 2, 6):
        assert call(c=cache(k_scale=A + off)) == ALIGN and call(c=cache(v_scale=A + off)) == ALIGN


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,D,cap", [(1, 2, 128, 192), (1, 1, 64, 64), (3, 1, 128, 320)])
def test_calls_on_one_layer(kvc, B, H, D, cap):
    """Every call, layer by layer on slices, against the same calls on the whole cache."""
    Ly, L, m = 5, cap - 20, 9
    whole, parts = kvc.KV8Cache(Ly, B, H, D, cap), kvc.KV8Cache(Ly, B, H, D, cap)
    layers = [kvc.KV8Cache.from_tensors(**{n: getattr(parts, n)[i:i + 1] for n in NAMES}) for i in range(Ly)]
    assert any(x.k_scale.data_ptr() % 16 for x in layers)
    u = (Ly, B, H)
    k, v, a, b = dev(rnd(u + (L, D), 1), rnd(u + (L, D), 2), rnd(u + (m, D), 3), rnd(u + (m, D), 4))
    q = rnd((Ly, B, 3 * H, D), 5, boost=False).cuda()
    votes = torch.rand(u + (L,), generator=torch.Generator().manual_seed(1)).cuda()
    kw = dict(keep_window=4, pool_kernel=7, budget=min(L - 1, 100))

    def every(c, s):
        kvc.snapkv_select_kv8(votes[s], k[s], v[s], c, **kw)
        got = [kvc.kv8_decode_attn(q[s], c)]
        kvc.kv8_write(k[s], v[s], c)
        kvc.kv8_append(a[s], b[s], c, new_pos=L)
        for t in range(9):
            got.append(kvc.kv8_decode_attn(q[s], c, k_new=a[s][..., t, :].contiguous(), v_new=b[s][..., t, :].contiguous(),
                                           new_pos=L + m + t))
        return got + list(kvc.kv8_read(c))

    want = every(whole, slice(None))
    for i, c in enumerate(layers):
        for x, y in zip(every(c, slice(i, i + 1)), want):
            assert torch.equal(x.view(torch.int16), y[i:i + 1].view(torch.int16))
    for n in NAMES[:8]:
        x, y = getattr(parts, n), getattr(whole, n)
        t = torch.int16 if x.dtype is BF else torch.int32 if x.element_size() == 4 else torch.uint8
        assert torch.equal(x.view(t), y.view(t)), n
    assert kvc.kvc_device_status() == 0

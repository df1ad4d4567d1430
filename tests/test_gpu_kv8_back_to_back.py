"""Calls on one cache issued back to back, so that each is launched while the one before still runs:
what they give is, bit for bit, what the same calls give with the GPU waited for in between."""

import pytest
import torch

from test_gpu_kv8 import dev, poison, rnd
from test_gpu_kv8_rollback import same, state

pytestmark = pytest.mark.gpu


def pair(kvc, shape, D, cap, n, seed):
    k, v = dev(rnd(shape + (max(int(n.max()), 1), D), seed), rnd(shape + (max(int(n.max()), 1), D), seed + 1))
    return [kvc.kv8_write(k, v, poison(kvc.KV8Cache(*shape, D, cap)), lengths=n.cuda()) for _ in range(2)]


def steps(shape, D, G, T, seed):
    return dev(rnd((T, shape[0], shape[1], shape[2] * G, D), seed, boost=False), rnd((T,) + shape + (D,), seed + 1, boost=False),
               rnd((T,) + shape + (D,), seed + 2, boost=False))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("shape,D,G", [((1, 1, 1), 128, 1), ((1, 2, 8), 128, 4), ((2, 4, 40), 64, 8), ((1, 3, 5), 64, 2)], ids=str)
def test_steps(kvc, shape, D, G, graph):
    """200 steps: every unit's open block fills three times."""
    T, cap = 200, 1024
    n = torch.randint(0, 600, shape, generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    n.view(-1)[0] = 63
    one, two = pair(kvc, shape, D, cap, n, 1)
    q, kn, vn = steps(shape, D, G, T, 3)
    outs = torch.empty_like(q)

    def run(c, out, wait):
        for t in range(T):
            kvc.kv8_decode_attn(q[t], c, k_new=kn[t], v_new=vn[t], new_pos=t, out=out[t])
            if wait:
                torch.cuda.synchronize()

    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(one, outs, False)
        g.replay()
    else:
        run(one, outs, False)
    want = torch.empty_like(q)
    run(two, want, True)
    assert torch.equal(outs.view(torch.int16), want.view(torch.int16))
    same(state(one), state(two))
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_every_call_behind_every_other(kvc, D):
    """Writes, appends, steps, reads and selections in a row, each reading what the one before wrote:
    outputs as the next call's rows, read rows written again, counts lowered in between."""
    shape, cap, G, L = (1, 2, 4), 512, 2, 300
    n = torch.tensor([0, 63, 64, 100, 127, 200, 255, 1], dtype=torch.int32).view(shape)
    one, two = pair(kvc, shape, D, cap, n, 11)
    a, b = dev(rnd(shape + (70, D), 21), rnd(shape + (70, D), 22))
    votes = torch.rand(shape + (L,), generator=torch.Generator().manual_seed(7)).cuda()
    q, kn, vn = steps(shape, D, G, 1, 31)

    def turn(c, wait):
        got = []
        hold = (lambda: torch.cuda.synchronize()) if wait else (lambda: None)
        for t in range(6):
            kvc.kv8_append(a, b, c, new_pos=t)
            hold()
            got.append(kvc.kv8_decode_attn(q[0], c, k_new=kn[0], v_new=vn[0], new_pos=t))
            hold()
            row = got[-1].view(shape + (G, D))[..., 0, :].contiguous()
            got.append(kvc.kv8_decode_attn(q[0], c, k_new=row, v_new=row, new_pos=t))
            hold()
            c.n_valid.sub_(2)
            k, v = kvc.kv8_read(c, n_rows=L)
            hold()
            got += [k, v]
            kvc.kv8_write(k, v, c)
            hold()
            got.append(kvc.kv8_decode_attn(got[1], c))
            hold()
            kvc.snapkv_select_kv8(votes, k, v, c, keep_window=8, pool_kernel=7, budget=100 + t)
            hold()
            got.append(kvc.kv8_decode_attn(q[0], c))
            hold()
            q[0].mul_(-1)
        return got

    torch.cuda.synchronize()
    x = turn(one, False)
    y = turn(two, True)
    for i, (s, t) in enumerate(zip(x, y)):
        assert torch.equal(s.view(torch.int16), t.view(torch.int16)), i
    same(state(one), state(two))
    assert kvc.kvc_device_status() == 0

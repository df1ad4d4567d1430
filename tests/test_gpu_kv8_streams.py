"""The 8-bit cache's calls on a stream of the caller's (stream=...), and what snapkv_compress_kv8 holds,
whatever order its votes were added up in."""

import pytest
import torch

from test_gpu_kv8 import BF, dev, poison, rnd
from test_gpu_kv8_rollback import bits, same, state

pytestmark = pytest.mark.gpu
SELECT = dict(keep_window=16, pool_kernel=7, budget=130)


def calls(kvc, x, c, s):
    """Each call once, on the current stream (s None) or on s; returns outputs."""
    got = []
    kvc.kv8_write(x["k"], x["v"], c, lengths=x["n"], stream=s)
    kvc.kv8_append(x["a"], x["b"], c, counts=x["m"], new_pos=3, stream=s)
    got += kvc.kv8_read(c, stream=s)
    got += kvc.kv8_read(c, n_rows=100, k_out=x["ko"], v_out=x["vo"], stream=s)
    got.append(kvc.kv8_decode_attn(x["q"], c, k_new=x["kn"], v_new=x["vn"], new_pos=9, stream=s))
    kvc.snapkv_select_kv8(x["votes"], x["k"], x["v"], c, stream=s, **SELECT)
    got += kvc.kv8_read(c, stream=s)
    kvc.snapkv_select_kv8(x["votes"], x["k"], x["pinned"], c, stream=s, **SELECT)
    got += kvc.kv8_read(c, stream=s)
    kvc.snapkv_compress_kv8(x["qw"], x["k"], x["v"], c, votes_out=x["votes_out"], stream=s, **SELECT)
    got += kvc.kv8_read(c, stream=s)
    return got


@pytest.mark.parametrize("D", [64, 128])
def test_calls_on_a_stream_of_their_own(kvc, D):
    """The other stream's inputs only come to be late in it, while the current stream is busy with
    something else: a call that ran on another stream than its own would see other rows."""
    Ly, B, H, G, L, cap = 1, 2, 2, 2, 600, 704
    u = (Ly, B, H)
    x = dict(zip(("k", "v", "a", "b"), dev(rnd(u + (L, D), 1), rnd(u + (L, D), 2), rnd(u + (40, D), 3), rnd(u + (40, D), 4))))
    x["q"], x["kn"], x["vn"] = dev(rnd((Ly, B, H * G, D), 5, boost=False), rnd(u + (D,), 6, boost=False), rnd(u + (D,), 7, boost=False))
    x["qw"] = rnd((Ly, B, H, 16, D), 8, boost=False).cuda()        # one row tile: votes add up in one order
    x["votes"] = torch.rand(u + (L,), generator=torch.Generator().manual_seed(1)).cuda()
    x["n"] = torch.tensor([600, 500, 64, 1], dtype=torch.int32).view(u).cuda()
    x["m"] = torch.tensor([40, 12, 0, 39], dtype=torch.int32).view(u).cuda()
    x["ko"], x["vo"] = (torch.full(u + (100, D), 3.0, dtype=BF, device="cuda") for _ in "kv")
    x["votes_out"] = torch.empty(u + (L,), device="cuda")
    x["pinned"] = x["v"].cpu().pin_memory()
    want_cache, got_cache = (poison(kvc.KV8Cache(*u, D, cap)) for _ in range(2))
    want = [t.clone() for t in calls(kvc, x, want_cache, None)] + [x["votes_out"].clone()]
    y = {n: t if n == "pinned" else torch.zeros_like(t) for n, t in x.items()}
    y["ko"].fill_(3.0), y["vo"].fill_(3.0)
    big = torch.ones(1 << 28, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late = torch.ones(1 << 28, device="cuda")
        for _ in range(20):
            late.mul_(1.0)
        for n, t in x.items():
            if n not in ("pinned", "ko", "vo", "votes_out"):
                y[n].copy_(t)
    for _ in range(40):
        big.mul_(1.0)
    got = calls(kvc, y, got_cache, s)
    with torch.cuda.stream(s):
        got = [t.clone() for t in got] + [y["votes_out"].clone()]
    s.synchronize()
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(bits(a), bits(b)), i
    same(state(want_cache), state(got_cache))
    torch.cuda.synchronize()
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("case", [  # Ly, B, Hq, Hkv, D, L, W, pool, budget, avg; the first three add votes up in several row tiles
    (2, 1, 32, 2, 128, 3000, 32, 7, 1024, False), (1, 1, 32, 1, 64, 2000, 64, 5, 300, True), (1, 2, 64, 2, 128, 700, 32, 1, 130, False),
    (1, 1, 4, 4, 64, 512, 8, 7, 64, False), (1, 1, 2, 2, 128, 60, 16, 7, 128, False)], ids=lambda c: "x".join(map(str, c)))
def test_what_a_compression_holds(kvc, case):
    """The positions are snapkv_select's of the votes that the call itself gives, the rows kv8_write's
    of those positions."""
    Ly, B, Hq, H, D, L, W, P, budget, avg = case
    u, cap = (Ly, B, H), (max(budget, 64) + 63) // 64 * 64
    k, v = dev(rnd(u + (L, D), 81), rnd(u + (L, D), 82))
    qw = rnd((Ly, B, Hq, min(W, L), D), 83, boost=False).cuda()
    kw = dict(keep_window=W, pool_kernel=P, budget=budget, pool_avg=avg)
    votes = torch.empty(u + (L,), device="cuda")
    got = poison(kvc.KV8Cache(*u, D, cap))
    kvc.snapkv_compress_kv8(qw, k, v, got, votes_out=votes, **kw)
    c = kvc.snapkv_select(votes, k, v, cap=cap, **kw)
    assert torch.equal(got.pos, c["pos"]) and torch.equal(got.n_valid, c["n_valid"])
    n = int(got.n_valid.view(-1)[0])
    assert n == min(budget, L) and (got.n_valid == n).all()
    want = poison(kvc.KV8Cache(*u, D, cap))
    kvc.kv8_write(k, v, want, rows=got.pos[..., :n].contiguous())
    same(state(got), state(want))
    assert kvc.kvc_device_status() == 0

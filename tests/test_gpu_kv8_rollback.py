"""Rows taken back from the 8-bit cache (a draft's rejected tokens) by lowering n_valid.  What is
held, read back and attended over afterwards is compared bit for bit with a cache that was given
only the rows that were kept: that one is checked against the oracle in test_gpu_kv8.py."""

import pytest
import torch

from test_gpu_kv8 import BF, check_unit, dev, poison, rnd, unit_of, units

pytestmark = pytest.mark.gpu
STATE = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "pos", "n_valid")


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.dtype == BF else torch.int32)


def state(cache):
    return {n: bits(getattr(cache, n)).clone() for n in STATE}


def same(a, b):
    for n in STATE:
        assert torch.equal(a[n], b[n]), n


def counts(values, shape):
    return torch.tensor(values, dtype=torch.int32).view(shape)


def rows_of(parts, u):
    """The rows that unit u holds: parts is a list of (rows [.., m, D], how many of them)."""
    return torch.cat([x[u][:int(n[u])] for x, n in parts])


def check_held(kvc, cache, kparts, vparts, q):
    """Everything a user reads of the cache against a cache written at once."""
    want = poison(kvc.KV8Cache(*cache.shape, cache.head_dim, cache.cap))
    L = cache.cap
    k, v = (torch.zeros(cache.shape + (L, cache.head_dim), dtype=BF) for _ in "kv")
    n = torch.zeros(cache.shape, dtype=torch.int32)
    for u in units(cache):
        a, b = rows_of(kparts, u), rows_of(vparts, u)
        k[u][:len(a)], v[u][:len(b)] = a, b
        n[u] = len(a)
    kvc.kv8_write(*dev(k, v), want, lengths=n.cuda())
    assert torch.equal(cache.n_valid.cpu(), n)
    for x, y in zip(kvc.kv8_read(cache), kvc.kv8_read(want)):
        assert torch.equal(bits(x), bits(y))
    for u in units(cache):
        b = int(n[u]) // 64
        for name in ("k_codes", "v_codes"):
            assert torch.equal(bits(getattr(cache, name))[u][:64 * b], bits(getattr(want, name))[u][:64 * b])
        for name in ("k_scale", "v_scale"):
            assert torch.equal(getattr(cache, name)[u][:b], getattr(want, name)[u][:b])
    assert torch.equal(kvc.kv8_decode_attn(q, cache), kvc.kv8_decode_attn(q, want))


@pytest.mark.parametrize("D,m", [(128, 1), (128, 5), (64, 5), (64, 64), (128, 63), (128, 700), (64, 333)])
def test_an_append_taken_back_and_repeated(kvc, D, m):
    """n_valid put back to where it was, the same rows again: the same cache, each time."""
    shape, cap = (1, 2, 8), 1280
    n0 = counts([0, 1, 63, 64, 62, 60, 59, 127, 128, 100, 500, 511, 512, 513, 540, 0], shape)
    k, v = rnd(shape + (540, D), 1), rnd(shape + (540, D), 2)
    a, b = rnd(shape + (m, D), 3), rnd(shape + (m, D), 4)
    cache = poison(kvc.KV8Cache(*shape, D, cap))
    kvc.kv8_write(*dev(k, v), cache, lengths=n0.cuda())
    kvc.kv8_append(*dev(a, b), cache, new_pos=9)
    first = state(cache)
    every = torch.full(shape, m, dtype=torch.int32)
    for _ in range(3):
        cache.n_valid.copy_(n0)
        kvc.kv8_append(*dev(a, b), cache, new_pos=9)
        same(state(cache), first)
    for u in units(cache):
        check_unit(cache, u, unit_of(rows_of([(k, n0), (a, every)], u)), unit_of(rows_of([(v, n0), (b, every)], u)))
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("by", ["append", "steps"])
@pytest.mark.parametrize("D,G,draft", [(128, 4, 5), (64, 8, 7), (128, 1, 64), (64, 2, 40)])
def test_rejected_drafts(kvc, by, D, G, draft):
    """Drafts appended at every place about a block's end, all or some of their tokens rejected,
    others appended in their place; what is held is looked at in between, with the rows taken
    back for good and for one look only."""
    shape, cap = (2, 2, 16), 384
    g = torch.Generator().manual_seed(draft)
    n0 = torch.arange(64, dtype=torch.int32).view(shape) + 96       # 96 .. 159
    k, v = rnd(shape + (160, D), 11), rnd(shape + (160, D), 12)
    q = rnd((shape[0], shape[1], shape[2] * G, D), 13, boost=False).cuda()
    cache = poison(kvc.KV8Cache(*shape, D, cap))
    kvc.kv8_write(*dev(k, v), cache, lengths=n0.cuda())
    kparts, vparts = [(k, n0)], [(v, n0)]

    def add(m, seed):
        a, b = rnd(shape + (m, D), seed, boost=False), rnd(shape + (m, D), seed + 1, boost=False)
        if by == "append":
            kvc.kv8_append(*dev(a, b), cache)
        else:
            for t in range(m):
                kvc.kv8_decode_attn(q, cache, k_new=a[..., t, :].contiguous().cuda(),
                                    v_new=b[..., t, :].contiguous().cuda())
        return a, b

    for t in range(3):
        a, b = add(draft, 20 + 4 * t)
        full = cache.n_valid.clone()
        whole = kvc.kv8_decode_attn(q, cache), *kvc.kv8_read(cache)
        keep = torch.randint(0, draft + 1, shape, generator=g, dtype=torch.int32)
        if t == 0:
            keep.zero_()
        cache.n_valid.copy_(full - (draft - keep).cuda())
        now_k, now_v = kparts + [(a, keep)], vparts + [(b, keep)]
        check_held(kvc, cache, now_k, now_v, q)
        cache.n_valid.copy_(full)                                   # a look back takes nothing away
        for x, y in zip((kvc.kv8_decode_attn(q, cache), *kvc.kv8_read(cache)), whole):
            assert torch.equal(bits(x), bits(y))
        cache.n_valid.copy_(full - (draft - keep).cuda())
        kparts, vparts = now_k, now_v
        a, b = add(3, 22 + 4 * t)                                   # other tokens in their place
        three = torch.full(shape, 3, dtype=torch.int32)
        kparts, vparts = kparts + [(a, three)], vparts + [(b, three)]
        check_held(kvc, cache, kparts, vparts, q)
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("U", [(1, 3, 40), (2, 20, 16)], ids=str)
def test_many_units_taken_back(kvc, U):
    """About one unit to a CTA, and more units than threads: every fourth taken back into its
    completed block, then attended over and added to."""
    D, G, cap, n0 = 64, 2, 192, 60
    k, v = rnd(U + (n0, D), 31), rnd(U + (n0, D), 32)
    a, b = rnd(U + (9, D), 33), rnd(U + (9, D), 34)
    q = rnd((U[0], U[1], U[2] * G, D), 35, boost=False).cuda()
    cache = poison(kvc.KV8Cache(*U, D, cap))
    kvc.kv8_write(*dev(k, v), cache)
    kvc.kv8_append(*dev(a, b), cache)
    keep = torch.full(U, 9, dtype=torch.int32)
    keep.view(-1)[::4] = torch.arange(keep.view(-1)[::4].numel(), dtype=torch.int32) % 5
    cache.n_valid.copy_(keep + n0)
    full = torch.full(U, n0, dtype=torch.int32)
    kparts, vparts = [(k, full), (a, keep)], [(v, full), (b, keep)]
    check_held(kvc, cache, kparts, vparts, q)
    kn, vn = rnd(U + (1, D), 36, boost=False), rnd(U + (1, D), 37, boost=False)
    kvc.kv8_decode_attn(q, cache, k_new=kn[..., 0, :].contiguous().cuda(), v_new=vn[..., 0, :].contiguous().cuda())
    one = torch.ones(U, dtype=torch.int32)
    check_held(kvc, cache, kparts + [(kn, one)], vparts + [(vn, one)], q)
    assert kvc.kvc_device_status() == 0


def test_rows_that_are_gone_are_reported(kvc):
    """A row count inside a block whose bf16 rows are no longer held; whole blocks are fine."""
    D, shape = 128, (1, 1, 2)
    k = rnd(shape + (300, D), 41).cuda()
    q = rnd((1, 1, 4, D), 42, boost=False).cuda()
    row = rnd(shape + (1, D), 43).cuda()
    calls = (lambda c: kvc.kv8_read(c), lambda c: kvc.kv8_decode_attn(q, c), lambda c: kvc.kv8_append(row, row, c),
             lambda c: kvc.kv8_decode_attn(q, c, k_new=row[..., 0, :].contiguous(), v_new=row[..., 0, :].contiguous()))
    for call in calls:
        cache = kvc.kv8_write(k, k, kvc.KV8Cache(*shape, D, 512))
        for n in (128, 192, 299):
            cache.n_valid.fill_(n)
            call(cache)
            assert kvc.kvc_device_status() == 0, n
            kvc.kv8_write(k, k, cache)
        cache.n_valid.fill_(100)                   # in the prompt
        call(cache)
        assert kvc.kvc_device_status() == kvc.DEV_BAD_STATE
        cache = kvc.kv8_write(k, k, kvc.KV8Cache(*shape, D, 512))
        kvc.kv8_append(k[..., :150, :].contiguous(), k[..., :150, :].contiguous(), cache)    # 300 + 150: blocks 4, 5, 6 fill
        cache.n_valid.fill_(310)                   # in block 4, which held rows before
        call(cache)
        assert kvc.kvc_device_status() == 0
        cache = kvc.kv8_write(k, k, kvc.KV8Cache(*shape, D, 512))
        kvc.kv8_append(k[..., :150, :].contiguous(), k[..., :150, :].contiguous(), cache)
        cache.n_valid.fill_(390)                   # in block 6
        call(cache)
        assert kvc.kvc_device_status() == kvc.DEV_BAD_STATE
    cache = kvc.kv8_write(k[..., :256, :].contiguous(), k[..., :256, :].contiguous(), kvc.KV8Cache(*shape, D, 512))
    kvc.kv8_append(k[..., :150, :].contiguous(), k[..., :150, :].contiguous(), cache)       # blocks 4 and 5, no rows before
    cache.n_valid.fill_(330)                       # in the last of them
    kvc.kv8_read(cache)
    assert kvc.kvc_device_status() == 0


def test_another_state_put_into_the_tensors(kvc):
    """A snapshot copied back, and another cache's rows copied in, under a cache that has gone on
    since: taken as they are, with and without blocks filled with -1."""
    D, shape, cap = 64, (1, 2, 4), 256
    q = rnd((1, 2, 8, D), 50, boost=False).cuda()
    n0 = counts([100, 120, 126, 127, 64, 65, 88, 1], shape)
    full = torch.full(shape, 40, dtype=torch.int32)
    k, v, k2, v2 = (rnd(shape + (130, D), 51 + i) for i in range(4))
    a, b = rnd(shape + (40, D), 55), rnd(shape + (40, D), 56)
    for reset in (False, True):
        cache = poison(kvc.KV8Cache(*shape, D, cap))
        kvc.kv8_write(*dev(k, v), cache, lengths=n0.cuda())
        snap = {n: getattr(cache, n).clone() for n in STATE}
        other = poison(kvc.KV8Cache(*shape, D, cap))
        kvc.kv8_write(*dev(k2, v2), other, lengths=n0.cuda())
        for rows, src in (((k, v), snap), ((k2, v2), {n: getattr(other, n) for n in STATE})):
            kvc.kv8_append(*dev(a, b), cache)
            for n in STATE:
                getattr(cache, n).copy_(src[n])
            if reset:
                cache.blocks.fill_(-1)
            check_held(kvc, cache, [(rows[0], n0)], [(rows[1], n0)], q)
            kvc.kv8_append(*dev(a, b), cache)
            check_held(kvc, cache, [(rows[0], n0), (a, full)], [(rows[1], n0), (b, full)], q)
    assert kvc.kvc_device_status() == 0


def test_a_selection_and_a_write_start_afresh(kvc):
    """What an earlier sequence left does not show in the next one's open block."""
    D, shape, L = 128, (1, 1, 2), 400
    k, v = rnd(shape + (L, D), 61), rnd(shape + (L, D), 62)
    q = rnd((1, 1, 4, D), 63, boost=False).cuda()
    votes = torch.rand(shape + (L,), generator=torch.Generator().manual_seed(3)).cuda()
    cache = poison(kvc.KV8Cache(*shape, D, 512))
    for n in (100, 70, 128, 1):
        kvc.kv8_write(*dev(k, v), cache)
        kvc.kv8_append(*dev(k[..., :60, :].contiguous(), v[..., :60, :].contiguous()), cache)
        kvc.snapkv_select_kv8(votes, *dev(k, v), cache, keep_window=min(n, 16), pool_kernel=7, budget=n)
        rows = cache.pos[..., :n].cpu().long().unsqueeze(-1).expand(shape + (n, D))
        m = torch.full(shape, n, dtype=torch.int32)
        check_held(kvc, cache, [(k.gather(3, rows), m)], [(v.gather(3, rows), m)], q)
        kvc.kv8_write(*dev(k[..., :n, :].contiguous(), v[..., :n, :].contiguous()), cache)
        check_held(kvc, cache, [(k, m)], [(v, m)], q)
    assert kvc.kvc_device_status() == 0


def test_captured_drafts_are_taken_back(kvc):
    """A draft, its rejection and a step in one graph, replayed: what the same calls give eagerly."""
    D, shape, cap = 128, (1, 2, 2), 512
    n0 = counts([100, 62, 125, 190], shape)
    caches = []
    for _ in range(2):
        c = poison(kvc.KV8Cache(*shape, D, cap))
        kvc.kv8_write(*dev(rnd(shape + (200, D), 71), rnd(shape + (200, D), 72)), c, lengths=n0.cuda())
        caches.append(c)
    q = rnd((1, 2, 8, D), 73, boost=False).cuda()
    a, b = dev(rnd(shape + (6, D), 74), rnd(shape + (6, D), 75))
    kn, vn = dev(rnd(shape + (D,), 76, boost=False), rnd(shape + (D,), 77, boost=False))
    take = counts([6, 5, 4, 3], shape).cuda()

    def turn(c):
        kvc.kv8_append(a, b, c, new_pos=3)
        c.n_valid.sub_(take)
        return kvc.kv8_decode_attn(q, c, k_new=kn, v_new=vn, new_pos=5)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = turn(caches[0])
    for t in range(40):
        g.replay()
        assert torch.equal(out, turn(caches[1])), t
        a.mul_(-1.0), q.mul_(-1.0)
    same(state(caches[0]), state(caches[1]))
    assert kvc.kvc_device_status() == 0


def test_a_c_call_without_the_kept_block(kvc):
    """k_last, v_last and blocks NULL: writes, appends, steps and reads as with them."""
    import ctypes

    from attention_score_kv_snapkv_gb300 import _binding as Bd
    D, shape, cap = 128, (1, 1, 3), 256
    k, v = dev(rnd(shape + (130, D), 81), rnd(shape + (130, D), 82))
    q = rnd((1, 1, 6, D), 83, boost=False).cuda()
    one, two = (poison(kvc.KV8Cache(*shape, D, cap)) for _ in range(2))
    c = Bd.KV8CacheC(*(getattr(one._c, n) for n, _ in Bd.KV8CacheC._fields_))
    c.k_last = c.v_last = c.blocks = None
    s = torch.cuda.current_stream().cuda_stream
    p = Bd.KV8Params(*shape[:2], 6, shape[2], D, cap, 7)
    x = [t[..., :60, :].contiguous() for t in (k, v)]
    out = torch.empty_like(q)
    assert Bd.lib().kv8_write(ctypes.byref(p), 130, 130, k.data_ptr(), v.data_ptr(), None, None, None, ctypes.byref(c), s) == 0
    assert Bd.lib().kv8_append(ctypes.byref(p), 60, x[0].data_ptr(), x[1].data_ptr(), None, ctypes.byref(c), s) == 0
    kvc.kv8_write(k, v, two)
    kvc.kv8_append(*x, two, new_pos=7)
    for t in range(5):
        kn, vn = (y[..., t, :].contiguous() for y in x)
        assert Bd.lib().kv8_decode_attn(ctypes.byref(p), q.data_ptr(), kn.data_ptr(), vn.data_ptr(), ctypes.byref(c),
                                        out.data_ptr(), s) == 0
        assert torch.equal(out, kvc.kv8_decode_attn(q, two, k_new=kn, v_new=vn, new_pos=7))
    same(state(one), state(two))
    assert (one.blocks == -1).all() and not one.k_last.any()
    assert kvc.kvc_device_status() == 0


def test_refusals(kvc):
    shape, D = (1, 1, 2), 64
    c = kvc.KV8Cache(*shape, D, 128)
    names = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "n_valid", "pos")
    t = {n: getattr(c, n) for n in names}
    more = {n: getattr(c, n) for n in ("k_last", "v_last", "blocks")}
    kvc.KV8Cache.from_tensors(**t, **more)
    for bad in ({"k_last": None}, {"v_last": None}, {"blocks": None}, {"k_last": c.k_tail}, {"v_last": c.v_last.float()},
                {"blocks": c.blocks[..., :1].contiguous()}, {"blocks": c.blocks.long()}, {"blocks": c.blocks.cpu()}):
        with pytest.raises((TypeError, ValueError)):
            kvc.KV8Cache.from_tensors(**t, **{**more, **bad})


def test_a_hundred_thousand_units_taken_back(kvc):
    """More units to a CTA than it keeps row counts for; a third are lowered into the block that the
    append completed, the others within the open one, or not at all."""
    U, D, cap, n0, m = (10, 100, 100), 64, 128, 60, 9
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn(U + (n0 + m, D), generator=g, device="cuda").to(BF) for _ in "kv"]
    cut = lambda a, b: [x[..., a:b, :].contiguous() for x in rows]  # noqa: E731
    cache = kvc.kv8_append(*cut(n0, n0 + m), kvc.kv8_write(*cut(0, n0), kvc.KV8Cache(*U, D, cap)))
    n = n0 + torch.randint(0, 12, U, generator=g, device="cuda", dtype=torch.int32).clamp(max=m)
    q = torch.randn(U[:2] + (U[2], D), generator=g, device="cuda").to(BF)
    kn, vn = (torch.randn(U + (D,), generator=g, device="cuda").to(BF) for _ in "kv")
    cache.n_valid.copy_(n)
    want = kvc.kv8_write(*rows, kvc.KV8Cache(*U, D, cap), lengths=n)
    for step in range(2):
        assert torch.equal(bits(kvc.kv8_decode_attn(q, cache)), bits(kvc.kv8_decode_attn(q, want)))
        for x, y in zip(kvc.kv8_read(cache), kvc.kv8_read(want)):
            assert torch.equal(bits(x), bits(y))
        if step == 0:
            a, b = (kvc.kv8_decode_attn(q, c, k_new=kn, v_new=vn, new_pos=5) for c in (cache, want))
            assert torch.equal(bits(a), bits(b))
    assert torch.equal(cache.n_valid, want.n_valid) and kvc.kvc_device_status() == 0


@pytest.mark.parametrize("by", ["append", "step"])
@pytest.mark.parametrize("D,cap", [(64, 64), (128, 256)])
def test_a_full_cache_taken_back(kvc, by, D, cap):
    """Filled to its capacity and past it, taken back by up to a block less one row, filled again; units
    that add nothing (counts of zero) stay as they were taken back."""
    shape, G = (1, 3, 7), 2
    k, v = rnd(shape + (cap - 5, D), 1), rnd(shape + (cap - 5, D), 2)
    a, b = rnd(shape + (9, D), 3, boost=False), rnd(shape + (9, D), 4, boost=False)
    q = rnd((1, 3, 7 * G, D), 5, boost=False).cuda()

    def add(x, y, c, m):
        if by == "append":
            kvc.kv8_append(*dev(x, y), c, counts=m.cuda())
        else:
            for t in range(x.shape[3]):
                kvc.kv8_decode_attn(q, c, k_new=x[..., t, :].contiguous().cuda(), v_new=y[..., t, :].contiguous().cuda())

    cache = kvc.kv8_write(*dev(k, v), poison(kvc.KV8Cache(*shape, D, cap)))
    full, five, nine = (torch.full(shape, n, dtype=torch.int32) for n in (cap - 5, 5, 9))
    add(a, b, cache, nine)
    assert kvc.kvc_device_status() == kvc.DEV_CACHE_FULL
    check_held(kvc, cache, [(k, full), (a, five)], [(v, full), (b, five)], q)
    back = torch.arange(21, dtype=torch.int32).view(shape) * 3                 # 0 .. 60 rows taken back
    cache.n_valid.copy_(cap - back)
    rows = [torch.cat([x, y[..., :5, :]], 3) for x, y in ((k, a), (v, b))]
    kept = cap - back
    check_held(kvc, cache, [(rows[0], kept)], [(rows[1], kept)], q)
    m = torch.where(torch.arange(21).view(shape) % 4 == 1, 0, 3).to(torch.int32) if by == "append" else torch.full(shape, 3, dtype=torch.int32)
    add(a[..., 6:9, :].contiguous(), b[..., 6:9, :].contiguous(), cache, m)
    took = torch.minimum(m, back)
    check_held(kvc, cache, [(rows[0], kept), (a[..., 6:9, :], took)], [(rows[1], kept), (b[..., 6:9, :], took)], q)
    assert kvc.kvc_device_status() == (kvc.DEV_CACHE_FULL if (took < m).any() else 0)

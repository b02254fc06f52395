"""Head norms, position rotation and the rotating append against fp64 (GPU)."""
import numpy as np
import pytest
import torch

from tests._rope import assert_bf16_rows, assert_codes, rope64

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "e4m3", "int8", "nvfp4"]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_476_b200 as m

    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _fused(T, Hq, Hkv, D, seed):
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=_gen(seed)).bfloat16().cuda()
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _rope(pkv, D, rot, inter, norm, seed=5, most=4096):
    w = [(1 + 0.2 * torch.randn(D, generator=_gen(seed + i))).cuda() for i in range(2)]
    return pkv.Rope(pkv.rope_cos_sin(most, rot) if rot else None, interleaved=inter,
                    q_norm_weight=w[0] if norm else None, k_norm_weight=w[1] if norm else None)


def _np(t):
    return t.detach().double().cpu().numpy()


def _expect(x, pos, rope, rot, which):
    w = getattr(rope, which + "_norm_weight")
    return rope64(_np(x), pos, rot, rope.interleaved, None if w is None else _np(w),
                  rope.norm_eps)


@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (128, 128, True), (128, 48, False),
                                         (128, 16, True), (64, 64, False), (64, 16, False),
                                         (64, 48, True), (128, 0, False)])
@pytest.mark.parametrize("T,Hq,Hkv,norm", [(1, 8, 2, True), (3, 5, 3, False), (67, 32, 8, True),
                                           (1029, 7, 1, True), (701, 32, 8, False)])
def test_norm_and_rotation(pkv, D, rot, inter, T, Hq, Hkv, norm):
    if not rot and not norm:
        norm = True
    q, k, _ = _fused(T, Hq, Hkv, D, T + rot)
    rope = _rope(pkv, D, rot, inter, norm)
    pos = np.random.default_rng(T).integers(0, 4096, T).astype(np.int32)
    qo, ko = pkv.pkv_qk_norm_rope(rope, q, k, torch.from_numpy(pos).cuda() if rot else None)
    assert qo.is_contiguous() and ko.is_contiguous()
    assert_bf16_rows(qo, *_expect(q, pos, rope, rot, "q"))
    assert_bf16_rows(ko, *_expect(k, pos, rope, rot, "k"))


def test_values_of_unlike_size_zeros_and_far_positions(pkv):
    D, T = 128, 40
    q, k, _ = _fused(T, 4, 2, D, 9)
    q, k = q.clone(), k.clone()
    q[0] = 0
    q[1] *= 1e-18
    q[2] *= 1e15
    k[3, 0, ::2] = 0
    rope = _rope(pkv, D, D, False, True, most=1 << 18)
    pos = np.linspace(0, (1 << 18) - 1, T).astype(np.int32)
    qo, ko = pkv.pkv_qk_norm_rope(rope, q, k, torch.from_numpy(pos).cuda())
    assert_bf16_rows(qo, *_expect(q, pos, rope, D, "q"))
    assert_bf16_rows(ko, *_expect(k, pos, rope, D, "k"))


def test_q_or_k_alone_in_place_and_bad_positions(pkv):
    D, T = 64, 33
    q, k, _ = _fused(T, 6, 2, D, 11)
    rope = _rope(pkv, D, 64, False, True, most=100)
    pos = torch.arange(T, dtype=torch.int32)
    both = pkv.pkv_qk_norm_rope(rope, q, k, pos.cuda())
    assert torch.equal(pkv.pkv_qk_norm_rope(rope, q, None, pos.cuda())[0], both[0])
    assert torch.equal(pkv.pkv_qk_norm_rope(rope, None, k, pos.cuda())[1], both[1])
    own = q.contiguous()
    assert pkv.pkv_qk_norm_rope(rope, own, None, pos.cuda(), q_out=own)[0] is own
    assert torch.equal(own, both[0])
    # positions outside the table: those rows stay, the flag says so
    pos[4], pos[9] = 100, -1
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(both[0], 7.0)
    ko = torch.full_like(both[1], 7.0)
    pkv.pkv_qk_norm_rope(rope, q, k, pos.cuda(), q_out=out, k_out=ko, error_flags=flags)
    ok = torch.ones(T, dtype=torch.bool)
    ok[[4, 9]] = False
    assert torch.equal(out[ok.cuda()], both[0][ok.cuda()]) and bool((out[[4, 9]] == 7).all())
    assert torch.equal(ko[ok.cuda()], both[1][ok.cuda()]) and bool((ko[[4, 9]] == 7).all())
    assert int(flags) == pkv.PKV_FLAG_BAD_LENGTH


class _Pool:
    """A cache of format fmt with sentinel bytes, and its rows by (page, head, slot)."""

    def __init__(self, pkv, fmt, pages, Hkv, P, D, seed=0):
        self.fmt, self.shape = fmt, (pages, Hkv, P, D)
        n = pages * Hkv * P
        self.row = {"bf16": 2 * D, "e4m3": D, "int8": D, "nvfp4": D // 2}[fmt]
        self.extra = D // 16 if fmt == "nvfp4" else 0
        self.k = torch.full((n * (self.row + self.extra),), 0x5A, dtype=torch.uint8, device="cuda")
        self.v = self.k.clone()
        div = {"bf16": 1, "e4m3": 448, "int8": 127, "nvfp4": 448 * 6}[fmt]
        s = (3 + 2 * torch.rand(2, pages, Hkv, generator=_gen(seed + 3))) / div
        self.ks, self.vs = (None, None) if fmt == "bf16" else (s[0].cuda(), s[1].cuda())
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")

        def shaped(x):
            if fmt == "bf16":
                return x.view(torch.bfloat16).view(self.shape)
            return x if fmt == "nvfp4" else x.view(self.shape)

        self.cache = pkv.PagedKVCache(shaped(self.k), shaped(self.v), fmt, self.ks, self.vs,
                                      self.flags, geometry=self.shape)

    def rows(self, x):
        """bytes [pages, Hkv, P, row + extra]"""
        a = x.cpu().numpy()
        n = int(np.prod(self.shape[:3]))
        codes = a[:n * self.row].reshape(*self.shape[:3], self.row)
        if not self.extra:
            return codes
        return np.concatenate([codes, a[n * self.row:].reshape(*self.shape[:3], self.extra)], -1)


def _batch(P, before, new, seed=1):
    need = [-(-(a + n) // P) for a, n in zip(before, new)]
    order = np.random.default_rng(seed).permutation(sum(need) + 2).astype(np.int32)
    table = np.full((len(new), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(before, new)]) if cu[-1] else \
        np.zeros(0, int)
    return table, cu, seq, pos, sum(need) + 2


def _cuda(*arrays):
    return [torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in arrays]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,P,rot,inter,norm,before,new", [
    (128, 64, 128, False, True, [0, 63, 64, 200], [1, 1, 1, 1]),       # a decode step
    (128, 128, 48, False, False, [5, 0, 300, 127, 9], [70, 0, 3, 2, 200]),  # ragged, one empty
    (64, 64, 16, True, True, [0, 1], [130, 65]),
    (64, 128, 64, False, True, [11] * 40, [3] * 40),
    (128, 64, 0, False, True, [62], [5]),
])
def test_append_rope(pkv, fmt, D, P, rot, inter, norm, before, new):
    Hq, Hkv = 6, 3
    table, cu, seq, pos, pages = _batch(P, before, new)
    T, pad = int(cu[-1]), 7
    q, k, v = _fused(T + pad, Hq, Hkv, D, T)
    rope = _rope(pkv, D, rot, inter, norm)
    pool = _Pool(pkv, fmt, pages, Hkv, P, D)
    dt, db, dc = _cuda(table, before, cu)
    q_out = torch.full((T + pad, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    pkv.paged_kv_append_rope(pool.cache, rope, dt, db, dc, k, v, q=q, q_out=q_out)
    torch.cuda.synchronize()
    assert int(pool.flags) == 0
    assert bool((q_out[T:] == 3).all())  # the padding's queries are left alone
    assert_bf16_rows(q_out[:T], *_expect(q[:T], pos, rope, rot, "q"))
    page, slot = table[seq, pos // P], pos % P
    # V: the bytes paged_kv_append writes; every other byte of the pools untouched
    ref = _Pool(pkv, fmt, pages, Hkv, P, D)
    pkv.paged_kv_append(ref.cache, dt, db, dc, k[:T].contiguous(), v[:T].contiguous())
    assert torch.equal(pool.v, ref.v)
    got = pool.rows(pool.k)
    held = np.zeros(pool.shape[:3], bool)
    held[page, :, slot] = True
    assert np.all(got[~held] == 0x5A)
    z, mag = _expect(k[:T], pos, rope, rot, "k")
    rows = got[page, :, slot]  # [T, Hkv, bytes]
    if fmt == "bf16":
        assert_bf16_rows(torch.from_numpy(rows.copy()).view(torch.bfloat16).view(T, Hkv, D), z, mag)
    else:
        scale = pool.ks.cpu().numpy()[page].reshape(-1)
        assert_codes(fmt, rows.reshape(T * Hkv, -1), scale, z.reshape(T * Hkv, D),
                     mag.reshape(T * Hkv, D))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_without_rotation_and_norm_it_is_the_plain_append(pkv, fmt, D):
    P, Hkv, before, new = 64, 2, [3, 100, 0], [2, 61, 129]
    table, cu, _, _, pages = _batch(P, before, new)
    _, k, v = _fused(int(cu[-1]), 1, Hkv, D, 3)
    k = k.clone()
    k[5] = 0
    k[6, :, ::3] *= 300
    dt, db, dc = _cuda(table, before, cu)
    a, b = _Pool(pkv, fmt, pages, Hkv, P, D), _Pool(pkv, fmt, pages, Hkv, P, D)
    assert pkv.paged_kv_append_rope(a.cache, pkv.Rope(), dt, db, dc, k, v) is None
    pkv.paged_kv_append(b.cache, dt, db, dc, k, v.contiguous())
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_append_rope_is_rotation_then_append(pkv):
    """bf16 pools: the same bits as pkv_qk_norm_rope and paged_kv_append, with
    positions of the caller's choice too."""
    P, Hkv, D, before, new = 64, 2, 128, [0, 70, 5], [90, 1, 33]
    table, cu, _, pos, pages = _batch(P, before, new)
    q, k, v = _fused(int(cu[-1]), 8, Hkv, D, 4)
    rope = _rope(pkv, D, 64, False, True)
    dt, db, dc = _cuda(table, before, cu)
    for where in (pos, (pos * 7 + 3) % 4096):
        dp, = _cuda(where)
        a, b = _Pool(pkv, "bf16", pages, Hkv, P, D), _Pool(pkv, "bf16", pages, Hkv, P, D)
        qa = pkv.paged_kv_append_rope(a.cache, rope, dt, db, dc, k, v, q=q,
                                      positions=None if where is pos else dp)
        qb, kb = pkv.pkv_qk_norm_rope(rope, q, k, dp)
        pkv.paged_kv_append(b.cache, dt, db, dc, kb, v.contiguous())
        assert torch.equal(qa, qb) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_append_rope_skips_what_it_cannot_place(pkv):
    P, Hkv, D = 64, 2, 64
    before, new = [60, 0, 10, 62], [8, 3, 2, 4]
    table, cu, seq, pos, pages = _batch(P, before, new)
    table[0, 1] = pages           # tokens 4.. of sequence 0: an id past the pool
    table[1, 0] = -5
    before = np.array(before, np.int32)
    before[3] = table.shape[1] * P - 1  # its last three tokens lie past the table
    table[3, -1] = table[3, 0]
    q, k, v = _fused(int(cu[-1]), 4, Hkv, D, 8)
    rope = _rope(pkv, D, 64, False, False)
    dt, db, dc = _cuda(table, before, cu)
    pool = _Pool(pkv, "bf16", pages, Hkv, P, D)
    q_out = pkv.paged_kv_append_rope(pool.cache, rope, dt, db, dc, k, v, q=q)
    assert int(pool.flags) == pkv.PKV_FLAG_BAD_PAGE | pkv.PKV_FLAG_BAD_LENGTH
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(before, new)])
    assert_bf16_rows(q_out, *_expect(q, pos, rope, 64, "q"))  # queries are rotated all the same
    held = np.zeros(pool.shape[:3], bool)
    for t, (b, p) in enumerate(zip(seq, pos)):
        if p < table.shape[1] * P and 0 <= table[b, p // P] < pages:
            held[table[b, p // P], :, p % P] = True
    assert held.sum() == Hkv * (4 + 2 + 1)
    for x in (pool.k, pool.v):
        assert np.array_equal((pool.rows(x) != 0x5A).any(-1), held)
    # a rotation position outside the table: the token is skipped whole
    pool = _Pool(pkv, "e4m3", pages, Hkv, P, D)
    short = pkv.Rope(pkv.rope_cos_sin(12, 64))
    table, cu, _, pos, _ = _batch(P, [10], [4])
    dt, db, dc = _cuda(table, [10], cu)
    q_out = torch.full((4, 4, D), 3.0, dtype=torch.bfloat16, device="cuda")
    pkv.paged_kv_append_rope(pool.cache, short, dt, db, dc, k[:4], v[:4], q=q[:4], q_out=q_out)
    assert int(pool.flags) == pkv.PKV_FLAG_BAD_LENGTH
    assert bool((q_out[2:] == 3).all()) and not bool((q_out[:2] == 3).all())
    for x in (pool.k, pool.v):
        assert (pool.rows(x) != 0x5A).any(-1).sum() == 2 * Hkv


def test_append_rope_captured_and_on_a_side_stream(pkv):
    P, Hkv, D, before, new = 64, 8, 128, [7] * 5, [1] * 5
    table, cu, _, pos, pages = _batch(P, before, new)
    q, k, v = _fused(5, 32, Hkv, D, 6)
    rope = _rope(pkv, D, 128, False, True)
    dt, db, dc = _cuda(table, before, cu)
    a = _Pool(pkv, "e4m3", pages, Hkv, P, D)
    want = pkv.paged_kv_append_rope(a.cache, rope, dt, db, dc, k, v, q=q)
    b = _Pool(pkv, "e4m3", pages, Hkv, P, D)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = pkv.paged_kv_append_rope(b.cache, rope, dt, db, dc, k, v, q=q, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(side, want) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    c = _Pool(pkv, "e4m3", pages, Hkv, P, D)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_kv_append_rope(c.cache, rope, dt, db, dc, k, v, q=q, q_out=out)
        db.add_(1)  # the next step's position
    db.copy_(torch.tensor(before, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(a.k, c.k) and torch.equal(a.v, c.v)
    g.replay()  # position 8 now: both tokens are in the cache
    torch.cuda.synchronize()
    held = (c.rows(c.k) != 0x5A).any(-1)
    assert held.sum() == 2 * 5 * Hkv


def test_step_driver_rotates(pkv):
    """StepDriver with a rotation against the same step with q and K rotated first."""
    P, Hkv, Hq, D = 64, 2, 8, 128
    rope = _rope(pkv, D, 128, False, True)
    res, pools = [], []
    for mode in ("driver", "before"):
        pool = _Pool(pkv, "bf16", 16, Hkv, P, D)
        alloc = pkv.PageAllocator(16, P, 4, 4)
        drv = pkv.StepDriver(pool.cache, alloc, 4, rope=rope if mode == "driver" else None)
        outs, lens = [], np.zeros(3, int)
        for dec, chunk in (([], [40, 70, 1]), ([0, 2], [20])):
            slots = [0, 1, 2] if not dec else [1]
            n = len(dec) + sum(chunk)
            q, k, v = (t.contiguous() for t in _fused(n, Hq, Hkv, D, n))
            rows, new = dec + slots, [1] * len(dec) + chunk
            pos = np.concatenate([np.arange(lens[r], lens[r] + m) for r, m in zip(rows, new)])
            for r, m in zip(rows, new):
                lens[r] += m
            if mode == "driver":
                st, d, c = drv.step(dec, slots, chunk, k, v, q=q)
            else:
                q, k = pkv.pkv_qk_norm_rope(rope, q, k, _cuda(pos)[0])
                st, d, c = drv.step(dec, slots, chunk, k, v, q[:len(dec)], q[len(dec):])
            assert st == 0
            outs += [t for pair in (d, c) if pair for t in pair]
        torch.cuda.synchronize()
        res.append(outs)
        pools.append(pool)
    assert all(torch.equal(a, b) for a, b in zip(*res)) and len(res[0]) == len(res[1])
    assert torch.equal(pools[0].k, pools[1].k) and torch.equal(pools[0].v, pools[1].v)
    with pytest.raises(ValueError):
        drv.step([0], [], [], k, v, q=q)


@pytest.mark.parametrize("T", [1, 37])
def test_calls_on_a_given_stream_give_the_same(pkv, T):
    """The binding's short way (this stream, its own results) and its long way."""
    q, k, v = _fused(T, 8, 2, 128, 3)
    rope = _rope(pkv, 128, 64, False, True)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    here = torch.cuda.current_stream()
    for a in ((q, k), (q, None), (None, k)):
        for x, y in zip(pkv.pkv_qk_norm_rope(rope, *a, pos),
                        pkv.pkv_qk_norm_rope(rope, *a, pos, stream=here)):
            assert (x is None and y is None) or torch.equal(x, y)
    pools = [_Pool(pkv, "bf16", 2, 2, 64, 128) for _ in range(2)]
    table = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    before = torch.tensor([5], dtype=torch.int32).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    x = pkv.paged_kv_append_rope(pools[0].cache, rope, table, before, cu, k, v, q=q)
    y = pkv.paged_kv_append_rope(pools[1].cache, rope, table, before, cu, k, v, q=q, stream=here)
    assert torch.equal(x, y) and torch.equal(pools[0].k, pools[1].k)
    assert torch.equal(pools[0].v, pools[1].v)
    assert pkv.paged_kv_append_rope(pools[0].cache, rope, table, before, cu, k, v) is None


def test_refusals_from_python(pkv):
    q, k, v = _fused(4, 8, 2, 128, 3)
    rope = _rope(pkv, 128, 64, False, True)
    pos = torch.arange(4, dtype=torch.int32).cuda()
    for a in ((None, None, pos), (q, k, None), (q, k, pos[:3]), (q, k, pos.long()),
              (q.float(), k, pos), (q, k[:3], pos), (q.cpu(), k, pos), (q[..., ::2], k, pos),
              (q[..., :64].contiguous(), k[..., :64].contiguous(), pos)):
        with pytest.raises(ValueError):
            pkv.pkv_qk_norm_rope(rope, *a)
    with pytest.raises(ValueError):
        pkv.Rope(q_norm_weight=torch.ones(128).cuda(), k_norm_weight=torch.ones(64).cuda())
    pool = _Pool(pkv, "bf16", 2, 2, 64, 128)
    table = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    before, cu = torch.zeros(1, dtype=torch.int32).cuda(), torch.tensor([0, 4]).int().cuda()
    good = [table, before, cu, k, v]
    for at, bad in ((0, table.long()), (0, table.repeat(2, 1)), (1, before.cpu()), (2, cu[:1]),
                    (3, k[:, :1]), (4, v[:3]), (4, v.half())):
        a = list(good)
        a[at] = bad
        with pytest.raises(ValueError):
            pkv.paged_kv_append_rope(pool.cache, rope, *a)
    for kw in ({"total_new_tokens": 5}, {"q": q[:3]}, {"q": q.float()}, {"positions": pos[:2]}):
        with pytest.raises(ValueError):
            pkv.paged_kv_append_rope(pool.cache, rope, *good, **kw)
    assert int(pool.flags) == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (128, 13, 5), (64, 21, 3), (128, 9, 0)])
@pytest.mark.parametrize("T", [150, 700, 1500, 3100, 9001])
def test_every_number_of_rows_an_item(pkv, D, Hq, Hkv, T):
    """Batches on both sides of where an item takes two, four and eight rows, with head
    counts that leave items short."""
    x = torch.randn(T, Hq + Hkv, D, generator=_gen(T)).bfloat16().cuda()
    q, k = x[:, :Hq], x[:, Hq:] if Hkv else None
    for inter, norm in ((False, True), (True, False)):
        rope = _rope(pkv, D, D, inter, norm)
        pos = np.random.default_rng(T).integers(0, 4096, T).astype(np.int32)
        qo, ko = pkv.pkv_qk_norm_rope(rope, q, k, torch.from_numpy(pos).cuda())
        assert_bf16_rows(qo, *_expect(q, pos, rope, D, "q"))
        if Hkv:
            assert_bf16_rows(ko, *_expect(k, pos, rope, D, "k"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,Hq,Hkv", [(400, 32, 8), (900, 24, 5), (2200, 16, 8), (5000, 8, 3)])
def test_large_appends(pkv, fmt, T, Hq, Hkv):
    """The same for the append: pools and queries against a call for each few tokens."""
    D, P = 128, 64
    q, k, v = _fused(T, Hq, Hkv, D, T)
    rope = _rope(pkv, D, 64, False, True, most=8192)
    n = -(-T // P)
    table = torch.randperm(n, generator=_gen(1)).int()[None].cuda()
    ints = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()
    pools = [_Pool(pkv, fmt, n, Hkv, P, D) for _ in range(2)]
    whole = pkv.paged_kv_append_rope(pools[0].cache, rope, table, ints(0), ints(0, T), k, v, q=q)
    for at in range(0, T, 16):  # (one row an item)
        m = min(16, T - at)
        part = pkv.paged_kv_append_rope(pools[1].cache, rope, table, ints(at), ints(0, m),
                                        k[at:at + m], v[at:at + m], q=q[at:at + m])
        assert torch.equal(whole[at:at + m], part)
    assert torch.equal(pools[0].k, pools[1].k) and torch.equal(pools[0].v, pools[1].v)
    z, mag = _expect(q, np.arange(T), rope, 64, "q")
    assert_bf16_rows(whole, z, mag)

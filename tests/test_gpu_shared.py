"""Decode attention over shared prefixes against fp64 (GPU)."""
import copy

import pytest
import torch

from tests._rope import rope64
from tests._shared import Batch, assert_exact

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "e4m3", "int8", "nvfp4"]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_476_b200 as m

    return m


def _check(pkv, batch, flags=0):
    cache = batch.cache(pkv)
    got = pkv.paged_decode_attention_shared(cache, *batch.args(), batch.scale)
    assert int(batch.flags) == flags
    assert_exact(got, batch)
    return cache, got


# lens, cu, prefix: small groups; a group of one, an empty one, sequences outside
SMALL = {
    "three": lambda P: ([2 * P + 1, 2 * P + 65, 3 * P], [0, 3], [2 * P]),
    "one token": lambda P: ([1, 1, 1], [0, 3], [0]),
    "two": lambda P: ([P + 1, P + 1], [0, 2], [P]),
    "mixed": lambda P: ([P + 5, 3 * P, 7, 2 * P + 9, 0, P, 4 * P + 3, 4 * P + 64, 4 * P + 1, 11],
                        [1, 2, 2, 4, 4, 9], [2 * P, P, 0, P, 4 * P + 3]),
    "nothing of their own": lambda P: ([5 * P] * 4, [0, 4], [5 * P]),
    "shorter members": lambda P: ([0, 1, P - 1, 3 * P - 1, 3 * P, 3 * P + 1, 2 * P], [0, 7], [3 * P]),
    "no member holds it": lambda P: ([0, P, 2 * P], [0, 3], [3 * P]),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 4), (64, 3, 1), (128, 1, 8), (64, 2, 2)])
@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("name", SMALL)
def test_small_groups(pkv, fmt, D, Hkv, G, page, name):
    lens, cu, prefix = SMALL[name](page)
    _check(pkv, Batch(lens, cu, prefix, Hkv, G, D, page, fmt, seed=len(name)))


# rows of a group around 128 and 256 (one, two and more Q tiles), odd prefixes
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G,D", [(16, 8, 128), (17, 8, 128), (32, 8, 128), (33, 8, 128),
                                   (70, 8, 64), (129, 1, 128), (131, 2, 64), (200, 4, 128)])
def test_many_rows(pkv, fmt, n, G, D):
    lens = [64 * 7 + (i * 37) % 90 for i in range(n)] + [30, 400]
    _check(pkv, Batch(lens, [0, n], [64 * 7], 2, G, D, 64, fmt, seed=n))


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_groups_of_unlike_sizes(pkv, fmt):
    sizes, lens, cu, prefix = [2, 40, 3, 1, 65, 5], [], [0], []
    for i, n in enumerate(sizes):
        prefix.append(128 * (1 + 5 * i % 7))
        lens += [prefix[-1] + (31 * j) % 300 for j in range(n)]
        cu.append(cu[-1] + n)
    _check(pkv, Batch(lens, cu, prefix, 2, 4, 128, 64, fmt, seed=3))


@pytest.mark.parametrize("fmt,n,prefix", [("bf16", 5, 20032), ("e4m3", 40, 9984),
                                          ("nvfp4", 3, 20032), ("int8", 3, 12800)])
def test_long_prefixes(pkv, fmt, n, prefix):
    _check(pkv, Batch([prefix + 3 + 50 * i for i in range(n)], [0, n], [prefix], 1, 8, 128, 64,
                      fmt, seed=7))


@pytest.mark.parametrize("fmt", FORMATS[1:])
def test_scales_of_unlike_size(pkv, fmt):
    """Page scales over 30 powers of two, in one batch and far from 1 as a whole."""
    for shift, spread in ((0, 30.0), (-60, 4.0), (-100, 2.0)):
        b = Batch([333, 350, 449, 320], [0, 4], [320], 2, 4, 128, 64, fmt, seed=5)
        r = 2.0 ** (torch.randint(0, int(spread) + 1, b.scales[1].shape,
                                  generator=torch.Generator().manual_seed(1)) - spread + shift)
        r = r.float().to(b.q.device)
        b.scales[1].mul_(r)
        b.values[1].mul_(r.double()[:, :, None, None])
        cache = b.cache(pkv)
        # sequences with nothing but the prefix: its part alone
        b.lens = [320] * 4
        got = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale)
        assert_exact(got, b)


def test_equals_plain_decode_and_itself(pkv):
    for fmt in FORMATS:
        b = Batch([700, 800, 650, 640, 1000], [0, 3, 5], [640, 512], 4, 4, 128, 64, fmt, seed=1)
        cache, (out, lse) = _check(pkv, b)
        plain, plain_lse = pkv.paged_decode_attention(cache, b.q, b.table, b.ints(b.lens), 1000,
                                                      b.scale)
        assert_exact((plain, plain_lse), b)
        again = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        none = torch.zeros(0, dtype=torch.int32, device="cuda")
        alone = pkv.paged_decode_attention_shared(cache, *b.args()[:4], b.ints([0]), none, b.scale)
        assert torch.equal(alone[0], plain) and torch.equal(alone[1], plain_lse)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_softmax_scales(pkv, scale):
    for fmt in FORMATS:
        b = Batch([200, 321, 192], [0, 3], [192], 2, 4, 64, 64, fmt, seed=8)
        b.scale = scale
        if scale:
            cache = b.cache(pkv)
            assert_exact(pkv.paged_decode_attention_shared(cache, *b.args(), scale), _abs_scale(b))
        else:
            _check(pkv, b)


def _abs_scale(b):
    """The batch with scale's sign moved to q (the error bounds want a positive scale)."""
    b = copy.copy(b)
    if b.scale < 0:
        b.q, b.scale = -b.q, -b.scale
    return b


def test_values_behind_a_short_member(pkv):
    """NaN in prefix tokens that one member does not hold stays out of that member."""
    b = Batch([300, 330, 200, 290], [0, 4], [256], 2, 2, 128, 64, seed=2)
    pid = int(b.table[0, 3])
    assert int(b.table[2, 3]) == pid
    for x in b.pools:
        x[pid, :, 20] = float("nan")
    cache = b.cache(pkv)
    got = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale)
    assert_exact(got, b, rows=[2])
    assert bool(got[0][[0, 1, 3]].isnan().all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_pages_and_scales(pkv, fmt):
    """Rejected pages are left out and flagged, as in plain decode."""
    b = Batch([400, 450, 420], [0, 3], [320], 2, 4, 128, 64, fmt, seed=4)
    b.table[:, 2] = b.pages
    b.table[:, 4] = -7
    b.table[1, 6] = b.pages + 3  # of its own
    want = pkv.PKV_FLAG_BAD_PAGE
    if fmt != "bf16":
        want |= pkv.PKV_FLAG_BAD_SCALE
        b.scales[1][b.table[0, 1].long()] = float("inf")
        b.scales[0][b.table[0, 3].long(), 1] = 0.0
    cache = b.cache(pkv)
    got = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale)
    assert int(b.flags) == want
    plain = pkv.paged_decode_attention(cache, b.q, b.table, b.ints(b.lens), 450, b.scale)
    # two evaluations, each within the bound of exact(): mean of |v| below 1, scores to 2^-9
    assert float((got[0].float() - plain[0].float()).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -8)
    assert float((got[1] - plain[1]).abs().max()) <= 2.0 ** -8


def test_bad_groups_are_flagged(pkv):
    b = Batch([200, 210, 220, 230], [0, 4], [128], 2, 4, 128, 64, seed=6)
    for cu, prefix in (([0, 5], [128]), ([-1, 4], [128]), ([3, 1, 4], [128, 128]), ([0, 4], [-64])):
        cache = b.cache(pkv)
        args = (*b.args()[:4], b.ints(cu), b.ints(prefix))
        got = pkv.paged_decode_attention_shared(cache, *args, b.scale)
        assert int(b.flags) == pkv.PKV_FLAG_BAD_LENGTH
        if len(prefix) == 1:  # the group is not one: everyone alone
            assert_exact(got, b)
    # a prefix past the page table ends at the table; nobody holds it all
    cache = b.cache(pkv)
    got = pkv.paged_decode_attention_shared(cache, *b.args()[:5], b.ints([1 << 30]), b.scale)
    assert int(b.flags) == 0
    assert_exact(got, b)


def test_lengths_out_of_range(pkv):
    b = Batch([200, 210, 220], [0, 3], [128], 2, 4, 128, 64, seed=6)
    lens = b.ints([200, -4, 220])
    cache = b.cache(pkv)
    got = pkv.paged_decode_attention_shared(cache, b.q, b.table, lens, 220, *b.args()[4:], b.scale)
    assert int(b.flags) == pkv.PKV_FLAG_BAD_LENGTH
    b.lens[1] = 0
    assert_exact(got, b)


def test_captured_and_replayed_with_new_lengths(pkv):
    b = Batch([300, 340, 300, 700, 800], [0, 3, 5], [256, 640], 2, 4, 128, 64, "e4m3", seed=9)
    cache = b.cache(pkv)
    q, table, lens, _, cu, prefix = b.args()
    work = pkv.decode_shared_workspace(cache, 5, 8, 800, 2)
    out, lse = torch.empty_like(q), torch.empty(5, 8, device="cuda")

    def call():
        pkv.paged_decode_attention_shared(cache, q, table, lens, 800, cu, prefix, b.scale, out,
                                          lse, work)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    work.fill_(0xFF)  # nothing is kept in it between calls
    for new in ([300, 340, 258, 700, 800], [290, 256, 0, 640, 799], [1, 300, 300, 10, 20]):
        lens.copy_(b.ints(new))
        b.lens = new
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert_exact((out, lse), b)
    # groups undone between replays
    cu.copy_(b.ints([0, 0, 0]))
    graph.replay()
    torch.cuda.synchronize()
    assert_exact((out, lse), b)


def test_two_streams_with_workspaces_of_their_own(pkv):
    bs = [Batch([600 + i, 640, 700], [0, 3], [576], 4, 4, 128, 64, "bf16", seed=i) for i in (1, 2)]
    caches = [b.cache(pkv) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    args = [b.args() for b in bs]  # made on the default stream, alive until the end
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, b in enumerate(bs):
            got[i] = pkv.paged_decode_attention_shared(caches[i], *args[i], b.scale,
                                                       stream=streams[i])
    torch.cuda.synchronize()
    for g, b in zip(got, bs):
        assert_exact(g, b)


def test_without_lse_and_given_results(pkv):
    b = Batch([200, 210], [0, 2], [128], 2, 2, 64, 64, seed=3)
    cache = b.cache(pkv)
    out = torch.empty_like(b.q)
    got, none = pkv.paged_decode_attention_shared(cache, *b.args(), out=out, want_lse=False)
    assert got is out and none is None
    assert torch.equal(out, pkv.paged_decode_attention_shared(cache, *b.args())[0])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_rotating_append_then_shared_decode(pkv, fmt):
    """A prompt appended once, forked to four sequences, a few decode steps of all."""
    Hkv, G, D, page, n, prompt = 2, 4, 128, 64, 4, 200
    gen = torch.Generator().manual_seed(12)
    pages = 4 + 3 * n
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    k_pool = torch.zeros(pages, Hkv, page, D, dtype=dt, device="cuda")
    v_pool = torch.zeros_like(k_pool)
    scale = None if fmt == "bf16" else torch.full((pages, Hkv), 6.0 / 448, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = pkv.PagedKVCache(k_pool, v_pool, fmt, scale, scale, flags)
    rope = pkv.Rope(pkv.rope_cos_sin(1024, D), q_norm_weight=torch.ones(D, device="cuda"),
                    k_norm_weight=torch.ones(D, device="cuda"))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def rows(t):
        x = torch.randn(t, Hkv * (G + 2), D, generator=gen).bfloat16().cuda()
        return x[:, :Hkv * G], x[:, Hkv * G:Hkv * (G + 1)], x[:, Hkv * (G + 1):]

    table = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
    table[:, :3] = ints([3, 1, 2])  # whole pages of the prompt, shared
    for b in range(n):
        table[b, 3:6] = ints([4 + 3 * b, 5 + 3 * b, 6 + 3 * b])
    _, k, v = rows(prompt)
    table[0, 3:6], first = ints([4, 5, 6]), table[:1]
    pkv.paged_kv_append_rope(cache, rope, first, ints([0]), ints([0, prompt]), k, v)
    for b in range(1, n):  # the prompt's last, partial page is copied, as a fork does
        for x in (k_pool, v_pool):
            x[4 + 3 * b] = x[4]
    ks, vs = [[k] for _ in range(n)], [[v] for _ in range(n)]
    for step in range(3):
        q, k, v = rows(n)
        for b in range(n):
            ks[b].append(k[b:b + 1])
            vs[b].append(v[b:b + 1])
        length = prompt + step
        qr = pkv.paged_kv_append_rope(cache, rope, table, ints([length] * n),
                                      ints(range(n + 1)), k, v, q=q)
        out, lse = pkv.paged_decode_attention_shared(cache, qr, table, ints([length + 1] * n),
                                                     length + 1, ints([0, n]), ints([prompt]))
    assert int(flags) == 0
    # exact from the inputs; K and q round to bf16 (2^-8 of a value: 2^-7 of |q||k| a score),
    # K and V of the FP8 cache by 2^-4, of scores of at most |q||k| / sqrt(D) = sqrt(D)
    for b in range(n):
        kk = torch.cat(ks[b]).double().cpu().numpy()
        z, _ = rope64(kk, range(length + 1), D, False, [1.0] * D)
        zq, _ = rope64(q[b:b + 1].double().cpu().numpy(), [length], D, False, [1.0] * D)
        z, zq = torch.from_numpy(z), torch.from_numpy(zq)[0].view(Hkv, G, D)
        vv = torch.cat(vs[b]).double().cpu().permute(1, 0, 2)
        s = torch.einsum("hgd,nhd->hgn", zq, z) / D ** 0.5
        mags = torch.einsum("hgd,nhd->hgn", zq.abs(), z.abs()) / D ** 0.5
        half = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -4 + 2.0 ** -8
        ds = (mags.amax(-1) * (half + 2.0 ** -8 + 2.0 ** -15))[..., None]
        p = torch.softmax(s, -1)
        want, mag = p @ vv, p @ vv.abs()
        tol = mag * (torch.expm1(2 * ds) + 2.0 ** -8 + (0 if fmt == "bf16" else 2.0 ** -4)) \
            + 2.0 ** -8 * want.abs() + 2.0 ** -8
        err = (out[b].double().cpu().view(Hkv, G, D) - want).abs()
        assert bool((err <= tol).all())
        assert bool(((lse[b].double().cpu().view(Hkv, G) - torch.logsumexp(s, -1)).abs()
                     <= ds[..., 0] + 2.0 ** -15).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_calls_on_a_given_stream_give_the_same(pkv, fmt):
    """The binding's short way (this stream, its own results) and its long way."""
    b = Batch([200, 210, 150], [0, 3], [128], 2, 4, 128, 64, fmt, seed=3)
    cache = b.cache(pkv)
    work = pkv.decode_shared_workspace(cache, 3, 8, 210, 1)
    here = torch.cuda.current_stream()
    short = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale, workspace=work)
    long = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale, workspace=work, stream=here)
    assert torch.equal(short[0], long[0]) and torch.equal(short[1], long[1])
    none = pkv.paged_decode_attention_shared(cache, *b.args(), workspace=work, want_lse=False)
    assert torch.equal(none[0], short[0]) and none[1] is None


def test_refusals_from_python(pkv):
    b = Batch([200, 210], [0, 2], [128], 2, 4, 128, 64, seed=3)
    cache = b.cache(pkv)
    work = pkv.decode_shared_workspace(cache, 2, 8, 210, 1)
    q, table, lens, n, cu, prefix = b.args()
    call = pkv.paged_decode_attention_shared
    assert call(cache, q, table, lens, n, cu, prefix, workspace=work)[0].shape == q.shape
    for args in ((q.float(), table, lens, n, cu, prefix), (q[:1], table, lens, n, cu, prefix),
                 (q.cpu(), table, lens, n, cu, prefix), (q[..., :64], table, lens, n, cu, prefix),
                 (q, table[:, ::2], lens, n, cu, prefix), (q, table.long(), lens, n, cu, prefix),
                 (q, table, lens[:1], n, cu, prefix), (q, table, lens, n, cu[:2], prefix[:0]),
                 (q, table, lens, n, cu, prefix.cpu())):
        with pytest.raises(ValueError):
            call(cache, *args, workspace=work)
    with pytest.raises(ValueError):
        call(cache, q, table, lens, n, cu, prefix, out=torch.empty_like(q)[:1])
    with pytest.raises(ValueError):
        call(cache, q, table, lens, n, cu, prefix, workspace=work.cpu())
    for kw in ({"workspace": work[:64]}, {"softmax_scale": float("nan"), "workspace": work}):
        with pytest.raises(pkv.PagedKVError):
            call(cache, q, table, lens, n, cu, prefix, **kw)
    with pytest.raises(pkv.PagedKVError):
        call(cache, q, table, lens, table.shape[1] * 64 + 1, cu, prefix)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,G,D,sizes", [(8, 1, 64, [2]), (4, 4, 128, [2]),
                                             (2, 8, 128, [2, 20, 33, 3]), (2, 4, 64, [3, 70, 40]),
                                             (3, 4, 128, [40, 2, 34, 2, 70])])
def test_many_short_prefixes_again_and_again(pkv, fmt, heads, G, D, sizes):
    """Many prefixes of one to five tiles for each CTA, against one and two Q tiles: its
    roles lead and lag across them, and what lies where changes between them."""
    groups = 40 if len(sizes) == 1 else 20
    cu, lens, prefix = [0], [], []
    for i in range(groups):
        n = sizes[i % len(sizes)]
        prefix.append(64 * (1 + (7 * i) % 10 // (2 if len(sizes) == 1 else 1)))
        lens += [prefix[-1] + 1 + (37 * (cu[-1] + j)) % 900 for j in range(n)]
        cu.append(cu[-1] + n)
    b = Batch(lens, cu, prefix, heads, G, D, 64, fmt, seed=2)
    cache = b.cache(pkv)
    args = b.args()
    work = pkv.decode_shared_workspace(cache, cu[-1], heads * G, max(lens), groups)
    first = pkv.paged_decode_attention_shared(cache, *args, b.scale, workspace=work)
    assert_exact(first, b)
    for _ in range(100):
        again = pkv.paged_decode_attention_shared(cache, *args, b.scale, workspace=work)
    torch.cuda.synchronize()
    assert int(b.flags) == 0
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_nobody_holds_a_token(pkv):
    """A padded batch: every length 0."""
    for fmt in FORMATS:
        b = Batch([0] * 5, [0, 3, 5], [64, 128], 2, 4, 128, 64, fmt, seed=1)
        cache = b.cache(pkv)
        out, lse = torch.full_like(b.q, 7), torch.zeros(5, 8, device="cuda")
        pkv.paged_decode_attention_shared(cache, *b.args(), b.scale, out, lse)
        assert int(b.flags) == 0
        assert not bool(out.any()) and bool((lse == -torch.inf).all())


@pytest.mark.parametrize("fmt,n", [("nvfp4", 4700), ("bf16", 700)])
def test_many_sequences(pkv, fmt, n):
    """More sequences than a CTA plans in shared memory (4,608 of FP4 at head_dim 64)."""
    prefix, cu = [64, 0, 128], [5, n // 2, n // 2, n - 9]
    lens = [(64 if i < n // 2 else 128) + i % 7 for i in range(n)]
    lens[3], lens[n - 20] = 0, 100
    _check(pkv, Batch(lens, cu, prefix, 1, 2, 64, 64, fmt, seed=4))

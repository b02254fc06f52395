"""Quantised pools whose V scales are small or unlike: no token is lost (GPU).

The bounds are those of tests._shared.exact without its term for tokens that
meet their page's V scale in f16: P times the scale keeps its 11 bits, in every
part of the batch, so what remains is the 2^-25 of the largest weight times the
largest value that exact() has for all tokens.
"""
import copy

import pytest
import torch

from tests._shared import Batch, assert_exact

pytestmark = pytest.mark.gpu
FORMATS = ["e4m3", "int8", "nvfp4"]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_476_b200 as m

    return m


def _strict(b):
    """The batch as exact() bounds it where no token has an f16 step of its own."""
    b = copy.copy(b)
    b.shared_tokens = lambda i: b.lens[i]
    return b


def _scale_v(b, factor):
    """V scales (and the exact values) times factor [pages, Hkv]."""
    b.scales[1].mul_(factor)
    b.values[1].mul_(factor.double()[:, :, None, None])


def _both(pkv, b, num_ctas=0):
    """Plain decode and (with the batch's groups) shared decode against fp64."""
    cache = b.cache(pkv)
    plain = pkv.paged_decode_attention(cache, b.q, b.table, b.ints(b.lens), max(b.lens), b.scale,
                                       num_ctas=num_ctas)
    assert int(b.flags) == 0
    assert_exact(plain, _strict(b))
    if b.prefix:
        shared = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale)
        assert int(b.flags) == 0
        assert_exact(shared, _strict(b))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,Hkv,G,page", [(128, 2, 4, 64), (64, 3, 1, 128), (128, 1, 8, 128)])
@pytest.mark.parametrize("shift,spread", [(0, 30), (-20, 0), (-60, 4), (-100, 2)])
def test_v_scales_far_from_one(pkv, fmt, D, Hkv, G, page, shift, spread):
    b = Batch([333, 350, 449, 1000, 70, 1], [0, 3], [320], Hkv, G, D, page, fmt, seed=5)
    g = torch.Generator().manual_seed(shift + G)
    r = 2.0 ** (torch.randint(0, spread + 1, b.scales[1].shape, generator=g).float()
                - spread + shift)
    _scale_v(b, r.to(b.q.device))
    _both(pkv, b)


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_tail_behind_one_token(pkv, fmt):
    """One token with weight 1 and value 0, 8,191 with weight 2^-14: half the mass."""
    D, n = 128, 8192
    b = Batch([n], [0], [], 1, 4, D, 64, fmt, seed=2)
    first = int(b.table[0, 0])
    k, v = b.pools[0], b.pools[1]
    k.zero_()
    v.zero_()
    b.scales[0].fill_(1.0)
    b.scales[1].fill_(2.0 ** -11)  # FP4 of values up to 1 has 3.7e-4
    if fmt == "nvfp4":
        codes = b.pages * 64 * D // 2
        k[codes:] = v[codes:] = 0x38                    # block scales 1
        v[:codes] = 0x22                                # 1.0
        rows = (first * 64) * D // 2
        k[rows] = 0x07                                  # 6 at d = 0 of token 0
        v[rows:rows + D // 2] = 0
        top = 6.0
    else:
        one = 0x38 if fmt == "e4m3" else 1
        v.fill_(one)
        k[first, 0, 0, 0] = 0x4C if fmt == "e4m3" else 6  # 6
        v[first, 0, 0] = 0
        top = 6.0
    b.values = [torch.zeros(b.pages, 1, 64, D, dtype=torch.float64, device="cuda"),
                torch.full((b.pages, 1, 64, D), 2.0 ** -11, dtype=torch.float64, device="cuda")]
    b.values[0][first, 0, 0, 0] = top
    b.values[1][first, 0, 0] = 0
    b.q.zero_()
    b.q[..., 0] = 14 * 0.693 / b.scale / top
    _both(pkv, b, num_ctas=1)  # one segment: all weights relative to that token's


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("zeros", [[0], [3], [9], [0, 1, 2, 3], [5, 6, 7, 8, 9], [0, 2, 4, 6, 8],
                                   list(range(10))])
@pytest.mark.parametrize("tiny,other", [(2.0 ** -126, 1.0), (1e-42, 1.0), (2.0 ** -126, 2.0 ** 18),
                                        (2.0 ** -80, 2.0 ** 18)])
def test_pages_of_zeros(pkv, fmt, zeros, tiny, other):
    """Pages whose V is 0 and whose scale is the smallest there is still weigh in the sum."""
    b = Batch([640, 700, 833, 2000], [0, 4], [640], 2, 4, 128, 64, fmt, seed=3)
    _scale_v(b, torch.full_like(b.scales[1], other))
    for j in zeros:
        pid = int(b.table[0, j])
        b.scales[1][pid] = tiny
        b.values[1][pid] = 0
        if fmt == "nvfp4":
            n = 2 * 64 * 128 // 2  # code bytes of a page
            b.pools[1][pid * n:(pid + 1) * n] = 0
        else:
            b.pools[1][pid] = 0
    _both(pkv, b)
    # one part alone: a prefix of these pages only, whatever the own tokens' scales are
    b.lens = [640] * 4
    _both(pkv, b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,Hkv,G,page", [(128, 2, 4, 64), (64, 3, 1, 128), (128, 1, 8, 128)])
@pytest.mark.parametrize("shift,spread", [(0, 30), (-20, 0), (-60, 4), (-100, 2)])
@pytest.mark.parametrize("L,n", [(700, 300), (65, 65), (1000, 1)])
def test_prefill_with_v_scales_far_from_one(pkv, fmt, D, Hkv, G, page, shift, spread, L, n):
    b = Batch([L], [0], [], Hkv, G, D, page, fmt, seed=6)
    g = torch.Generator().manual_seed(shift + G)
    r = 2.0 ** (torch.randint(0, spread + 1, b.scales[1].shape, generator=g).float()
                - spread + shift)
    _scale_v(b, r.to(b.q.device))
    cache = b.cache(pkv)
    q = torch.randn(n, Hkv * G, D, generator=g).bfloat16().cuda()
    got = pkv.paged_prefill_chunk_attention(cache, q, b.ints([0, n]), b.table, b.ints([L]), n,
                                            b.scale)
    assert int(b.flags) == 0
    # each query as a sequence of its own, of the tokens up to it
    rows = _strict(b)
    rows.q, rows.lens, rows.table = q, list(range(L - n + 1, L + 1)), b.table.expand(n, -1)
    assert_exact(got, rows)

"""Refusals of the rotation entry points, and the fp64 rotation's own pins (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

from tests._rope import rope64, table64

OK, NULL, SHAPE, PAGE_SIZE, HEAD_DIM, ALIGN = 0, -1, -2, -3, -4, -9
A = 0x10000  # a fake aligned device address; never dereferenced


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__

    __graft_entry__._builder().build()
    import paged_kv_cache_476_b200 as m

    return m


def _rope(pkv, **kw):
    r = pkv.PkvRope(A, 100, 64, 0, A, None, 1e-6)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


BAD_ROPE = [
    ({"rotary_dim": 8}, SHAPE), ({"rotary_dim": 144}, SHAPE), ({"rotary_dim": -16}, SHAPE),
    ({"cos_sin": None}, NULL), ({"cos_sin": A + 4}, ALIGN), ({"max_positions": 0}, SHAPE),
    ({"q_norm_weight": A + 8}, ALIGN), ({"k_norm_weight": A + 4}, ALIGN),
    ({"norm_eps": -1.0}, SHAPE), ({"norm_eps": float("nan")}, SHAPE),
]


def _norm_rope(pkv, rope=None, q=A, qs=32 * 128, Hq=32, k=A, ks=8 * 128, Hkv=8, D=128, pos=A, T=3,
               qo=A, ko=A):
    r = rope if rope is not None else _rope(pkv)
    return pkv.lib().pkv_qk_norm_rope(ctypes.byref(r), q, qs, Hq, k, ks, Hkv, D, pos, T, qo, ko,
                                      None, None)


def _append(pkv, rope=None, cache=None, table=A, maxp=4, before=A, cu=A, batch=2, T=5, k=A,
            ks=8 * 128, v=A, vs=8 * 128, q=A, qs=32 * 128, Hq=32, qo=A, pos=None):
    c = cache or pkv.PkvCache(A, A, None, None, 16, 64, 8, 128, pkv.PKV_KV_BF16, None)
    r = rope if rope is not None else _rope(pkv)
    return pkv.lib().paged_kv_append_rope(ctypes.byref(c), ctypes.byref(r), table, maxp, before,
                                          cu, batch, T, k, ks, v, vs, q, qs, Hq, qo, pos, None)


@pytest.mark.parametrize("kw,status", BAD_ROPE)
def test_bad_rotation(pkv, kw, status):
    assert _norm_rope(pkv, rope=_rope(pkv, **kw)) == status
    assert _append(pkv, rope=_rope(pkv, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({"D": 96}, HEAD_DIM), ({"T": -1}, SHAPE), ({"Hq": -1}, SHAPE), ({"Hkv": -2}, SHAPE),
    ({"q": None}, NULL), ({"k": None}, NULL), ({"qo": None}, NULL), ({"ko": None}, NULL),
    ({"pos": None}, NULL), ({"q": A + 2}, ALIGN), ({"ko": A + 8}, ALIGN),
    ({"qs": 32 * 128 + 4}, ALIGN), ({"qs": 31 * 128}, SHAPE), ({"ks": 0}, SHAPE),
    ({"T": 0, "q": None}, OK), ({"Hq": 0, "Hkv": 0, "q": None, "k": None}, OK),
])
def test_norm_rope_rejects(pkv, kw, status):
    assert _norm_rope(pkv, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"batch": -1}, SHAPE), ({"T": -1}, SHAPE), ({"maxp": 0}, SHAPE), ({"Hq": -1}, SHAPE),
    ({"maxp": (1 << 31) // 64}, SHAPE), ({"table": None}, NULL), ({"before": None}, NULL),
    ({"cu": None}, NULL), ({"k": None}, NULL), ({"v": None}, NULL), ({"q": None}, NULL),
    ({"qo": None}, NULL), ({"k": A + 8}, ALIGN), ({"vs": 8 * 128 + 2}, ALIGN),
    ({"ks": 7 * 128}, SHAPE), ({"qo": A + 4}, ALIGN), ({"T": 0, "k": None}, OK),
    ({"batch": 0, "table": None}, OK),
])
def test_append_rope_rejects(pkv, kw, status):
    assert _append(pkv, **kw) == status


def test_append_rope_rejects_a_bad_cache(pkv):
    bad = pkv.PkvCache(A, A, None, None, 16, 48, 8, 128, pkv.PKV_KV_BF16, None)
    assert _append(pkv, cache=bad) == PAGE_SIZE
    null = pkv.lib().paged_kv_append_rope(None, None, A, 4, A, A, 2, 5, A, 1024, A, 1024, None, 0,
                                          0, None, None, None)
    assert null == NULL


def test_binding_refuses_host_tensors(pkv):
    with pytest.raises(ValueError):
        pkv.Rope(torch.zeros(4, 16))
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.pkv_qk_norm_rope(pkv.Rope(), x, None)
    with pytest.raises(ValueError):
        pkv.pkv_qk_norm_rope(pkv.Rope(), None, None)
    with pytest.raises(ValueError):
        pkv.rope_cos_sin(4, 16, inv_freq=torch.ones(7), device="cpu")


def test_table_is_fp64_rounded_once(pkv):
    t = pkv.rope_cos_sin(1 << 18, 64, device="cpu").double().numpy()
    pos = np.array([0, 1, 77, 65535, (1 << 18) - 1])
    c, s = table64(pos, 64)
    # numpy's and torch's fp64 cos may differ in the last place before rounding
    assert np.abs(t[pos, :32] - c).max() <= 2.0 ** -24 + 1e-12
    assert np.abs(t[pos, 32:] - s).max() <= 2.0 ** -24 + 1e-12


def test_plain_rotation_is_a_rotation():
    """Scores depend on the distance of two positions alone, and norms stay."""
    x = np.random.default_rng(0).normal(size=(1, 2, 64))
    for inter in (False, True):
        for rot in (16, 64):
            a, _ = rope64(np.repeat(x, 2, 0), [5, 105], rot, inter)
            b, _ = rope64(np.repeat(x[:, ::-1], 2, 0), [9, 109], rot, inter)
            d = (a * b).sum(-1)
            assert np.allclose(d[0], d[1], atol=1e-5)
            assert np.allclose((a * a).sum(-1), (x * x).sum(-1), rtol=1e-6)
            assert np.array_equal(a[..., rot:], np.repeat(x, 2, 0)[..., rot:])
    y, _ = rope64(x, [0], 64, False, weight=np.ones(64), eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0)

"""Refusals of the shared-prefix decode, and its fp64 reference's own pins (CPU)."""
import ctypes

import pytest
import torch

from tests._shared import Batch, exact

OK, NULL, SHAPE, GQA, ALIGN = 0, -1, -2, -5, -9
A = 0x10000  # a fake aligned device address; never dereferenced


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__

    __graft_entry__._builder().build()
    import paged_kv_cache_476_b200 as m

    return m


def _call(pkv, cache=None, q=A, Hq=32, G=4, table=A, maxp=4, lens=A, batch=2, max_len=200, cu=A,
          prefix=A, groups=1, scale=0.1, out=A, lse=None, ws=A, nbytes=1 << 30):
    c = cache or pkv.PkvCache(A, A, None, None, 16, 64, 8, 128, pkv.PKV_KV_BF16, None)
    return pkv.lib().paged_decode_attention_shared(ctypes.byref(c), q, Hq, G, table, maxp, lens,
                                                   batch, max_len, cu, prefix, groups, scale, out,
                                                   lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    ({"groups": -1}, SHAPE), ({"cu": None}, NULL), ({"prefix": None}, NULL),
    ({"batch": -1}, SHAPE), ({"maxp": 0}, SHAPE), ({"max_len": 257}, SHAPE),
    ({"max_len": -1}, SHAPE), ({"scale": float("nan")}, SHAPE), ({"scale": float("inf")}, SHAPE),
    ({"G": 3, "Hq": 24}, GQA), ({"Hq": 16}, GQA), ({"q": None}, NULL), ({"out": None}, NULL),
    ({"table": None}, NULL), ({"lens": None}, NULL), ({"q": A + 8}, ALIGN), ({"out": A + 2}, ALIGN),
    ({"batch": 0, "cu": None, "prefix": None, "q": None}, OK),
    ({"maxp": 1 << 26}, SHAPE),
])
def test_rejects(pkv, kw, status):
    assert _call(pkv, **kw) == status


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8", "nvfp4"])
def test_reference_reads_the_table(fmt):
    """exact() against a loop over tokens, on a shared batch."""
    b = Batch([70, 64, 130, 0], [0, 3], [64], 2, 2, 64, 64, fmt, device="cpu")
    assert int(b.table[0, 0]) == int(b.table[1, 0]) == int(b.table[2, 0])
    assert int(b.table[0, 1]) != int(b.table[2, 1])
    out, lse, tol, tol_lse = exact(b)
    assert bool((out[3] == 0).all()) and bool(torch.isinf(lse[3]).all())
    for h in (0, 3):
        num, den = torch.zeros(64, dtype=torch.float64), 0.0
        for t in range(70):
            p, slot = int(b.table[0, t // 64]), t % 64
            w = torch.exp((b.q[0, h].double() * b.values[0][p, h // 2, slot]).sum() * b.scale)
            num += w * b.values[1][p, h // 2, slot]
            den += w
        assert float((out[0, h] - num / den).abs().max()) < 1e-12
        assert abs(float(lse[0, h] - torch.log(den))) < 1e-12
    assert bool((tol[:3] > 0).all()) and bool((tol_lse[:3] > 0).all())

"""The CPython module's short way for the rotation and shared-prefix calls (GPU):
that it takes ordinary calls, and that no status makes a call run twice."""
import ctypes

import pytest
import torch

from tests._shared import Batch

pytestmark = pytest.mark.gpu
SHAPE, CUDA = -2, -8


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_476_b200 as m

    return m


class _Calls:
    """One call of each entry point: the binding's arguments, and the public call."""

    def __init__(self, pkv):
        gen = torch.Generator().manual_seed(4)
        D, T = 128, 3
        x = torch.randn(T, 14, D, generator=gen).bfloat16().cuda()
        q, k, v = x[:, :8], x[:, 8:10], x[:, 10:12]
        ints = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()
        rope = pkv.Rope(pkv.rope_cos_sin(256, 64), q_norm_weight=torch.ones(D).cuda())
        pos = ints(1, 9, 200)
        pools = [torch.zeros(2, 2, 64, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cache = pkv.PagedKVCache(*pools, "bf16")
        table, before, cu = ints(1, 0)[None], ints(5), ints(0, T)
        b = Batch([200, 210, 150], [0, 3], [128], 2, 4, 128, 64, "bf16", seed=3)
        bc = b.cache(pkv)
        work = pkv.decode_shared_workspace(bc, 3, 8, 210, 1)
        a = b.args()
        self.keep = (b, bc, a)
        self.short = {
            "norm_rope": lambda m: m.norm_rope(rope._args, q, k, pos, None),
            "append_rope": lambda m: m.append_rope(cache._args, rope._args, table, before, cu, k, v,
                                                   q, None, None),
            "decode_shared": lambda m: m.decode_shared(bc._args, *a, b.scale, work, True),
        }
        self.public = {
            "norm_rope": lambda **kw: pkv.pkv_qk_norm_rope(rope, q, k, pos, **kw),
            "append_rope": lambda **kw: pkv.paged_kv_append_rope(cache, rope, table, before, cu, k,
                                                                 v, q=q, **kw),
            "decode_shared": lambda **kw: pkv.paged_decode_attention_shared(
                bc, *a, b.scale, workspace=work, **kw),
        }


NAMES = {"norm_rope": "pkv_qk_norm_rope", "append_rope": "paged_kv_append_rope",
         "decode_shared": "paged_decode_attention_shared"}


def _same(x, y):
    x, y = (z if isinstance(z, tuple) else (z,) for z in (x, y))
    assert len(x) == len(y) and all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.parametrize("name", NAMES)
def test_ordinary_calls_take_the_short_way(pkv, name):
    calls = _Calls(pkv)
    got = calls.short[name](pkv._binding)
    assert got is not NotImplemented
    _same(got, calls.public[name](stream=torch.cuda.current_stream()))


@pytest.fixture
def fakes(pkv):
    """Stand-ins for the three entry points that return `status` and count their calls."""
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    real = [getattr(pkv.lib(), n) for n in NAMES.values()]
    made = []

    def bind(status):
        count = [0]

        def fake(*args):
            count[0] += 1
            return status

        made.extend(ctypes.CFUNCTYPE(ctypes.c_int, *f.argtypes)(fake) for f in real)
        pkv._binding.bind(*map(address, made[-3:]), pkv.PagedKVError)
        return count

    yield bind
    pkv._binding.bind(*map(address, real), pkv.PagedKVError)


@pytest.mark.parametrize("name", NAMES)
def test_a_cuda_error_is_raised_and_nothing_runs_twice(pkv, fakes, monkeypatch, name):
    calls = _Calls(pkv)
    torch.cuda.synchronize()
    count = fakes(CUDA)

    def again(*args, **kw):
        raise AssertionError("the wrapper launched the call again")

    monkeypatch.setattr(pkv, "_on", again)
    with pytest.raises(pkv.PagedKVError) as e:
        calls.public[name]()
    assert e.value.status == CUDA and NAMES[name] in str(e.value) and count == [1]


@pytest.mark.parametrize("name", NAMES)
def test_a_refusal_goes_the_long_way(pkv, fakes, name):
    calls = _Calls(pkv)
    want = calls.public[name]()
    count = fakes(SHAPE)
    _same(calls.public[name](), want)
    assert count == [1]

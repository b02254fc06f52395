"""Streams given to the rotation and shared-prefix calls as the older calls take them:
objects, raw handles, and 0 for the default stream (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_476_b200 as m

    return m


class _Handle:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


def test_the_call_goes_to_the_stream_that_is_given(pkv):
    dev = torch.device("cuda", torch.cuda.current_device())
    side = torch.cuda.Stream()
    on = lambda stream: pkv._on(dev, stream, lambda raw: (raw, torch.cuda.current_stream().cuda_stream))
    for given in (side, side.cuda_stream, _Handle(side.cuda_stream)):
        raw, current = on(given)
        assert raw == side.cuda_stream and current == raw
    for given in (0, torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream, _Handle(0)):
        with torch.cuda.stream(side):
            raw, current = on(given)
        assert raw == 0 and current == 0
    with torch.cuda.stream(side):
        assert on(None)[0] == side.cuda_stream


@pytest.mark.parametrize("handle", [0, None])
def test_ordered_behind_the_default_streams_work(pkv, handle):
    """Values written on the default stream right before the call are the ones it reads."""
    D, T = 128, 4096
    rope = pkv.Rope(q_norm_weight=torch.ones(D, device="cuda"), norm_eps=0.0)
    q = torch.zeros(T, 32, D, dtype=torch.bfloat16, device="cuda")
    big = torch.ones(1 << 28, device="cuda")
    for i in range(5):
        torch.cuda.synchronize()
        for _ in range(10):
            big.mul_(1.0)      # keeps the default stream busy
        q.fill_(float(i + 1))  # norms to 1
        out, _ = pkv.pkv_qk_norm_rope(rope, q, None, stream=handle)
        q.zero_()
        assert bool((out == 1).all())

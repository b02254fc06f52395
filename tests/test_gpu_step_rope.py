"""A rotating step that is refused leaves the allocator as it was (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_476_b200 as m

    return m


def test_refused_steps_change_nothing(pkv):
    P, Hkv, Hq, D = 64, 2, 8, 128
    pools = [torch.zeros(8, Hkv, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    alloc = pkv.PageAllocator(8, P, 4, 4)
    rope = pkv.Rope(pkv.rope_cos_sin(256, D))
    drv = pkv.StepDriver(pkv.PagedKVCache(*pools, "bf16"), alloc, 4, rope=rope)
    x = torch.randn(70, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    for kw in ({"q": q[:69]}, {"q": q.float()}, {"q": q[..., :64]}, {"q": q.cpu()}, {"q": q[:, :7]},
               {"k_new": k[:69], "v_new": v[:69]}, {"v_new": v[:, :1]}, {"k_new": k.half()}):
        args = {"k_new": k, "v_new": v, "q": q, **kw}
        with pytest.raises(ValueError):
            drv.step([], [0, 1], [40, 30], **args)
        assert [alloc.seq_len(s) for s in (0, 1)] == [0, 0]
        assert len(alloc.free_pages()) == 8
    st, dec, chk = drv.step([], [0, 1], [40, 30], k, v, q=q)
    assert st == 0 and dec is None and chk[0].shape == (70, Hq, D)
    assert [alloc.seq_len(s) for s in (0, 1)] == [40, 30]

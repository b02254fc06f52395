"""Shared decode of batches whose groups have members without the whole prefix: right,
and not slowed down by the rows that are not there (GPU)."""
import pytest
import torch

from tests._shared import Batch, assert_exact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_476_b200 as m

    return m


# which members of a group hold its prefix: none but some in the middle, the ends, gaps
# longer than the lengths a lane looks at together
HOLD = {
    "one in the middle": [0] * 9 + [1] + [0] * 12,
    "the first": [1] + [0] * 20,
    "the last": [0] * 20 + [1],
    "both ends": [1] + [0] * 30 + [1],
    "every other": [0, 1] * 9,
    "a padded tail": [1] * 5 + [0] * 40,
    "nobody": [0] * 17,
    "all": [1] * 8,
}


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D", [(4, 128), (8, 64)])
@pytest.mark.parametrize("short", [0, 1, 255])
@pytest.mark.parametrize("first", HOLD)
def test_members_without_the_prefix(pkv, fmt, G, D, short, first):
    """Several groups, each with another pattern of holders."""
    names = list(HOLD)
    at = names.index(first)
    lens, cu, prefix = [70], [1], []
    for i, name in enumerate(names[at:at + 3]):
        lens += [256 + (37 * j) % 200 if x else short for j, x in enumerate(HOLD[name])]
        cu.append(len(lens))
        prefix.append(256)
    b = Batch(lens, cu, prefix, 2, G, D, 64, fmt, seed=at)
    got = pkv.paged_decode_attention_shared(b.cache(pkv), *b.args(), b.scale)
    assert int(b.flags) == 0
    assert_exact(got, b)


@pytest.mark.parametrize("fmt,D,groups,large", [("nvfp4", 64, 1200, 40), ("nvfp4", 64, 900, 0),
                                                ("e4m3", 64, 70, 300), ("bf16", 64, 30, 40)])
def test_many_groups(pkv, fmt, D, groups, large):
    """More groups than a block has warps, and than fit where it plans them (1,152 for FP4
    at head_dim 64, fewer beside the decode kernel's lengths); one of them large."""
    lens, cu, prefix = [], [0], []
    for g in range(groups):
        n = large if g == groups // 2 and large else 2 + g % 2
        # every fifth group is held by nobody, others have short members first or last
        lens += [63 if g % 5 == 0 or (j == g % 7 and j != 1) else 64 + (5 * g + j) % 70
                 for j in range(n)]
        cu.append(len(lens))
        prefix.append(64)
    b = Batch(lens, cu, prefix, 1, 2, D, 64, fmt, seed=groups)
    cache = b.cache(pkv)
    work = pkv.decode_shared_workspace(cache, len(lens), 2, max(lens), groups)
    work.fill_(0xFF)
    got = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale, workspace=work)
    assert int(b.flags) == 0
    assert_exact(got, b)
    again = pkv.paged_decode_attention_shared(cache, *b.args(), b.scale, workspace=work)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def _time(pkv, lens, cu, prefix, Hkv=8, G=4, D=128, page=64):
    """Microseconds of one shared and one plain call (bf16; own pages of their own)."""
    need = [-(-n // page) for n in lens]
    shared = [0] * len(lens)
    for g, n in enumerate(prefix):
        for b in range(cu[g], cu[g + 1]):
            shared[b] = min(n // page, need[b])
    pages = sum(need) + 1
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()
    k, of_group = 0, {}
    for b, n in enumerate(need):
        g = next((g for g in range(len(prefix)) if cu[g] <= b < cu[g + 1]), None)
        for j in range(n):
            key = (g, j) if j < shared[b] else (b, j, "own")
            if key not in of_group:
                of_group[key] = int(order[k])
                k += 1
            table[b, j] = of_group[key]
    pools = [torch.randn(pages, Hkv, page, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    cache = pkv.PagedKVCache(*pools, "bf16")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q = torch.randn(len(lens), Hkv * G, D, device="cuda").bfloat16()
    table, n = table.cuda(), max(lens)
    dl, dc, dp = ints(lens), ints(cu), ints(prefix)
    work = pkv.decode_shared_workspace(cache, len(lens), Hkv * G, n, len(prefix))
    own = pkv.decode_workspace(cache, len(lens), Hkv * G, n)
    out, lse = torch.empty_like(q), torch.empty(len(lens), Hkv * G, device="cuda")
    calls = (lambda: pkv.paged_decode_attention_shared(cache, q, table, dl, n, dc, dp, out=out,
                                                       lse=lse, workspace=work),
             lambda: pkv.paged_decode_attention(cache, q, table, dl, n, out=out, lse=lse,
                                                workspace=own))
    got = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                call()
        best = 1e9
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 1e3 / 4)
        got.append(best)
    print(f"shared {got[0]:.1f} us, plain {got[1]:.1f} us")
    return got


CHATS = [4096 + (211 * i) % 1024 for i in range(64)]


@pytest.mark.parametrize("pad", [8, 16, 192])
def test_padded_rows_cost_next_to_nothing(pkv, pad):
    """A batch captured for more sequences than live in it: the group's padded rows have
    length 0.  (Counted as work, they left one SM of 148 for the own tokens: 64 times.)"""
    alone = _time(pkv, CHATS, [0, 64], [4096])[0]
    padded = _time(pkv, CHATS + [0] * pad, [0, 64 + pad], [4096])[0]
    assert padded < 1.5 * alone, (padded, alone)


@pytest.mark.parametrize("lens,prefix", [
    ([8256 + 32 * (i % 7) for i in range(32)] + [8000] * 32, 8192),   # half of them shorter
    ([8256, 8300] + [8000] * 62, 8192),                               # two hold it
    ([9000] * 64, 9472),                                              # nobody does
])
def test_members_just_under_the_prefix(pkv, lens, prefix):
    """Members that share nothing are read by the decode kernel, with the SMs for it."""
    shared, plain = _time(pkv, lens, [0, len(lens)], [prefix])
    assert shared < 1.5 * plain, (shared, plain)

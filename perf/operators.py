"""Cases of the position-rotation, rotating-append and shared-prefix decode operators.

``run`` computes each in plain torch (32 bits, rounded once at the end), or,
where ``own`` is true, through the package's entry points.  ``exact`` is the
same in 64 bits, written from the definitions.
"""
import math
import random

import torch

own = False

# (kv heads, q heads per kv head, head_dim) of this repository's workloads and tests
HEADS = {"tiny": (8, 1, 64), "small": (2, 4, 128), "8b": (8, 4, 128), "70b": (8, 8, 128),
         "narrow": (4, 2, 64)}
ELEM = {"bf16": 2.0, "e4m3": 1.0, "int8": 1.0, "nvfp4": 0.5625}


# --------------------------------------------------------------------- the cases
def listed():
    return [
        # decode step of a few sequences: the rotation's latency
        {"name": "rope_decode_4", "op": "rope", "tokens": 4, "heads": "8b", "rotary": 128,
         "interleaved": False, "norm": True},
        # prefill batch of a model with per-head q/k norms
        {"name": "rope_prefill_16k", "op": "rope", "tokens": 16384, "heads": "8b", "rotary": 128,
         "interleaved": False, "norm": True},
        # odd token count, partial interleaved rotation, no norms
        {"name": "rope_partial_1531", "op": "rope", "tokens": 1531, "heads": "narrow",
         "rotary": 32, "interleaved": True, "norm": False},
        # decode step: one new token of each of 64 sequences
        {"name": "append_decode_64", "op": "append", "seqs": 64, "new": 1, "context": 1024,
         "heads": "8b", "page": 64, "fmt": "bf16", "rotary": 128, "interleaved": False,
         "norm": False},
        # prefill chunks of up to 1024 tokens, head norms
        {"name": "append_prefill_16", "op": "append", "seqs": 16, "new": 1024, "context": 2048,
         "heads": "8b", "page": 64, "fmt": "bf16", "rotary": 128, "interleaved": False,
         "norm": True},
        # one-byte cache, 256 decode rows with a few tokens each (speculative decoding)
        {"name": "append_e4m3_256", "op": "append", "seqs": 256, "new": 5, "context": 512,
         "heads": "70b", "page": 64, "fmt": "e4m3", "rotary": 64, "interleaved": False,
         "norm": True},
        # three samples of one short prompt: the latency of a call
        {"name": "shared_tiny", "op": "shared", "seqs": 3, "groups": 1, "prefix": 128,
         "suffix": 65, "heads": "tiny", "page": 64, "fmt": "bf16"},
        # 64 chats behind one system prompt
        {"name": "shared_chat_64", "op": "shared", "seqs": 64, "groups": 1, "prefix": 4096,
         "suffix": 1024, "heads": "8b", "page": 64, "fmt": "bf16"},
        # 8 requests with 4 parallel samples each, FP8 cache
        {"name": "shared_samples_32", "op": "shared", "seqs": 32, "groups": 8, "prefix": 2048,
         "suffix": 256, "heads": "70b", "page": 64, "fmt": "e4m3"},
        # 16 questions about one long document
        {"name": "shared_long_16", "op": "shared", "seqs": 16, "groups": 1, "prefix": 65536,
         "suffix": 512, "heads": "8b", "page": 128, "fmt": "bf16"},
        # few-shot evaluation: a wide batch behind one prompt, FP8 cache
        {"name": "shared_wide_256", "op": "shared", "seqs": 256, "groups": 1, "prefix": 8192,
         "suffix": 512, "heads": "70b", "page": 64, "fmt": "e4m3"},
        # several prompts of unlike lengths, FP4 cache
        {"name": "shared_fp4_48", "op": "shared", "seqs": 48, "groups": 3, "prefix": 6144,
         "suffix": 384, "heads": "8b", "page": 64, "fmt": "nvfp4"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "shared", "shared"])
    heads = rng.choice(sorted(HEADS))
    hkv, group, d = HEADS[heads]
    if op == "shared":
        seqs = _log(rng, 1, 256)
        prefix = _log(rng, 64, 32768)
        # no dearer than 256 sequences of 8192 tokens over 8 kv heads
        prefix = max(64, min(prefix, (256 * 8192 * 8 * 128) // (seqs * hkv * d)))
        return {"op": op, "seqs": seqs, "groups": _log(rng, 1, max(1, seqs // 2)),
                "prefix": prefix, "suffix": _log(rng, 1, 512), "heads": heads,
                "page": rng.choice([64, 128]), "fmt": rng.choice(sorted(ELEM))}
    rotary = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
    case = {"op": op, "heads": heads, "rotary": rotary, "interleaved": rng.random() < 0.3,
            "norm": rng.random() < 0.6}
    if op == "rope":
        return {**case, "tokens": _log(rng, 1, 16384)}
    new = _log(rng, 1, 1024)
    return {**case, "seqs": _log(rng, 1, min(256, 16384 // new)), "new": new,
            "context": _log(rng, 1, 2048), "page": rng.choice([64, 128]),
            "fmt": rng.choice(["bf16", "e4m3"])}


def _lengths(case):
    """The ragged lengths of a case: the same for every seed."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["seqs"]
    if case["op"] == "append":
        new = [case["new"] if case["new"] == 1 else r.randint(1, case["new"]) for _ in range(n)]
        return [r.randint(0, case["context"]) for _ in range(n)], new
    cuts = sorted(r.sample(range(1, n), case["groups"] - 1)) if case["groups"] > 1 else []
    cu = [0, *cuts, n]
    page = case["page"]
    most = max(1, case["prefix"] // page)
    pages = [most if g == 0 else r.randint(max(1, most // 3), most) for g in range(len(cu) - 1)]
    lens = [p * page + r.randint(1, case["suffix"])
            for g, p in enumerate(pages) for _ in range(cu[g + 1] - cu[g])]
    return cu, [p * page for p in pages], lens


# ------------------------------------------------------------------ the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _rotation(case, gen, most):
    """cos and sin of the positions (a table that a program keeps) and the norms' weights."""
    hkv, group, d = HEADS[case["heads"]]
    half = case["rotary"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * inv
    s = {"cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(), "eps": 1e-6,
         "interleaved": case["interleaved"], "qw": None, "kw": None}
    if case["norm"]:
        s["qw"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=gen)
        s["kw"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=gen)
    return s


def _projection(case, gen, tokens):
    """q, k, v as slices of one fused projection's output."""
    hkv, group, d = HEADS[case["heads"]]
    hq = hkv * group
    x = torch.randn(tokens, hq + 2 * hkv, d, device="cuda", generator=gen).bfloat16()
    return {"q": x[:, :hq], "k": x[:, hq:hq + hkv], "v": x[:, hq + hkv:]}


def _pool_values(case, gen, pages):
    """A pool of K or V as a running program left it, and its scales."""
    hkv, group, d = HEADS[case["heads"]]
    shape, fmt = (pages, hkv, case["page"], d), case["fmt"]
    scale = 0.5 + torch.rand(pages, hkv, device="cuda", generator=gen)
    if fmt == "bf16":
        return torch.randn(shape, device="cuda", generator=gen, dtype=torch.bfloat16), None
    if fmt == "e4m3":
        x = 40 * torch.randn(shape, device="cuda", generator=gen, dtype=torch.bfloat16)
        return x.clamp_(-448, 448).to(torch.float8_e4m3fn), scale / 40
    if fmt == "int8":
        x = 40 * torch.randn(shape, device="cuda", generator=gen, dtype=torch.bfloat16)
        return x.clamp_(-127, 127).to(torch.int8), scale / 40
    rows = pages * hkv * case["page"]
    codes = torch.randint(0, 256, (rows * d // 2,), device="cuda", generator=gen,
                          dtype=torch.uint8)
    blocks = torch.randint(0x60, 0x7F, (rows * d // 16,), device="cuda", generator=gen,
                           dtype=torch.uint8)  # E4M3 bytes of 32 to 448
    return torch.cat([codes, blocks]), scale / 400


def prepare(case, seed):
    gen = _generator(seed)
    hkv, group, d = HEADS[case["heads"]]
    s = {"case": case}
    if case["op"] == "rope":
        s |= _rotation(case, gen, 32768) | _projection(case, gen, case["tokens"])
        s["positions"] = torch.randint(0, 32768, (case["tokens"],), device="cuda", generator=gen,
                                       dtype=torch.int32)
    elif case["op"] == "append":
        before, new = _lengths(case)
        total, page = sum(new), case["page"]
        need = [-(-(a + b) // page) for a, b in zip(before, new)]
        s |= _rotation(case, gen, 4096) | _projection(case, gen, total)
        order = torch.randperm(sum(need), device="cuda", generator=gen).int()
        table = torch.full((len(new), max(need)), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(max(need), device="cuda") < _ints(need)[:, None]
        table[held] = order
        s |= {"table": table, "before": _ints(before), "total": total,
              "cu": _ints([sum(new[:i]) for i in range(len(new) + 1)])}
        dt = torch.bfloat16 if case["fmt"] == "bf16" else torch.float8_e4m3fn
        for x in ("k", "v"):
            s[x + "_pool"] = torch.zeros(sum(need), hkv, page, d, device="cuda",
                                         dtype=torch.uint8 if case["fmt"] == "e4m3" else dt).view(dt)
            s[x + "_scale"] = None
            if case["fmt"] == "e4m3":
                s[x + "_scale"] = (4 + torch.rand(sum(need), hkv, device="cuda",
                                                  generator=gen)) / 448
    else:
        cu, prefix, lens = _lengths(case)
        page = case["page"]
        need = [-(-n // page) for n in lens]
        shared = [p // page for p in prefix]
        total = sum(shared) + sum(n - shared[g] for g in range(len(shared))
                                  for n in need[cu[g]:cu[g + 1]])
        order = torch.randperm(total, device="cuda", generator=gen).int()
        table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for g, p in enumerate(shared):
            table[cu[g]:cu[g + 1], :p] = order[at:at + p]
            at += p
            for b in range(cu[g], cu[g + 1]):
                table[b, p:need[b]] = order[at:at + need[b] - p]
                at += need[b] - p
        s |= {"table": table, "lens": _ints(lens), "max_len": max(lens), "cu_groups": _ints(cu),
              "prefix": _ints(prefix), "scale": 1 / math.sqrt(d)}
        s["q"] = torch.randn(len(lens), hkv * group, d, device="cuda", generator=gen).bfloat16()
        for x in ("k", "v"):
            s[x + "_pool"], s[x + "_scale"] = _pool_values(case, gen, total)
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    """What a program on the package keeps: the cache, the rotation, the workspace."""
    import paged_kv_cache_476_b200 as pkv

    hkv, group, d = HEADS[case["heads"]]
    s["flags"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] != "rope":
        pages = int(s["table"].max()) + 1
        s["cache"] = pkv.PagedKVCache(
            s["k_pool"], s["v_pool"], case["fmt"], s["k_scale"], s["v_scale"], s["flags"],
            geometry=(pages, hkv, case["page"], d) if case["fmt"] == "nvfp4" else None)
    if case["op"] == "shared":
        s["work"] = pkv.decode_shared_workspace(s["cache"], case["seqs"], hkv * group,
                                                s["max_len"], case["groups"])
    else:
        s["rope"] = pkv.Rope(s["cos_sin"], interleaved=s["interleaved"], q_norm_weight=s["qw"],
                             k_norm_weight=s["kw"], norm_eps=s["eps"])


# --------------------------------------------------------------- the operators
def run(s):
    case = s["case"]
    if own:
        import paged_kv_cache_476_b200 as pkv

        if case["op"] == "rope":
            return pkv.pkv_qk_norm_rope(s["rope"], s["q"], s["k"], s["positions"],
                                        error_flags=s["flags"])
        if case["op"] == "append":
            q = pkv.paged_kv_append_rope(s["cache"], s["rope"], s["table"], s["before"], s["cu"],
                                         s["k"], s["v"], q=s["q"], total_new_tokens=s["total"])
            return q, s["k_pool"], s["v_pool"]
        return pkv.paged_decode_attention_shared(s["cache"], s["q"], s["table"], s["lens"],
                                                 s["max_len"], s["cu_groups"], s["prefix"],
                                                 s["scale"], workspace=s["work"])
    if case["op"] == "rope":
        return (_rotated(s, s["q"], s["qw"], s["positions"]).bfloat16(),
                _rotated(s, s["k"], s["kw"], s["positions"]).bfloat16())
    if case["op"] == "append":
        return _append(s, case["page"])
    return _shared(s, case)


def _rotated(s, x, weight, positions):
    """Norm and rotation of every head of x, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight
    rot = s["cos_sin"].shape[1]
    at = s["cos_sin"][positions.long()][:, None]
    c, sn = at[..., :rot // 2], at[..., rot // 2:]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _append(s, page):
    token = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:], token, right=True)
    pos = s["before"][seq].long() + token - s["cu"][seq]
    at, slot = s["table"][seq, pos // page].long(), pos % page
    for x, new in (("k", _rotated(s, s["k"], s["kw"], pos)), ("v", s["v"].float())):
        pool, scale = s[x + "_pool"], s[x + "_scale"]
        if scale is None:
            pool[at, :, slot] = new.bfloat16()
        else:
            code = (new / scale[at][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            pool.view(torch.uint8)[at, :, slot] = code.view(torch.uint8)
    return _rotated(s, s["q"], s["qw"], pos).bfloat16(), s["k_pool"], s["v_pool"]


def _values(s, x, case, at, dtype):
    """The cached K or V of the pages `at` [n, pages]: [n, kv heads, tokens, head_dim]."""
    hkv, group, d = HEADS[case["heads"]]
    page, pool = case["page"], s[x + "_pool"]
    if case["fmt"] == "nvfp4":
        rows = pool.numel() // (d // 2 + d // 16)
        codes = pool[:rows * d // 2].view(-1, hkv, page, d // 2)[at]
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
        blocks = pool[rows * d // 2:].view(torch.float8_e4m3fn).view(-1, hkv, page, d // 16)
        e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                            dtype=dtype, device=pool.device)
        v = e2m1[codes] * blocks.to(dtype)[at].repeat_interleave(16, -1)
    elif case["fmt"] == "e4m3":
        v = pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).to(dtype)
    else:
        v = pool[at].to(dtype)
    if s[x + "_scale"] is not None:
        v = v * s[x + "_scale"].to(dtype)[at][..., None, None]
    n, pages = at.shape
    return v.transpose(1, 2).reshape(n, hkv, pages * page, d)


def _shared(s, case):
    hkv, group, d = HEADS[case["heads"]]
    at = s["table"].clamp(min=0).long()
    q = s["q"].float().view(-1, hkv, group, d)
    scores = (q @ _values(s, "k", case, at, torch.float32).transpose(-1, -2)) * s["scale"]
    seen = torch.arange(scores.shape[-1], device="cuda") < s["lens"][:, None]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ _values(s, "v", case, at, torch.float32)) / total
    lse = (top + torch.log(total)).squeeze(-1)
    return out.flatten(1, 2).bfloat16(), lse.flatten(1, 2)


# ----------------------------------------------------------- the work of a pass
def work(case):
    hkv, group, d = HEADS[case["heads"]]
    hq = hkv * group
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": t * (2 * (hq + hkv) * d * 2 + case["rotary"] * 4 + 4),
                "flops": t * (hq + hkv) * d * (7 if case["norm"] else 3)}
    eb = ELEM[case["fmt"]]
    if case["op"] == "append":
        t = sum(_lengths(case)[1])
        return {"bytes": t * ((2 * hq + 2 * hkv) * d * 2 + 2 * hkv * d * eb + case["rotary"] * 4),
                "flops": t * (hq + hkv) * d * (7 if case["norm"] else 3)}
    cu, prefix, lens = _lengths(case)
    own_tokens = sum(n - prefix[g] for g in range(len(prefix)) for n in lens[cu[g]:cu[g + 1]])
    return {"bytes": (sum(prefix) + own_tokens) * hkv * d * 2 * eb
            + len(lens) * hq * (d * 4 + 4),
            "flops": 4 * hq * d * sum(lens)}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    hkv, group, d = HEADS[case["heads"]]

    def turn(x, weight, where):
        x = x.double().clone()
        if weight is not None:
            x = x / (x.square().sum(-1, keepdim=True) / d + s["eps"]).sqrt() * weight.double()
        rows, half = s["cos_sin"].double()[where.long()], case["rotary"] // 2
        for i in range(half):
            i0, i1 = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            z = torch.complex(x[..., i0], x[..., i1]) * torch.complex(
                rows[:, i], rows[:, half + i])[:, None]
            x[..., i0], x[..., i1] = z.real, z.imag
        return x

    if case["op"] == "rope":
        return turn(s["q"], s["qw"], s["positions"]), turn(s["k"], s["kw"], s["positions"])
    if case["op"] == "append":
        before, new = _lengths(case)
        pos = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(before, new)])
        seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"),
                                      torch.tensor(new, device="cuda"))
        page = case["page"]
        row = s["table"].long()[seq, pos // page], pos % page
        pools = []
        for x, y in (("k", turn(s["k"], s["kw"], pos)), ("v", s["v"].double())):
            pool = torch.zeros(s[x + "_pool"].shape, dtype=torch.float64, device="cuda")
            if case["fmt"] == "e4m3":
                y = y / s[x + "_scale"].double()[row[0]][..., None]
            pool.permute(0, 2, 1, 3)[row[0], row[1]] = y
            pools.append(pool)
        return turn(s["q"], s["qw"], pos), *pools
    # one sequence at a time, page by page
    out, lse = [], []
    for b, n in enumerate(s["lens"].tolist()):
        at = s["table"][b:b + 1, :-(-n // case["page"])].long()
        k, v = (_values(s, x, case, at, torch.float64)[0, :, :n] for x in ("k", "v"))
        a = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(hkv, group, d), k) * s["scale"]
        lse.append(torch.logsumexp(a, -1).flatten())
        out.append(torch.einsum("hgn,hnd->hgd", torch.softmax(a, -1), v).reshape(-1, d))
    return torch.stack(out), torch.stack(lse)

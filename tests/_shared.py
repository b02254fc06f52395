"""Batches whose sequences share pages, and decode attention over them in 64 bits
(plain torch, any device; shares nothing with the library)."""
from __future__ import annotations

import random

import torch

E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


class Batch:
    """Sequences of `lens` tokens; group g (cu[g] .. cu[g + 1] - 1) shares the pages of
    its first prefix[g] tokens.  The pages lie in random order; all that no
    sequence holds is NaN (or the format's largest bytes), table entries past a
    sequence's last page are -1."""

    def __init__(self, lens, cu, prefix, Hkv, G, D, page, fmt="bf16", seed=0, device="cuda",
                 spread=1.0):
        r = random.Random(seed)
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.cu, self.prefix = list(lens), list(cu), list(prefix)
        self.Hkv, self.G, self.D, self.page, self.fmt = Hkv, G, D, page, fmt
        B = len(lens)
        need = [-(-n // page) for n in lens]
        shared = [0] * B
        for g, p in enumerate(prefix):
            for b in range(cu[g], cu[g + 1]):
                shared[b] = min(p // page, need[b])
        owner, rows = {}, []
        for b in range(B):
            g = next((g for g in range(len(prefix)) if cu[g] <= b < cu[g + 1]), None)
            rows.append([owner.setdefault((g, j) if j < shared[b] else (b, j, "own"), len(owner))
                         for j in range(need[b])])
        self.pages = len(owner) + 2  # two pages nobody holds
        order = list(range(self.pages))
        r.shuffle(order)
        self.table = torch.full((B, max([1, *need]) + 1), -1, dtype=torch.int32)
        live = torch.zeros(self.pages, page, dtype=torch.bool)
        for b, row in enumerate(rows):
            for j, p in enumerate(row):
                self.table[b, j] = order[p]
                live[order[p], :lens[b] - j * page] = True
        shape = (self.pages, Hkv, page, D)
        dead = ~live[:, None, :, None].expand(shape)
        self.scales = [None, None]
        self.pools, self.values = [], []
        for i in range(2):
            s = 2.0 ** (spread * (torch.rand(self.pages, Hkv, generator=gen) - 0.5)).float()
            if fmt == "bf16":
                pool = torch.randn(shape, generator=gen).bfloat16()
                pool[dead] = float("nan")
                v = pool.double()
            elif fmt == "nvfp4":
                s = s / 300
                codes = torch.randint(0, 256, (*shape[:3], D // 2), generator=gen, dtype=torch.uint8)
                blocks = torch.randint(0x60, 0x7F, (*shape[:3], D // 16), generator=gen,
                                       dtype=torch.uint8)
                blocks[~live[:, None, :].expand(shape[:3])] = 0x7F  # NaN
                pool = torch.cat([codes.flatten(), blocks.flatten()])
                nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
                v = torch.tensor(E2M1, dtype=torch.float64)[nib] * \
                    blocks.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
            else:
                x = torch.randn(shape, generator=gen) * 40
                if fmt == "e4m3":
                    pool = x.clamp(-448, 448).to(torch.float8_e4m3fn)
                    v = pool.double()
                    pool = pool.view(torch.uint8)
                    pool[dead] = 0x7F  # NaN
                else:
                    pool = x.round().clamp(-127, 127).to(torch.int8)
                    v = pool.double()
                    pool[dead] = 127
                s = s / 40
            if fmt != "bf16":
                self.scales[i] = s.to(device)
                v = v * s.double()[:, :, None, None]
            v[dead] = 0.0
            self.pools.append(pool.to(device))
            self.values.append(v.to(device))
        self.q = torch.randn(B, Hkv * G, D, generator=gen).bfloat16().to(device)
        self.table = self.table.to(device)
        self.scale = D ** -0.5

    def cache(self, pkv):
        self.flags = torch.zeros(1, dtype=torch.int32, device=self.q.device)
        return pkv.PagedKVCache(*self.pools, self.fmt, *self.scales, self.flags,
                                geometry=(self.pages, self.Hkv, self.page, self.D)
                                if self.fmt == "nvfp4" else None)

    def shared_tokens(self, b):
        """Tokens of sequence b that are read for its group."""
        for g, p in enumerate(self.prefix):
            if self.cu[g] <= b < self.cu[g + 1]:
                n = p // self.page * self.page
                return n if self.lens[b] >= n and self.cu[g + 1] - self.cu[g] > 1 else 0
        return 0

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.q.device)

    def args(self):
        """(q, table, lens, max_len, cu_groups, prefix_lens) of the shared entry point."""
        return (self.q, self.table, self.ints(self.lens), max(self.lens), self.ints(self.cu),
                self.ints(self.prefix))


def exact(batch):
    """out [B, Hq, D], lse [B, Hq] in fp64, and the bounds of their errors.

    The kernels' error: a score's products are exact in fp32 and their sum of D
    <= 128 terms, its scale and its reference cost at most 131 half-ulps
    (2^-24): ds = 2^-16 sum |q k| scale.  INT8 pools may see q in 13-bit fixed
    point, off by 2^-14 of its row's largest value: ds += 2^-14 amax sum |k|
    scale.  A weight then errs by 2 ds (itself and the sum), by its rounding
    to bf16 (2^-8), by 2^-18 for the exponentials and the joins of parts, and
    by 2^-25 of the largest weight where it is small in f16; the output rounds
    to bf16 once more.  The logarithm of the sum errs by ds, 2^-18, and 2^-22 of
    itself.

    Tokens that go through paged_decode_attention's kernel (all but the prefix)
    have their weight times the page's V scale vs in f16: below 2^-14 that is a
    multiple of 2^-24, so off by 2^-25 whatever vs is.  With weights relative
    to the largest (l >= 1 / its softmax value pmax) such a token adds
    2^-25 (|v| / vs) pmax to the error, which is more than the 2^-25 |v| pmax
    above where vs < 1.
    """
    b0 = batch
    dev = b0.q.device
    B, Hq, D = b0.q.shape
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, Hq), -torch.inf, dtype=torch.float64, device=dev)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(b0.lens):
        if n == 0:
            continue
        at = b0.table[b, :-(-n // b0.page)].long()
        k, v = (x[at].transpose(0, 1).reshape(b0.Hkv, -1, D)[:, :n] for x in b0.values)
        q = b0.q[b].double().view(b0.Hkv, b0.G, D)
        s = (q @ k.transpose(1, 2)) * b0.scale
        ds = 2.0 ** -16 * (q.abs() @ k.abs().transpose(1, 2)).amax(-1) * b0.scale
        if b0.fmt == "int8":
            ds = ds + 2.0 ** -14 * q.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None] * b0.scale
        p = torch.softmax(s, -1)
        o = p @ v
        mag = p @ v.abs()
        vmax = v.abs().amax((1, 2))[:, None, None]
        err = mag * (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -18) \
            + n * 2.0 ** -25 * p.amax(-1)[..., None] * vmax
        own = b0.shared_tokens(b)
        if b0.fmt != "bf16" and own < n:
            vs = b0.scales[1][at].double().T.repeat_interleave(b0.page, 1)[:, own:n].clamp(max=1)
            per = (v[:, own:].abs().amax(-1) / vs).amax(-1)
            err = err + (n - own) * 2.0 ** -25 * p[..., own:].amax(-1)[..., None] * per[:, None, None]
        out[b] = o.view(Hq, D)
        tol[b] = (err + 2.0 ** -8 * (o.abs() + err)).view(Hq, D)
        lse[b] = torch.logsumexp(s, -1).flatten()
        tol_lse[b] = (ds + 2.0 ** -18).flatten() + 2.0 ** -22 * lse[b].abs()
    return out, lse, tol, tol_lse


def assert_exact(got, batch, rows=None):
    out, lse, tol, tol_lse = exact(batch)
    rows = slice(None) if rows is None else rows
    o, l = got[0].double()[rows], got[1].double()[rows]
    out, lse, tol, tol_lse = out[rows], lse[rows], tol[rows], tol_lse[rows]
    err = (o - out).abs()
    assert bool((err <= tol).all()), (int((~(err <= tol)).sum()), float((err / tol).nan_to_num(9e9).max()))
    empty = torch.isinf(lse)
    assert torch.equal(l[empty], lse[empty])
    err = (l - lse)[~empty].abs()
    assert bool((err <= tol_lse[~empty]).all()), float((err / tol_lse[~empty]).max())

"""Plain fp64 head norm and position rotation, and the check of pool codes
against it (numpy; shares nothing with the library)."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def table64(positions, rot, base=10000.0):
    """cos, sin [T, rot/2] as the fp32 values the table holds."""
    inv = base ** (-np.arange(rot // 2, dtype=np.float64) / max(rot // 2, 1))
    a = np.asarray(positions, np.float64)[:, None] * inv
    return np.cos(a).astype(np.float32).astype(np.float64), \
        np.sin(a).astype(np.float32).astype(np.float64)


def rope64(x, positions, rot, interleaved, weight=None, eps=1e-6):
    """x [T, H, D] fp64 -> (z, mag): the exact rows, and per value the sum of the
    magnitudes that enter it (what an fp32 evaluation's error scales with)."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x * np.asarray(weight, np.float64) / np.sqrt(
            np.mean(x * x, -1, keepdims=True) + np.float64(np.float32(eps)))
    z, mag = x.copy(), np.abs(x)
    if rot:
        c, s = (t[:, None, :] for t in table64(positions, rot))
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        z[..., a] = x[..., a] * c - x[..., b] * s
        z[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return z, mag


# Relative error of the fp32 evaluation, against the magnitudes above: the sum
# of D <= 128 squares in a tree of depth <= 16 + 3 adds at most 19 half-ulps
# (2^-24 each) and a product's 1, of which the root keeps half (10); mean and
# eps 2 more halved (1); the root's reciprocal <= 2 ulps (4); two products with
# the weight (2); the rotation's product and fused add (2): 19 * 2^-24 < 2^-19.
FP32_REL = 2.0 ** -19


def assert_bf16_rows(out, z, mag):
    """bf16 results: half a step (2^-8 of the value) off the fp32 evaluation."""
    o = out.detach().float().cpu().numpy().astype(np.float64)
    err32 = FP32_REL * mag
    tol = err32 + 2.0 ** -8 * (np.abs(z) + err32) + 2.0 ** -133
    bad = np.abs(o - z) > tol
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(o - z) / tol)))


def assert_codes(fmt, rows, scale, z, mag):
    """Codes of K rows: `rows` [N, bytes] (FP4: codes then block scales), `scale`
    [N], exact values z [N, D].  Each code is within half a step of the exact
    quotient, moved by at most the fp32 error (and the quotient's rounding)."""
    s = scale[:, None].astype(np.float64)
    y, err = z / s, (FP32_REL * mag + 2.0 ** -23 * np.abs(z)) / s
    if fmt == "e4m3":
        v = torch.from_numpy(rows.copy()).view(torch.float8_e4m3fn).double().numpy()
        half = np.maximum(2.0 ** -4 * (np.abs(y) + err), 2.0 ** -10)  # subnormal step 2^-9
        y = np.clip(y, -448, 448)
        assert np.all(np.abs(v - y) <= half + err)
    elif fmt == "int8":
        v = rows.view(np.int8).astype(np.float64)
        assert np.all(np.abs(v - np.clip(y, -127, 127)) <= 0.5 + err)
    else:
        D = z.shape[1]
        codes, blocks = rows[:, :D // 2], rows[:, D // 2:]
        v = np.empty_like(z)
        for par, nib in ((0, codes & 15), (1, codes >> 4)):
            v[:, par::2] = np.where(nib & 8, -1, 1) * E2M1[nib & 7]
        sb = torch.from_numpy(blocks.copy()).view(torch.float8_e4m3fn).double().numpy()
        amax = np.abs(y).reshape(len(y), -1, 16).max(-1) / 6
        aerr = err.reshape(len(y), -1, 16).max(-1) / 6 + 2.0 ** -22 * amax
        half = np.maximum(2.0 ** -4 * (amax + aerr), 2.0 ** -10)
        assert np.all(np.abs(sb - np.minimum(amax, 448)) <= half + aerr)
        d = np.repeat(sb, 16, axis=1)
        with np.errstate(divide="ignore", invalid="ignore"):
            w, werr = np.where(d > 0, y / d, 0.0), np.where(d > 0, (err + 2.0 ** -23 * np.abs(y)) / d, 0)
        top = np.abs(w) + werr  # half a step at the larger magnitude; 6 and beyond saturate
        half = np.where(top <= 2, 0.25, np.where(top <= 4, 0.5, 1.0))
        assert np.all(np.abs(v - np.clip(w, -6, 6)) <= half + werr)

"""The training and 8-bit operators in 64 bits (torch, float64), and the error
bounds that their tests hold the kernels to.

Each reference returns (value, size) pairs: `size` is the same sum with every
product taken positive.  A kernel that rounds a factor of the sum n times and
its result once, each by at most u = eps / 2 of the value, and adds K products
in fp32, is off by at most

    (n u + (K + SLACK) 2^-24) size + u |value|

to first order.  SLACK covers the gate's exponential, reciprocal and products.
Over many outputs such errors have either sign, so the 2-norm of the
difference is also held to (n + 1) u + (K + SLACK) 2^-24 of the result's.
"""
from __future__ import annotations

import torch

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SLACK = 64


def assert_close(name, got, ref, size, K, dtype, inner=0, floor=1e-37, split=0.0):
    """got against the 64-bit ref; inner: roundings of the factors on the way (of `dtype`);
    floor: what is lost to fp32's smallest numbers; split: what a factor held as two bf16
    values is off by (2^-8 of the residual, itself 2^-8 of the value)."""
    u, v = U[dtype], 2.0 ** -24 * (K + SLACK) + split
    got, diff = got.double(), (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    bound = (inner * u + v) * size + u * ref.abs() + floor
    bad = diff > bound
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values over their bound, worst "
                           f"{float((diff / bound).max()):.3g} times at {int((diff / bound).argmax())}")
    norm = float(ref.norm())
    rel = float(diff.norm()) / norm if norm else float(diff.norm())
    far = (inner + 1) * u + v * float(size.norm()) / max(norm, 1e-300)
    assert rel <= far, f"{name}: 2-norm error {rel:.3g}, bound {far:.3g}"
    return rel


def silu_parts(g):
    s = torch.sigmoid(g)
    return s, s * (1 + g * (1 - s))


def ffn_train(x, offsets, w1, w3, w2):
    """gate, up, h as (value, size), rows past the last group zero."""
    n, d, F = x.shape[0], x.shape[1], w1.shape[1]
    z = lambda c: torch.zeros((n, c), dtype=torch.float64, device=x.device)  # noqa: E731
    out = {k: (z(c), z(c)) for k, c in (("gate", F), ("up", F), ("h", d))}
    for e in range(w1.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        X, A, B, C = (t.double() for t in (x[a:b], w1[e], w3[e], w2[e]))
        g, u = X @ A.T, X @ B.T
        sg, su = X.abs() @ A.abs().T, X.abs() @ B.abs().T
        act = g * torch.sigmoid(g) * u
        out["gate"][0][a:b], out["gate"][1][a:b] = g, sg
        out["up"][0][a:b], out["up"][1][a:b] = u, su
        out["h"][0][a:b], out["h"][1][a:b] = act @ C.T, act.abs() @ C.abs().T
        # errors of the fp32 sums g and u move act by at most 1.1 |u| sg + |silu(g)| su a unit
        move = 1.1 * u.abs() * sg + (g * torch.sigmoid(g)).abs() * su
        out.setdefault("h_move", z(d))[a:b] = move @ C.abs().T
    return out


def ffn_backward(x, offsets, w1, w3, w2, gate, up, dh):
    """dx_perm, dw1, dw3, dw2 as (value, size)."""
    n, d, F, E = x.shape[0], x.shape[1], w1.shape[1], w1.shape[0]
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=x.device)  # noqa: E731
    shapes = {"dx_perm": (n, d), "dw1": (E, F, d), "dw3": (E, F, d), "dw2": (E, d, F)}
    out = {k: (z(*s), z(*s)) for k, s in shapes.items()}
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        X, A, B, C, g, u, H = (t.double() for t in (x[a:b], w1[e], w3[e], w2[e], gate[a:b], up[a:b], dh[a:b]))
        s, slope = silu_parts(g)
        da, ada = H @ C, H.abs() @ C.abs()
        act, dg, du = g * s * u, da * u * slope, da * g * s
        # sizes: da by its own sum (its fp32 error enters dg and du), slope by its largest terms
        sdg, sdu = ada * u.abs() * (s * (1 + g.abs())), ada * (g * s).abs()
        for k, v, size in (("dw2", H.T @ act, H.abs().T @ act.abs()),
                           ("dw1", dg.T @ X, dg.abs().T @ X.abs()), ("dw3", du.T @ X, du.abs().T @ X.abs())):
            out[k][0][e], out[k][1][e] = v, size
        out["dx_perm"][0][a:b] = dg @ A + du @ B
        out["dx_perm"][1][a:b] = dg.abs() @ A.abs() + du.abs() @ B.abs()
        # what the fp32 error of da adds, a unit of 2^-24 (d + SLACK) each
        out.setdefault("dx_move", z(n, d))[a:b] = sdg @ A.abs() + sdu @ B.abs()
        out.setdefault("dw1_move", z(E, F, d))[e] = sdg.T @ X.abs()
        out.setdefault("dw3_move", z(E, F, d))[e] = sdu.T @ X.abs()
    return out


def quantize(v):
    """int8 values (as float64) and fp32 scales of the rows of v."""
    amax = v.abs().amax(-1, keepdim=True).float()
    scale = torch.clamp(amax / torch.full_like(amax, 127.0), min=2.0 ** -126)
    return torch.round(v.double() / scale.double()), scale

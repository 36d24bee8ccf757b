"""Orthogonalisation and the Muon step on the GPU against the definition in 64 bits.

Tolerances.  A step's factors are rounded: X, A and B each by half a step u of what the
products read (2^-11 relative in fp16; `precise`: 2^-21, for two parts and the product of
the lower ones that is left out), sums of K products in fp32 by at most K 2^-24 of the sum of
their magnitudes.  With the norms of the exact X_k, A_k and B_k that gives what a step adds
to the error of X_{k+1} in the 2-norm of all elements (`step_error`); what is there already
grows by at most the largest slope of the polynomial on the values that occur, since the
derivative of such a matrix function is bounded by its divided differences.
"""
import math
import struct

import numpy as np
import pytest
import torch

import zero_partitioned_mixed_shard_amd as Z

pytestmark = pytest.mark.gpu

A, B, C, EPS = 3.4445, -4.7750, 2.0315, 1e-7
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def half_step(t):
    return torch.finfo(t).eps / 2


def polynomial(g, precise=False, steps=5, a=A, b=B, c=C, eps=EPS):
    """(orth(g), bound of the kernel's error in the 2-norm) in 64 bits on the CPU."""
    g = g.double().cpu()
    x = g if g.shape[0] <= g.shape[1] else g.t()
    x = x / (x.norm() + eps)
    m, n = x.shape
    u = 2.0 ** -21 if precise else 2.0 ** -11
    err = 2.0 ** -21 * float(x.norm())          # X_0's two parts, the factor's rounding
    for _ in range(steps):
        s = x @ x.t()
        q = b * s + c * s @ s
        top = float(torch.linalg.matrix_norm(x, 2))
        xf, sf, qf = float(x.norm()), float(s.norm()), float(q.norm())
        # sums of K products, in each element at most K 2^-24 |row| |row|
        d_s = 2 * u * top * xf + n * 2.0 ** -24 * xf * xf + u * sf
        d_q = (abs(b) + 2 * abs(c) * top ** 2) * d_s + abs(c) * m * 2.0 ** -24 * sf * sf + u * qf \
            + 4 * 2.0 ** -24 * (abs(b) * sf + abs(c) * sf * top ** 2)
        d_x = d_q * top + u * float(torch.linalg.matrix_norm(q, 2)) * xf + m * 2.0 ** -24 * qf * xf \
            + 2.0 ** -21 * abs(a) * xf
        v = torch.linspace(0, max(top, 1e-3) * 1.02, 4001, dtype=torch.float64)
        slope = float((a + 3 * b * v ** 2 + 5 * c * v ** 4).abs().max())
        err = slope * err + d_x
        x = a * x + q @ x
    return (x if g.shape[0] <= g.shape[1] else x.t()), 1.05 * err


def update(rows, cols, seed, kind="normal"):
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn(rows, cols, generator=gen, dtype=torch.float64)
    if kind == "low":
        k = max(1, min(rows, cols) // 16)
        g = torch.randn(rows, k, generator=gen, dtype=torch.float64) @ \
            torch.randn(k, cols, generator=gen, dtype=torch.float64) / math.sqrt(k) + 0.05 * g
    return g * 0.01


def workspace(plan):
    # whatever it holds does not matter
    return torch.full((max(1, Z.zero_matrix_workspace_bytes(plan)),), 0xFF, dtype=torch.uint8,
                      device="cuda")


def check(got, g, out_type, precise, **ns):
    want, bound = polynomial(g, precise, **ns)
    off = float((got.double().cpu() - want).norm())
    size = float(want.norm())
    least = 2.0 ** -25 * math.sqrt(want.numel()) if out_type == torch.float16 else 0.0
    limit = bound + half_step(out_type) * (size + bound) + least
    assert off <= limit, (off / size, limit / size)
    return off / size if size else 0.0


SIZES = [(64, 40000), (40001, 5), (1, 1), (1, 7), (7, 1), (1, 1000), (3, 200), (16, 1025), (1025, 16), (63, 65), (64, 64), (65, 64),
         (64, 130), (128, 128), (129, 500), (500, 129), (256, 1030), (1025, 1100), (1300, 1025)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("precise", [False, True])
def test_sizes(rows, cols, precise):
    g = update(rows, cols, rows * 31 + cols).float().cuda()
    out = torch.full((rows, cols), 7.0, device="cuda")
    plan = Z.zero_matrix_plan([g], out=[out], precise=precise)
    Z.zero_orthogonalize(plan, workspace(plan))
    check(out, g, torch.float32, precise)


@pytest.mark.parametrize("src", sorted(TYPES))
@pytest.mark.parametrize("dst", sorted(TYPES))
@pytest.mark.parametrize("kind", ["normal", "low"])
def test_types(src, dst, kind):
    shapes = [(200, 333), (70, 40), (333, 200), (129, 130)]
    g = [update(r, c, k, kind).to(TYPES[src]).cuda() for k, (r, c) in enumerate(shapes)]
    out = [torch.zeros(s, dtype=TYPES[dst], device="cuda") for s in shapes]
    plan = Z.zero_matrix_plan(g, out=out)
    assert plan.precise == (dst == "fp32")
    Z.zero_orthogonalize(plan, workspace(plan))
    for x, y in zip(g, out):
        check(y, x, TYPES[dst], plan.precise)


def result(sumsq=0.0, overflow=0, inv=1.0):
    return torch.frombuffer(bytearray(struct.pack("<dIf", sumsq, overflow, inv)), dtype=torch.int32).cuda()


def muon_state(matrices, count, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    p = torch.randn(count, generator=gen) * 0.02
    m = torch.randn(count, generator=gen) * 1e-3
    g = torch.zeros(count)
    for k, (at, r, c) in enumerate(matrices):
        g[at:at + r * c] = update(r, c, seed + k, "low").float().reshape(-1)
    return p.cuda(), m.cuda(), p.to(TYPES[dtype]).cuda(), (g * 0.1).to(TYPES[dtype]).cuda()


def muon_reference(p, m, g, matrices, hp, inv, coef, precise=False):
    """(p, m, bound of |error of p| in the 2-norm, per matrix) in 64 bits on the CPU."""
    p, m, g = p.double().cpu().clone(), m.double().cpu().clone(), g.double().cpu()
    found = []
    for at, r, c in matrices:
        s = slice(at, at + r * c)
        gg = g[s] * inv * coef
        m[s] = hp.momentum * m[s] + gg
        u = gg + hp.momentum * m[s] if hp.nesterov else m[s]
        o, bound = polynomial(u.view(r, c), precise)
        alpha = {0: 1.0, 1: math.sqrt(max(1.0, r / c)), 2: 0.2 * math.sqrt(max(r, c))}[hp.scaling]
        # the update itself is rounded too: u to 3 half steps of fp32, which 5 steps
        # multiply by at most 3.45 each
        bound += 3 * 2.0 ** -24 * 3.45 ** 5
        size = float(p[s].norm())
        p[s] = p[s] * (1.0 - hp.lr * hp.weight_decay) - hp.lr * alpha * o.reshape(-1)
        found.append((s, hp.lr * alpha * (bound + 2.0 ** -23 * float(o.norm())) + 3 * 2.0 ** -24 * size))
    return p, m, found


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nesterov,scaling,clip,precise", [(True, "rms", 0.0, False), (False, None, 0.5, False),
                                                           (True, "aspect", 2.0, True)])
def test_muon_step(dtype, nesterov, scaling, clip, precise):
    # odd offsets, gaps between the matrices, wide and tall, small and beyond one tile
    matrices, at = [], 3
    for r, c in [(64, 200), (300, 130), (1, 50), (40, 1), (257, 257), (129, 1025)]:
        matrices.append((at, r, c))
        at += r * c + 5
    p, m, p16, g = muon_state(matrices, at, dtype, 5)
    inv = 0.25
    before = [x.clone() for x in (p, m, p16, g)]
    sumsq = float((g.float() * inv).double().square().sum())
    coef = min(1.0, clip / (math.sqrt(sumsq) + 1e-6)) if clip else 1.0
    hp = Z.zero_muon_hparams(lr=0.01, momentum=0.9, weight_decay=0.1, max_grad_norm=clip,
                             nesterov=nesterov, scaling=scaling)
    plan = Z.zero_muon_plan(matrices, precise=precise)
    assert plan.extent == at - 5
    Z.zero_muon_step(p, m, p16, g, plan, hp, result(sumsq, 0, inv), workspace(plan))
    wp, wm, bounds = muon_reference(before[0], before[1], g, matrices, hp, inv, coef, precise)
    off = (m.double().cpu() - wm).abs()
    assert bool((off <= 4 * 2.0 ** -24 * (before[1].double().cpu().abs() + (g.double().cpu() * inv).abs())
                 + 1e-45).all())
    for s, bound in bounds:
        assert float((p[s].double().cpu() - wp[s]).norm()) <= bound, s
    assert torch.equal(p16.view(torch.int16).cpu(), torch.where(
        torch.zeros(at, dtype=torch.bool).index_fill_(0, torch.cat([torch.arange(a, a + r * c) for a, r, c in matrices]), True),
        p.to(TYPES[dtype]).cpu().view(torch.int16), before[2].cpu().view(torch.int16)))
    # nothing between the matrices changes, nor the gradient
    inside = torch.zeros(at, dtype=torch.bool)
    for a, r, c in matrices:
        inside[a:a + r * c] = True
    for x, y in ((p, before[0]), (m, before[1])):
        assert torch.equal(x.cpu()[~inside], y.cpu()[~inside])
    assert torch.equal(g, before[3])

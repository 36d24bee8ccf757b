"""The Muon step, alone and in ShardStep, against its definition in 64 bits, in limits that a step
without decay, of the other momentum or 5 % too long or short would miss.

Limits.  An update to 32 bits is off by at most 5e-5 of its norm (the header's, for these
matrices; of shorter sides up to 64 by the 24 bits of its factors, amplified by at most 3.45
a step), of one fp16 part by 2e-3; a weight's step is two products and a difference in fp32,
each off by 2^-24 of its operands.
"""
import math
import struct

import numpy as np
import pytest
import torch

import zero_partitioned_mixed_shard_amd as Z
from zero_partitioned_mixed_shard_amd.shard import ShardStep

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def single(x):
    return float(np.float32(x))


A, B, C, EPS = single(3.4445), single(-4.7750), single(2.0315), single(1e-7)


def orth64(g):
    x = g.double()
    x = x / (x.norm() + EPS)
    wide = x if x.shape[0] <= x.shape[1] else x.t()
    for _ in range(5):
        s = wide @ wide.t()
        wide = A * wide + (B * s + C * s @ s) @ wide
    return wide if g.shape[0] <= g.shape[1] else wide.t()


def gradient(rows, cols, gen):
    """A part of low rank and noise."""
    k = max(1, min(rows, cols) // 8)
    return torch.randn(rows, k, generator=gen) @ torch.randn(k, cols, generator=gen) / math.sqrt(k) + \
        0.5 * torch.randn(rows, cols, generator=gen)


SHAPES = [(64, 200), (300, 130), (1, 50), (40, 1), (257, 257), (129, 1025), (1100, 300)]


def flat(seed, dtype, gap=5):
    """(matrices, master, momentum, gradient) with odd offsets and gaps."""
    gen, matrices, at = torch.Generator().manual_seed(seed), [], 3
    for r, c in SHAPES:
        matrices.append((at, r, c))
        at += r * c + gap
    p, m, g = torch.randn(at, generator=gen) * 0.02, torch.zeros(at), torch.zeros(at)
    for o, r, c in matrices:
        m[o:o + r * c] = gradient(r, c, gen).reshape(-1) * 3e-3
        g[o:o + r * c] = gradient(r, c, gen).reshape(-1) * 1e-3
    return matrices, p, m, (g * 64).to(TYPES[dtype])


def reference(p, m, g, matrices, hp, inv, coef, **change):
    """(p, m) in 64 bits; change: nesterov, decay or a factor of the step, as a mistake would."""
    p, m, g = p.double().clone(), m.double().clone(), g.double()
    for o, r, c in matrices:
        s = slice(o, o + r * c)
        gg = g[s] * inv * coef
        m[s] = hp.momentum * m[s] + gg
        u = gg + hp.momentum * m[s] if change.get("nesterov", hp.nesterov) else m[s]
        alpha = {0: 1.0, 1: math.sqrt(max(1.0, r / c)), 2: 0.2 * math.sqrt(max(r, c))}[hp.scaling]
        o64 = orth64(u.view(r, c)).reshape(-1)
        p[s] = p[s] * (1.0 - hp.lr * change.get("decay", hp.weight_decay)) - \
            hp.lr * alpha * change.get("factor", 1.0) * o64
    return p, m


def step_limit(p, o, s, hp, precise):
    """Of the 2-norm of a matrix's weights after the step."""
    r, c = s
    update = hp.lr * {0: 1.0, 1: math.sqrt(max(1.0, r / c)), 2: 0.2 * math.sqrt(max(r, c))}[hp.scaling] * o
    own = 3.45 ** 5 * 2.0 ** -22 if min(r, c) <= 64 else 5e-5 if precise else 2e-3
    return own * update + 2.0 ** -23 * (p + update)


def result(sumsq, overflow=0, inv=1.0):
    return torch.frombuffer(bytearray(struct.pack("<dIf", sumsq, overflow, inv)), dtype=torch.int32).cuda()


def test_shard_step_takes_32_bits_on_request():
    o, r, c = 0, 200, 260
    start = (torch.randn(r * c, generator=torch.Generator().manual_seed(1)) * 0.02).half()
    grad = (gradient(r, c, torch.Generator().manual_seed(2)) * 0.05).half().reshape(-1)
    off = []
    for precise in (False, True):
        st = ShardStep(0, r * c, [(0, r * c)], Z.ZERO_FP16, lr=0.01, matrices=[(o, r, c)], muon_precise=precise)
        assert st.muon_plan.precise == precise
        st.load_param16(start.cuda())
        assert st.step([grad.cuda()]).applied
        want, _ = reference(start, torch.zeros(r * c), grad, [(o, r, c)], st.muon_hp, 1.0, 1.0)
        update = float((want - start.double() * (1 - st.muon_hp.lr * st.muon_hp.weight_decay)).norm())
        off.append(float((st.master.double().cpu() - want).norm()) / update)
    assert off[0] <= 2e-3 and off[1] <= 1e-5


def test_shard_step_clips_matrices_and_the_rest_alike():
    """A clip given to the step, none to muon: the matrices take it too.  The momentum after the
    first step is the clipped gradient, element by element."""
    rows, cols, rest = 40, 70, 500
    n = rows * cols + rest
    gen = torch.Generator().manual_seed(3)
    start = (torch.randn(n, generator=gen) * 0.02).half()
    grad = (torch.randn(n, generator=gen) * 0.1).half()
    clip = 0.25
    coef = clip / (float(grad.double().norm()) + 1e-6)
    assert coef < 0.1
    muon = Z.zero_muon_hparams(lr=0.01, weight_decay=0.1)
    st = ShardStep(0, n, [(0, n)], Z.ZERO_FP16, lr=0.01, weight_decay=0.1, max_grad_norm=clip,
                   matrices=[(0, rows, cols)], muon=muon)
    assert st.muon_hp is muon and muon.max_grad_norm == 0
    st.load_param16(start.cuda())
    assert st.step([grad.cuda()]).applied
    g = grad.double() * coef
    got = st.exp_avg.double().cpu()
    inside, beta1 = slice(0, rows * cols), single(0.9)
    # two products, the coefficient's own rounding, and AdamW's (1 - beta1)
    assert bool(((got - g)[inside].abs() <= 4 * 2.0 ** -24 * g[inside].abs() + 1e-45).all())
    assert bool(((got - (1 - beta1) * g)[rows * cols:].abs() <= 2.0 ** -20 * g[rows * cols:].abs()).all())
    want, _ = reference(start, torch.zeros(n), grad, [(0, rows, cols)], muon, 1.0, coef)
    o = float(orth64(g[inside].view(rows, cols)).norm())
    off = float((st.master.double().cpu() - want)[inside].norm())
    assert off <= step_limit(float(start.double()[inside].norm()), o, (rows, cols), muon, False)
    # the clip follows the step's own, and the learning rate muon's
    before, st.hp.max_grad_norm, muon.lr, muon.weight_decay = st.exp_avg.clone(), 0.0, 0.0, 0.0
    master = st.master.clone()
    assert st.step([grad.cuda()]).applied
    want = single(0.95) * before.double().cpu()[inside] + grad.double()[inside]
    assert bool(((st.exp_avg.double().cpu()[inside] - want).abs() <= 2.0 ** -22 * (want.abs() + grad.double()[inside].abs())).all())
    assert torch.equal(st.master[inside], master[inside])


def test_two_clips_are_refused():
    kw = dict(matrices=[(0, 8, 9)])
    for step_clip, muon_clip in ((1.0, 0.5), (0.0, 1.0)):
        with pytest.raises(ValueError, match="clip"):
            ShardStep(0, 72, [(0, 72)], Z.ZERO_FP16, max_grad_norm=step_clip,
                      muon=Z.zero_muon_hparams(max_grad_norm=muon_clip), **kw)
    for step_clip, muon_clip in ((1.0, 1.0), (0.1, 0.1), (1.0, 0.0), (0.0, 0.0), (0.0, -1.0)):
        ShardStep(0, 72, [(0, 72)], Z.ZERO_FP16, max_grad_norm=step_clip,
                  muon=Z.zero_muon_hparams(max_grad_norm=muon_clip), **kw)


def test_captured_step_clips():
    """Captured and replayed, the clip is the capture's; with an active one every replay is the
    eager step's."""
    matrices, p, m, g = flat(4, "bf16")
    n = p.numel()
    kw = dict(lr=0.01, max_grad_norm=0.01, matrices=matrices, device_control=True, own_ranks=True, world=1)
    steps = [ShardStep(0, n, [(0, n)], Z.ZERO_BF16, muon=Z.zero_muon_hparams(lr=0.01), **kw) for _ in range(2)]
    for st in steps:
        st.load_param16(p.bfloat16().cuda())
        st.rank_bufs[0].copy_(g)
    graph = steps[0].capture()
    for k in range(3):
        for st in steps:
            st.rank_bufs[0].copy_(g * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        steps[1].step()
        for x, y in zip((steps[0].master, steps[0].exp_avg, steps[0].param16),
                        (steps[1].master, steps[1].exp_avg, steps[1].param16)):
            assert torch.equal(x, y), k
    assert float((steps[1].exp_avg[matrices[1][0]:matrices[2][0]]).norm()) < 0.05


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("nesterov,scaling,clip", [(True, "rms", 0.0), (False, "rms", 0.01), (True, "aspect", 0.01),
                                                   (False, None, 0.0), (True, None, 1e9)])
def test_step(dtype, precise, nesterov, scaling, clip):
    matrices, p, m, g = flat(11, dtype)
    inv = 2.0 ** -6
    # the norm is of the whole gradient, of all owners: larger than these matrices'
    sumsq = 9.0 * float((g.double() * inv).square().sum())
    clip, inv = single(clip), single(inv)
    coef = min(1.0, clip / (math.sqrt(sumsq) + 1e-6)) if clip > 0 else 1.0
    assert (coef < 0.1) == (clip == single(0.01))
    coef = single(coef)
    hp = Z.zero_muon_hparams(lr=0.01, momentum=0.9, weight_decay=0.5, max_grad_norm=clip, nesterov=nesterov,
                             scaling=scaling)
    plan = Z.zero_muon_plan(matrices, precise=precise)
    ws = torch.full((plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    dp, dm, dg, p16 = p.cuda(), m.cuda(), g.cuda(), p.to(TYPES[dtype]).cuda()
    Z.zero_muon_step(dp, dm, p16, dg, plan, hp, result(sumsq, 0, inv), ws)
    wp, wm = reference(p, m, g, matrices, hp, inv, coef)
    got, mom = dp.double().cpu(), dm.double().cpu()
    assert bool(((mom - wm).abs() <= 4 * 2.0 ** -24 * (m.double().abs() + (g.double() * inv * coef).abs()) + 1e-45).all())
    wrong = [reference(p, m, g, matrices, hp, inv, coef, **c)[0] for c in
             (dict(decay=0.0), dict(nesterov=not nesterov), dict(factor=1.05), dict(factor=0.95))]
    inside = torch.zeros(p.numel(), dtype=torch.bool)
    for o, r, c in matrices:
        s = slice(o, o + r * c)
        inside[s] = True
        size = float(p[s].double().norm())
        alpha = {0: 1.0, 1: math.sqrt(max(1.0, r / c)), 2: 0.2 * math.sqrt(max(r, c))}[hp.scaling]
        o64 = float((p[s].double() * (1 - hp.lr * hp.weight_decay) - wp[s]).norm()) / (hp.lr * alpha)
        limit = step_limit(size, o64, (r, c), hp, precise)
        assert float((got[s] - wp[s]).norm()) <= limit, (r, c)
        # what a mistake would have given lies outside (a clipped gradient is little beside the
        # momentum, and the two forms' updates nearer)
        for w in wrong:
            assert float((w[s] - wp[s]).norm()) > limit, (r, c)
        assert torch.equal(p16.cpu()[s].view(torch.int16), dp.cpu()[s].to(TYPES[dtype]).view(torch.int16))
    assert torch.equal(dp.cpu()[~inside], p[~inside]) and torch.equal(dm.cpu()[~inside], m[~inside])


@pytest.mark.parametrize("precise", [False, True])
def test_step_of_large_tiles(precise):
    """256 wide tiles, one step at a time and two to a pass, with momentum, decay and the rms
    factor; the products in 64 bits on the device."""
    shapes = [(2100, 3300), (2300, 2200), (2048, 300)]
    gen = torch.Generator(device="cuda").manual_seed(2)
    n = sum(r * c for r, c in shapes)
    p = torch.randn(n, device="cuda", generator=gen) * 0.02
    m, g = (torch.randn(n, device="cuda", generator=gen) * 1e-2 for _ in range(2))
    g = g.bfloat16()
    hp = Z.zero_muon_hparams(lr=0.01, momentum=0.9, weight_decay=0.5, max_grad_norm=0.5)
    sumsq = float(g.double().square().sum())
    coef = single(hp.max_grad_norm / (math.sqrt(sumsq) + 1e-6))
    assert coef < 0.1
    matrices, at = [], 0
    for r, c in shapes:
        matrices.append((at, r, c))
        at += r * c
    plan = Z.zero_muon_plan(matrices, precise=precise)
    ws = torch.full((plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    dp, dm, p16 = p.clone(), m.clone(), p.bfloat16()
    Z.zero_muon_step(dp, dm, p16, g, plan, hp, result(sumsq), ws)
    gg = g.double() * coef
    wm = hp.momentum * m.double() + gg
    u = gg + hp.momentum * wm
    assert bool(((dm.double() - wm).abs() <= 4 * 2.0 ** -24 * (m.double().abs() + gg.abs()) + 1e-45).all())
    for o, r, c in matrices:
        s = slice(o, o + r * c)
        x = u[s].view(r, c)
        x = x / (torch.linalg.vector_norm(x) + EPS)
        x = x if r <= c else x.t().contiguous()
        for _ in range(5):
            q = x.mm(x.t().contiguous())
            x = A * x + (B * q + C * q.mm(q)).mm(x)
        x = (x if r <= c else x.t()).reshape(-1)
        step = hp.lr * 0.2 * math.sqrt(max(r, c))
        want = p[s].double() * (1 - hp.lr * hp.weight_decay) - step * x
        size, norm = float(p[s].double().norm()), float(x.norm())
        limit = step_limit(size, norm, (r, c), hp, precise)
        assert float((dp[s].double() - want).norm()) <= limit
        assert hp.lr * hp.weight_decay * size > 2 * limit and 0.05 * step * norm > 2 * limit
    assert torch.equal(p16, dp.bfloat16())

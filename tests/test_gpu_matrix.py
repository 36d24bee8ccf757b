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


# Five steps' roundings taken as independent: each is u / sqrt(3) (rms, u = 2^-11) of a term
# that the polynomial weighs by at most |b| + 2 |c|, and later slopes are below 2 where the
# singular values are by then; added in squares.
TYPICAL = 2.0 ** -11 / math.sqrt(3) * (abs(B) + 2 * abs(C)) * math.sqrt(5)


@pytest.mark.parametrize("rows,cols", [(65, 66), (96, 300), (512, 512), (1376, 512), (1024, 4096), (1300, 1300),
                                       (1040, 2800)])
@pytest.mark.parametrize("kind", ["normal", "low"])
def test_error_is_that_of_the_roundings(rows, cols, kind):
    g = update(rows, cols, 3, kind).float().cuda()
    out = torch.empty_like(g)
    plan = Z.zero_matrix_plan([g], out=[out], precise=False)
    Z.zero_orthogonalize(plan, workspace(plan))
    want, _ = polynomial(g)
    assert float((out.double().cpu() - want).norm()) <= TYPICAL * float(want.norm())
    # and to 32 bits, where a product's fp32 sums of K terms weigh most: rms sqrt(K) 2^-24
    plan = Z.zero_matrix_plan([g], out=[out], precise=True)
    Z.zero_orthogonalize(plan, workspace(plan))
    k = max(rows, cols)
    limit = (2.0 ** -21 + math.sqrt(k) * 2.0 ** -24) * (abs(B) + 2 * abs(C)) * math.sqrt(5) * 4
    assert float((out.double().cpu() - want).norm()) <= limit * float(want.norm())


@pytest.mark.parametrize("steps,a,b,c", [(1, A, B, C), (2, A, B, C), (3, 1.5, -0.5, 0.0), (6, A, B, C),
                                         (4, 1.875, -1.25, 0.375)])
@pytest.mark.parametrize("rows,cols", [(20, 90), (130, 500), (300, 140), (1030, 1040)])
def test_coefficients_and_steps(steps, a, b, c, rows, cols):
    g = update(rows, cols, 8).float().cuda()
    out = torch.empty_like(g)
    for precise in (False, True):
        plan = Z.zero_matrix_plan([g], out=[out], precise=precise)
        Z.zero_orthogonalize(plan, workspace(plan), ns=Z.zero_newton_schulz(a, b, c, 1e-7, steps))
        check(out, g, torch.float32, precise, steps=steps, a=a, b=b, c=c)


def test_strides_transposes_and_in_place():
    gen = torch.Generator().manual_seed(6)
    wide = (torch.randn(300, 3 * 200 + 7, generator=gen) * 0.01).cuda()
    q, k, v = (wide[:, 7 + 200 * i:7 + 200 * (i + 1)] for i in range(3))
    tall = (torch.randn(150, 410, generator=gen) * 0.01).bfloat16().cuda()
    t = tall.t()                                             # columns of consecutive elements
    rows = (torch.randn(500, 90, generator=gen) * 0.01).half().cuda()[3:400:2]
    every = [q, k, v, t, rows]
    want = [polynomial(x, True) for x in every]
    outs = [torch.zeros(300, 200, device="cuda"), torch.zeros(300, 200, device="cuda", dtype=torch.bfloat16), v,
            torch.zeros(150, 410, device="cuda").t(), rows]
    keep = wide.clone()
    plan = Z.zero_matrix_plan(every, out=outs)
    Z.zero_orthogonalize(plan, workspace(plan))
    for y, (w, bound) in zip(outs, want):
        limit = bound + half_step(y.dtype) * float(w.norm()) * 1.01 + 1e-6
        assert float((y.double().cpu() - w).norm()) <= limit
    assert torch.equal(wide[:, :407], keep[:, :407])         # all but v, which is in place
    one = q.clone()
    plan = Z.zero_matrix_plan([one])
    Z.zero_orthogonalize(plan, workspace(plan))
    # another plan may cut its sums elsewhere: both are within the bound of the same matrix
    assert float((one.double() - outs[0].double()).norm()) <= 2 * want[0][1]
    again = q.clone()
    Z.zero_orthogonalize(Z.zero_matrix_plan([again]), workspace(plan))
    assert torch.equal(one, again)


def test_special_matrices():
    shapes = [(70, 90), (20, 300), (200, 200), (40, 8), (300, 70)]
    g = [update(r, c, k).float() for k, (r, c) in enumerate(shapes)]
    g[1].zero_()                                             # of zeros
    g[2][3, 7] = float("inf")
    g[3][1, 1] = float("nan")
    dev = [x.cuda() for x in g]
    out = [torch.full_like(x, 7.0) for x in dev]
    plan = Z.zero_matrix_plan(dev, out=out)
    Z.zero_orthogonalize(plan, workspace(plan))
    assert not bool(out[1].any())
    assert bool(out[2].isnan().all()) and bool(out[3].isnan().all())
    check(out[0], g[0], torch.float32, True)
    check(out[4], g[4], torch.float32, True)
    # a matrix of zeros among the larger ones
    z = torch.zeros(100, 130, device="cuda")
    plan = Z.zero_matrix_plan([z], out=[torch.ones_like(z)])
    Z.zero_orthogonalize(plan, workspace(plan))
    assert not bool(plan.out[0].any())


@pytest.mark.parametrize("scale", [1e-18, 1e18])
@pytest.mark.parametrize("shape", [(30, 200), (129, 300)])
def test_any_magnitude(scale, shape):
    # the norm is far above eps, or eps is given as small
    g = (update(*shape, 2) * scale).float().cuda()
    out = torch.empty_like(g)
    plan = Z.zero_matrix_plan([g], out=[out])
    Z.zero_orthogonalize(plan, workspace(plan), ns=Z.zero_newton_schulz(eps=1e-28))
    check(out, g, torch.float32, True, eps=1e-28)


def test_many_matrices_and_whole_tiles():
    # more 256-wide tiles than a round of blocks, a cut rest, several groups, small ones between
    shapes = ([(1024, 1030)] * 30 + [(16, 700), (700, 16)] * 20 + [(513, 512)] * 150 + [(1500, 1200)])
    g = [update(r, c, k % 7, "low").bfloat16().cuda() for k, (r, c) in enumerate(shapes)]
    out = [torch.empty_like(x) for x in g]
    plan = Z.zero_matrix_plan(g, out=out)
    ws = workspace(plan)
    Z.zero_orthogonalize(plan, ws)
    for k in (0, 29, 30, 31, 69, 70, 100, 219, 220):
        want, _ = polynomial(g[k])
        off = float((out[k].double().cpu() - want).norm())
        assert off <= (TYPICAL + half_step(torch.bfloat16)) * float(want.norm()), k
    # the same matrices agree wherever they are in the list (whole or cut tiles)
    seen = {}
    for k, (x, y) in enumerate(zip(g, out)):
        other = seen.setdefault((tuple(x.shape), k % 7), y)
        off = float((y.double() - other.double()).norm())
        assert off <= 2 * (TYPICAL + half_step(torch.bfloat16)) * float(y.double().norm()), k
    again = [y.clone() for y in out]
    ws.fill_(0x3C)
    Z.zero_orthogonalize(plan, ws)
    assert all(torch.equal(x, y) for x, y in zip(out, again))


def test_nothing_else_is_written():
    shapes = [(65, 129), (300, 70), (5, 33), (1300, 257)]
    pad = 256
    total = sum(r * c + pad for r, c in shapes) + pad
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        src = torch.randn(total, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        dst = torch.full((total,), 3.0, dtype=dtype, device="cuda")
        g, out, at, inside = [], [], pad + 1, torch.zeros(total, dtype=torch.bool)
        for r, c in shapes:
            g.append(src[at:at + r * c].view(r, c))
            out.append(dst[at:at + r * c].view(r, c))
            inside[at:at + r * c] = True
            at += r * c + pad - 1
        keep = src.clone()
        plan = Z.zero_matrix_plan(g, out=out)
        size = Z.zero_matrix_workspace_bytes(plan)
        ws = torch.full((size + 8192,), 0x55, dtype=torch.uint8, device="cuda")
        Z.zero_orthogonalize(plan, ws[4096:4096 + size])
        assert torch.equal(src, keep)
        assert bool((dst.cpu()[~inside] == 3.0).all())
        assert bool((ws[:4096] == 0x55).all()) and bool((ws[4096 + size:] == 0x55).all())


def test_muon_skips_on_overflow():
    matrices = [(0, 30, 50), (1500, 200, 130)]
    p, m, p16, g = muon_state(matrices, 27500, "fp16", 3)
    before = [x.clone() for x in (p, m, p16)]
    plan = Z.zero_muon_plan(matrices)
    ws = workspace(plan)
    Z.zero_muon_step(p, m, p16, g, plan, Z.zero_muon_hparams(lr=1.0), result(1.0, 1, 1.0), ws)
    for x, y in zip((p, m, p16), before):
        assert torch.equal(x, y)


def test_graph_streams_and_two_graphs_of_one_workspace():
    matrices = [(1, 40, 70), (3000, 260, 300), (90000, 140, 129)]
    hp = Z.zero_muon_hparams(lr=0.01, max_grad_norm=0.5)
    plan = Z.zero_muon_plan(matrices)
    ws = workspace(plan)
    states = [muon_state(matrices, 110000, "bf16", 7 + k) for k in range(2)]
    eager = [[x.clone() for x in st] for st in states]
    res = [result(2.0), result(3.0)]
    skip = result(1.0, 1)

    def step(st, k, use=None):
        Z.zero_muon_step(*st, plan, hp, res[k] if use is None else use, ws)

    side = torch.cuda.Stream()
    graphs = []
    for k in range(2):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            warm = [x.clone() for x in states[k]]
            step(warm, k)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(states[k], k)
        graphs.append(graph)
    for n in range(4):
        for k in range(2):
            if n == 2 and k == 1:                            # a skipped step among the replays
                saved = res[1].clone()
                res[1].copy_(skip)
                graphs[1].replay()
                torch.cuda.synchronize()
                res[1].copy_(saved)
                continue
            graphs[k].replay()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):                    # eager work between, on another stream
                side.wait_stream(torch.cuda.current_stream())
                step(eager[k], k)
            side.synchronize()
            for x, y in zip(states[k], eager[k]):
                assert torch.equal(x, y), (n, k)


def test_python_refusals():
    g = torch.zeros(8, 9, device="cuda")
    with pytest.raises(ValueError):
        Z.zero_matrix_plan([g.view(-1)])
    with pytest.raises(ValueError):
        Z.zero_matrix_plan([torch.zeros(8, 9)])
    with pytest.raises(ValueError):
        Z.zero_matrix_plan([g], out=[])
    with pytest.raises(ValueError):
        Z.zero_matrix_plan([g], out=[torch.zeros(9, 8, device="cuda")])
    with pytest.raises(ValueError):
        Z.zero_matrix_plan([g], out=[torch.zeros(9, 8, device="cuda").t()])     # rows here, columns there
    with pytest.raises(ValueError):
        Z.zero_matrix_plan([torch.zeros(8, 18, device="cuda")[:, ::2]])
    with pytest.raises(ValueError):
        Z.zero_matrix_plan([torch.zeros(1, 9, device="cuda").expand(8, 9)])
    with pytest.raises(TypeError):
        Z.zero_matrix_plan([g.double()])
    with pytest.raises(TypeError):
        Z.zero_matrix_plan([None])
    with pytest.raises(Z.ZeroError):
        Z.zero_matrix_plan([g, g], out=[torch.zeros_like(g)] * 2)
    plan, ranges = Z.zero_matrix_plan([g]), Z.zero_muon_plan([(0, 8, 9)])
    ws = workspace(ranges)
    with pytest.raises(ValueError):
        Z.zero_orthogonalize(plan, torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        Z.zero_orthogonalize(plan, torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(TypeError):
        Z.zero_orthogonalize(ranges, ws)
    p, h, r = torch.zeros(72, device="cuda"), torch.zeros(72, device="cuda", dtype=torch.half), result()
    hp = Z.zero_muon_hparams()
    with pytest.raises(TypeError):
        Z.zero_muon_step(p, p.clone(), h, h.clone(), plan, hp, r, ws)
    with pytest.raises(TypeError):
        Z.zero_muon_step(p, p.clone(), h, h.bfloat16(), ranges, hp, r, ws)
    for bad in (p[:71], p.double(), torch.zeros(144, device="cuda")[::2], p.cpu()):
        with pytest.raises(ValueError):
            Z.zero_muon_step(bad, p.clone(), h, h.clone(), ranges, hp, r, ws)
    with pytest.raises(ValueError):
        Z.zero_muon_step(p, p.clone(), h, h.clone(), ranges, hp, r[:3], ws)
    with pytest.raises(ValueError):
        Z.zero_muon_step(p, p.clone(), h, h.clone(), ranges, hp, r, ws[:-1][:16])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(graph, stream=side):
            Z.zero_muon_plan([(0, 8, 9)])


def test_empty_lists():
    for plan in (Z.zero_matrix_plan([], device="cuda"), Z.zero_matrix_plan([torch.zeros(0, 5, device="cuda")])):
        Z.zero_orthogonalize(plan, workspace(plan))
    plan = Z.zero_muon_plan([(0, 0, 9)])
    p, h = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda", dtype=torch.half)
    Z.zero_muon_step(p, p, h, h, plan, Z.zero_muon_hparams(), result(), workspace(plan))


def orth64(g):
    """On the device, for large ones: the polynomial in 64 bits."""
    x = g.double()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    wide = x if x.shape[0] <= x.shape[1] else x.t().contiguous()
    for _ in range(5):
        s = wide.mm(wide.t().contiguous())
        wide = A * wide + (B * s + C * s.mm(s)).mm(wide)
    return wide if g.shape[0] <= g.shape[1] else wide.t().contiguous()


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("shapes", [
    [(2300, 2400)],                         # 256 wide tiles, none of a whole round: all cut
    [(2300, 5000)],                         # in pairs (not in 32 bits)
    [(3000, 2350), (2350, 3000)],
    [(1500, 1700), (300, 260), (900, 2000), (64, 70)],   # one group for all, and a small one
    [(5000, 4100)],                         # whole tiles and cut ones
])
def test_large_tiles(shapes, precise):
    limit = TYPICAL if not precise else (2.0 ** -21 + math.sqrt(max(map(max, shapes))) * 2.0 ** -24) * \
        (abs(B) + 2 * abs(C)) * math.sqrt(5) * 4
    # the update is the gradient, in 32 bits and as the step takes it
    g16 = [update(r, c, 5).cuda().half() for r, c in shapes]
    want = [orth64(g) for g in g16]
    outs = [torch.empty(g.shape, device="cuda") for g in g16]
    plan = Z.zero_matrix_plan(g16, out=outs, precise=precise)
    Z.zero_orthogonalize(plan, workspace(plan))
    for o, w in zip(outs, want):
        assert float((o.double() - w).norm()) <= limit * float(w.norm())
    ends = [0]
    for r, c in shapes:
        ends.append(ends[-1] + r * c)
    matrices = [(at, r, c) for at, (r, c) in zip(ends, shapes)]
    grad = torch.cat([g.reshape(-1) for g in g16])
    master, momentum = torch.ones(ends[-1], device="cuda"), torch.zeros(ends[-1], device="cuda")
    p16 = torch.zeros(ends[-1], device="cuda", dtype=torch.half)
    plan = Z.zero_muon_plan(matrices, precise=precise)
    hp = Z.zero_muon_hparams(lr=2.0, weight_decay=0.0, nesterov=False, scaling=None)
    Z.zero_muon_step(master, momentum, p16, grad, plan, hp, result(), workspace(plan))
    for (at, r, c), w in zip(matrices, want):
        o = (1.0 - master[at:at + r * c].double().view(r, c)) / 2
        # the weights' own rounding: 2^-24 of at most 1 + 2 |w|, each
        own = 2.0 ** -24 * (math.sqrt(r * c) + 2 * float(w.norm())) / 2
        assert float((o - w).norm()) <= limit * float(w.norm()) + own
    assert torch.equal(momentum, grad.float()) and torch.equal(p16, master.half())

"""The errors that the header states for orthogonalisation, on the matrices where they are
largest: of exactly and almost low rank, of two levels of singular values, of equal entries.

Limits.  A step's planes are rounded entry by entry, half a step of fp16 at most; off the
diagonals nothing makes up for it.  Independent roundings e of the entries of an m x m plane
of 2-norm 1 and of X's rows are, over the directions that a matrix of rank r does have, an
error of e sqrt(r / m) of the result, and over the m - r others one that later steps multiply by
a each, of e / sqrt(m) or less: with e = 2^-11 / sqrt(3) (rms), |b| + 2 |c| = 8.8 and what two
steps between make of it, 0.06 / sqrt(m) in all (one direction, whose roundings are fewest and
weigh most: 0.08); two steps to a pass multiply planes once more, 0.1.  Entries that are all
alike are all rounded alike: 2^-11 (|b| + 2 |c|) in a step, 2.2e-2 over five, and in pairs of steps
again once more of a's square, 3e-2.  To 32 bits the same with 2^-21, and with X's own last bit, 2^-22 of the entries,
which 485 times in the m directions that a matrix of low rank does not have is 485 2^-22 / sqrt(3)
of what is there, and the fp32 sums' 2^-24 sqrt(n / 32) with it.
"""
import math

import pytest
import torch

import zero_partitioned_mixed_shard_amd as Z

pytestmark = pytest.mark.gpu


def single(x):
    return torch.tensor(x, dtype=torch.float32).double().item()


A, B, C, EPS = single(3.4445), single(-4.7750), single(2.0315), single(1e-7)


def orth64(g):
    x = g.double()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    wide = x if x.shape[0] <= x.shape[1] else x.t().contiguous()
    for _ in range(5):
        s = wide.mm(wide.t().contiguous())
        wide = A * wide + (B * s + C * s.mm(s)).mm(wide)
    return wide if g.shape[0] <= g.shape[1] else wide.t().contiguous()


def of_rank(rows, cols, rank, gen, noise=0.0):
    g = torch.randn(rows, rank, generator=gen, dtype=torch.float64) @ \
        torch.randn(rank, cols, generator=gen, dtype=torch.float64)
    return g / math.sqrt(rank) + noise * torch.randn(rows, cols, generator=gen, dtype=torch.float64)


def of_levels(rows, cols, rank, level, gen):
    """`rank` singular values of 1, the others of `level`."""
    m, n = min(rows, cols), max(rows, cols)
    u = torch.linalg.qr(torch.randn(m, m, generator=gen, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(n, m, generator=gen, dtype=torch.float64))[0]
    s = torch.full((m,), level, dtype=torch.float64)
    s[:rank] = 1.0
    g = (u * s) @ v.t()
    return g if rows <= cols else g.t().contiguous()


def matrix(kind, rows, cols):
    gen, m = torch.Generator().manual_seed(rows * 31 + cols), min(rows, cols)
    if kind == "normal":
        return torch.randn(rows, cols, generator=gen, dtype=torch.float64)
    if kind == "noise":
        return of_rank(rows, cols, max(1, m // 16), gen, 0.5)
    if kind == "alike":
        return torch.full((rows, cols), 0.37, dtype=torch.float64)
    if kind == "one":
        return of_rank(rows, cols, 1, gen)
    if kind == "almost one":
        return of_rank(rows, cols, 1, gen, 1e-3)
    if kind == "two levels":
        return of_levels(rows, cols, m // 2, 1e-3, gen)
    return of_rank(rows, cols, max(2, m // int(kind)), gen)


def error(g, precise, out=torch.float32, **kw):
    y = torch.zeros(g.shape, dtype=out, device="cuda")
    plan = Z.zero_matrix_plan([g], out=[y], precise=precise, **kw)
    ws = torch.full((max(1, Z.zero_matrix_workspace_bytes(plan)),), 0xFF, dtype=torch.uint8, device="cuda")
    Z.zero_orthogonalize(plan, ws)
    want = orth64(g)
    return float((y.double() - want).norm() / want.norm())


def limits(kind, rows, cols):
    """(in fp16 products, to 32 bits) of the header."""
    m, n = min(rows, cols), max(rows, cols)
    if kind in ("normal", "noise"):
        return 2e-3, 1e-5
    if kind == "alike":
        return 3e-2 if m >= 2048 and 2 * n >= 3 * m else 2.2e-2, 1e-3
    if kind in ("one", "almost one"):
        return 0.08 / math.sqrt(m), 1e-3
    return (0.1 if m >= 2048 and 2 * n >= 3 * m else 0.06) / math.sqrt(m), 5e-5


KINDS = ["normal", "noise", "2", "4", "16", "one", "almost one", "two levels", "alike"]


@pytest.mark.parametrize("rows,cols", [(65, 66), (65, 200), (512, 128), (256, 256), (300, 400), (512, 1376),
                                       (768, 2100), (1024, 1024), (2800, 1040), (1500, 1700)])
@pytest.mark.parametrize("kind", KINDS)
def test_errors_are_as_stated(kind, rows, cols):
    g = matrix(kind, rows, cols).float().cuda()
    fast, precise = limits(kind, rows, cols)
    assert error(g, False) <= fast
    assert error(g, True) <= precise


@pytest.mark.parametrize("kind", ["noise", "4", "16", "one", "alike"])
def test_errors_of_two_steps_to_a_pass(kind):
    rows, cols = 2048, 4096
    gen = torch.Generator(device="cuda").manual_seed(3)
    if kind == "alike":
        g = torch.full((rows, cols), 0.37, device="cuda")
    else:
        k = 1 if kind == "one" else 2048 // (16 if kind == "noise" else int(kind))
        g = torch.randn(rows, k, device="cuda", generator=gen) @ torch.randn(k, cols, device="cuda", generator=gen)
        if kind == "noise":
            g = g / math.sqrt(k) + 0.5 * torch.randn(rows, cols, device="cuda", generator=gen)
    fast, precise = limits(kind, rows, cols)
    assert error(g, False) <= fast
    assert error(g, True) <= precise


def test_a_gradient_of_few_tokens():
    """What a first step meets: the product of 48 tokens' activations and errors, in bf16, of
    which the update is a multiple."""
    rows, cols = 320, 768
    gen = torch.Generator().manual_seed(5)
    g = of_rank(rows, cols, 48, gen).bfloat16().cuda()
    assert error(g, False) <= 0.06 / math.sqrt(320)
    m = torch.zeros(rows * cols, device="cuda")
    p = torch.zeros(rows * cols, device="cuda")
    p16 = torch.zeros(rows * cols, device="cuda", dtype=torch.bfloat16)
    plan = Z.zero_muon_plan([(0, rows, cols)])
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    one = torch.zeros(4, dtype=torch.int32, device="cuda")
    one.view(torch.float32)[3] = 1.0
    hp = Z.zero_muon_hparams(lr=1.0, weight_decay=0.0, scaling=None)
    Z.zero_muon_step(p, m, p16, g.reshape(-1), plan, hp, one, ws)
    want = orth64(g)
    assert float((-p.double().view(rows, cols) - want).norm()) <= 0.06 / math.sqrt(320) * float(want.norm())


@pytest.mark.parametrize("kind", ["normal", "noise", "4", "two levels"])
@pytest.mark.parametrize("rows,cols", [(65, 200), (300, 400), (1024, 700), (1500, 1700)])
def test_float16_results_are_off_by_their_rounding(kind, rows, cols):
    """A rounding is off by at most half of 2^-10 of its binade's first value, evenly spread: in the
    2-norm by 2^-10 / sqrt(12) of the result, and the products' 5e-5 beside it."""
    g = matrix(kind, rows, cols).half().cuda()
    assert error(g, None, torch.float16) <= 2.0 ** -10 / math.sqrt(12) + 5e-5


def test_who_takes_two_parts():
    g = torch.ones(70, 80, device="cuda")
    half, bf, f32 = (torch.empty(70, 80, device="cuda", dtype=t) for t in
                     (torch.float16, torch.bfloat16, torch.float32))
    for outs, precise, want in (([half], None, (False, 2)), ([bf], None, (False, 1)), ([f32], None, (True, 2)),
                                ([half, bf], None, (False, 2)), ([half], False, (False, 1)),
                                ([half], True, (True, 2)), ([f32], False, (False, 1))):
        plan = Z.zero_matrix_plan([g] * len(outs), out=outs, precise=precise)
        assert (plan.precise, plan.parts) == want and plan.c.precise == plan.parts - 1
    assert Z.zero_muon_plan([(0, 70, 80)]).parts == 1 and Z.zero_muon_plan([(0, 70, 80)], precise=True).parts == 2


@pytest.mark.parametrize("rows,cols,kind", [(65, 200000, "normal"), (200000, 130, "normal"), (130, 100000, "alike"),
                                            (1100, 70000, "normal"), (70, 4000000, "alike"), (4000000, 65, "normal")])
def test_long_sums(rows, cols, kind):
    """A's diagonal is a sum of as many positive terms as there are columns: in chains of at
    most 1024 fp32 sums, and these added up, its error does not grow with them."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    g = torch.full((rows, cols), 0.37, device="cuda") if kind == "alike" else \
        torch.randn(rows, cols, device="cuda", generator=gen)
    fast, precise = limits(kind, rows, cols)
    assert error(g, False) <= fast
    assert error(g, True) <= precise


def test_long_ones_among_others():
    """A long matrix is a group of its own, whatever is beside it."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    shapes = [(200, 300), (66, 40000), (20, 50000), (33000, 70), (1030, 200), (90, 32768), (90, 32769)]
    g = [torch.randn(s, device="cuda", generator=gen) for s in shapes]
    for precise in (False, True):
        out = [torch.zeros_like(x) for x in g]
        plan = Z.zero_matrix_plan(g, out=out, precise=precise)
        ws = torch.full((plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        Z.zero_orthogonalize(plan, ws)
        for x, y in zip(g, out):
            want = orth64(x)
            assert float((y.double() - want).norm()) <= limits("normal", *x.shape)[precise] * float(want.norm())


@pytest.mark.parametrize("rows,cols", [(16, 300), (64, 40000), (3000, 30), (70, 300), (500, 400)])
@pytest.mark.parametrize("largest", [3.3e38, 2.0 ** 100, 2.0 ** 60])
def test_values_at_the_end_of_the_range(rows, cols, largest):
    """The norm is beyond fp32's range, or its reciprocal subnormal; the result is what it is for
    any other multiple of the matrix."""
    g = matrix("normal", rows, cols)
    g = (g * (largest / float(g.abs().max()))).float().cuda()
    assert bool(g.isfinite().all())
    assert error(g, True) <= limits("normal", rows, cols)[1]
    if min(rows, cols) > 64:
        assert error(g, False) <= limits("normal", rows, cols)[0]


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (7, 1), (1, 1000), (3, 200), (16, 1025), (1025, 16), (17, 33),
                                       (63, 65), (64, 64), (64, 40000), (40001, 5)])
@pytest.mark.parametrize("kind", ["normal", "4", "one", "alike"])
def test_small_sides_are_in_32_bits(rows, cols, kind):
    """The polynomial of the Gram matrix is made in 64 bits, P (its 2-norm at most 3.4445^5 = 485)
    rounded to fp32, and P U is a sum of up to 64 fp32 products: 2^-24 of |P| |U| each, of
    independent signs, 4 times that at most over all of a row.  Entries that are all alike have
    no independent signs: P is 485 on the diagonal and about -485 / m beside it, so a row's
    partial sums are the same in all columns and go from 485 u down to the result, of m sums each
    rounded by up to 2^-24 of 485 u / 2 on the average; the result is at least 0.68 u."""
    g = matrix(kind, rows, cols).float().cuda()
    limit = 3.4445 ** 5 * 2.0 ** -22
    if kind == "alike":
        limit = max(limit, (min(rows, cols) / 2 + 1) * 3.4445 ** 5 * 2.0 ** -24 / 0.68)
    for precise in (False, True):
        assert error(g, precise) <= limit


@pytest.mark.parametrize("count,rows,cols", [(41, 1024, 1024), (43, 1024, 1024), (80, 600, 620), (17, 1000, 1024),
                                             (19, 1000, 1024)])
def test_lists_on_both_sides_of_the_tiles_rule(count, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(count)
    src = torch.randn(count, rows, cols, device="cuda", generator=gen).bfloat16()
    for precise in (False, True):
        out = torch.zeros(count, rows, cols, device="cuda")
        plan = Z.zero_matrix_plan(list(src), out=list(out), precise=precise)
        ws = torch.full((plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        Z.zero_orthogonalize(plan, ws)
        for k in (0, count // 2, count - 1):
            want = orth64(src[k])
            off = float((out[k].double() - want).norm())
            assert off <= limits("normal", rows, cols)[precise] * float(want.norm()), (precise, k)


@pytest.mark.parametrize("rows,cols,value", [(1926, 10327, 2.964), (3754, 6598, 7.826), (3282, 5389, 5.498)])
def test_lower_parts_are_added_up_first(rows, cols, value):
    """Equal entries: a tile's sums are rounded alike, and otherwise in a tile that is cut; what
    differs is no multiple of the matrix, and later steps multiply it by a each.  With the large
    products first there would be three times as many such roundings (5.8e-3)."""
    assert error(torch.full((rows, cols), value, device="cuda"), True) <= 1e-3

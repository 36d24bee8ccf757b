"""The operators over tensor tables on the GPU against their definitions in 64
bits: norms, clipping, accumulation, their fused forms, and a run of them
together.

Tolerances, from the rounding of each step (half a step of a type: fp32 2^-24,
bf16 2^-8, fp16 2^-11 relative; below the type's normal range half its
smallest step):
  sumsq   sums of n non-negative fp64 terms, two orders: 2 n 2^-53; inv^2 and its
          product 3 more roundings
  norms   as sumsq (half of it, after the root), then one rounding to fp32
  clip    the factor's rounding to fp32 and the product's: 2 * 2^-24, then one
          to the output's type (for fp32 the product's is that one)
  add     one fused multiply-add in fp32: 2^-24, then one to the output's type
"""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import zero_partitioned_mixed_shard_amd as Z

pytestmark = pytest.mark.gpu

HALF, BF, F32 = torch.float16, torch.bfloat16, torch.float32
U = {F32: 2.0 ** -24, HALF: 2.0 ** -11, BF: 2.0 ** -8}
TINY = {F32: 2.0 ** -150, HALF: 2.0 ** -25, BF: 2.0 ** -134}   # half the smallest step
SIZES = [1, 2, 7, 8, 9, 63, 64, 65, 511, 2047, 2048, 2049, 4100, 8191, 16383, 16384, 16385,
         40000, 131072 + 3]
GUARD = 64                                                     # elements around every output


def f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


class Set:
    """Tensors at chosen element offsets, each inside a guarded buffer."""

    def __init__(self, sizes, types, offsets, seed=0, scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bufs, self.t = [], []
        for n, dt, off in zip(sizes, types, offsets):
            buf = torch.full((n + 2 * GUARD + 8,), 77.0, dtype=dt, device="cuda")
            v = buf[GUARD + off:GUARD + off + n]
            v.normal_(0.0, scale, generator=g)
            self.bufs.append((buf, GUARD + off, n))
            self.t.append(v)

    def assert_guards(self):
        for buf, a, n in self.bufs:
            assert bool((buf[:a] == 77.0).all()) and bool((buf[a + n:] == 77.0).all())


def host64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def make_res(sumsq=0.0, overflow=0, inv=1.0):
    raw = bytearray(struct.pack("<dIf", sumsq, overflow, inv))
    return torch.frombuffer(raw, dtype=torch.int32).clone().cuda()


def workspace(plan):
    # filled with NaN: the calls need no initialisation
    return torch.full((-(-plan.workspace_bytes // 8),), float("nan"), dtype=torch.float64,
                      device="cuda")


def ref_norms(arrays, kind, inv):
    """(sumsq, per-tensor norms) in 64 bits."""
    if kind == "max":
        each = [float(np.abs(a).max()) if a.size else 0.0 for a in arrays]
        return (max(each, default=0.0) * inv) ** 2, np.array(each) * inv
    sq = [math.fsum((a * a).tolist()) if a.size < 50000 else float(np.dot(a, a)) for a in arrays]
    return math.fsum(sq) * inv * inv, np.sqrt(np.array(sq)) * inv


def check_norm(res, norms, arrays, kind, inv):
    r = Z.read_result(res)
    want, each = ref_norms(arrays, kind, inv)
    n = sum(a.size for a in arrays) if kind == "l2" else 0
    assert r.overflow == 0 and r.inv_scale == inv
    assert abs(r.sumsq - want) <= (2 * n + 8) * 2.0 ** -53 * want
    if norms is not None:
        got = norms.double().cpu().numpy()
        size = np.array([a.size if kind == "l2" else 0 for a in arrays])
        assert (np.abs(got - each) <= (2.0 ** -24 + (size + 8) * 2.0 ** -53) * each + TINY[F32]).all()


def assert_rounded(got, want, dt, steps=0.0, what=""):
    """got = want rounded to dt after `steps` relative error before it."""
    g = host64(got)
    tol = np.abs(want) * (U[dt] * (1 + steps) + steps) + TINY[dt]
    bad = np.flatnonzero(~(np.abs(g - want) <= tol))
    assert not bad.size, f"{what}: {bad.size} of {g.size} off, first {bad[:4]}: {g[bad[:4]]} {want[bad[:4]]}"


def clip_steps(dt):
    # the factor's rounding and, unless that is the output's own, the product's
    # (2^-40 covers the second order and the fp64 steps of the factor)
    return 2.0 ** -24 * (1 if dt == F32 else 2) + 2.0 ** -40


def clip_want(x, norm, max_norm, inv):
    c = max_norm / (norm + 1e-6) if max_norm > 0 else 1.0
    return x * (min(c, 1.0) * inv)


# ------------------------------------------------------------------- table --
@pytest.mark.parametrize("seed", range(6))
def test_table_covers_every_element_once(seed):
    """The expanded table against a plain cut of every tensor."""
    rng = np.random.default_rng(seed)
    count = [0, 1, 5, 40, 300, 3000][seed]
    sizes = [int(n) for n in rng.choice([0, 1, 7, 4095, 4096, 4097, 16384, 16385, 70001], count)]
    src, dst = ([(F32, HALF, BF)[k] for k in rng.integers(0, 3, count)] for _ in range(2))
    flat = torch.zeros(4 * sum(sizes) + 64 * count + 8, dtype=torch.uint8, device="cuda")
    outs, at = [], 0
    for n, d in zip(sizes, dst):
        at += int(rng.integers(0, 8)) * 4
        outs.append(flat[at:at + n * d.itemsize].view(d))
        at += -(-n * d.itemsize // 4) * 4
    tensors = [torch.zeros(n, dtype=d, device="cuda") for n, d in zip(sizes, src)]
    plan = Z.zero_tensor_plan(tensors, out=outs, device="cuda")
    assert plan.c.writable == 1
    code = {F32: Z.ZERO_FP32, HALF: Z.ZERO_FP16, BF: Z.ZERO_BF16}
    runs, rests, pieces, dsts = [], [], [], []
    for k, (t, o) in enumerate(zip(tensors, outs)):
        def record(begin, n):
            return (t.data_ptr() + begin * t.element_size(), k,
                    n | code[t.dtype] << 24 | code[o.dtype] << 28)
        n, b = t.numel(), 0
        while n - b >= 16384:
            runs.append(record(b, 16384))
            b += 16384
        rests += [record(a, min(4096, n - a)) for a in range(b, n, 4096)]
        lead = o.data_ptr() % 128 // o.element_size()
        b = 0
        while b < n:
            c = min(n - b, 4096 - (lead if b == 0 else 0))
            pieces.append(record(b, c))
            dsts.append(o.data_ptr() + b * o.element_size())
            b += c
    raw = plan.table.cpu().numpy()[plan.c.head_bytes:]
    rec = np.dtype([("src", np.uint64), ("tensor", np.int32), ("info", np.uint32)])
    every = np.array(runs + rests + pieces, dtype=rec)
    assert (plan.c.n_runs, plan.c.n_rests, plan.c.n_pieces) == (len(runs), len(rests), len(pieces))
    assert raw[:every.nbytes].tobytes() == every.tobytes()
    assert raw[every.nbytes:].tobytes() == np.array(dsts, dtype=np.uint64).tobytes()


# ------------------------------------------------------------------- norms --
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dt", [F32, HALF, BF])
def test_norm_sizes_and_alignments(dt, kind):
    inv = f32(1.0 / 3.0)
    sizes = SIZES + [0, 5]
    s = Set(sizes, [dt] * len(sizes), [k % 8 for k in range(len(sizes))], seed=1)
    for n, t in zip(sizes, s.t):
        plan = Z.zero_tensor_plan([t])
        res, norms = make_res(9.0, 1, 5.0), torch.full((1,), -1.0, device="cuda")
        Z.zero_tensor_norm(plan, inv, res, workspace(plan), kind=kind, norms=norms)
        check_norm(res, norms, [host64(t)], kind, inv)
    plan = Z.zero_tensor_plan(s.t)
    res, norms = make_res(), torch.full((len(sizes),), -1.0, device="cuda")
    Z.zero_tensor_norm(plan, inv, res, workspace(plan), kind=kind, norms=norms)
    check_norm(res, norms, [host64(t) for t in s.t], kind, inv)
    again = make_res()
    Z.zero_tensor_norm(plan, inv, again, workspace(plan), kind=kind)
    assert torch.equal(again, res)                       # the same bits, with or without norms


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dt", [F32, HALF, BF])
def test_norm_bits_do_not_depend_on_the_place(dt, kind):
    """The same values at every start in a 16-byte access: the same bits, and nothing
    read beyond them counts (NaN on both sides)."""
    sizes = [16384 * 3 + 4099, 16384, 5, 16385]
    values = [torch.randn(n, device="cuda").to(dt) for n in sizes]
    first = None
    for off in range(9):
        bufs = [torch.full((n + 32,), float("nan"), dtype=dt, device="cuda") for n in sizes]
        tensors = [b[8 + off:8 + off + n].copy_(v) for b, v, n in zip(bufs, values, sizes)]
        plan = Z.zero_tensor_plan(tensors)
        res, norms = make_res(), torch.zeros(len(sizes), device="cuda")
        Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), kind=kind, norms=norms)
        if first is None:
            first = res.clone(), norms.clone()
            check_norm(res, norms, [host64(v) for v in values], kind, 1.0)
        assert torch.equal(res, first[0]) and torch.equal(norms, first[1]), off


@pytest.mark.parametrize("kind", ["l2", "max"])
def test_norm_mixed_types_and_empty_tables(kind):
    for sizes in ([], [0], [0, 0, 3], [300, 0, 70001, 1, 0, 16384, 2]):
        types = [(F32, HALF, BF)[k % 3] for k in range(len(sizes))]
        s = Set(sizes, types, [(3 * k) % 8 for k in range(len(sizes))], seed=2)
        plan = Z.zero_tensor_plan(s.t, device="cuda")
        res = make_res(3.0, 1, 2.0)
        norms = torch.full((len(sizes),), -1.0, device="cuda")
        Z.zero_tensor_norm(plan, 0.5, res, workspace(plan), kind=kind, norms=norms)
        check_norm(res, norms, [host64(t) for t in s.t], kind, 0.5)


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("count", [40000, 60000])
def test_norm_of_many_tensors(kind, count):
    """At 60000 more partials than one block joins; half of the tensors empty or of
    one element."""
    rng = np.random.default_rng(5)
    sizes = [int(n) for n in rng.choice([0, 1, 3, 40], count)]
    flat = torch.empty(sum(sizes), dtype=HALF, device="cuda").normal_(
        generator=torch.Generator(device="cuda").manual_seed(3))
    tensors = list(flat.split(sizes))
    plan = Z.zero_tensor_plan(tensors)
    res, norms = make_res(), torch.full((len(sizes),), -1.0, device="cuda")
    Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), kind=kind, norms=norms)
    host = host64(flat)
    ends = np.cumsum(sizes)
    check_norm(res, norms, [host[e - n:e] for e, n in zip(ends, sizes)], kind, 1.0)


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dt", [F32, HALF, BF])
def test_overflow_is_found_anywhere(dt, kind):
    n = 20011
    for value in (float("inf"), float("-inf"), float("nan")):
        for at in (0, 1, 8, 2047, 2048, 16383, 16384, n - 1):
            s = Set([5, n, 9], [dt] * 3, [0, 3, 1], seed=4)
            s.t[1][at] = value
            plan = Z.zero_tensor_plan(s.t)
            res, norms = make_res(), torch.zeros(3, device="cuda")
            Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), kind=kind, norms=norms)
            r = Z.read_result(res)
            assert r.overflow == 1 and not math.isfinite(r.sumsq), (value, at)
            assert [math.isfinite(x) for x in norms.tolist()] == [True, False, True]
            before = [t.clone() for t in s.t]
            Z.zero_tensor_clip(plan, 0.1, res)
            Z.zero_tensor_clip(plan, 0.1, res, norms=norms)
            for t, b in zip(s.t, before):                 # a skipped step writes nothing
                assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
            # a later finite table keeps the flag
            clean = Z.zero_tensor_plan([s.t[0]])
            Z.zero_tensor_norm(clean, 1.0, res, workspace(clean), kind=kind, accumulate=True)
            assert Z.read_result(res).overflow == 1


def test_extreme_finite_values_do_not_overflow():
    """The largest and smallest finite values of each type: squares and sums stay
    finite and exact enough in 64 bits, and no flag is raised."""
    for dt in (F32, HALF, BF):
        fi = torch.finfo(dt)
        small = 2.0 ** -149 if dt == F32 else TINY[dt] * 2
        for value in (fi.max, fi.min, small):
            t = torch.full((5000,), value, dtype=dt, device="cuda")
            for kind in ("l2", "max"):
                plan = Z.zero_tensor_plan([t])
                res = make_res()
                Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), kind=kind)
                check_norm(res, None, [host64(t)], kind, 1.0)


def test_accumulated_tables_give_one_norm():
    s = Set([1000, 20000, 33], [F32, BF, HALF], [1, 2, 3], seed=6)
    host = [host64(t) for t in s.t]
    for kind in ("l2", "max"):
        res = make_res(1e30, 1, 1.0)
        for k, t in enumerate(s.t):
            p = Z.zero_tensor_plan([t])
            Z.zero_tensor_norm(p, 0.25, res, workspace(p), kind=kind, accumulate=k > 0)
        check_norm(res, None, host, kind, 0.25)


def test_norm_past_32_bit_offsets():
    n = (1 << 31) + 16391
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[-1], t[1 << 31], t[5] = 3.0, -4.0, 12.0
    plan = Z.zero_tensor_plan([t])
    for kind, want in (("l2", 169.0), ("max", 144.0)):
        res = make_res()
        Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), kind=kind)
        assert Z.read_result(res).sumsq == want
    res = make_res(169.0, 0, 1.0)
    Z.zero_tensor_clip(plan, 13.0 + 1e-6, res)           # factor 1 up to 2^-24 of rounding
    Z.zero_tensor_clip(plan, 6.5, res)                    # and about a half
    assert [float(t[k]) for k in (5, 1 << 31, n - 1)] == [6.0, -2.0, 1.5]


def test_tables_longer_than_one_launch():
    """More pieces than a grid holds (6.9e10 elements in one tensor): values at the
    ends and on both sides of the launches' border."""
    border = ((1 << 24) - 1) * 4096                       # elements of a launch's pieces
    n = border + 5000
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("not enough device memory")
    t = torch.zeros(n, dtype=BF, device="cuda")
    at = [0, border - 1, border, n - 1]
    for k, v in zip(at, (1.0, -2.0, 4.0, -10.0)):
        t[k] = v
    plan = Z.zero_tensor_plan([t])
    assert plan.c.n_pieces == (1 << 24) + 1
    ws = workspace(plan)
    for kind, want in (("l2", 121.0), ("max", 100.0)):
        res = make_res()
        Z.zero_tensor_norm(plan, 1.0, res, ws, kind=kind)
        assert Z.read_result(res).sumsq == want
    Z.zero_tensor_clip(plan, 0.0, make_res(1.0, 0, 0.5))
    assert [float(t[k]) for k in at] == [0.5, -1.0, 2.0, -5.0]
    res = make_res()
    Z.zero_tensor_accumulate(plan, 1.0, res=res, workspace=ws)
    assert [float(t[k]) for k in at] == [1.0, -2.0, 4.0, -10.0]
    assert Z.read_result(res).sumsq == 121.0


# -------------------------------------------------------------------- clip --
@pytest.mark.parametrize("dst", [None, F32, HALF, BF])
@pytest.mark.parametrize("src", [F32, HALF, BF])
def test_clip_sizes_and_alignments(src, dst):
    sizes = SIZES + [0, 4]
    for shift in (0, 3):
        s = Set(sizes, [src] * len(sizes), [(k + shift) % 8 for k in range(len(sizes))], seed=7)
        o = s if dst is None else Set(sizes, [dst] * len(sizes), [k % 8 for k in range(len(sizes))])
        host = [host64(t) for t in s.t]
        plan = Z.zero_tensor_plan(s.t, out=None if dst is None else o.t)
        inv, max_norm, sumsq = f32(0.3), f32(2.5), 81.0
        Z.zero_tensor_clip(plan, max_norm, make_res(sumsq, 0, inv))
        for t, x in zip(o.t, host):
            assert_rounded(t, clip_want(x, 9.0, max_norm, inv), t.dtype, clip_steps(t.dtype))
        o.assert_guards()
        if dst is not None:
            s.assert_guards()
            for t, x in zip(s.t, host):
                assert np.array_equal(host64(t), x)       # the input stays


@pytest.mark.parametrize("max_norm", [0.0, -1.0, 100.0, float("inf")])
def test_clip_off_leaves_values(max_norm):
    s = Set([5000, 17], [BF, F32], [0, 1], seed=8)
    before = [t.clone() for t in s.t]
    plan = Z.zero_tensor_plan(s.t)
    Z.zero_tensor_clip(plan, max_norm, make_res(25.0, 0, 1.0))
    assert all(torch.equal(t, b) for t, b in zip(s.t, before))
    out = [torch.zeros_like(t) for t in s.t]              # elsewhere: copied
    Z.zero_tensor_clip(Z.zero_tensor_plan(s.t, out=out), max_norm, make_res(25.0, 0, 1.0))
    assert all(torch.equal(t, b) for t, b in zip(out, before))


@pytest.mark.parametrize("sizes", [[70, 5], [900] * 12, [9, 70000, 5], [3000] * 1100])
def test_clip_norm_off_leaves_values(sizes):
    """In place with a factor of 1, on every path: the same bits, and the norm."""
    tensors = list(torch.randn(sum(sizes), device="cuda").split(sizes))
    before = [t.clone() for t in tensors]
    plan = Z.zero_tensor_plan(tensors)
    for max_norm in (0.0, 1e9):
        for norms in (None, torch.zeros(len(sizes), device="cuda")):
            res = make_res()
            Z.zero_tensor_clip_norm(plan, max_norm, 1.0, res, workspace(plan), norms=norms,
                                    per_tensor=norms is not None)
            assert all(torch.equal(t, b) for t, b in zip(tensors, before))
            check_norm(res, norms, [host64(t) for t in tensors], "l2", 1.0)
    Z.zero_tensor_clip_norm(plan, 0.0, 0.5, res, workspace(plan))   # and halved
    assert all(torch.equal(t, b * 0.5) for t, b in zip(tensors, before))


def test_clip_next_to_the_border():
    """Norms a few roundings around max_norm - 1e-6, where the ratio turns from 1 to
    below: in place gives the bits of the same clip into other tensors."""
    x = torch.randn(5000, device="cuda")
    for max_norm in (1.0, 1e-6, 2e-6, 1e3, 5e-7):
        top = f32(max_norm) - 1e-6
        for step in (-1e-3, -3e-16, -1e-16, 0.0, 1e-16, 3e-16, 1e-9, 1e-7, 1e-3):
            norm = abs(top) * (1.0 + step)
            mine, out = x.clone(), torch.empty_like(x)
            res = make_res(norm * norm, 0, 1.0)
            Z.zero_tensor_clip(Z.zero_tensor_plan([mine]), max_norm, res)
            Z.zero_tensor_clip(Z.zero_tensor_plan([x], out=[out]), max_norm, res)
            assert torch.equal(mine, out), (max_norm, step)
            norms = torch.tensor([norm], device="cuda")
            mine.copy_(x)
            Z.zero_tensor_clip(Z.zero_tensor_plan([mine]), max_norm, res, norms=norms)
            Z.zero_tensor_clip(Z.zero_tensor_plan([x], out=[out]), max_norm, res, norms=norms)
            assert torch.equal(mine, out), (max_norm, step)


def test_clip_each_by_its_own_norm():
    sizes = [1, 100, 0, 16384, 50001]
    s = Set(sizes, [F32, BF, HALF, HALF, F32], [0, 1, 0, 5, 2], seed=9)
    host = [host64(t) for t in s.t]
    out = [torch.empty_like(t) for t in s.t]
    plan = Z.zero_tensor_plan(s.t, out=out)
    given = [0.25, 4.0, 7.0, 0.0, 1e20]                   # any norms: they are taken as they are
    Z.zero_tensor_clip(plan, 0.5, make_res(1.0, 0, 0.5), norms=torch.tensor(given, device="cuda"))
    for t, x, n in zip(out, host, given):
        assert_rounded(t, clip_want(x, f32(n), 0.5, 0.5), t.dtype, clip_steps(t.dtype))


def test_norms_beyond_fp32():
    """A tensor whose norm fp32 does not hold: finite in the result, inf among the
    norms, and clipped to zeros by it; by the result's norm as defined."""
    t = torch.full((5000,), 3e38, device="cuda")
    out = torch.ones(5000, device="cuda")
    plan = Z.zero_tensor_plan([t], out=[out])
    res, norms = make_res(), torch.zeros(1, device="cuda")
    Z.zero_tensor_clip_norm(plan, 1.0, 1.0, res, workspace(plan), norms=norms, per_tensor=True)
    assert Z.read_result(res).overflow == 0 and norms.item() == float("inf")
    assert bool((out == 0).all())
    check_norm(res, None, [host64(t)], "l2", 1.0)
    Z.zero_tensor_clip(plan, 1e6, res)
    assert_rounded(out, clip_want(host64(t), math.sqrt(Z.read_result(res).sumsq), 1e6, 1.0), F32,
                   clip_steps(F32))


def test_clip_rounds_to_nearest_even_and_to_inf():
    x = torch.tensor([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 3.4e38, -3.4e38, 0.0, -0.0], device="cuda")
    out = [torch.empty(6, dtype=BF, device="cuda")]
    Z.zero_tensor_clip(Z.zero_tensor_plan([x], out=out), 0.0, make_res(1.0, 0, 1.0))
    inf = float("inf")
    assert out[0].tolist() == [1.0, 1 + 4 * 2.0 ** -8, inf, -inf, 0.0, 0.0]
    assert math.copysign(1.0, out[0][5].item()) == -1.0
    out = [torch.empty(6, dtype=HALF, device="cuda")]
    x = torch.tensor([1 + 2.0 ** -11, 1 + 3 * 2.0 ** -11, 65519.0, 65520.0, 2.0 ** -25, 2.0 ** -24],
                     device="cuda")
    Z.zero_tensor_clip(Z.zero_tensor_plan([x], out=out), 0.0, make_res(1.0, 0, 1.0))
    assert out[0].tolist() == [1.0, 1 + 4 * 2.0 ** -11, 65504.0, inf, 0.0, 2.0 ** -24]


# --------------------------------------------------------------- clip_norm --
@pytest.mark.parametrize("per_tensor", [False, True])
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_norm_is_norm_then_clip(kind, per_tensor, in_place):
    """The fused call gives the two calls' bits, at few pieces and many."""
    for sizes in ([], [0], [3], [4096, 70, 1, 0, 9], [4096] * 4, [4097] * 4, [3] * 5, [100] * 16,
                  [100] * 17, [16384], SIZES, [30000] * 40, [5] * 17000, [4096] * 1024,
                  [16384] * 1025, [1 << 22, (1 << 21) + 3, 77]):
        types = [(F32, BF, HALF)[k % 3] for k in range(len(sizes))]
        s = Set(sizes[:64], types[:64], [k % 8 for k in range(64)], seed=10)
        tensors = s.t
        if len(sizes) > 64:
            tensors = list(torch.randn(sum(sizes), device="cuda").split(sizes))
        host = [host64(t) for t in tensors]
        n, inv = len(tensors), f32(0.2)
        outs = [[torch.zeros(t.numel(), dtype=(BF, F32, HALF)[k % 3], device="cuda")
                 for k, t in enumerate(tensors)] for _ in range(2)]
        two = Z.zero_tensor_plan(tensors, out=outs[0], device="cuda")
        res, norms = [make_res(), make_res()], [torch.zeros(n, device="cuda") for _ in range(2)]
        Z.zero_tensor_norm(two, inv, res[0], workspace(two), kind=kind, norms=norms[0])
        if in_place:
            outs = [[t.clone() for t in tensors], tensors]
            two = Z.zero_tensor_plan(outs[0], device="cuda")
            one = Z.zero_tensor_plan(tensors, device="cuda")
        else:
            one = Z.zero_tensor_plan(tensors, out=outs[1], device="cuda")
        Z.zero_tensor_clip(two, 0.05, res[0], norms=norms[0] if per_tensor else None)
        Z.zero_tensor_clip_norm(one, 0.05, inv, res[1], workspace(one), kind=kind, norms=norms[1],
                                per_tensor=per_tensor)
        check_norm(res[1], norms[1], host, kind, inv)
        assert torch.equal(res[0], res[1]) and torch.equal(norms[0], norms[1])
        for a, b in zip(outs[0], outs[1]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        # and the definition's values
        total = math.sqrt(ref_norms(host, kind, inv)[0])
        for k in range(0, n, max(1, n // 50)):
            norm = norms[1][k].item() if per_tensor else total
            assert_rounded(outs[1][k], clip_want(host[k], norm, f32(0.05), inv), outs[1][k].dtype,
                           clip_steps(outs[1][k].dtype))
        if not per_tensor and not in_place:               # without the tensors' norms: same bits
            bare = make_res()
            again = [t.clone().zero_() for t in outs[1]]
            plan = Z.zero_tensor_plan(tensors, out=again, device="cuda")
            Z.zero_tensor_clip_norm(plan, 0.05, inv, bare, workspace(plan), kind=kind)
            assert torch.equal(bare, res[0])
            for a, b in zip(outs[0], again):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("sizes", [[40], [9, 70000, 5], [1 << 20, 3]])
@pytest.mark.parametrize("per_tensor", [False, True])
def test_clip_norm_overflow_writes_nothing(sizes, per_tensor):
    s = Set(sizes, [HALF] * len(sizes), [1] * len(sizes), seed=11)
    s.t[-1][-1] = float("nan")
    out = [torch.full_like(t, 3.0) for t in s.t]
    plan = Z.zero_tensor_plan(s.t, out=out)
    res, norms = make_res(), torch.zeros(len(sizes), device="cuda")
    Z.zero_tensor_clip_norm(plan, 1.0, 1.0, res, workspace(plan), norms=norms, per_tensor=per_tensor)
    assert Z.read_result(res).overflow == 1
    assert all(bool((o == 3.0).all()) for o in out)
    if not per_tensor:
        for kind in ("l2", "max"):
            res = make_res()
            Z.zero_tensor_clip_norm(plan, 1.0, 1.0, res, workspace(plan), kind=kind)
            assert Z.read_result(res).overflow == 1
            assert all(bool((o == 3.0).all()) for o in out)


@pytest.mark.parametrize("sizes", [[40, 3], [900] * 12, [9, 70000, 5], [3000] * 1100, [1 << 20, 3]])
def test_unscale_factor_from_the_step_control(sizes):
    """Every call and path with the factor read on the device gives the bits of the
    same call with it as an argument."""
    tensors = list(torch.randn(sum(sizes), device="cuda").split(sizes))
    ctl = Z.control_to_device(Z.zero_step_control_init(8.0, 1.0, 1000, 3.0, 0.9, 0.999))
    inv = Z.read_control(ctl).inv_scale
    assert inv == f32(1.0 / 24.0)
    for kind in ("l2", "max"):
        for norms in (None, torch.zeros(len(sizes), device="cuda")):
            got = []
            for args in ((inv, {}), (1.0, {"ctl_dev": ctl})):
                out = [torch.zeros_like(t) for t in tensors]
                acc = [torch.zeros_like(t) for t in tensors]
                plan, add = (Z.zero_tensor_plan(tensors, out=o) for o in (out, acc))
                res, ws = [make_res() for _ in range(3)], workspace(plan)
                kw = dict(kind=kind, norms=norms, **args[1])
                Z.zero_tensor_norm(plan, args[0], res[0], ws, **kw)
                Z.zero_tensor_clip_norm(plan, 0.1, args[0], res[1], ws, **kw)
                Z.zero_tensor_accumulate(add, 0.5, overwrite=True, res=res[2], workspace=ws,
                                         inv_scale=args[0], **kw)
                got.append(res + out + acc + ([norms.clone()] if norms is not None else []))
            for a, b in zip(*got):
                assert torch.equal(a, b)
            assert torch.equal(got[0][0], got[0][1])
            check_norm(got[0][0], None, [host64(t) for t in tensors], kind, inv)


def test_clip_by_the_flat_checks_result():
    """Tensors clipped by the norm that the flat buffer's check found."""
    sizes = [700, 33, 20000]
    flat = torch.randn(sum(sizes), device="cuda").to(BF)
    pieces = list(flat.split(sizes))
    out = [torch.empty(n, device="cuda") for n in sizes]
    res = make_res()
    ws = torch.empty(-(-Z.zero_check_workspace_bytes(flat.numel()) // 8), dtype=torch.float64,
                     device="cuda")
    Z.zero_unscale_check_norm(flat, 0.125, res, ws)
    Z.zero_tensor_clip(Z.zero_tensor_plan(pieces, out=out), 1.0, res)
    host = host64(flat)
    assert_rounded(torch.cat(out), clip_want(host, float(np.linalg.norm(host)) * 0.125, 1.0, 0.125),
                   F32, clip_steps(F32) + 21000 * 2.0 ** -53)


@pytest.mark.parametrize("seed", range(12))
def test_random_tables(seed):
    """Tables of random lengths, types and places: norm, clip_norm and accumulation
    against 64 bits, guard bands around every output."""
    rng = np.random.default_rng(100 + seed)
    count = int(2 ** rng.uniform(0, 8))
    sizes = [int(2 ** rng.uniform(0, 17)) - int(rng.integers(0, 2)) for _ in range(count)]
    pick = [F32, HALF, BF]
    src = Set(sizes, [pick[k] for k in rng.integers(0, 3, count)], rng.integers(0, 8, count), seed=seed,
              scale=10.0 ** rng.uniform(-3, 1))
    dst = Set(sizes, [pick[k] for k in rng.integers(0, 3, count)], rng.integers(0, 8, count),
              seed=1000 + seed)
    plan = Z.zero_tensor_plan(src.t, out=dst.t)
    x, y = [host64(t) for t in src.t], [host64(t) for t in dst.t]
    kind, inv, w = ("l2", "max")[seed % 2], f32(2.0 ** rng.uniform(-6, 2)), f32(rng.uniform(-2, 2))
    res, norms, ws = make_res(), torch.zeros(count, device="cuda"), workspace(plan)
    Z.zero_tensor_accumulate(plan, w, res=res, workspace=ws, inv_scale=inv, kind=kind, norms=norms)
    check_norm(res, norms, [host64(t) for t in dst.t], kind, inv)
    for t, a, b in zip(dst.t, x, y):
        assert_rounded(t, w * a + b, t.dtype, 2.0 ** -50 + (0 if t.dtype == F32 else 2.0 ** -24))
    limit = f32(10.0 ** rng.uniform(-2, 2))
    each = bool(rng.integers(0, 2))
    Z.zero_tensor_clip_norm(plan, limit, inv, res, ws, kind=kind, norms=norms, per_tensor=each)
    check_norm(res, norms, x, kind, inv)
    total = math.sqrt(Z.read_result(res).sumsq)
    for t, a, n in zip(dst.t, x, norms.tolist()):
        assert_rounded(t, clip_want(a, n if each else total, limit, inv), t.dtype, clip_steps(t.dtype))
    src.assert_guards()
    dst.assert_guards()


def test_clip_norm_matches_torch_clip_grad_norm():
    gen = torch.Generator(device="cuda").manual_seed(12)
    params = [torch.nn.Parameter(torch.zeros(sh, device="cuda"))
              for sh in ((64, 33), (33,), (1,), (257, 129))]
    for p in params:
        p.grad = torch.empty_like(p).normal_(generator=gen)
    mine = [p.grad.clone() for p in params]
    plan = Z.zero_tensor_plan(mine)
    for kind, p in (("l2", 2.0), ("max", float("inf"))):
        res = make_res()
        norm = torch.nn.utils.clip_grad_norm_(params, 0.5, norm_type=p, foreach=False)
        Z.zero_tensor_clip_norm(plan, 0.5, 1.0, res, workspace(plan), kind=kind)
        # torch sums in fp32 (33,153 terms, pairwise) and rounds its norms to fp32
        assert abs(math.sqrt(Z.read_result(res).sumsq) - norm.item()) <= 1e-5 * norm.item()
        for q, m in zip(params, mine):
            assert torch.allclose(q.grad, m, rtol=2e-5, atol=0.0)


# -------------------------------------------------------------- accumulate --
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("dst", [F32, HALF, BF])
@pytest.mark.parametrize("src", [F32, HALF, BF])
def test_accumulate(src, dst, first):
    sizes = SIZES + [0, 12]
    w = f32(0.7)
    s = Set(sizes, [src] * len(sizes), [(k + 2) % 8 for k in range(len(sizes))], seed=13)
    for kind in (None, "l2", "max"):
        o = Set(sizes, [dst] * len(sizes), [k % 8 for k in range(len(sizes))], seed=14)
        plan = Z.zero_tensor_plan(s.t, out=o.t)
        x, y = [host64(t) for t in s.t], [host64(t) for t in o.t]
        if kind is None:
            Z.zero_tensor_accumulate(plan, w, overwrite=first)
        else:
            res, norms = make_res(5.0, 1, 3.0), torch.zeros(len(sizes), device="cuda")
            Z.zero_tensor_accumulate(plan, w, overwrite=first, res=res, workspace=workspace(plan),
                                     inv_scale=0.125, kind=kind, norms=norms)
            check_norm(res, norms, [host64(t) for t in o.t], kind, 0.125)
        for t, a, b in zip(o.t, x, y):
            want = w * a + (0.0 if first else b)
            assert_rounded(t, want, dst, 2.0 ** -50 if dst == F32 else 2.0 ** -24 + 2.0 ** -50)
        o.assert_guards()
        s.assert_guards()


def test_accumulate_in_place_and_overflow():
    s = Set([3000, 9], [F32, BF], [1, 0], seed=15)
    host = [host64(t) for t in s.t]
    plan = Z.zero_tensor_plan(s.t)
    Z.zero_tensor_accumulate(plan, 0.5)                   # x + x/2, exact but for the rounding
    for t, x in zip(s.t, host):
        assert_rounded(t, 1.5 * x, t.dtype, 2.0 ** -24)
    # a sum beyond a 16-bit type's range is an overflow of what is stored
    big = [torch.full((20,), 60000.0, dtype=HALF, device="cuda")]
    acc = [torch.full((20,), 60000.0, dtype=HALF, device="cuda")]
    p = Z.zero_tensor_plan(big, out=acc)
    for kind in ("l2", "max"):
        res = make_res()
        Z.zero_tensor_accumulate(p, 1.0, res=res, workspace=workspace(p), kind=kind)
        assert Z.read_result(res).overflow == 1 and bool(torch.isinf(acc[0]).all())
    Z.zero_tensor_accumulate(p, 1.0, overwrite=True, res=res, workspace=workspace(p))
    assert Z.read_result(res).overflow == 0               # the old values are not read
    acc[0].fill_(float("nan"))
    Z.zero_tensor_accumulate_norm(p, 1.0, res, workspace(p), overwrite=True)
    assert Z.read_result(res).overflow == 0 and float(acc[0][0]) == 60000.0


# ----------------------------------------------- tables, streams, graphs ----
def test_dense_permutations_and_refusals():
    base = torch.randn(6, 10, 7, device="cuda")
    t = base.permute(2, 0, 1)
    out = torch.zeros(6, 10, 7, device="cuda").permute(2, 0, 1)
    plan = Z.zero_tensor_plan([t], out=[out])
    Z.zero_tensor_clip(plan, 0.0, make_res(1.0, 0, 2.0))
    assert torch.equal(out, t * 2)
    with pytest.raises(ValueError, match="order"):
        Z.zero_tensor_plan([t], out=[torch.zeros(7, 6, 10, device="cuda")])
    with pytest.raises(ValueError, match="dense"):
        Z.zero_tensor_plan([base[:, ::2]])
    with pytest.raises(ValueError, match="order"):
        Z.zero_tensor_plan([base], out=[base.reshape(-1)[1:]])
    with pytest.raises(ValueError, match="one tensor for each"):
        Z.zero_tensor_plan([base], out=[])
    with pytest.raises(TypeError):
        Z.zero_tensor_plan([base.double()])
    with pytest.raises(ValueError, match="on cuda"):
        Z.zero_tensor_plan([base, torch.zeros(3)])
    with pytest.raises(ValueError, match="strided"):
        Z.zero_tensor_plan([torch.eye(3, device="cuda").to_sparse()])
    with pytest.raises(ValueError, match="negated"):
        Z.zero_tensor_plan([torch.ones(1, dtype=torch.complex64, device="cuda").conj().imag])
    flat = torch.zeros(100, device="cuda")
    twice = Z.zero_tensor_plan([flat, flat[50:]])         # read only
    res = make_res()
    Z.zero_tensor_norm(twice, 1.0, res, workspace(twice))
    for call in (lambda: Z.zero_tensor_clip(twice, 1.0, res),
                 lambda: Z.zero_tensor_clip_norm(twice, 1.0, 1.0, res, workspace(twice)),
                 lambda: Z.zero_tensor_accumulate(twice),
                 lambda: Z.zero_tensor_norm(plan, float("nan"), res, workspace(plan)),
                 lambda: Z.zero_tensor_norm(plan, 0.0, res, workspace(plan)),
                 lambda: Z.zero_tensor_clip(plan, float("nan"), res),
                 lambda: Z.zero_tensor_accumulate(plan, float("inf"))):
        with pytest.raises(Z.ZeroError, match="invalid"):
            call()
    for call in (lambda: Z.zero_tensor_norm(plan, 1.0, res[:3], workspace(plan)),
                 lambda: Z.zero_tensor_norm(plan, 1.0, res.cpu(), workspace(plan)),
                 lambda: Z.zero_tensor_norm(plan, 1.0, res, workspace(plan)[:0]),
                 lambda: Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), kind="l1"),
                 lambda: Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), norms=flat.half()),
                 lambda: Z.zero_tensor_norm(plan, 1.0, res, workspace(plan), norms=flat[:0]),
                 lambda: Z.zero_tensor_clip(plan, 1.0, res, norms=flat[::2]),
                 lambda: Z.zero_tensor_accumulate(plan, norms=flat),
                 lambda: Z.zero_tensor_accumulate(plan, accumulate=True),
                 lambda: Z.zero_tensor_accumulate(plan, res=res),
                 lambda: Z.zero_tensor_clip_norm(plan, 1.0, 1.0, res, workspace(plan),
                                                 per_tensor=True)):
        with pytest.raises(ValueError):
            call()


def test_other_streams():
    """Two calls at once on two streams, each with a workspace of its own."""
    tensors = [torch.randn(n, device="cuda") for n in (100, 300_001, 7)]
    plan = Z.zero_tensor_plan(tensors)
    want = make_res()
    Z.zero_tensor_norm(plan, 1.0, want, workspace(plan))
    streams = [torch.cuda.Stream() for _ in range(2)]
    res, ws = [make_res() for _ in streams], [workspace(plan) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, r, w in zip(streams, res, ws):
            Z.zero_tensor_norm(plan, 1.0, r, w, stream=s)
    with torch.cuda.stream(streams[0]):
        Z.zero_tensor_norm(plan, 1.0, res[0], ws[0])
    Z.zero_tensor_norm(plan, 1.0, res[1], ws[1], stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(r, want) for r in res)
    with torch.cuda.stream(streams[0]):                   # built there, called on the default one
        plan = Z.zero_tensor_plan(tensors)
    Z.zero_tensor_norm(plan, 1.0, res[0].zero_(), ws[0])
    Z.zero_tensor_norm(plan, 1.0, res[1].zero_(), ws[1], stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(r, want) for r in res)


def test_no_plan_inside_a_capture():
    t = torch.ones(1000, device="cuda")
    plan, res = Z.zero_tensor_plan([t]), make_res()
    ws, said = workspace(plan), []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_tensor_norm(plan, 1.0, res, ws)
        try:
            Z.zero_tensor_plan([t])
        except RuntimeError as e:
            said.append(str(e))
    assert said == ["build the plan before the capture"]
    for k in (1.0, 2.0, 3.0):                             # the capture is whole
        t.fill_(k)
        graph.replay()
        assert Z.read_result(res).sumsq == 1000.0 * k * k


@pytest.mark.parametrize("per_tensor", [False, True])
def test_graph_replays(per_tensor):
    """Accumulate, norm and clip captured once and replayed on new gradients,
    with eager calls that use other buffers in between."""
    sizes = [70, 20000, 0, 300_000]
    g16 = [torch.zeros(n, dtype=BF, device="cuda") for n in sizes]
    acc = [torch.zeros(n, device="cuda") for n in sizes]
    out = [torch.zeros(n, dtype=HALF, device="cuda") for n in sizes]
    p_acc, p_out = Z.zero_tensor_plan(g16, out=acc), Z.zero_tensor_plan(acc, out=out)
    res, norms = make_res(), torch.zeros(len(sizes), device="cuda")
    ctl = Z.control_to_device(Z.zero_step_control_init(8.0, 1.0, 2, 1.0, 0.9, 0.999))
    ws = workspace(p_out)

    def step(p_acc, p_out, res, norms, ws, ctl):
        Z.zero_tensor_accumulate(p_acc, 0.5, overwrite=True)
        Z.zero_tensor_accumulate(p_acc, 0.25, res=res, workspace=ws, norms=norms, ctl_dev=ctl)
        Z.zero_tensor_clip_norm(p_out, 0.3, 1.0, res, ws, norms=norms, per_tensor=per_tensor,
                                ctl_dev=ctl)
        Z.zero_step_control_update(ctl, res)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p_acc, p_out, res, norms, ws, ctl)
    e_g16, e_acc, e_out = ([t.clone() for t in x] for x in (g16, acc, out))
    e_plans = Z.zero_tensor_plan(e_g16, out=e_acc), Z.zero_tensor_plan(e_acc, out=e_out)
    e_res, e_norms, e_ws, e_ctl = make_res(), torch.zeros_like(norms), workspace(p_out), ctl.clone()
    gen = torch.Generator(device="cuda").manual_seed(16)
    for k in range(6):
        for t, e in zip(g16, e_g16):
            t.normal_(generator=gen)
            e.copy_(t)
        if k == 3:
            g16[1][7] = e_g16[1][7] = float("inf")        # a skipped step among them
        graph.replay()
        step(*e_plans, e_res, e_norms, e_ws, e_ctl)
        torch.cuda.synchronize()
        assert torch.equal(res, e_res) and torch.equal(ctl, e_ctl)
        assert torch.equal(norms.view(torch.int32), e_norms.view(torch.int32))
        for a, b in zip(acc + out, e_acc + e_out):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert Z.read_result(res).overflow == (k == 3)
    assert Z.read_control(ctl).skipped == 1


def test_a_step_from_micro_batches_to_adamw():
    """The operators as a step uses them: three micro-batches accumulate in fp32
    (the last with the norm), the result is cast into the flat 16-bit gradient,
    and AdamW unscales and clips by that norm; against the same step in 64 bits
    up to AdamW's input and torch's AdamW after it."""
    shapes = [(64, 48), (48,), (129, 31), (5,)]
    sizes = [math.prod(s) for s in shapes]
    total, scale, max_norm = sum(sizes), 1024.0, 0.5
    gen = torch.Generator(device="cuda").manual_seed(17)
    acc = [torch.full((n,), float("nan"), device="cuda") for n in sizes]
    flat = torch.zeros(total, dtype=BF, device="cuda")
    pieces = list(flat.split(sizes))
    to_flat = Z.zero_tensor_plan(acc, out=pieces)
    res = make_res()
    want = [np.zeros(n) for n in sizes]
    for k in range(3):
        grads = [torch.empty(s, device="cuda").normal_(0.0, 0.02 * scale, generator=gen).to(BF)
                 for s in shapes]
        plan = Z.zero_tensor_plan([g.reshape(-1) for g in grads], out=acc)
        norm = dict(res=res, workspace=workspace(plan), inv_scale=1.0 / scale) if k == 2 else {}
        Z.zero_tensor_accumulate(plan, 1.0 / 3.0, overwrite=k == 0, **norm)
        want = [w + f32(1.0 / 3.0) * host64(g) for w, g in zip(want, grads)]
    for a, w in zip(acc, want):                           # three roundings of partial sums
        lim = 3 * U[F32] * (np.abs(w) + 0.2 * scale)
        assert (np.abs(host64(a) - w) <= lim).all()
    check_norm(res, None, [host64(a) for a in acc], "l2", 1.0 / scale)
    norm = math.sqrt(Z.read_result(res).sumsq)
    assert norm > max_norm                                # the clip is active
    Z.zero_tensor_clip(to_flat, 0.0, make_res(0.0, 0, 1.0))   # a cast: scaled, unclipped
    assert torch.equal(flat, torch.cat(acc).to(BF))
    p16 = torch.randn(total, device="cuda", generator=gen).to(BF)
    master = p16.float()
    m, v, new16 = torch.zeros_like(master), torch.zeros_like(master), torch.zeros_like(p16)
    hp = Z.zero_adamw_hparams(1e-3, 0.9, 0.999, 1e-8, 0.01, max_norm, 1)
    start = master.clone()
    Z.zero_adamw_step(master, m, v, new16, flat, hp, res)
    g = flat.double().cpu() / scale * (max_norm / (norm + 1e-6))
    q = torch.nn.Parameter(start.double().cpu())
    q.grad = g
    torch.optim.AdamW([q], lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01).step()
    # fp32 AdamW's first step: the update is lr * g / (|g| + eps), a few roundings
    # of values of at most |p| and lr
    lim = 4 * U[F32] * q.detach().abs() + 16 * U[F32] * 1e-3
    # the ratio g / (|g| + eps) moves with g's own rounding only where |g| ~ eps
    lim += 1e-3 * 8 * U[F32] * 1.0
    assert bool(((master.double().cpu() - q.detach()).abs() <= lim).all())
    assert torch.equal(new16, master.to(BF))
    # the same clip done by the table call gives the gradient AdamW used
    clipped = [torch.empty(n, device="cuda") for n in sizes]
    Z.zero_tensor_clip(Z.zero_tensor_plan(pieces, out=clipped), max_norm, res)
    assert_rounded(torch.cat(clipped), g.numpy(), F32, clip_steps(F32))


# ------------------------------------------------------ which path is taken ----
def call_ms(call, reps=20):
    """The shortest of `reps` calls, by events."""
    call()
    times = []
    for _ in range(reps):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("per_tensor", [False, True])
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_few_elements_among_empty_tensors(kind, per_tensor):
    """Tables of empty tensors but for one or a few, on both sides of the number of
    tensors that one block gives norms to: the two calls' bits and the definition's
    values."""
    for count in (17, 127, 128, 129, 5000):
        sizes = [0] * count
        sizes[0], sizes[count // 2], sizes[-1] = 3, 4097, 70
        s = Set([n for n in sizes if n], [F32, BF, HALF], [1, 2, 3], seed=18)
        held = iter(s.t)
        tensors = [next(held) if n else torch.zeros(0, device="cuda") for n in sizes]
        host = [host64(t) for t in tensors]
        outs = [[torch.zeros_like(t) for t in tensors] for _ in range(2)]
        two, one = (Z.zero_tensor_plan(tensors, out=o) for o in outs)
        res = [make_res(), make_res()]
        norms = [torch.full((count,), -1.0, device="cuda") for _ in range(2)]
        Z.zero_tensor_norm(two, 0.5, res[0], workspace(two), kind=kind, norms=norms[0])
        check_norm(res[0], norms[0], host, kind, 0.5)
        Z.zero_tensor_clip(two, 0.1, res[0], norms=norms[0] if per_tensor else None)
        Z.zero_tensor_clip_norm(one, 0.1, 0.5, res[1], workspace(one), kind=kind, norms=norms[1],
                                per_tensor=per_tensor)
        assert torch.equal(res[0], res[1]) and torch.equal(norms[0], norms[1])
        total = math.sqrt(ref_norms(host, kind, 0.5)[0])
        for k in (0, count // 2, count - 1):
            assert torch.equal(outs[0][k], outs[1][k])
            norm = norms[1][k].item() if per_tensor else total
            assert_rounded(outs[1][k], clip_want(host[k], norm, f32(0.1), 0.5), outs[1][k].dtype,
                           clip_steps(outs[1][k].dtype))


def test_many_empty_tensors_are_not_one_blocks_work():
    """200,000 tensors' norms, all but one of them empty: 45 us by all of the GPU, 8.2 ms
    where one block takes them in turn."""
    tensors = [torch.zeros(0, device="cuda")] * 200_000 + [torch.full((5,), 2.0, device="cuda")]
    plan = Z.zero_tensor_plan(tensors)
    res, ws = make_res(), workspace(plan)
    norms = torch.full((len(tensors),), -1.0, device="cuda")
    ms = call_ms(lambda: Z.zero_tensor_norm(plan, 1.0, res, ws, norms=norms))
    assert Z.read_result(res).sumsq == 20.0
    assert bool((norms[:-1] == 0).all()) and norms[-1].item() == f32(math.sqrt(20.0))
    assert ms < 2.0
    ms = call_ms(lambda: Z.zero_tensor_clip_norm(plan, 1e9, 1.0, res, ws, norms=norms,
                                                 per_tensor=True))
    assert bool((tensors[-1] == 2.0).all()) and ms < 2.0


def test_overwriting_16_bit_accumulators_runs_as_a_clip_does():
    """The first micro-batch of 2.2e8 bf16 values into bf16 accumulators, with the norm, and
    their clip move the same bytes: 142 and 134 us.  With the blocks per CU that adding
    to fp32 accumulators takes it was 228."""
    n = 220_000_000
    x, y = torch.zeros(n, dtype=BF, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    plan = Z.zero_tensor_plan(list(x.split(1_000_000)), out=list(y.split(1_000_000)))
    res, given, ws = make_res(), make_res(4.0, 0, 0.5), workspace(plan)
    first, clip = [], []
    for _ in range(10):                                   # in turn
        first.append(call_ms(lambda: Z.zero_tensor_accumulate(plan, 0.5, overwrite=True, res=res,
                                                              workspace=ws), 4))
        clip.append(call_ms(lambda: Z.zero_tensor_clip(plan, 1.0, given), 4))
    assert min(first) < 1.35 * min(clip), (min(first), min(clip))


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("few", [3, 128, 129, 600])
def test_tensors_of_many_partials(few, kind):
    """A tensor of over 1024 partials, whose norm a block joins where there are few tensors
    and a wave otherwise (1027 partials of the norm and 4108 of the accumulation: up to
    128 and 513 tensors): every call that gives norms, against 64 bits."""
    sizes = [5] * few
    sizes[1], sizes[-1] = 1027 * 16384 + 4099, 0
    flat = torch.randn(sum(sizes) + 1, generator=torch.Generator(device="cuda").manual_seed(few),
                       device="cuda").to(BF)[1:]
    tensors = list(flat.split(sizes))
    host = [host64(t) for t in tensors]
    out = torch.zeros(sum(sizes), device="cuda")
    plan = Z.zero_tensor_plan(tensors, out=list(out.split(sizes)))
    ws, inv = workspace(plan), f32(0.3)
    res, norms = make_res(), torch.full((few,), -1.0, device="cuda")
    Z.zero_tensor_norm(plan, inv, res, ws, kind=kind, norms=norms)
    check_norm(res, norms, host, kind, inv)
    again, each = make_res(), torch.full((few,), -1.0, device="cuda")
    Z.zero_tensor_clip_norm(plan, 0.5, inv, again, ws, kind=kind, norms=each, per_tensor=True)
    assert torch.equal(again, res) and torch.equal(each, norms)
    for y, x, n in zip(out.split(sizes), host, each.tolist()):
        assert_rounded(y, clip_want(x, n, 0.5, inv), F32, clip_steps(F32))
    Z.zero_tensor_accumulate(plan, 1.0, overwrite=True, res=res, workspace=ws, inv_scale=inv,
                             kind=kind, norms=norms)
    assert torch.equal(out, flat.float())
    check_norm(res, norms, host, kind, inv)
    flat[sizes[0] + 12_345_678] = float("nan")
    Z.zero_tensor_norm(plan, inv, res, ws, kind=kind, norms=norms)
    assert Z.read_result(res).overflow == 1
    assert [k for k, x in enumerate(norms.tolist()) if not math.isfinite(x)] == [1]


def test_a_large_tensor_beside_many_small_ones():
    """The norms of 4.3e9 elements (262,144 partials, 1,048,576 of the accumulation) beside
    5000 tensors: joined by blocks, though the average tensor has few partials."""
    n, few = 1 << 32, 5000
    if torch.cuda.mem_get_info()[0] < 2 * n + (4 << 30):
        pytest.skip("not enough device memory")
    flat = torch.zeros(n + 64 * few, dtype=BF, device="cuda")
    flat[5], flat[n - 1], flat[n], flat[-1] = 3.0, -4.0, 12.0, 2.0
    plan = Z.zero_tensor_plan(list(flat.split([n] + [64] * few)))
    ws = workspace(plan)
    for add, scale in ((False, 1.0), (True, 2.0)):
        res, norms = make_res(), torch.full((few + 1,), -1.0, device="cuda")
        if add:
            Z.zero_tensor_accumulate(plan, 1.0, res=res, workspace=ws, norms=norms)
        else:
            Z.zero_tensor_norm(plan, 1.0, res, ws, norms=norms)
        assert Z.read_result(res).sumsq == 173.0 * scale * scale
        assert [norms[k].item() / scale for k in (0, 1, -1)] == [5.0, 12.0, 2.0]
        assert not norms[2:-1].any()


def test_a_stream_destroyed_before_the_plan():
    """Calls on a stream that the caller made, by its handle and as torch's current
    stream, which is then destroyed: the plan goes later, and its memory is used again."""
    paths = [ln.split()[-1] for ln in open("/proc/self/maps") if "libamdhip64" in ln]
    hip = ctypes.CDLL(paths[0])
    hip.hipStreamDestroy.argtypes = [ctypes.c_void_p]
    tensors = [torch.randn(n, device="cuda") for n in (100, 300_001, 7)]
    plan, want = Z.zero_tensor_plan(tensors), make_res()
    Z.zero_tensor_norm(plan, 1.0, want, workspace(plan))
    recorded = []
    plan.table.record_stream = recorded.append
    res, ws = make_res(), workspace(plan)
    torch.cuda.synchronize()
    handles = [ctypes.c_void_p() for _ in range(2)]
    for handle in handles:
        assert hip.hipStreamCreateWithFlags(ctypes.byref(handle), 1) == 0    # non-blocking
    for external, handle in enumerate(handles):
        res.zero_()
        torch.cuda.synchronize()
        if external:
            with torch.cuda.stream(torch.cuda.ExternalStream(handle.value)):
                Z.zero_tensor_norm(plan, 1.0, res, ws)
        else:
            Z.zero_tensor_norm(plan, 1.0, res, ws, stream=handle.value)
        torch.cuda.synchronize()
        assert torch.equal(res, want)
        assert not recorded                               # before the stream is gone
        assert hip.hipStreamDestroy(handle) == 0
    side = torch.cuda.Stream()                            # torch's own is recorded, once
    for _ in range(2):
        Z.zero_tensor_norm(plan, 1.0, res, ws, stream=side)
    side.synchronize()
    assert recorded == [side] and torch.equal(res, want)
    del plan
    assert bool((torch.zeros(4096, dtype=torch.uint8, device="cuda") == 0).all())


@pytest.mark.parametrize("per_tensor", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_of_tables_beyond_the_cache(in_place, per_tensor):
    """Tables of over 256 MiB have a kernel of their own: every type pair, ragged sizes and
    starts give the bits of small plans over the same tensors, the guards stay, a
    skipped step writes nothing, and so does a factor of 1 in place."""
    large = [5_000_001, 70, 4_500_017, 16385, 3_999_999, 4_194_309, 6_000_007, 4_100_003,
             4_194_304, 6_500_003, 5_500_012, 5_300_005, 4_096_000, 4_800_008, 4_700_003]
    sizes = [n for pair in zip(SIZES, large + SIZES) for n in pair] + [0, 5_100_001]
    count = len(sizes)
    pick = [F32, HALF, BF]
    s = Set(sizes, [pick[k % 3] for k in range(count)], [k % 8 for k in range(count)], seed=19)
    if in_place:
        o = s
        plan = Z.zero_tensor_plan(s.t)
    else:
        o = Set(sizes, [pick[k // 3 % 3] for k in range(count)], [(5 * k + 1) % 8 for k in range(count)],
                seed=20)
        plan = Z.zero_tensor_plan(s.t, out=o.t)
    assert plan.c.bytes > 256 << 20
    inv, max_norm = f32(0.7), f32(0.9)
    norms = torch.rand(count, generator=torch.Generator(device="cuda").manual_seed(21),
                       device="cuda") * 2.0
    given = norms if per_tensor else None
    before = [t.clone() for t in o.t]
    Z.zero_tensor_clip(plan, max_norm, make_res(1.5625, 1, inv), norms=given)
    assert all(torch.equal(t, b) for t, b in zip(o.t, before))
    if in_place:
        for off in (0.0, 100.0):
            Z.zero_tensor_clip(plan, off, make_res(1.5625, 0, 1.0), norms=given)
            assert all(torch.equal(t, b) for t, b in zip(o.t, before))
    res = make_res(1.5625, 0, inv)                        # norm 1.25
    want = [torch.zeros_like(t) for t in o.t]
    for k, (x, w) in enumerate(zip(s.t, want)):
        small = Z.zero_tensor_plan([x], out=[w])
        assert small.c.bytes < 256 << 20
        Z.zero_tensor_clip(small, max_norm, res, norms=norms[k:k + 1] if per_tensor else None)
    host = [host64(x) if n < 1 << 20 or k == 1 else None for k, (n, x) in enumerate(zip(sizes, s.t))]
    Z.zero_tensor_clip(plan, max_norm, res, norms=given)
    for k, (t, w) in enumerate(zip(o.t, want)):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8)), k
        if host[k] is not None:
            norm = norms[k].item() if per_tensor else 1.25
            assert_rounded(t, clip_want(host[k], norm, max_norm, inv), t.dtype, clip_steps(t.dtype))
    o.assert_guards()
    s.assert_guards()

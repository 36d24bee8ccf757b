"""Embedding lookup and its gradient on the GPU against the definition in 64 bits.

Tolerances.  A lookup is one product in fp32 (half a step of fp32, u = 2^-24) and one
rounding to the result's type.  A gradient's sum of k rows takes at most k additions, each
off by u of the magnitudes' sum; then one fused product and sum, rounded to fp32, and to
the type.
"""
import numpy as np
import pytest
import torch

import zero_partitioned_mixed_shard_amd as Z

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24
LEAST = {"fp32": 2.0 ** -149, "fp16": 2.0 ** -25, "bf16": 2.0 ** -134}   # half the last subnormal


def half_step(t):
    return torch.finfo(TYPES[t]).eps / 2


def workspace(n, vocab, dim):
    # whatever it holds does not matter
    return torch.full((max(256, Z.zero_embedding_workspace_bytes(n, vocab, dim)),), 0xFF,
                      dtype=torch.uint8, device="cuda")


def table_of(vocab, dim, begin, count, values):
    """The whole table in 64 bits, 0 outside the slice."""
    w = torch.zeros(vocab * dim, dtype=torch.float64)
    w[begin:begin + count] = values.double().cpu().reshape(-1)
    return w.view(vocab, dim)


def lookup_ref(ids, vocab, dim, begin, values, scale):
    w = table_of(vocab, dim, begin, values.numel(), values)
    ids = ids.cpu().long()
    ok = (ids >= 0) & (ids < vocab)
    return torch.where(ok[..., None], w[torch.where(ok, ids, 0)] * scale, 0.0)


def grad_ref(ids, dy, vocab, dim, begin, old, scale, overwrite, padding):
    """(the slice's gradient, the bound of its error before the last rounding)."""
    count = old.numel()
    ids, dy = ids.cpu().long().reshape(-1), dy.double().cpu().reshape(-1, dim)
    ok = (ids >= 0) & (ids < vocab) & (ids != (-1 if padding is None else padding))
    total = torch.zeros(vocab, dim, dtype=torch.float64)
    size, times = torch.zeros_like(total), torch.zeros(vocab, 1, dtype=torch.float64)
    total.index_add_(0, ids[ok], dy[ok])
    size.index_add_(0, ids[ok], dy[ok].abs())
    times.index_add_(0, ids[ok], torch.ones(int(ok.sum()), 1, dtype=torch.float64))
    want = total * scale
    bound = abs(scale) * size * times * U32
    part = slice(begin, begin + count)
    want, bound = want.reshape(-1)[part], bound.reshape(-1)[part]
    if not overwrite:
        want = want + old.double().cpu().reshape(-1)
    return want, bound + U32 * want.abs()


def check_grad(got, kind, want, bound):
    off = (got.double().cpu().reshape(-1) - want).abs()
    limit = bound + half_step(kind) * (want.abs() + bound) + LEAST[kind]
    assert bool((off <= limit).all()), float((off - limit).max())


def inputs(n, vocab, dim, src, seed, spread="zipf", ids_type=torch.int64):
    gen = torch.Generator().manual_seed(seed)
    if spread == "zipf":
        ids = (torch.exp(torch.rand(n, generator=gen, dtype=torch.float64) * np.log(vocab + 1.0)) - 1).long()
        ids = ids.clamp(0, vocab - 1)
    elif spread == "one":
        ids = torch.full((n,), vocab - 1)
    else:
        ids = torch.randint(-2, vocab + 2, (n,), generator=gen)       # some of no row
    dy = torch.randn(n, dim, generator=gen).to(TYPES[src])
    return ids.to(ids_type).cuda(), dy.cuda()


@pytest.mark.parametrize("src", sorted(TYPES))
@pytest.mark.parametrize("dst", sorted(TYPES))
@pytest.mark.parametrize("ids_type", [torch.int32, torch.int64])
def test_lookup_types(src, dst, ids_type):
    vocab, dim, n, scale = 37, 515, 41, 0.3
    ids, _ = inputs(n, vocab, dim, src, 3, "any", ids_type)
    w = torch.randn(vocab * dim, generator=torch.Generator().manual_seed(1)).to(TYPES[src]).cuda()
    out = torch.full((n, dim), 7.0, dtype=TYPES[dst], device="cuda")
    Z.zero_embedding_lookup(out, ids, w, vocab, dim, scale=scale)
    want = lookup_ref(ids, vocab, dim, 0, w, np.float32(scale).item())
    off = (out.double().cpu() - want).abs()
    assert bool((off <= (U32 + half_step(dst)) * 1.0001 * want.abs() + LEAST[dst]).all())


@pytest.mark.parametrize("dim", [1, 7, 8, 9, 64, 511, 512, 513, 1024, 1031])
@pytest.mark.parametrize("begin,end", [(0, 0), (5, 3), (1, 0), (0, 1)])
def test_lookup_slices(dim, begin, end):
    vocab, n = 23, 70
    total = vocab * dim
    begin, end = min(begin * dim + 3, total - 1) if begin else 0, min(end * dim + 5, total) if end else 0
    count = max(0, total - begin - end)
    ids, _ = inputs(n, vocab, dim, "bf16", 5, "any")
    w = torch.randn(count, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    ids = ids.view(7, 10)
    out = torch.full((7, 10, dim), 7.0, device="cuda")
    Z.zero_embedding_lookup(out, ids, w, vocab, dim, begin=begin)
    assert torch.equal(out.double().cpu(), lookup_ref(ids, vocab, dim, begin, w, 1.0))


GRADS = [
    # tokens, vocab, dim, ids
    (1, 1, 1, "zipf"), (1, 50, 9, "zipf"), (2, 3, 512, "one"), (7, 5, 513, "any"), (64, 11, 64, "zipf"),
    (65, 1000, 72, "any"), (300, 17, 33, "zipf"), (1000, 512, 130, "zipf"), (1025, 511, 100, "any"),
    (4096, 70001, 16, "zipf"), (8192, 300, 8, "one"), (8192, 3000, 24, "zipf"), (8193, 3000, 24, "zipf"),
    (12289, 7, 40, "any"), (20000, 300000, 9, "zipf"), (70000, 2, 12, "any"), (70000, 50000, 5, "zipf"),
]


@pytest.mark.parametrize("n,vocab,dim,spread", GRADS)
@pytest.mark.parametrize("overwrite", [False, True])
def test_grad_sizes(n, vocab, dim, spread, overwrite):
    ids, dy = inputs(n, vocab, dim, "bf16", n + vocab, spread)
    grad = torch.randn(vocab, dim, generator=torch.Generator().manual_seed(9)).cuda()
    old = grad.clone()
    ws = workspace(n, vocab, dim)
    Z.zero_embedding_grad(grad, ids, dy, vocab, dim, ws, scale=0.5, overwrite=overwrite)
    want, bound = grad_ref(ids, dy, vocab, dim, 0, old, 0.5, overwrite, None)
    check_grad(grad, "fp32", want, bound)
    # a row that no token has stays as it was, bit for bit; or is zero
    has = torch.zeros(vocab + 1, dtype=torch.bool)
    has[torch.where((ids >= 0) & (ids < vocab), ids, vocab).cpu().long()] = True
    rest = ~has[:vocab]
    assert torch.equal(grad.cpu()[rest], torch.zeros_like(old.cpu()[rest]) if overwrite else old.cpu()[rest])
    # the same call, the same bits
    again = old.clone()
    Z.zero_embedding_grad(again, ids, dy, vocab, dim, ws, scale=0.5, overwrite=overwrite)
    assert torch.equal(again, grad)


@pytest.mark.parametrize("src", sorted(TYPES))
@pytest.mark.parametrize("dst", sorted(TYPES))
@pytest.mark.parametrize("overwrite", [False, True])
def test_grad_types_and_slices(src, dst, overwrite):
    vocab, dim, n = 203, 261, 900
    for begin, end, padding in ((0, 0, None), (4 * dim + 7, 3 * dim + 1, 9), (100 * dim + 3, 102 * dim + 9, 2)):
        count = vocab * dim - begin - end
        ids, dy = inputs(n, vocab, dim, src, 11 + begin, "zipf", torch.int32)
        # rows of a wider buffer; what ignored tokens hold is not read
        wide = torch.full((n, dim + 11), float("nan"), dtype=TYPES[src], device="cuda")
        wide[:, :dim] = dy
        if padding is not None:
            wide[ids == padding] = float("nan")
            dy = torch.where((ids == padding)[:, None], torch.zeros_like(dy), dy)
        grad = torch.randn(count, generator=torch.Generator().manual_seed(4)).to(TYPES[dst]).cuda()
        old = grad.clone()
        Z.zero_embedding_grad(grad, ids, wide[:, :dim], vocab, dim, workspace(n, vocab, dim), begin=begin,
                              scale=2.0, overwrite=overwrite, padding_id=padding)
        want, bound = grad_ref(ids, dy, vocab, dim, begin, old, 2.0, overwrite, padding)
        check_grad(grad, dst, want, bound)




def test_special_values_stay_in_their_rows():
    vocab, dim, n = 20, 70, 64
    ids = torch.arange(n, device="cuda") % 10
    dy = torch.ones(n, dim, device="cuda")
    dy[3, 5], dy[14, 6], dy[24, 6] = float("nan"), float("inf"), float("-inf")
    grad = torch.zeros(vocab, dim, device="cuda")
    Z.zero_embedding_grad(grad, ids, dy, vocab, dim, workspace(n, vocab, dim))
    got = grad.cpu()
    assert bool(got[3, 5].isnan()) and bool(got[4, 6].isnan())
    got[3, 5] = got[4, 6] = 0.0
    assert bool(torch.isfinite(got).all()) and not bool(got[10:].any())
    w = torch.full((vocab, dim), 60000.0, device="cuda")
    out = torch.empty(n, dim, dtype=torch.float16, device="cuda")
    Z.zero_embedding_lookup(out, ids, w, vocab, dim, scale=2.0)
    assert bool(out.isinf().all())                           # past fp16's range


def test_nothing_else_is_written():
    vocab, dim, n, pad = 61, 77, 500, 512
    for kind in TYPES:
        for begin, count in ((0, vocab * dim), (dim * 3 + 5, dim * 20 + 9), (7, 3)):
            buf = torch.full((count + 2 * pad + 1,), 3.0, dtype=TYPES[kind], device="cuda")
            grad = buf[pad + 1:pad + 1 + count]
            ids, dy = inputs(n, vocab, dim, "bf16", 3, "any")
            size = Z.zero_embedding_workspace_bytes(n, vocab, dim)
            ws = torch.full((size + 8192,), 0x55, dtype=torch.uint8, device="cuda")
            keep = dy.clone()
            for overwrite in (True, False):
                Z.zero_embedding_grad(grad, ids, dy, vocab, dim, ws[4096:4096 + size], begin=begin,
                                      overwrite=overwrite)
            assert bool((buf[:pad + 1] == 3.0).all()) and bool((buf[pad + 1 + count:] == 3.0).all())
            assert bool((ws[:4096] == 0x55).all()) and bool((ws[4096 + size:] == 0x55).all())
            assert torch.equal(dy, keep)
            # lookup into rows of a wider buffer
            wide = torch.full((n, dim + 9), 3.0, dtype=TYPES[kind], device="cuda")
            Z.zero_embedding_lookup(wide[:, 4:4 + dim], ids, grad, vocab, dim, begin=begin)
            assert bool((wide[:, :4] == 3.0).all()) and bool((wide[:, 4 + dim:] == 3.0).all())


def test_slices_lie_side_by_side():
    """Owners' lookups add up to the whole one, their gradients are its pieces."""
    vocab, dim, n = 101, 37, 333
    ids, dy = inputs(n, vocab, dim, "fp32", 9)
    w = torch.randn(vocab * dim, generator=torch.Generator().manual_seed(5)).cuda()
    whole, total = torch.empty(n, dim, device="cuda"), torch.zeros(n, dim, device="cuda")
    Z.zero_embedding_lookup(whole, ids, w, vocab, dim, scale=0.5)
    grad = torch.zeros(vocab * dim, device="cuda")
    ws = workspace(n, vocab, dim)
    Z.zero_embedding_grad(grad, ids, dy, vocab, dim, ws, overwrite=True)
    size = -(-vocab * dim // 8)
    for k in range(8):
        a, b = k * size, min((k + 1) * size, vocab * dim)
        part = torch.empty(n, dim, device="cuda")
        Z.zero_embedding_lookup(part, ids, w[a:b], vocab, dim, begin=a, scale=0.5)
        total += part
        piece = torch.full((b - a,), 9.0, device="cuda")
        Z.zero_embedding_grad(piece, ids, dy, vocab, dim, ws, begin=a, overwrite=True)
        want, bound = grad_ref(ids, dy, vocab, dim, a, piece, 1.0, True, None)
        check_grad(piece, "fp32", want, bound)
    assert torch.equal(whole, total)


def test_no_tokens():
    vocab, dim = 30, 20
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    dy = torch.empty(0, dim, device="cuda")
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    grad = torch.ones(vocab, dim, device="cuda")
    Z.zero_embedding_grad(grad, ids, dy, vocab, dim, none)
    assert bool((grad == 1).all())
    Z.zero_embedding_grad(grad, ids, dy, vocab, dim, none, overwrite=True)
    assert not bool(grad.any())
    Z.zero_embedding_lookup(torch.empty(0, dim, device="cuda"), ids, grad, vocab, dim)
    # all of them of no row
    ids = torch.full((9000,), -100, device="cuda")
    grad.fill_(2.0)
    Z.zero_embedding_grad(grad, ids, torch.ones(9000, dim, device="cuda"), vocab, dim, workspace(9000, vocab, dim))
    assert bool((grad == 2).all())


def test_graph_and_streams():
    vocab, dim = 300, 100
    for n in (500, 20000):
        ids, dy = inputs(n, vocab, dim, "bf16", 1)
        w = torch.randn(vocab, dim, generator=torch.Generator().manual_seed(5)).cuda()
        out, grad = torch.empty(n, dim, device="cuda"), torch.zeros(vocab, dim, device="cuda")
        ws = workspace(n, vocab, dim)

        def run():
            Z.zero_embedding_lookup(out, ids, w, vocab, dim)
            Z.zero_embedding_grad(grad, ids, dy, vocab, dim, ws)

        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        side = torch.cuda.Stream()
        for k in range(4):
            new_ids, new_dy = inputs(n, vocab, dim, "bf16", 2 + k, "any")
            ids.copy_(new_ids)
            dy.copy_(new_dy)
            grad.zero_()
            graph.replay()
            got = (out.clone(), grad.clone())
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                grad.zero_()
                run()
            side.synchronize()
            assert torch.equal(got[0], out) and torch.equal(got[1], grad), (n, k)


def test_offsets_past_32_bits():
    """A table and rows of dy beyond 2^31 elements."""
    vocab, dim, n = 70000, 32768, 9
    w = torch.zeros(vocab * dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, vocab - 1, 65536, vocab - 1, 65535, -1, vocab, 3, 69999], device="cuda")
    for r in (0, 3, 65535, 65536, vocab - 1):
        w[r * dim:(r + 1) * dim] = float(r % 251 + 1)
    out = torch.empty(n, dim, device="cuda")
    Z.zero_embedding_lookup(out, ids, w, vocab, dim)
    want = torch.tensor([r % 251 + 1 if 0 <= r < vocab else 0 for r in ids.tolist()], dtype=torch.float32)
    assert torch.equal(out.cpu(), want[:, None].expand(n, dim))
    dy = torch.ones(n, dim, dtype=torch.bfloat16, device="cuda")
    Z.zero_embedding_grad(w, ids, dy, vocab, dim, workspace(n, vocab, dim), overwrite=True)
    sums = w.view(vocab, dim).float()[[0, 3, 65535, 65536, vocab - 1, 1, 69998]]
    assert torch.equal(sums[:, 0].cpu(), torch.tensor([1.0, 1, 1, 1, 3, 0, 0]))
    assert bool((sums == sums[:, :1]).all())
    assert int((w != 0).sum()) == 5 * dim


def test_python_refusals():
    vocab, dim, n = 10, 16, 6
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    out, w = torch.zeros(n, dim, device="cuda"), torch.zeros(vocab, dim, device="cuda")
    ws = workspace(n, vocab, dim)
    ok = (out, ids, w, vocab, dim)
    Z.zero_embedding_lookup(*ok)
    for k, bad in ((0, out[:5]), (0, out.t()), (0, out.cpu()), (1, ids.cpu()), (1, ids[::2].repeat(1)[::2]),
                   (2, w.t()), (2, w.cpu())):
        args = list(ok)
        args[k] = bad
        with pytest.raises(ValueError):
            Z.zero_embedding_lookup(*args)
    for k, bad in ((0, out.double()), (1, ids.float()), (2, w.double())):
        args = list(ok)
        args[k] = bad
        with pytest.raises(TypeError):
            Z.zero_embedding_lookup(*args)
    with pytest.raises(Z.ZeroError):
        Z.zero_embedding_lookup(*ok, begin=1)
    with pytest.raises(Z.ZeroError):
        Z.zero_embedding_grad(w, ids, out, vocab, dim, ws[:256])
    with pytest.raises(ValueError):
        Z.zero_embedding_grad(w, ids, out, vocab, dim, ws.cpu())
    with pytest.raises(ValueError):
        Z.zero_embedding_grad(w, ids, out[:, :8], vocab, dim, ws)

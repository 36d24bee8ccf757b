"""The owner-shard step with Muon matrices, and a training step in which embedding rows,
accumulation, the shard step and Muon follow each other."""
import math

import numpy as np
import pytest
import torch

import zero_partitioned_mixed_shard_amd as Z
from zero_partitioned_mixed_shard_amd.shard import ShardStep

pytestmark = pytest.mark.gpu

# a group of whole tensors: matrices, vectors, a table
TENSORS = [(96, 160), (160,), (160, 96), (33,), (70, 70), (500, 48), (300, 64), (7,)]
MATRICES = (0, 2, 4, 6)
OFFS = np.concatenate([[0], np.cumsum([math.prod(s) for s in TENSORS])])
TOTAL = int(OFFS[-1])


def ranks(n, seed, scale=1.0, dtype=torch.float16):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(TOTAL, generator=gen) * 0.01 * scale).to(dtype).cuda() for _ in range(n)]


def matrices():
    return [(int(OFFS[k]), *TENSORS[k]) for k in MATRICES]


def inside():
    m = torch.zeros(TOTAL, dtype=torch.bool)
    for o, r, c in matrices():
        m[o:o + r * c] = True
    return m


@pytest.mark.parametrize("device_control", [False, True])
@pytest.mark.parametrize("owners", [1, 3])
def test_shard_step_with_matrices(device_control, owners):
    cuts = [0, TOTAL] if owners == 1 else [0, int(OFFS[3]), int(OFFS[5]), TOTAL]
    spans = list(zip(cuts[:-1], cuts[1:]))
    kw = dict(lr=1e-3, max_grad_norm=1.0, scale0=4.0, device_control=device_control)
    both = ShardStep(0, TOTAL, spans, Z.ZERO_FP16, matrices=matrices(), **kw)
    plain = ShardStep(0, TOTAL, spans, Z.ZERO_FP16, **kw)
    start = (torch.randn(TOTAL, generator=torch.Generator().manual_seed(2)) * 0.02).half().cuda()
    for st in (both, plain):
        st.load_param16(start)
    master, momentum, p16 = both.master.clone(), both.exp_avg.clone(), both.param16.clone()
    plan = Z.zero_muon_plan(matrices())
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    hp = Z.zero_muon_hparams(lr=1e-3, weight_decay=0.01, max_grad_norm=1.0)
    mine = inside().cuda()
    for s in range(4):
        bufs = ranks(2, 10 + s, scale=both.scale)
        if s == 2:
            bufs[0][int(OFFS[4]) + 5] = float("inf")         # in a matrix: the whole step is skipped
        infos = [st.step(bufs) for st in (both, plain)]
        assert infos[0].overflow == infos[1].overflow == int(s == 2)
        # the rest is AdamW's, bit for bit; the matrices are one call's
        Z.zero_muon_step(master, momentum, p16, both.reduced(bufs), plan, hp, both.res, ws)
        for x, y, z in ((both.master, plain.master, master), (both.exp_avg, plain.exp_avg, momentum),
                        (both.param16, plain.param16, p16)):
            assert torch.equal(x[~mine], y[~mine])
            assert torch.equal(x[mine], z[mine])
        assert not torch.equal(both.master[mine], plain.master[mine])
        assert not bool(both.exp_avg_sq[mine].any())


def test_captured_shard_step_with_matrices():
    st = ShardStep(0, TOTAL, [(0, TOTAL)], Z.ZERO_BF16, matrices=matrices(), device_control=True, own_ranks=True,
                   world=2)
    eager = ShardStep(0, TOTAL, [(0, TOTAL)], Z.ZERO_BF16, matrices=matrices(), device_control=True, own_ranks=True,
                      world=2)
    start = (torch.randn(TOTAL, generator=torch.Generator().manual_seed(2)) * 0.02).bfloat16().cuda()
    for s in (st, eager):
        s.load_param16(start)
        for r, buf in enumerate(s.rank_bufs):
            buf.copy_(ranks(2, 3, dtype=torch.bfloat16)[r])
    graph = st.capture()
    for k in range(4):
        for s in (st, eager):
            for r, buf in enumerate(s.rank_bufs):
                buf.copy_(ranks(2, 20 + k, dtype=torch.bfloat16)[r])
        graph.replay()
        torch.cuda.synchronize()
        eager.step()
        for x, y in ((st.master, eager.master), (st.exp_avg, eager.exp_avg), (st.param16, eager.param16)):
            assert torch.equal(x, y), k


def test_matrices_have_to_be_whole():
    with pytest.raises(ValueError, match="whole"):
        ShardStep(0, 100, [(0, 50), (50, 100)], Z.ZERO_FP16, matrices=[(40, 4, 5)])
    with pytest.raises(ValueError):
        ShardStep(0, 100, [(0, 100)], Z.ZERO_FP16, matrices=[(90, 4, 5)])
    with pytest.raises(ValueError):
        ShardStep(0, 100, [(0, 100)], Z.ZERO_FP16, matrices=[(0, 4, 5), (10, 4, 5)])
    with pytest.raises(ValueError):
        ShardStep(0, 100, [(0, 40), (60, 100)], Z.ZERO_FP16, matrices=[(44, 2, 5)])


def test_a_training_step():
    """Lookup from the 16-bit copy, a linear layer, its gradients and the table's by tokens into
    accumulators over two micro-batches, the cast into the bucket, reduce and check, Muon on the
    layer's matrix and AdamW on the table and the bias: against the same step in 64 bits."""
    vocab, dim, out_dim, n = 50, 64, 96, 200
    sizes = [vocab * dim, out_dim * dim, out_dim]
    offs = [0, sizes[0], sizes[0] + sizes[1]]
    total = sum(sizes)
    gen = torch.Generator().manual_seed(4)
    step = ShardStep(0, total, [(0, total)], Z.ZERO_BF16, lr=1e-3, matrices=[(offs[1], out_dim, dim)])
    step.load_param16((torch.randn(total, generator=gen) * 0.05).bfloat16().cuda())
    p0 = step.master.double().cpu()
    acc = [torch.empty(s, device="cuda") for s in sizes]
    bucket = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    ids_all = [torch.randint(0, vocab, (n,), generator=gen) for _ in range(2)]
    dy_all = [torch.randn(n, out_dim, generator=gen) * 1e-2 for _ in range(2)]
    ws = torch.empty(Z.zero_embedding_workspace_bytes(n, vocab, dim), dtype=torch.uint8, device="cuda")
    want = [torch.zeros(s, dtype=torch.float64) for s in sizes]
    table, weight = step.param16[:offs[1]], step.param16[offs[1]:offs[2]].view(out_dim, dim)
    t64, w64 = table.double().cpu().view(vocab, dim), weight.double().cpu()
    for k in range(2):
        ids, dy = ids_all[k].cuda(), dy_all[k].cuda()
        h = torch.empty(n, dim, device="cuda")
        Z.zero_embedding_lookup(h, ids, table, vocab, dim, scale=8.0)
        assert torch.equal(h.double().cpu(), t64[ids_all[k]] * 8.0)
        grads = [dy.t().contiguous().mm(h).reshape(-1), dy.sum(0)]
        dh = dy.mm(weight.float())
        Z.zero_embedding_grad(acc[0], ids, dh, vocab, dim, ws, scale=8.0, overwrite=k == 0)
        add = Z.zero_tensor_plan(grads, out=acc[1:])
        Z.zero_tensor_accumulate(add, overwrite=k == 0)
        h64, dy64 = t64[ids_all[k]] * 8.0, dy_all[k].double()
        want[0] += torch.zeros(vocab, dim, dtype=torch.float64).index_add_(0, ids_all[k], dy64 @ w64 * 8.0).reshape(-1)
        want[1] += (dy64.t() @ h64).reshape(-1)
        want[2] += dy64.sum(0)
    pieces = [bucket[o:o + s] for o, s in zip(offs, sizes)]
    cast = Z.zero_tensor_plan(acc, out=pieces)
    one = torch.zeros(4, dtype=torch.int32, device="cuda")
    one.view(torch.float32)[3] = 1.0
    Z.zero_tensor_clip(cast, 0.0, one)
    # sums of at most 400 terms in fp32, then one rounding to bf16
    for x, y in zip(pieces, want):
        size = float(y.abs().max())
        assert bool(((x.double().cpu() - y).abs() <= 2.0 ** -8 * y.abs() + 2000 * 2.0 ** -24 * size).all())
    info = step.step([bucket])
    assert info.applied
    g = bucket.double().cpu()
    # AdamW's first step: p (1 - lr wd) - lr g / (|g| + eps); Muon's from its own formula
    adam = p0 * (1 - 1e-3 * 0.01) - 1e-3 * g / (g.abs() + 1e-8)
    rest = torch.ones(total, dtype=torch.bool)
    rest[offs[1]:offs[2]] = False
    got = step.master.double().cpu()
    assert bool(((got - adam).abs()[rest] <= 2e-6 * adam.abs()[rest] + 1e-8).all())
    u = (g + 0.95 * g)[offs[1]:offs[2]].view(out_dim, dim)
    x = u.t() / (u.norm() + 1e-7)
    for _ in range(5):
        s = x @ x.t()
        x = 3.4445 * x + (-4.775 * s + 2.0315 * s @ s) @ x
    muon = p0[offs[1]:offs[2]] * (1 - 1e-3 * 0.01) - 1e-3 * 0.2 * math.sqrt(out_dim) * x.t().reshape(-1)
    # the shorter side is 64: all in 32 bits or more
    assert float((got[offs[1]:offs[2]] - muon).norm()) <= 1e-6 * float(muon.norm())

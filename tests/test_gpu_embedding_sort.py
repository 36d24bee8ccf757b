"""The embedding gradient's sorts on both sides of their rules: up to 64 blocks of 2048 tokens add
up the counts by themselves, more by a scan in rounds of 4096 counts; keys of one to four passes in
one block and in many.

Tolerances are those of the sums: k rows are k additions in fp32, each off by half a step
(2^-24) of the magnitudes' sum, then one product and sum.
"""
import pytest
import torch

import zero_partitioned_mixed_shard_amd as Z

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def ids_of(n, vocab, spread, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if spread == "even":
        return torch.randint(-1, vocab + 1, (n,), device="cuda", generator=gen)      # some of no row
    u = torch.rand(n, device="cuda", dtype=torch.float64, generator=gen)
    return ((torch.exp(u * torch.tensor(vocab + 1.0, dtype=torch.float64).log().item()) - 1).long()).clamp(0, vocab - 1)


def check(n, vocab, dim, spread, overwrite, padding=None, begin=0, count=None):
    count = vocab * dim - begin if count is None else count
    ids = ids_of(n, vocab, spread, n + vocab)
    dy = torch.randn(n, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).bfloat16()
    grad = torch.randn(count, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    old = grad.clone()
    ws = torch.full((Z.zero_embedding_workspace_bytes(n, vocab, dim),), 0xFF, dtype=torch.uint8, device="cuda")
    Z.zero_embedding_grad(grad, ids, dy, vocab, dim, ws, begin=begin, scale=0.5, overwrite=overwrite, padding_id=padding)
    ok = (ids >= 0) & (ids < vocab)
    if padding is not None:
        ok &= ids != padding
    total, size = (torch.zeros(vocab, dim, dtype=torch.float64, device="cuda") for _ in range(2))
    total.index_add_(0, ids[ok], dy[ok].double())
    size.index_add_(0, ids[ok], dy[ok].double().abs())
    times = torch.zeros(vocab, dtype=torch.float64, device="cuda")
    times.index_add_(0, ids[ok], torch.ones(int(ok.sum()), dtype=torch.float64, device="cuda"))
    part = slice(begin, begin + count)
    want = 0.5 * total.reshape(-1)[part]
    bound = 0.5 * U32 * (size * times[:, None]).reshape(-1)[part]
    if not overwrite:
        want = want + old.double()
    bound = bound + 2 * U32 * (want.abs() + bound)
    off = (grad.double() - want).abs()
    assert bool((off <= bound).all()), float((off - bound).max())
    rest = (times == 0)[:, None].expand(vocab, dim).reshape(-1)[part]
    assert torch.equal(grad[rest], torch.zeros_like(old[rest]) if overwrite else old[rest])
    again = old.clone()
    Z.zero_embedding_grad(again, ids, dy, vocab, dim, ws, begin=begin, scale=0.5, overwrite=overwrite,
                          padding_id=padding)
    assert torch.equal(again, grad)


# 64 blocks, one token more, several rounds of the scan, and a block that is not full
@pytest.mark.parametrize("n", [131072, 131073, 300001, 1048577])
@pytest.mark.parametrize("vocab,dim", [(400, 8), (200000, 4), (300000, 5)])
@pytest.mark.parametrize("overwrite", [False, True])
def test_many_tokens(n, vocab, dim, overwrite):
    check(n, vocab, dim, "zipf", overwrite)


def test_many_tokens_of_a_slice():
    vocab, dim = 150001, 7
    check(200003, vocab, dim, "even", True, padding=17, begin=30 * dim + 3, count=70000 * dim + 1)
    check(200003, vocab, dim, "even", False, padding=17, begin=30 * dim + 3, count=70000 * dim + 1)


# one block: a pass is at most 9 bits, so 511, 2^18 - 1 and 2^27 - 1 ids and one more (dim 1)
@pytest.mark.parametrize("vocab", [511, 512, 262143, 262144, 1000003, 134217727, 134217728])
@pytest.mark.parametrize("n", [1, 700, 8192])
def test_passes_of_one_block(vocab, n):
    check(n, vocab, 1, "even", False)


@pytest.mark.parametrize("vocab", [262143, 262144, 134217728])
def test_passes_of_many_blocks(vocab):
    check(8193, vocab, 1, "zipf", False)
    check(140000, vocab, 1, "even", True)


def test_all_tokens_are_one_id():
    vocab, dim, n = 200000, 4, 140001
    ids = torch.full((n,), 199999, device="cuda")
    dy = torch.ones(n, dim, device="cuda", dtype=torch.float16)
    grad = torch.zeros(vocab, dim, device="cuda")
    ws = torch.empty(Z.zero_embedding_workspace_bytes(n, vocab, dim), dtype=torch.uint8, device="cuda")
    Z.zero_embedding_grad(grad, ids, dy, vocab, dim, ws)
    assert bool((grad[-1] == n).all()) and not bool(grad[:-1].any())       # sums of ones below 2^24 are exact

"""Cases of the operators over whole matrices and over rows of the vocabulary table: orthogonalisation,
the Muon step of an owner's matrices, embedding lookup, and the embedding's gradient.

  orth      O = X_steps for every matrix G of a list, by Newton-Schulz products on its wide form:
            X_0 = G / (||G||_F + eps);  A = X X^T,  X <- a X + (b A + c A^2) X.
  muon      the owner's step over the matrices of its flat shard: g = grad * inv * clip,
            M = mu M + g,  U = g + mu M,  p = p (1 - lr wd) - lr alpha orth(U) with
            alpha = 0.2 sqrt(max(rows, cols)), and the 16-bit copy of p.
  lookup    y[t] = scale * W[id_t], W the vocabulary table or an owner's slice of it: elements
            [begin, begin + count) of the flat table (a partition cuts through rows); what lies
            outside gives 0, so that the owners' results add up.
  grad      dW[v] = (dW[v] +) scale * sum of dy[t] over the tokens t with id_t = v, for the same slice;
            ids outside the vocabulary, and the padding id, give nothing.
"""
import math
import random
import struct

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
_A, _B, _C, _EPS, _STEPS = 3.4445, -4.7750, 2.0315, 1e-7, 5
_MU, _WD = 0.95, 0.1


def listed():
    """The listed cases; each comment says what it stands for."""
    return [
        # a low-rank adapter's 56 pairs of factors: little work, latency counts
        _orth("orth_adapters", "bf16", "bf16", kind="adapter", count=56, rows=16, cols=2048),
        # 24 matrices of odd sizes, as rows of wider buffers, wide and tall
        _orth("orth_odd", "fp16", "fp16", kind="ragged", count=24, rows=1, cols=1500, extra=5),
        # two 32-bit updates, orthogonalised to 32 bits
        _orth("orth_fp32", "fp32", "fp32", kind="same", count=2, rows=2048, cols=5504, extra=0),
        # one owner's matrices, of 8 owners, of 12 layers of width 1024 whose feed-forward is 4 times as wide
        _muon("muon_encoder", "fp16", kind="encoder", count=1, rows=1024, cols=4, inv=2.0 ** -12),
        # four layers of a billion-parameter decoder
        _muon("muon_decoder_1b", "bf16", kind="decoder", count=4, rows=2048, cols=5504),
        # one layer of a 7e9-parameter decoder
        _muon("muon_decoder_7b", "bf16", kind="decoder", count=1, rows=4096, cols=11008),
        # one matrix of a 70e9-parameter decoder's layer, the largest
        _muon("muon_decoder_70b", "bf16", kind="same", count=1, rows=28672, cols=8192),
        # the tokens of one decoding step of eight sequences: the smallest call
        _rows("lookup_decode", "lookup", 8, 32000, 4096, "bf16", "bf16"),
        # a micro-batch of 4 sequences of 4096 tokens, scaled by sqrt(width), into 32 bits
        _rows("lookup_batch", "lookup", 16384, 32000, 4096, "bf16", "fp32", scale=64.0),
        # the same micro-batch's gradient into the 32-bit accumulators
        _rows("grad_batch", "grad", 16384, 32000, 4096, "bf16", "fp32", scale=0.25),
        # a padded batch's gradient over a small encoder's whole table, in 16 bits
        _rows("grad_encoder", "grad", 32768, 30522, 768, "fp16", "fp16", overwrite=True,
              padding=0.4),
        # an owner's slice of a large vocabulary, whose ends cut through rows
        _rows("grad_slice", "grad", 65537, 128003, 4095, "bf16", "bf16", overwrite=True,
              part=8, of=3),
    ]


def _f32(x):
    """The value as the calls take it, in 32 bits."""
    return struct.unpack("f", struct.pack("f", x))[0]


def _orth(name, src, dst, **more):
    c = {"name": name, "op": "orth", "src": src, "dst": dst, "kind": "same", "count": 1, "rows": 1,
         "cols": 1, "extra": 0}
    c.update(more)
    return c


def _muon(name, dtype, **more):
    c = {"name": name, "op": "muon", "dtype": dtype, "kind": "same", "count": 1, "rows": 1,
         "cols": 1, "inv": 1.0, "lr": _f32(1e-4), "max_norm": 1.0}
    c.update(more)
    return c


def _rows(name, op, tokens, vocab, dim, src, dst, **more):
    """src, dst: of lookups the table's and the result's type, of gradients dy's and the table's."""
    c = {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "src": src,
         "dst": dst, "scale": 1.0, "overwrite": False, "padding": 0.0, "part": 1, "of": 0}
    c.update(more)
    return c


def draw(rng):
    """One more case: matrices of 1 to 4096 on the shorter side, 1 to 2^17 tokens."""
    def spread(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))

    op = rng.choice(["orth", "muon", "muon", "lookup", "grad", "grad"])
    if op in ("orth", "muon"):
        kind = rng.choice(["same", "same", "ragged", "adapter"] if op == "orth" else
                          ["same", "decoder", "encoder"])
        m = spread(4, 64) if kind == "adapter" else spread(96, 2500) if kind == "ragged" else \
            spread(64, 1024) if kind == "encoder" else spread(200, 4096)
        n = min(16384, int(m * rng.uniform(1, 4))) if kind != "adapter" else spread(512, 8192)
        flops = _STEPS * (3.0 * m * m * n + m ** 3) * (1 if kind != "ragged" else 0.1)
        count = max(1, min(64, int(rng.uniform(0.1, 1.0) * 4e12 / flops)))
        if kind == "decoder":
            count = max(1, count // 6)
        if kind == "encoder":
            count, n = 1, rng.choice([2, 3, 4, 6])
        if kind == "same" and rng.random() < 0.5:
            m, n = n, m
        if op == "muon":
            t = rng.choice(["bf16", "bf16", "fp16"])
            c = _muon("", t, kind=kind, count=count, rows=m, cols=n,
                      inv=2.0 ** -rng.randint(4, 14) if t == "fp16" else 1.0,
                      max_norm=rng.choice([0.0, 1.0]), lr=_f32(10 ** rng.uniform(-5, -4)))
        else:
            dst = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            c = _orth("", rng.choice(["bf16", "fp16", "fp32"]), dst, kind=kind, rows=m, cols=n,
                      count=count if dst != "fp32" else max(1, count // 3),
                      extra=rng.choice([0, 0, 8, rng.randint(1, 70)]))
    else:
        vocab, dim = spread(1000, 200000), spread(64, 8192)
        if rng.random() < 0.7:
            dim = -(-dim // 64) * 64
        tokens = spread(1, min(1 << 17, (1 << 28) // dim))
        part = rng.choice([1, 1, 2, 8]) if vocab * dim < 1 << 29 else 8
        src, dst = rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice(["bf16", "fp16", "fp32", "fp32"])
        overwrite = op == "grad" and (dst == "fp16" or rng.random() < 0.5)
        c = _rows("", op, tokens, vocab, dim, src, dst, scale=_f32(rng.choice([1.0, 0.25, math.sqrt(dim)])),
                  overwrite=overwrite, padding=rng.choice([0.0, 0.0, 0.3]), part=part,
                  of=rng.randrange(part))
    del c["name"]
    return c


# -------------------------------------------------------------- geometry --
def _shapes(case):
    """(rows, cols) of every matrix."""
    r, c, n = case["rows"], case["cols"], case["count"]
    if case["kind"] == "adapter":
        return [(r, c) if k % 2 == 0 else (c, r) for k in range(n)]
    if case["kind"] == "ragged":
        rng = random.Random(n * 7919 + r * 31 + c)
        return [(rng.randint(max(1, r // 8), max(r, c)), rng.randint(max(1, r // 8), max(r, c)))
                for _ in range(n)]
    if case["kind"] == "decoder":
        return [(r, r), (r, r), (r, r), (r, r), (c, r), (c, r), (r, c)] * n
    if case["kind"] == "encoder":           # whole tensors 0, 8, 16, ... of 12 layers
        layer = [(r, r), (r, r), (r, r), (r, r), (c * r, r), (r, c * r)]
        return (layer * 12)[::8]
    return [(r, c)] * n


def _slice(case):
    """First element and elements of the part of the flat table that the case has."""
    total = case["vocab"] * case["dim"]
    size = -(-total // case["part"])
    begin = size * case["of"]
    return begin, min(size, total - begin)


def _fro(r, c):
    """Operations of the products of one matrix: A and A^2 are symmetric and count half."""
    m, n = min(r, c), max(r, c)
    return _STEPS * (3.0 * m * m * n + 1.0 * m ** 3)


def work(case):
    if case["op"] in ("orth", "muon"):
        shapes = _shapes(case)
        e = sum(r * c for r, c in shapes)
        b = _SIZE[case["src"]] + _SIZE[case["dst"]] if case["op"] == "orth" else 20
        return {"bytes": e * b, "flops": sum(_fro(r, c) for r, c in shapes)}
    t, d = case["tokens"], case["dim"]
    # tokens are spread evenly over the vocabulary's logarithm: the rows that some token has
    distinct = sum(1.0 - (1.0 - math.log1p(1.0 / v) / math.log(case["vocab"])) ** t
                   for v in range(1, min(case["vocab"], 4096)))
    if case["vocab"] > 4096:
        steps = 200
        span = math.log(case["vocab"] / 4096.0) / steps
        for k in range(steps):
            v = 4096.0 * math.exp((k + 0.5) * span)
            distinct += v * span * (1.0 - (1.0 - math.log1p(1.0 / v) / math.log(case["vocab"])) ** t)
    share = _slice(case)[1] / (case["vocab"] * d)
    read, rows = t * d * share, min(distinct, case["vocab"]) * d * share
    s, o = _SIZE[case["src"]], _SIZE[case["dst"]]
    if case["op"] == "lookup":
        return {"bytes": 8 * t + rows * s + t * d * o, "flops": t * d}
    read *= 1.0 - case["padding"]
    write = _slice(case)[1] * o if case["overwrite"] else 2 * rows * o
    return {"bytes": 8 * t + read * s + write, "flops": 2 * read}


# ---------------------------------------------------------------- inputs --
def _update(r, c, gen):
    """A gradient's values: a part of low rank and noise, entries about 1."""
    k = max(1, min(r, c) // 16)
    x = torch.randn(r, k, device="cuda", generator=gen) @ torch.randn(k, c, device="cuda", generator=gen)
    return x.mul_(k ** -0.5).add_(torch.randn(r, c, device="cuda", generator=gen), alpha=0.5)


def _prepare_orth(case, gen, st):
    src, dst = [], []
    shapes, extra = _shapes(case), case["extra"]
    x = torch.zeros(sum(r * (c + extra) for r, c in shapes), dtype=_TYPES[case["src"]], device="cuda")
    y = torch.zeros(sum(r * c for r, c in shapes), dtype=_TYPES[case["dst"]], device="cuda")
    at = to = 0
    for r, c in shapes:
        src.append(x[at:at + r * (c + extra)].view(r, c + extra)[:, :c])
        dst.append(y[to:to + r * c].view(r, c))
        src[-1].copy_(_update(r, c, gen).mul_(0.01))
        at, to = at + r * (c + extra), to + r * c
    st.update(src=src, dst=dst, out=y)
    if own:
        Z = st["Z"]
        st["plan"] = Z.zero_matrix_plan(src, out=dst)
        st["ws"] = torch.empty(Z.zero_matrix_workspace_bytes(st["plan"]), dtype=torch.uint8, device="cuda")


def _prepare_muon(case, gen, st):
    shapes, t = _shapes(case), _TYPES[case["dtype"]]
    total = sum(r * c for r, c in shapes)
    st["grad"] = torch.empty(total, dtype=t, device="cuda")
    st["momentum"] = torch.empty(total, device="cuda")
    st["master"] = torch.empty(total, device="cuda").normal_(0.0, 0.02, generator=gen)
    at, st["matrices"] = 0, []
    for r, c in shapes:
        st["matrices"].append((at, r, c))
        g = _update(r, c, gen).mul_(1e-3)
        st["grad"][at:at + r * c] = (g / case["inv"]).reshape(-1).to(t)
        # the momentum of earlier steps: partly the same directions
        st["momentum"][at:at + r * c] = g.mul_(6.0).add_(_update(r, c, gen), alpha=4e-3).reshape(-1)
        at += r * c
    st["param16"] = st["master"].to(t)
    # the norm over all owners: the check's result, which the step is given
    sumsq = 3.0 * float((st["grad"].float() * case["inv"]).square().sum(dtype=torch.float64))
    st["coef"] = min(1.0, case["max_norm"] / (math.sqrt(sumsq) + 1e-6)) if case["max_norm"] > 0 else 1.0
    st["res"] = torch.frombuffer(bytearray(struct.pack("<dIf", sumsq, 0, case["inv"])),
                                 dtype=torch.int32).cuda()
    if own:
        Z = st["Z"]
        st["plan"] = Z.zero_muon_plan(st["matrices"])
        st["ws"] = torch.empty(Z.zero_matrix_workspace_bytes(st["plan"]), dtype=torch.uint8, device="cuda")
        st["hp"] = Z.zero_muon_hparams(lr=case["lr"], momentum=_MU, weight_decay=_WD,
                                       max_grad_norm=case["max_norm"])


def _prepare_rows(case, gen, st):
    t, v, d = case["tokens"], case["vocab"], case["dim"]
    begin, count = _slice(case)
    st.update(begin=begin, size=count)
    # the k-th most frequent token is about k times rarer than the first
    u = torch.rand(t, device="cuda", dtype=torch.float64, generator=gen)
    ids = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1)
    st["pad"] = None
    if case["padding"]:
        st["pad"] = v // 3
        ids[torch.rand(t, device="cuda", generator=gen) < case["padding"]] = st["pad"]
    st["ids"] = ids
    if case["op"] == "lookup":
        st["table"] = torch.empty(count, dtype=_TYPES[case["src"]], device="cuda").normal_(0.0, 0.02, generator=gen)
        st["out"] = torch.zeros(t, d, dtype=_TYPES[case["dst"]], device="cuda")
    else:
        st["dy"] = torch.empty(t, d, dtype=_TYPES[case["src"]], device="cuda").normal_(0.0, 1e-2, generator=gen)
        st["grad"] = torch.empty(count, dtype=_TYPES[case["dst"]], device="cuda").normal_(0.0, 1e-2, generator=gen)
        if own:
            st["ws"] = torch.empty(st["Z"].zero_embedding_workspace_bytes(t, v, d), dtype=torch.uint8,
                                   device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case)
    if own:
        import zero_partitioned_mixed_shard_amd as Z
        st["Z"] = Z
    {"orth": _prepare_orth, "muon": _prepare_muon}.get(case["op"], _prepare_rows)(case, gen, st)
    return st


# ----------------------------------------------------------- plain forms --
def _by_shape(shapes):
    found = {}
    for k, s in enumerate(shapes):
        found.setdefault(s, []).append(k)
    return found


def _orthogonal(x):
    """Newton-Schulz on a batch of matrices of one shape."""
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (torch.sqrt(torch.sum(x * x, dim=(1, 2), keepdim=True)) + _EPS)
    for _ in range(_STEPS):
        a = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = _A * x + torch.matmul(_B * a + _C * torch.matmul(a, a), x)
    return x.transpose(1, 2) if tall else x


def _plain_orth(st):
    for which in _by_shape([tuple(x.shape) for x in st["src"]]).values():
        o = _orthogonal(torch.stack([st["src"][k] for k in which]).float())
        for j, k in enumerate(which):
            st["dst"][k].copy_(o[j])
    return st["out"]


def _plain_muon(st):
    for (r, c), which in _by_shape([m[1:] for m in st["matrices"]]).items():
        spans = [slice(st["matrices"][k][0], st["matrices"][k][0] + r * c) for k in which]
        g = torch.stack([st["grad"][s] for s in spans]).float() * st["inv"] * st["coef"]
        m = torch.stack([st["momentum"][s] for s in spans]) * _MU + g
        o = _orthogonal((g + _MU * m).view(-1, r, c)).reshape(len(which), r * c)
        p = torch.stack([st["master"][s] for s in spans])
        p = p * (1.0 - st["lr"] * _WD) - (st["lr"] * 0.2 * math.sqrt(max(r, c))) * o
        for j, s in enumerate(spans):
            st["momentum"][s] = m[j]
            st["master"][s] = p[j]
            st["param16"][s] = p[j].to(st["param16"].dtype)
    return {"master": st["master"], "momentum": st["momentum"], "param16": st["param16"]}


def _row_range(st):
    """The rows that the slice touches, and where it begins in the first of them."""
    d = st["dim"]
    first = st["begin"] // d
    return first, -(-(st["begin"] + st["size"]) // d), st["begin"] - first * d


def _plain_lookup(st):
    first, last, lead = _row_range(st)
    d, w = st["dim"], st["table"]
    if lead or (last - first) * d != st["size"]:
        w = w.new_zeros((last - first) * d)
        w[lead:lead + st["size"]] = st["table"]
    ids = st["ids"]
    mine = (ids >= first) & (ids < last)
    rows = w.view(-1, d)[torch.where(mine, ids - first, torch.zeros_like(ids))].float() * st["scale"]
    st["out"].copy_(torch.where(mine[:, None], rows, torch.zeros_like(rows)))
    return st["out"]


def _plain_grad(st):
    first, last, lead = _row_range(st)
    d, ids = st["dim"], st["ids"]
    dy = st["dy"]
    if st["pad"] is not None or st["part"] > 1:
        mine = (ids >= first) & (ids < last)
        if st["pad"] is not None:
            mine = mine & (ids != st["pad"])
        ids, dy = ids[mine], dy[mine]
    full = torch.zeros((last - first) * d, device="cuda")
    full.view(-1, d).index_add_(0, ids - first, dy.float())
    full = full[lead:lead + st["size"]] * st["scale"]
    st["grad"].copy_(full if st["overwrite"] else st["grad"].float() + full)
    return st["grad"]


# ------------------------------------------------------- the library's calls --
def _own(st):
    Z, op = st["Z"], st["op"]
    if op == "orth":
        Z.zero_orthogonalize(st["plan"], st["ws"])
        return st["out"]
    if op == "muon":
        Z.zero_muon_step(st["master"], st["momentum"], st["param16"], st["grad"], st["plan"],
                         st["hp"], st["res"], st["ws"])
        return {"master": st["master"], "momentum": st["momentum"], "param16": st["param16"]}
    if op == "lookup":
        Z.zero_embedding_lookup(st["out"], st["ids"], st["table"], st["vocab"], st["dim"],
                                begin=st["begin"], scale=st["scale"])
        return st["out"]
    Z.zero_embedding_grad(st["grad"], st["ids"], st["dy"], st["vocab"], st["dim"], st["ws"],
                          begin=st["begin"], scale=st["scale"], overwrite=st["overwrite"],
                          padding_id=st["pad"])
    return st["grad"]


def run(state):
    if own:
        return _own(state)
    return {"orth": _plain_orth, "muon": _plain_muon, "lookup": _plain_lookup,
            "grad": _plain_grad}[state["op"]](state)


# -------------------------------------------------------------- in 64 bits --
def _exact_orth(g):
    """One matrix: its wide form, and the products fused with their sums."""
    g = g.double()
    wide = g if g.shape[0] <= g.shape[1] else g.t().contiguous()
    x = wide / (torch.linalg.vector_norm(wide) + _EPS)
    for _ in range(_STEPS):
        s = x.mm(x.t().contiguous())
        x = torch.addmm(x, torch.addmm(s, s, s, beta=_B, alpha=_C), x, beta=_A)
    return x if g.shape[0] <= g.shape[1] else x.t()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "orth":
        return torch.cat([_exact_orth(g).reshape(-1) for g in st["src"]])
    if case["op"] == "muon":
        g = st["grad"].double() * (case["inv"] * st["coef"])
        m = st["momentum"].double() * _MU + g
        u, p = g + _MU * m, st["master"].double() * (1.0 - case["lr"] * _WD)
        for at, r, c in st["matrices"]:
            o = _exact_orth(u[at:at + r * c].view(r, c)).reshape(-1)
            p[at:at + r * c] -= case["lr"] * 0.2 * math.sqrt(max(r, c)) * o
        return {"master": p, "momentum": m, "param16": p}
    begin, count = _slice(case)
    d, ids = case["dim"], st["ids"]
    if case["op"] == "lookup":
        # element by element: where in the slice it lies
        y = torch.zeros(case["tokens"], d, dtype=torch.float64, device="cuda")
        for a in range(0, case["tokens"], 4096):
            at = ids[a:a + 4096, None] * d + torch.arange(d, device="cuda") - begin
            ok = (at >= 0) & (at < count)
            y[a:a + 4096] = torch.where(ok, st["table"][at.clamp(0, count - 1)].double() * case["scale"], 0.0)
        return y
    y = torch.zeros(count, dtype=torch.float64, device="cuda") if case["overwrite"] else st["grad"].double()
    for a in range(0, case["tokens"], 4096):
        at = ids[a:a + 4096, None] * d + torch.arange(d, device="cuda") - begin
        ok = (at >= 0) & (at < count) & (ids[a:a + 4096, None] != (-1 if st["pad"] is None else st["pad"]))
        y.index_add_(0, at[ok], st["dy"][a:a + 4096].double()[ok] * case["scale"])
    return y

"""Cases of the operators over tables of gradient tensors: norm, clip, both at once, and accumulation.

A table is a list of tensors of any sizes and a mix of types, as a model's
parameters have gradients.  x is an element of a gradient, E all elements:

  norm        S = sum x^2 over the table (or M = max |x|), the overflow flag
              "some x is inf or NaN", and where asked every tensor's own norm;
              everything is unscaled by `inv`.  sumsq = inv^2 S or (inv M)^2.
  clip        y = x * inv * c with c = max_norm / (norm + 1e-6) where that is
              below 1, else 1; c from the table's norm or from each tensor's
              own; y stays as it was where the flag is set.  y is another
              tensor (of another type, it may be) or x itself.
  clip_norm   a norm, and the clip by it.
  accumulate  y = y + w x (first: y = w x), and where asked the norm of the
              new y.

A case's tensors are pieces of one or two flat buffers, back to back (as
a bucket of contiguous gradients holds them: their starts are then aligned to
nothing but their elements) or each at a multiple of 256 bytes (as separate
allocations lie), so the plain forms run on whole buffers.
"""
import math
import random
import struct

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    """The listed cases; each comment says what it stands for."""
    def ragged(name, op, tensors, lo, hi, src, dst="", **more):
        return _case(name, op, src, dst, tensors=tensors, lo=lo, hi=hi, **more)

    def decoder(name, op, layers, width, ffn, vocab, src, dst="", **more):
        return _case(name, op, src, dst, layers=layers, width=width, ffn=ffn, vocab=vocab, **more)

    return [
        # the norm of a handful of biases and gains: latency alone
        ragged("norm_few_small", "norm", 8, 64, 4096, "fp32", pad=True),
        # the norm of a 7e9-parameter decoder's 16-bit gradients, the largest
        # group that the benchmark's workloads flatten
        decoder("norm_decoder_7b", "norm", 32, 4096, 11008, 32000, "bf16", pad=True),
        # a fragmented bucket of 10,000 loss-scaled gradients, each one's norm
        # reported too
        ragged("norm_each_of_10000", "norm", 10000, 64, 1 << 20, "fp16", per_tensor=True,
               inv=2.0 ** -16),
        # the largest magnitude of a model whose vectors have 32-bit gradients
        decoder("norm_max_mixed", "norm", 16, 2048, 5504, 32000, "mixed", kind="max", pad=True),
        # an in-place clip of a billion-parameter model by a norm that is
        # known (summed over ranks, for instance)
        decoder("clip_in_place", "clip", 16, 2048, 5504, 32000, "bf16", "same", pad=True,
                max_norm=1.0, inv=0.5),
        # accumulated 32-bit gradients into a 16-bit bucket, unscaled and
        # clipped on the way
        ragged("clip_into_bucket", "clip", 997, 1, 1 << 20, "fp32", "bf16", max_norm=1.0,
               inv=1.0 / 12),
        # every tensor clipped by its own norm
        ragged("clip_each", "clip", 3000, 0, 1 << 17, "fp16", "fp32", per_tensor=True,
               max_norm=0.05, inv=2.0 ** -10),
        # norm and clip of an adapter's gradients: a few small matrices
        ragged("clip_norm_adapter", "clip_norm", 28, 4096, 65536, "bf16", "bf16", pad=True,
               max_norm=1.0),
        # norm and clip of the ToyModel's gradients (1e8 parameters), which
        # the last-level cache can hold between the two
        decoder("clip_norm_100m", "clip_norm", 12, 1024, 2816, 32000, "fp32", "fp32", pad=True,
                max_norm=1.0),
        # norm and clip of a billion-parameter model, 16-bit, from loss-scaled
        # gradients into a bucket
        decoder("clip_norm_1b", "clip_norm", 16, 2048, 5504, 32000, "fp16", "fp16",
                max_norm=1.0, inv=2.0 ** -12),
        # a micro-batch's 16-bit gradients into 32-bit accumulators
        decoder("accumulate_1b", "accumulate", 16, 2048, 5504, 32000, "bf16", "fp32", pad=True,
                weight=0.25),
        # the last micro-batch of a fragmented bucket, with the norm of the sum
        ragged("accumulate_norm", "accumulate", 4001, 1, 1 << 18, "fp16", "fp32", weight=1.0,
               inv=2.0 ** -16, with_norm=True),
    ]


def _case(name, op, src, dst, **more):
    c = {"name": name, "op": op, "src": src, "dst": dst, "kind": "l2", "per_tensor": False,
         "pad": False, "inv": 1.0, "max_norm": 0.0, "weight": 1.0, "first": False,
         "with_norm": False, "layers": 0, "width": 0, "ffn": 0, "vocab": 0, "tensors": 0, "lo": 0,
         "hi": 0}
    c.update(more)
    for k in ("inv", "max_norm", "weight"):   # the calls take these in 32 bits
        c[k] = struct.unpack("f", struct.pack("f", c[k]))[0]
    return c


def draw(rng):
    """One more case: 1 to 4096 tensors, 2^10 to 2^28 elements in all."""
    def spread(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))

    op = rng.choice(["norm", "clip", "clip_norm", "accumulate"])
    n = spread(1, 4096)
    mean = max(1.0, spread(1 << 10, 1 << 28) / n)
    src = rng.choice(["fp32", "bf16", "fp16", "mixed"])
    dst = "" if op == "norm" else rng.choice(["fp32", "bf16", "fp16"])
    if op == "clip" and rng.random() < 0.25:
        dst = "same"
    with_norm = op == "accumulate" and rng.random() < 0.5
    c = _case("", op, src, dst, tensors=n, lo=int(mean / rng.uniform(4, 40)),
              hi=max(1, int(mean * rng.uniform(1.1, 2.5))), pad=rng.random() < 0.5,
              kind=rng.choice(["l2", "l2", "max"]),
              per_tensor=(op != "accumulate" or with_norm) and rng.random() < 0.4,
              inv=rng.choice([1.0, 2.0 ** -8, 1.0 / rng.randint(2, 9)]),
              max_norm=0.0 if op in ("norm", "accumulate") else 10.0 ** rng.uniform(-2, 1),
              weight=rng.uniform(0.1, 1.0) if op == "accumulate" else 1.0,
              first=op == "accumulate" and rng.random() < 0.3, with_norm=with_norm)
    del c["name"]
    return c


# ---------------------------------------------------------------- the table --
def _numels(case):
    """Elements of every tensor, in the table's order, and which are vectors."""
    if case["layers"]:
        d, f = case["width"], case["ffn"]
        layer = [d * d, d * d, d * d, d * d, f * d, f * d, f * d, d, d]
        sizes = [case["vocab"] * d] + layer * case["layers"] + [d, case["vocab"] * d]
        return sizes, [s == d for s in sizes]
    rng = random.Random(case["tensors"] * 7919 + case["hi"])
    lo, hi = case["lo"], case["hi"]
    span = math.log((hi + 1) / max(lo, 0.5))
    sizes = [min(hi, int(max(lo, 0.5) * math.exp(rng.random() * span)))
             for _ in range(case["tensors"])]
    return sizes, [k % 3 == 1 for k in range(len(sizes))]


def _src_types(case):
    """The type of every tensor's gradient."""
    sizes, vector = _numels(case)
    if case["src"] != "mixed":
        return sizes, [case["src"]] * len(sizes)
    return sizes, ["fp32" if v else "bf16" for v in vector]


def _total(case):
    """(elements, bytes of the gradients, bytes of the outputs, tensors)."""
    sizes, types = _src_types(case)
    read = sum(s * _SIZE[t] for s, t in zip(sizes, types))
    write = read if case["dst"] == "same" else sum(sizes) * _SIZE.get(case["dst"], 0)
    return sum(sizes), read, write, len(sizes)


def work(case):
    e, read, write, n = _total(case)
    each = 4 * n if case["per_tensor"] else 0
    if case["op"] == "norm":
        return {"bytes": read + 16 + each, "flops": 2 * e}
    if case["op"] == "clip":
        return {"bytes": read + write + 16 + each, "flops": e}
    if case["op"] == "clip_norm":
        return {"bytes": read + write + 16 + each, "flops": 3 * e}
    again = 0 if case["first"] else write
    norm = 2 * e if case["with_norm"] else 0
    return {"bytes": read + write + again + (16 + each if norm else 0), "flops": 2 * e + norm}


def _lay_out(sizes, members, pad):
    """Starts of the member tensors in their flat buffer, and its elements."""
    starts, at = [], 0
    for k in members:
        starts.append(at)
        at += -(-sizes[k] // 128) * 128 if pad else sizes[k]
    return starts, at


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    sizes, types = _src_types(case)
    st = dict(case, parts=[], n=len(sizes))
    src, dst = [None] * len(sizes), [None] * len(sizes)
    for t in sorted(set(types)):
        members = [k for k in range(len(sizes)) if types[k] == t]
        starts, count = _lay_out(sizes, members, case["pad"])
        x = torch.zeros(count, dtype=_TYPES[t], device="cuda")
        y = x if case["dst"] in ("", "same") else torch.zeros(count, dtype=_TYPES[case["dst"]],
                                                               device="cuda")
        for k, at in zip(members, starts):
            # layers' gradients lie some binades apart; unscaled they are
            # about 1e-5 to 1e-2
            sigma = 10.0 ** rng.uniform(-5, -2) / case["inv"]
            src[k] = x[at:at + sizes[k]].normal_(0.0, sigma, generator=gen)
            dst[k] = y[at:at + sizes[k]]
            if case["op"] == "accumulate" and not case["first"]:
                dst[k].normal_(0.0, 2.0 * sigma, generator=gen)
        ends = torch.tensor([a + sizes[k] for k, a in zip(members, starts)], device="cuda")
        st["parts"].append({
            "x": x, "y": y, "which": torch.tensor(members, device="cuda"),
            "starts": torch.tensor(starts, device="cuda"), "ends": ends,
            "lengths": torch.tensor(starts[1:] + [count], device="cuda")
            - torch.tensor(starts, device="cuda")})
    st["res"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    st["norms"] = torch.zeros(len(sizes), dtype=torch.float32, device="cuda")
    if case["op"] == "clip":                # the norms come from an earlier call
        sumsq, norms = _norm(st, [p["x"] for p in st["parts"]])
        st["res"].copy_(torch.frombuffer(bytearray(
            struct.pack("<dIf", float(sumsq), 0, case["inv"])), dtype=torch.int32))
        if case["per_tensor"]:
            st["norms"].copy_(norms)
    st["sumsq"] = st["res"].view(torch.float64)[:1]
    st["overflow"] = st["res"][2:3]
    if own:
        import zero_partitioned_mixed_shard_amd as Z
        st["Z"] = Z
        st["plan"] = Z.zero_tensor_plan(src, out=None if case["dst"] in ("", "same") else dst)
        st["ws"] = torch.empty(-(-Z.zero_tensor_workspace_bytes(st["plan"]) // 8),
                               dtype=torch.float64, device="cuda")
    return st


# ------------------------------------------------------------- plain forms --
def _square_sums(x, part, each):
    """Sum of squares of a buffer (a square of 16-bit values is exact in 32
    bits), or of each of its tensors; the sums are long: 64 bits."""
    if each:
        total = torch.cat([x.new_zeros(1, dtype=torch.float64),
                           torch.cumsum(x.double().square(), 0)])
        return total[part["ends"]] - total[part["starts"]]
    if x.dtype == torch.float32:
        return x.double().square().sum()
    x = x.float()
    return torch.sum(x * x, dtype=torch.float64)


def _maxima(x, part, each):
    x = x.float().abs()
    if not each:
        return x.max().double() if x.numel() else x.new_zeros((), dtype=torch.float64)
    found = x.new_zeros(part["ends"].numel())
    tensor = torch.repeat_interleave(torch.arange(found.numel(), device="cuda"), part["lengths"])
    return found.scatter_reduce(0, tensor, x, "amax").double()


def _norm(st, buffers):
    """The square of the unscaled norm and, where asked, each tensor's norm."""
    each, largest, inv = st["per_tensor"], st["kind"] == "max", st["inv"]
    found = [(_maxima if largest else _square_sums)(x, p, each)
             for x, p in zip(buffers, st["parts"])]
    norms = None
    if each:
        norms = torch.zeros(st["n"], dtype=torch.float32, device="cuda")
        norms[torch.cat([p["which"] for p in st["parts"]])] = \
            (torch.cat(found) * inv if largest else torch.cat(found).clamp(min=0).sqrt() * inv).float()
        found = [f.max() if largest else f.sum() for f in found]
    total = torch.stack(found)
    return ((total.max() * inv).square() if largest else total.sum() * (inv * inv)), norms


def _clip(st, sumsq, norms, overflow):
    def factor(norm):
        c = st["max_norm"] / (norm + 1e-6)
        return (torch.where(c < 1.0, c, torch.ones_like(c)) * st["inv"]).float()

    f = [factor(norms.double())[p["which"]].repeat_interleave(p["lengths"])
         if st["per_tensor"] else factor(sumsq.sqrt()) for p in st["parts"]]
    return [p["y"].copy_(torch.where(overflow != 0, p["y"], (p["x"].float() * g).to(p["y"].dtype)))
            for p, g in zip(st["parts"], f)]


def _accumulate(st):
    w = st["weight"]
    return [p["y"].copy_(p["x"].float() * w if st["first"] else p["y"].float() + p["x"].float() * w)
            for p in st["parts"]]


def _plain(st):
    out = {}
    if st["op"] == "accumulate":
        out["y"] = _accumulate(st)
    if st["op"] in ("norm", "clip_norm") or st["with_norm"]:
        sumsq, norms = _norm(st, out["y"] if "y" in out else [p["x"] for p in st["parts"]])
        out["sumsq"] = sumsq.reshape(1)
        out["overflow"] = (~torch.isfinite(out["sumsq"])).int()
        if st["per_tensor"]:
            out["norms"] = norms
    if st["op"] in ("clip", "clip_norm"):
        out["y"] = _clip(st, out.get("sumsq", st["sumsq"]), out.get("norms", st["norms"]),
                         out.get("overflow", st["overflow"]))
    return out


# ------------------------------------------------------- the library's calls --
def _own(st):
    Z, op, plan = st["Z"], st["op"], st["plan"]
    norms = st["norms"] if st["per_tensor"] else None
    if op == "norm":
        Z.zero_tensor_norm(plan, st["inv"], st["res"], st["ws"], kind=st["kind"], norms=norms)
    elif op == "clip":
        Z.zero_tensor_clip(plan, st["max_norm"], st["res"], norms=norms)
    elif op == "clip_norm":
        Z.zero_tensor_clip_norm(plan, st["max_norm"], st["inv"], st["res"], st["ws"],
                                kind=st["kind"], norms=norms, per_tensor=st["per_tensor"])
    elif st["with_norm"]:
        Z.zero_tensor_accumulate(plan, st["weight"], overwrite=st["first"], res=st["res"],
                                 workspace=st["ws"], inv_scale=st["inv"], kind=st["kind"],
                                 norms=norms)
    else:
        Z.zero_tensor_accumulate(plan, st["weight"], overwrite=st["first"])
    out = {}
    if op != "norm":
        out["y"] = [p["y"] for p in st["parts"]]
    if op in ("norm", "clip_norm") or st["with_norm"]:
        out["sumsq"], out["overflow"] = st["sumsq"], st["overflow"]
        if st["per_tensor"]:
            out["norms"] = norms
    return out


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    """The definition in 64 bits, tensor by tensor."""
    st = prepare(case, seed)
    inv, largest, w, limit = case["inv"], case["kind"] == "max", case["weight"], case["max_norm"]
    spans = [list(zip(p["which"].tolist(), p["starts"].tolist(), p["ends"].tolist()))
             for p in st["parts"]]
    res = {}
    y = [p["y"].double() for p in st["parts"]] if case["op"] != "norm" else None
    if case["op"] == "accumulate":
        y = [p["x"].double() * w + (0.0 if case["first"] else b) for p, b in zip(st["parts"], y)]
        res["y"] = y
    if case["op"] != "accumulate" or case["with_norm"]:
        one = torch.zeros(st["n"], dtype=torch.float64, device="cuda")
        for i, p in enumerate(st["parts"]):
            b = p["x"]
            if case["op"] == "accumulate":  # the norm of what the accumulators hold
                b = y[i].to(p["y"].dtype)
            for k, a, z in spans[i]:
                if z > a:
                    v = b[a:z].double().abs()
                    one[k] = v.max() if largest else torch.dot(v, v)
        total = one.max().square() if largest else one.sum()
        each = (one if largest else one.sqrt()) * inv
        sumsq = total * inv * inv
        if case["op"] == "clip":            # the call is given these, rounded
            sumsq, each = st["sumsq"][0], st["norms"].double()
        else:
            res["sumsq"] = sumsq.reshape(1)
            res["overflow"] = None
            if case["per_tensor"]:
                res["norms"] = each
        if case["op"] in ("clip", "clip_norm"):
            norm = each if case["per_tensor"] else sumsq.sqrt().expand(st["n"])
            f = torch.clamp(limit / (norm + 1e-6), max=1.0) * inv
            for i, p in enumerate(st["parts"]):
                y[i] = p["x"].double()
                for k, a, z in spans[i]:
                    y[i][a:z] *= f[k]
            res["y"] = y
    return res

"""Tensor-table plans on the CPU: sizes, the head of the device table, which plans
may be written to, and the refusals of every zero_tensor_* call (no device
pointer is ever read: a refused call launches nothing)."""
import ctypes

import numpy as np
import pytest

import zero_partitioned_mixed_shard_amd as Z
from zero_partitioned_mixed_shard_amd import tensors as T

FP16, BF16, FP32 = Z.ZERO_FP16, Z.ZERO_BF16, Z.ZERO_FP32
SIZE = {FP16: 2, BF16: 2, FP32: 4}


def entries(rows):
    """rows: (src, dst, numel, src_dtype, dst_dtype)."""
    e = np.zeros(max(1, len(rows)), dtype=T._ENTRY)
    if rows:
        e[:len(rows)] = rows
    return e


def init(rows, n=None):
    plan = T.zero_tensor_plan_t()
    rc = Z.lib().zero_tensor_plan_init(entries(rows).ctypes.data, len(rows) if n is None else n,
                                       ctypes.byref(plan))
    return rc, plan


def head(rows, plan):
    """The table's head: entries, and every tensor's first run, rest and piece."""
    buf = np.full(plan.head_bytes // 8 + 2, -7, dtype=np.int64)
    rc = Z.lib().zero_tensor_plan_head(entries(rows).ctypes.data, ctypes.byref(plan),
                                       buf.ctypes.data)
    assert rc == Z.ZERO_OK and (buf[plan.head_bytes // 8:] == -7).all()
    n = len(rows)
    assert plan.head_bytes % 16 == 0 and 0 <= plan.head_bytes // 8 - (4 * n + 3 * (n + 1)) <= 1
    firsts = buf[4 * n:4 * n + 3 * (n + 1)].reshape(3, n + 1)
    return buf[:4 * n].view(T._ENTRY), *firsts


def test_entry_and_plan_sizes():
    assert T._ENTRY.itemsize == 32 and ctypes.sizeof(T.zero_tensor_plan_t) == 80


@pytest.mark.parametrize("seed", range(20))
def test_head_counts_every_tensors_parts(seed):
    rng = np.random.default_rng(seed)
    rows, at = [], 1 << 20
    for _ in range(int(rng.integers(0, 12))):
        n = int(rng.choice([0, 1, 7, 100, 4095, 4096, 4097, 16383, 16384, 16385, 70000, 1000003]))
        s, d = (int(x) for x in rng.choice([FP16, BF16, FP32], 2))
        dst = at + n * SIZE[s] + (-(at + n * SIZE[s])) % 4
        rows.append((at, dst, n, s, d))
        at = dst + n * SIZE[d] + 64
        at += -at % 4
    rc, plan = init(rows)
    assert rc == Z.ZERO_OK and plan.writable == 1
    assert plan.n_tensors == len(rows) and plan.numel == sum(r[2] for r in rows)
    assert plan.bytes == sum(r[2] * (SIZE[r[3]] + SIZE[r[4]]) for r in rows)
    assert plan.fp32_out == (sum(r[2] for r in rows if r[4] == FP32) > plan.numel // 2)
    even = sum(r[2] for r in rows if r[3] != FP32 and r[0] % 4 == 0)
    assert plan.even16 == (plan.numel > 0 and even >= plan.numel // 8 * 7)
    assert plan.table_bytes - plan.head_bytes == 16 * (plan.n_runs + plan.n_rests) + 24 * plan.n_pieces
    e, run, rest, piece = head(rows, plan)
    assert (e == entries(rows)[:len(rows)]).all()
    for f, a, n in ((run, 0, plan.n_runs), (rest, plan.n_runs, plan.n_rests),
                    (piece, 0, plan.n_pieces)):
        assert f[0] == a and f[-1] == a + n
    for k, (src, dst, n, s, d) in enumerate(rows):
        # runs of 16384 elements, the rest in rests of 4096: by the count alone
        assert run[k + 1] - run[k] == n // 16384
        assert rest[k + 1] - rest[k] == -(-(n % 16384) // 4096)
        # pieces end at multiples of 128 bytes past the one the output begins in
        lead = dst % 128 // SIZE[d]
        assert piece[k + 1] - piece[k] == (-(-(n + lead) // 4096) if n else 0)


def test_large_tensors():
    n = (1 << 36) + 5
    rc, plan = init([(1 << 40, (1 << 42) + 4, n, BF16, FP32)])
    assert rc == Z.ZERO_OK and plan.numel == n and plan.bytes == 6 * n
    assert (plan.n_runs, plan.n_rests) == (n // 16384, 1) and plan.n_pieces == (1 << 24) + 1


def test_largest_tensor():
    """The largest tensor decides how the tensors' norms are joined."""
    for numels in ([], [0], [4095], [5, 1 << 30, 70000, 0], [1 << 40], [1 << 45, 1 << 44]):
        rows = [(1 << 50, (k + 1) << 51, n, BF16, BF16) for k, n in enumerate(numels)]
        rc, plan = init(rows)
        assert rc == Z.ZERO_OK
        assert plan.largest == min(max(numels, default=0) // 4096, 2 ** 31 - 1)


@pytest.mark.parametrize("rows,writable", [
    ([(4096, 4096, 10, FP16, FP16)], 1),                                   # in place
    ([(4096, 4096, 10, FP16, BF16)], 0),                                   # in place, other type
    ([(4096, 4098, 10, FP16, FP16)], 0),                                   # shifted onto itself
    ([(4096, 4116, 10, FP16, FP16)], 1),                                   # right after itself
    ([(4096, 4096, 10, FP32, FP16)], 0),                                   # narrowed onto itself
    ([(4096, 8192, 10, FP16, FP32), (8192 + 36, 4096 * 4, 5, FP16, FP16)], 0),  # out over next input
    ([(4096, 8192, 10, FP16, FP32), (8192 + 40, 4096 * 4, 5, FP16, FP16)], 1),
    ([(4096, 8192, 10, FP16, FP16), (6000, 8210, 5, FP16, FP16)], 0),      # outputs overlap
    ([(4096, 4096, 10, FP16, FP16), (4096, 4096, 10, FP16, FP16)], 0),     # the same tensor twice
    ([(4096, 8192, 10, FP16, FP16), (4096, 9000, 10, FP16, FP16)], 1),     # one input, two outputs
    ([(4096, 4096, 0, FP16, FP16), (4096, 4096, 3, FP16, FP16)], 1),       # an empty one beside it
    ([], 1),
])
def test_writable(rows, writable):
    rc, plan = init(rows)
    assert rc == Z.ZERO_OK and plan.writable == writable


def test_init_refusals():
    ok = (4096, 8192, 10, FP16, FP32)
    bad = {"negative count": (4096, 8192, -1, FP16, FP32), "null src": (0, 8192, 10, FP16, FP32),
           "null dst": (4096, 0, 10, FP16, FP32), "type 0": (4096, 8192, 10, 0, FP32),
           "type 4": (4096, 8192, 10, FP16, 4), "odd fp16": (4097, 8192, 10, FP16, FP32),
           "fp32 at 2": (4096, 8194, 10, FP16, FP32)}
    for what, row in bad.items():
        assert init([ok, row])[0] == Z.ZERO_EINVAL, what
    for row in ((4096, 8192, 1 << 62, FP16, FP32), (2 ** 64 - 8, 8192, 10, FP16, FP32)):
        assert init([row])[0] == Z.ZERO_ERANGE
    # more than an int64 of elements, and more pieces than any memory holds
    assert init([(4096, 4096, (1 << 62) - 1, FP16, FP16)] * 3)[0] == Z.ZERO_ERANGE
    assert init([(4096, 4096, 1 << 55, FP16, FP16)])[0] == Z.ZERO_ERANGE
    assert init([(4096, 4096, 0, FP16, FP16)], n=1 << 24)[0] == Z.ZERO_ERANGE   # tensors
    # pointers and types of nothing: only the types are looked at
    assert init([(0, 0, 0, FP16, FP32)])[0] == Z.ZERO_OK
    L, plan = Z.lib(), T.zero_tensor_plan_t()
    assert L.zero_tensor_plan_init(None, 1, ctypes.byref(plan)) == Z.ZERO_EINVAL
    assert L.zero_tensor_plan_init(entries([ok]).ctypes.data, -1, ctypes.byref(plan)) == Z.ZERO_EINVAL
    assert L.zero_tensor_plan_init(entries([ok]).ctypes.data, 1, None) == Z.ZERO_EINVAL
    assert L.zero_tensor_plan_init(None, 0, ctypes.byref(plan)) == Z.ZERO_OK
    rc, plan = init([ok])
    buf = np.zeros(plan.head_bytes, np.uint8)
    e = entries([ok])
    assert L.zero_tensor_plan_head(e.ctypes.data, None, buf.ctypes.data) == Z.ZERO_EINVAL
    assert L.zero_tensor_plan_head(e.ctypes.data, ctypes.byref(plan), None) == Z.ZERO_EINVAL
    assert L.zero_tensor_plan_head(None, ctypes.byref(plan), buf.ctypes.data) == Z.ZERO_EINVAL
    other = entries([(4096, 8192, 100_000, FP16, FP32)])   # another plan's entries
    assert L.zero_tensor_plan_head(other.ctypes.data, ctypes.byref(plan),
                                   buf.ctypes.data) == Z.ZERO_EINVAL
    for args in ((None, 4096), (ctypes.byref(plan), None), (ctypes.byref(plan), 4096 + 8)):
        assert L.zero_tensor_plan_expand(*args, None) == Z.ZERO_EINVAL


def test_head_refuses_another_plans_entries():
    """Entries with the same counts as the plan's but not its: types, starts, and outputs
    that overlap (a plan that may be written through would stand for them)."""
    L = Z.lib()
    mine = [(4096, 8192, 100, FP16, FP16), (4400, 12288, 100, FP16, FP16)]
    rc, plan = init(mine)
    assert rc == Z.ZERO_OK and plan.writable == 1 and plan.even16 == 1
    buf = np.zeros(plan.head_bytes, np.uint8)

    def refused(rows):
        return L.zero_tensor_plan_head(entries(rows).ctypes.data, ctypes.byref(plan),
                                       buf.ctypes.data) == Z.ZERO_EINVAL and not buf.any()

    assert refused([mine[0], (4400, 8200, 100, FP16, FP16)])              # outputs overlap
    assert refused([mine[0], (8192, 12288, 100, FP16, FP16)])             # an input under an output
    assert refused([(4098, *mine[0][1:]), mine[1]])                       # starts between dwords
    assert refused([(4096, 8192, 100, FP16, FP32), mine[1]])              # another type
    assert refused([(4096, 8192, 99, FP16, FP16), mine[1]])               # another size
    plan.n_tensors = 1 << 24
    assert refused(mine)
    plan.n_tensors = 2
    assert not refused(mine) and buf.any()


def test_workspace_bytes():
    assert Z.lib().zero_tensor_workspace_bytes(None) == 0
    for rows in ([], [(4096, 4096, 1, FP16, FP16)], [(4096, 4096, 1 << 33, FP16, FP16)],
                 [(4096, 4096, 1 << 40, FP16, FP16)]):
        rc, plan = init(rows)
        ws = Z.lib().zero_tensor_workspace_bytes(ctypes.byref(plan))
        assert max(16, 8 * plan.n_pieces) <= ws <= 8 * (plan.n_pieces + plan.n_pieces // 4096 + 2)


def test_call_refusals():
    """Bad arguments of the device calls; the pointers are never read."""
    L = Z.lib()
    fake = 1 << 12
    nan, inf = float("nan"), float("inf")
    _, good = init([(4096, 8192, 100, FP16, FP32)])
    _, closed = init([(4096, 8192, 10, FP16, FP32)] * 2)
    assert closed.writable == 0
    g, c = ctypes.byref(good), ctypes.byref(closed)
    ws = L.zero_tensor_workspace_bytes(g)
    L2 = Z.ZERO_NORM_L2

    def norm(plan=g, table=fake, kind=L2, inv=1.0, ctl=None, res=fake, w=fake, wb=ws):
        return L.zero_tensor_norm(plan, table, kind, inv, ctl, res, None, w, wb, 0, None)

    def fused(plan=g, table=fake, kind=L2, clip=1.0, inv=1.0, res=fake, norms=None, each=0, w=fake,
              wb=ws):
        return L.zero_tensor_clip_norm(plan, table, kind, clip, inv, None, res, norms, each, w, wb,
                                       None)

    def add(plan=g, table=fake, weight=1.0, kind=L2, inv=1.0, res=fake, w=fake, wb=ws):
        return L.zero_tensor_accumulate_norm(plan, table, weight, 0, kind, inv, None, res, None, w,
                                             wb, 0, None)

    shared = [dict(plan=None), dict(table=None), dict(table=fake + 8), dict(kind=0), dict(kind=3),
              dict(inv=0.0), dict(inv=-1.0), dict(inv=nan), dict(inv=inf), dict(res=None),
              dict(w=None), dict(w=fake + 4), dict(wb=ws - 1)]
    for call in (norm, fused, add):
        for bad in shared:
            assert call(**bad) == Z.ZERO_EINVAL, (call.__name__, bad)
    for bad in (dict(plan=c), dict(clip=nan), dict(each=1)):
        assert fused(**bad) == Z.ZERO_EINVAL, bad
    for bad in (dict(plan=c), dict(weight=nan), dict(weight=inf)):
        assert add(**bad) == Z.ZERO_EINVAL, bad
    for args in ((None, fake, 1.0, fake, None), (g, None, 1.0, fake, None), (c, fake, 1.0, fake, None),
                 (g, fake, nan, fake, None), (g, fake, 1.0, None, None)):
        assert L.zero_tensor_clip(*args, None) == Z.ZERO_EINVAL, args
    for args in ((None, fake, 1.0), (g, None, 1.0), (c, fake, 1.0), (g, fake, nan), (g, fake, -inf)):
        assert L.zero_tensor_accumulate(*args, 0, None) == Z.ZERO_EINVAL, args


def test_binding_refuses_host_tensors():
    import torch
    for t in (torch.zeros(4), torch.zeros(4, dtype=torch.float64)):
        with pytest.raises(ValueError, match="device"):
            Z.zero_tensor_plan([t])
    for bad in ([None], [torch.zeros(4), None], [np.zeros(4)]):
        with pytest.raises(TypeError, match="tensors expected"):
            Z.zero_tensor_plan(bad)
    with pytest.raises(TypeError, match="tensors expected"):
        Z.zero_tensor_plan([torch.zeros(4)], out=[None])


@pytest.mark.parametrize("capturing", [0, 1, 2])
def test_no_plan_inside_a_capture_on_either_device(monkeypatch, capturing):
    """A plan for device 1 built with device 0 current: refused where the current stream
    of either captures, not for another device's."""
    import torch
    current = [0]

    class device:
        def __init__(self, d):
            self.d = torch.device(d).index

        def __enter__(self):
            self.was, current[0] = current[0], self.d

        def __exit__(self, *exc):
            current[0] = self.was

    class Built(Exception):
        pass

    def build(*args, **kw):
        raise Built

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] == capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", build)
    want = Built if capturing == 2 else RuntimeError
    with pytest.raises(want, match=None if capturing == 2 else "before the capture"):
        Z.zero_tensor_plan([], device="cuda:1")
    assert current == [0]


def test_a_callers_streams_are_not_recorded(monkeypatch):
    """torch's allocator uses the streams recorded for the table when the plan goes, and
    a stream that the caller made may be gone by then: torch's own are recorded, once
    each, handles and streams around handles are not."""
    import torch
    from types import SimpleNamespace as NS

    dev = torch.device("cuda", 0)

    def stream(handle, stream_id):
        return NS(device=dev, cuda_stream=handle, stream_id=stream_id)

    default, pool, other = stream(0, 0), stream(0x5000, 35), stream(0x5100, 67)
    external = stream(0x6000, 0x6000)                     # as torch.cuda.ExternalStream
    current, seen, ran = [default], [], []
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: current[0].cuda_stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: current[0])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d=None: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: stream(raw, raw))
    plan = object.__new__(Z.zero_tensor_plan)
    plan.device, plan._index, plan._args, plan._streams = dev, 0, (), {0x4000}
    plan.table = NS(record_stream=lambda s: seen.append(s.cuda_stream))

    def call(s, now=default):
        current[0] = now
        plan._call(lambda raw: ran.append(raw) or 0, (), s)

    for s, now in ((None, default), (pool, default), (0x5000, default), (None, other),
                   (external, default), (None, external), (0x7000, default), (0x7000, other),
                   (0, pool), (default, pool), (stream(0x7000, 99), default)):
        call(s, now)                                      # the last: the handle is torch's now
    assert ran == [0, 0x5000, 0x5000, 0x5100, 0x6000, 0x6000, 0x7000, 0x7000, 0, 0, 0x7000]
    assert seen == [0, 0x5000, 0x5100, 0x7000]


def test_dense_orders():
    import torch
    x = torch.zeros(4, 6, 5)
    assert T._order(x) is None and T._order(x[:, :1].contiguous()) is None
    assert T._order(x.permute(2, 0, 1)) == (1, 30, 5)
    assert T._order(torch.zeros(0, 3)) is None and T._order(torch.zeros(())) is None
    assert T._order(x.transpose(0, 1)[:, :, None]) == (5, 30, 1)
    for bad in (x[:, ::2], x[:, :, 1:], x[:1].expand(4, 6, 5), x.transpose(0, 2)[1:]):
        with pytest.raises(ValueError, match="dense"):
            T._order(bad)


def test_unknown_norm_kind():
    with pytest.raises(ValueError, match="kind"):
        T._kind("l1")

"""Plans of matrices and the refusals of the calls over matrices and embedding rows, on the
CPU: nothing is launched."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import zero_partitioned_mixed_shard_amd as Z
from zero_partitioned_mixed_shard_amd import build
from zero_partitioned_mixed_shard_amd.matrix import _ENTRY, zero_matrix_plan_t

L = Z.lib()
OK, EINVAL, ERANGE = Z.ZERO_OK, Z.ZERO_EINVAL, Z.ZERO_ERANGE
MIB = 1 << 20


def entry(src=MIB, dst=2 * MIB, rows=4, cols=8, src_ld=None, dst_ld=None, st=3, dt=3):
    e = np.zeros(1, dtype=_ENTRY)
    e[0] = (src, dst, rows, cols, cols if src_ld is None else src_ld, cols if dst_ld is None else dst_ld, st, dt)
    return e


def init(entries, precise=0):
    e = np.concatenate(entries) if entries else np.zeros(1, dtype=_ENTRY)
    c = zero_matrix_plan_t()
    rc = L.zero_matrix_plan_init(e.ctypes.data, len(entries), precise, ctypes.byref(c))
    return rc, c, e


def muon(ranges, precise=0):
    r = np.array(ranges or [(0, 0, 0)], dtype=np.int64)
    c = zero_matrix_plan_t()
    return L.zero_muon_plan_init(r.ctypes.data, len(ranges), precise, ctypes.byref(c)), c, r


def test_plan_counts():
    rc, c, _ = init([])
    assert rc == OK and (c.n_matrices, c.numel, c.workspace_bytes, c.kind) == (0, 0, 0, 1)
    rc, c, _ = init([entry(rows=0), entry(cols=0), entry(rows=5, cols=7)])
    assert rc == OK and (c.n_matrices, c.numel) == (3, 35)
    rc, c, _ = muon([(3, 5, 7), (38, 200, 300), (100000, 0, 9)])
    assert rc == OK and (c.n_matrices, c.numel, c.extent, c.kind) == (3, 60035, 60038, 2)


@pytest.mark.parametrize("precise", [0, 1])
def test_workspace_holds_the_planes(precise):
    for rows, cols in ((65, 65), (300, 100), (1024, 4096), (4096, 1100)):
        rc, c, _ = muon([(0, rows, cols)], precise)
        assert rc == OK
        m, n = sorted((rows, cols))
        assert c.workspace_bytes >= 8 * m * n + (8 if precise else 4) * m * m
        # padding to tiles, partials and cut tiles: at most 256 parts of 256 x 256 sums
        mp, np_ = -(-m // 256) * 256, -(-n // 256) * 256
        assert c.workspace_bytes <= 8 * mp * np_ + 8 * mp * mp + 2 * 512 * 256 * 256 * 4 + 64 * mp + (1 << 20)


BAD = [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(src=0), EINVAL), (dict(dst=0), EINVAL),
    (dict(src=MIB + 2), EINVAL), (dict(dst=MIB + 1, dt=1), EINVAL), (dict(st=0), EINVAL),
    (dict(dt=4), EINVAL), (dict(src_ld=7), EINVAL), (dict(dst_ld=7), EINVAL),
    (dict(rows=4194241), ERANGE), (dict(cols=1 << 40), ERANGE), (dict(rows=65537, cols=65537), ERANGE),
    (dict(src_ld=1 << 61), ERANGE), (dict(src=(1 << 63) - 8), ERANGE),
    # results that overlap the matrix but are not in its place
    (dict(dst=MIB + 4), EINVAL), (dict(dst=MIB, dt=1), EINVAL), (dict(dst=MIB, dst_ld=9), EINVAL),
]


@pytest.mark.parametrize("bad,rc", BAD)
def test_entries_refused(bad, rc):
    assert init([entry(**bad)])[0] == rc
    assert init([entry(src=8 * MIB, dst=9 * MIB), entry(**bad)])[0] == rc


def test_empty_matrices_are_not_looked_at():
    assert init([entry(src=0, dst=0, rows=0)])[0] == OK
    assert init([entry(src=1, dst=3, cols=0, src_ld=0, dst_ld=0)])[0] == OK


def test_overlaps():
    a, b = entry(), entry(src=3 * MIB, dst=4 * MIB)
    assert init([a, b])[0] == OK
    assert init([a, entry(src=3 * MIB, dst=2 * MIB + 64)])[0] == EINVAL        # two results
    assert init([a, entry(src=2 * MIB + 64, dst=4 * MIB)])[0] == EINVAL        # a result in a matrix
    assert init([a, entry(src=MIB, dst=4 * MIB)])[0] == OK                     # one matrix, two results
    assert init([entry(dst=MIB), b])[0] == OK                                  # in place
    # blocks of columns of one buffer lie between each other's rows
    left = entry(src=MIB, dst=MIB, src_ld=24, dst_ld=24)
    mid = entry(src=MIB + 32, dst=MIB + 32, src_ld=24, dst_ld=24)
    right = entry(src=MIB + 64, dst=MIB + 64, src_ld=24, dst_ld=24)
    assert init([right, left, mid])[0] == OK
    assert init([left, entry(src=MIB + 28, dst=MIB + 28, src_ld=24, dst_ld=24)])[0] == EINVAL
    assert init([left, entry(src=MIB + 64, dst=MIB + 64, cols=9, src_ld=24, dst_ld=24)])[0] == EINVAL


@pytest.mark.parametrize("ranges,rc", [
    ([(-1, 2, 2)], EINVAL), ([(0, -2, 2)], EINVAL), ([(0, 2, 2), (3, 2, 2)], EINVAL),
    ([(0, 70000, 70000)], ERANGE), ([(0, 4194241, 1)], ERANGE), ([(1 << 62, 2, 2)], ERANGE),
    ([(4, 2, 2), (0, 2, 2)], OK), ([(0, 4194240, 1)], OK), ([(0, 1, 65537)], OK),
])
def test_ranges(ranges, rc):
    assert muon(ranges)[0] == rc


def test_tables():
    rc, c, e = init([entry(), entry(src=3 * MIB, dst=4 * MIB, rows=100, cols=70)])
    table = np.zeros(c.table_bytes, dtype=np.uint8)
    assert L.zero_matrix_plan_table(e.ctypes.data, ctypes.byref(c), table.ctypes.data) == OK
    assert table.any()
    other = zero_matrix_plan_t.from_buffer_copy(bytes(c))
    other.numel += 1
    assert L.zero_matrix_plan_table(e.ctypes.data, ctypes.byref(other), table.ctypes.data) == EINVAL
    assert L.zero_matrix_plan_table(e.ctypes.data, ctypes.byref(c), None) == EINVAL
    assert L.zero_matrix_plan_table(None, ctypes.byref(c), table.ctypes.data) == EINVAL
    r = np.array([(0, 5, 7)], dtype=np.int64)
    assert L.zero_muon_plan_table(r.ctypes.data, ctypes.byref(c), table.ctypes.data) == EINVAL   # another kind
    assert L.zero_matrix_plan_init(None, 1, 0, ctypes.byref(c)) == EINVAL
    assert L.zero_matrix_plan_init(e.ctypes.data, -1, 0, ctypes.byref(c)) == EINVAL
    assert L.zero_matrix_plan_init(e.ctypes.data, 1, 0, None) == EINVAL


def call(kind="orth", ns=None, host=True, table=4096, ws=4096, ws_bytes=None, hp=None, **bufs):
    """An entry point with addresses of nothing: it has to refuse before a launch."""
    if kind == "orth":
        rc, c, e = init([entry(rows=100, cols=70)])
        t = np.zeros(c.table_bytes, dtype=np.uint8)
        assert L.zero_matrix_plan_table(e.ctypes.data, ctypes.byref(c), t.ctypes.data) == OK
    else:
        rc, c, r = muon([(0, 100, 70)])
        t = np.zeros(c.table_bytes, dtype=np.uint8)
        assert L.zero_muon_plan_table(r.ctypes.data, ctypes.byref(c), t.ctypes.data) == OK
    tail = (ctypes.byref(c), t.ctypes.data if host is True else host, table)
    size = c.workspace_bytes if ws_bytes is None else ws_bytes
    if bufs.pop("as_orth", kind == "orth"):
        return L.zero_orthogonalize(*tail, ctypes.byref(ns or Z.zero_newton_schulz()), ws, size, None)
    b = dict(master=MIB, momentum=2 * MIB, param16=3 * MIB, grad16=4 * MIB, dtype=1, res=5 * MIB)
    b.update(bufs)
    return L.zero_muon_step(b["master"], b["momentum"], b["param16"], b["grad16"], b["dtype"], *tail,
                            ctypes.byref(hp or Z.zero_muon_hparams()), b["res"], ws, size, None)


NS = [dict(steps=0), dict(steps=33), dict(eps=0.0), dict(eps=float("nan")), dict(a=float("inf")),
      dict(steps=11), dict(a=2.0, b=0.0, c=0.0), dict(b=4.775), dict(a=40.0, b=-80.0, c=40.0)]


@pytest.mark.parametrize("ns", NS)
def test_coefficients_refused(ns):
    ns = Z.zero_newton_schulz(**ns)
    assert call(ns=ns) == EINVAL
    assert call("muon", hp=Z.zero_muon_hparams(ns=ns)) == EINVAL


@pytest.mark.parametrize("kind", ["orth", "muon"])
def test_calls_refused(kind):
    assert call(kind, host=None) == EINVAL
    assert call(kind, table=None) == EINVAL
    assert call(kind, table=4100) == EINVAL
    assert call(kind, ws=None) == EINVAL
    assert call(kind, ws=4096 + 128) == EINVAL
    assert call(kind, ws_bytes=16) == EINVAL
    junk = np.zeros(4096, dtype=np.uint8)
    assert call(kind, host=junk.ctypes.data) == EINVAL
    assert call(kind, as_orth=kind != "orth") == EINVAL                          # the other kind's plan


@pytest.mark.parametrize("bad", [dict(master=None), dict(momentum=None), dict(param16=None), dict(grad16=None),
                                 dict(res=None), dict(res=MIB + 4), dict(master=MIB + 2), dict(momentum=MIB + 1),
                                 dict(param16=MIB + 1), dict(grad16=MIB + 1), dict(dtype=3), dict(dtype=0)])
def test_muon_refused(bad):
    assert call("muon", **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(lr=float("nan")), dict(momentum=float("inf")),
                                 dict(weight_decay=float("nan")), dict(max_grad_norm=float("nan"))])
def test_muon_parameters_refused(bad):
    assert call("muon", hp=Z.zero_muon_hparams(**bad)) == EINVAL
    hp = Z.zero_muon_hparams()
    hp.scaling = 3
    assert call("muon", hp=hp) == EINVAL
    with pytest.raises(ValueError):
        Z.zero_muon_hparams(scaling="max")


def lookup(**k):
    a = dict(out=MIB, out_ld=64, out_dtype=3, ids=2 * MIB, id_bytes=8, n=4, table=3 * MIB, table_dtype=2, vocab=100,
             dim=64, begin=0, count=6400, scale=1.0)
    a.update(k)
    return L.zero_embedding_lookup(*a.values(), None)


def grad(**k):
    a = dict(grad=MIB, grad_dtype=3, ids=2 * MIB, id_bytes=8, n=4, dy=3 * MIB, dy_ld=64, dy_dtype=2, vocab=100,
             dim=64, begin=0, count=6400, padding=-1, scale=1.0, overwrite=0, ws=4 * MIB, ws_bytes=1 << 30)
    a.update(k)
    return L.zero_embedding_grad(*a.values(), None)


COMMON = [(dict(n=-1), EINVAL), (dict(vocab=0), EINVAL), (dict(dim=0), EINVAL), (dict(n=1 << 31), ERANGE),
          (dict(vocab=(1 << 31) - 1), ERANGE), (dict(dim=1 << 29), ERANGE), (dict(id_bytes=2), EINVAL),
          (dict(ids=None), EINVAL), (dict(ids=MIB + 4), EINVAL), (dict(begin=-1), EINVAL),
          (dict(begin=6401), EINVAL), (dict(count=-1), EINVAL), (dict(count=6401), EINVAL),
          (dict(begin=1, count=6400), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL)]


@pytest.mark.parametrize("bad,rc", COMMON + [
    (dict(out=None), EINVAL), (dict(table=None), EINVAL), (dict(out=MIB + 2), EINVAL), (dict(table=MIB + 1), EINVAL),
    (dict(out_ld=63), EINVAL), (dict(out_dtype=0), EINVAL), (dict(table_dtype=5), EINVAL),
    (dict(out_ld=1 << 62), ERANGE), (dict(n=0, out=None, ids=None, table=None), OK)])
def test_lookup_refused(bad, rc):
    assert lookup(**bad) == rc


@pytest.mark.parametrize("bad,rc", COMMON + [
    (dict(grad=None), EINVAL), (dict(dy=None), EINVAL), (dict(grad=MIB + 2), EINVAL), (dict(dy=MIB + 1), EINVAL),
    (dict(dy_ld=63), EINVAL), (dict(grad_dtype=0), EINVAL), (dict(dy_dtype=5), EINVAL), (dict(dy_ld=1 << 62), ERANGE),
    (dict(ws=None), EINVAL), (dict(ws=MIB + 128), EINVAL), (dict(ws_bytes=100), EINVAL),
    (dict(n=0, ids=None, dy=None, ws=None, ws_bytes=0), OK), (dict(count=0), OK)])
def test_grad_refused(bad, rc):
    assert grad(**bad) == rc


def test_workspace_grows_with_the_tokens():
    assert Z.zero_embedding_workspace_bytes(-1, 10, 10) == 0
    assert Z.zero_embedding_workspace_bytes(10, 0, 10) == 0
    for dim in (1, 100, 512, 513, 4096, 30000):
        last = 0
        for n in sorted({int(1.3 ** k) for k in range(70)} | {8 * 4096 // (-(-dim // 512)) + k for k in (-1, 0, 1, 2)}):
            now = Z.zero_embedding_workspace_bytes(n, 1000, dim)
            assert now >= last, (n, dim)
            last = now


def test_accumulators_stay_in_place(tmp_path):
    """The products are written as instructions the compiler takes for something else: from a
    kernel's first product to the wait after its last nothing else may touch the
    accumulators (they are registers a..., and would be moved with v_accvgpr_* or spilled)."""
    src = os.path.join(build.PKG, "csrc", "zero_matrix.hip")
    out = str(tmp_path / "zero_matrix.s")
    flags = [f for f in build.FLAGS if f != "-shared"]
    subprocess.run([build.HIPCC, *flags, "-S", "--cuda-device-only", "-o", out, src], check=True, capture_output=True)
    name, inside, products, kernels, bad = None, False, 0, set(), []
    for line in open(out):
        if re.match(r"_ZN\S+:", line):
            name, inside = line.split(":")[0], False
        if name is None or "matrix_product_kernel" not in name:
            continue
        if re.search(r"\bv_mfma_", line):
            inside = True
            products += 1
            kernels.add(name)
        elif "s_nop 15" in line:
            inside = False
        elif inside and re.search(r"v_accvgpr_|scratch_|\ba\[?\d", line):
            bad.append((name, line.strip()))
    assert len(kernels) == 28 and products >= 28 * 64
    assert not bad, bad[:5]


def test_a_plans_table_stays_for_torchs_streams(monkeypatch):
    """A plan that is dropped while a call on another stream runs: the table's memory waits for
    that stream.  torch's own streams are recorded, once each; a caller's, which may be gone by
    then, are not."""
    import contextlib
    from types import SimpleNamespace as NS

    import torch

    dev = torch.device("cuda", 0)

    def stream(handle, stream_id):
        return NS(device=dev, cuda_stream=handle, stream_id=stream_id)

    default, pool, other, external = stream(0, 0), stream(0x5000, 35), stream(0x5100, 67), stream(0x6000, 0x6000)
    current, seen, ran = [default], [], []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: current[0])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d=None: default)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    for kind in (Z.zero_matrix_plan, Z.zero_muon_plan):
        plan = object.__new__(kind)
        plan.device, plan._streams = dev, {0x4000}
        plan.table = NS(record_stream=lambda s: seen.append(s.cuda_stream))
        seen.clear(), ran.clear()
        for s, now in ((None, default), (pool, default), (0x5000, default), (None, other), (external, default),
                       (None, external), (0x7000, default), (0, pool), (default, pool)):
            current[0] = now
            plan._call(lambda raw: ran.append(raw) or 0, (), s)
        assert ran == [0, 0x5000, 0x5000, 0x5100, 0x6000, 0x6000, 0x7000, 0, 0]
        assert seen == [0, 0x5000, 0x5100]


def bytes_of(at, rows, cols, ld):
    return {at + 4 * (r * ld + c) + b for r in range(rows) for c in range(cols) for b in range(4)}


def test_single_rows_beside_blocks():
    """A row's distance to the next is nothing that a list of one row has: it may lie between
    the rows of a block of columns.  Against the bytes themselves."""
    block = entry(src=MIB, dst=MIB, rows=4, cols=8, src_ld=24, dst_ld=24)
    assert init([block, entry(src=MIB + 4 * 32, dst=MIB + 4 * 32, rows=1, cols=16)])[0] == OK
    assert init([block, entry(src=MIB + 4 * 32, dst=MIB + 4 * 32, rows=1, cols=17)])[0] == EINVAL
    own = bytes_of(MIB, 4, 8, 24)
    for cols in (1, 3, 16, 17, 24, 40):
        for at in range(-45, 90):
            where = MIB + 4 * at
            row = entry(src=where, dst=where, rows=1, cols=cols, src_ld=cols + at % 5, dst_ld=cols + at % 5)
            free = own.isdisjoint(bytes_of(where, 1, cols, 0))
            for order in ([block, row], [row, block]):
                assert init(order)[0] == (OK if free else EINVAL), (cols, at)
    # two single rows, of any distances
    for at, free in ((7, False), (8, True), (-8, True), (-7, False), (0, False)):
        other = entry(src=MIB + 4 * at, dst=MIB + 4 * at, rows=1, cols=8, src_ld=30, dst_ld=30)
        assert (init([entry(src=MIB, dst=MIB, rows=1, cols=8), other])[0] == OK) == free, at


def registers(operand):
    """The vector registers that an operand names."""
    m = re.fullmatch(r"v(\d+)|v\[(\d+):(\d+)\]", operand.strip())
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def wait_states(text):
    m = re.match(r"s_nop (\d+)", text)
    return 1 + int(m[1]) if m else 1


def written_too_late(lines):
    """Products whose operands a vector instruction writes less than two wait states before, on
    any way to them: [(vector instruction, product)]."""
    code = [ln.split(";")[0].strip() for ln in lines]
    code = [ln for ln in code if ln and (not ln.startswith(".") or ln.endswith(":"))]
    labels = {ln[:-1]: k for k, ln in enumerate(code) if ln.endswith(":")}
    jumps = {}
    for k, ln in enumerate(code):
        m = re.match(r"s_c?branch\w* (\S+)", ln)
        if m and m[1] in labels:
            jumps.setdefault(labels[m[1]], []).append(k)
    bad = []

    def back(k, states, reads, product):
        """Looks at what is before code[k], `states` wait states before the product."""
        while k > 0 and states < 2:
            k -= 1
            if code[k].endswith(":"):
                for j in jumps.get(k, []):
                    back(j, states + 1, reads, product)      # the jump itself is a wait state
                continue
            if re.match(r"s_(branch|endpgm|setpc)", code[k]):
                return
            if code[k].startswith("v_") and not code[k].startswith(("v_mfma", "v_cmp", "v_readfirstlane", "v_readlane")):
                first = code[k].split(None, 1)[1].split(",")[0] if " " in code[k] else ""
                if registers(first) & reads:
                    bad.append((code[k], product))
            states += wait_states(code[k])

    for k, ln in enumerate(code):
        m = re.match(r"v_mfma_\S+ (.*)", ln)
        if m:
            ops = re.findall(r"[av]\[\d+:\d+\]|[av]\d+", m[1])
            back(k, 0, set().union(*(registers(o) for o in ops[1:3])), ln)
    return bad


def test_written_too_late_is_found():
    mfma = "\tv_mfma_f32_16x16x32_f16 a[0:3], v[4:7], v[8:11], a[0:3]"
    assert written_too_late(["\tv_mov_b32_e32 v5, v1", mfma])
    assert written_too_late(["\tv_mov_b32_e32 v5, v1", "\ts_nop 0", mfma])
    assert written_too_late(["\tv_lshlrev_b64 v[10:11], 1, v[2:3]", ".LBB0_1:", mfma])
    assert not written_too_late(["\tv_mov_b32_e32 v5, v1", "\ts_nop 1", mfma])
    assert not written_too_late(["\tv_mov_b32_e32 v5, v1", "\ts_add_u32 s0, s0, 1", "\ts_nop 0", mfma])
    assert not written_too_late(["\tv_mov_b32_e32 v12, v5", mfma])
    assert not written_too_late(["\tds_read_b128 v[4:7], v1", mfma])
    loop = [".LBB0_1:", mfma, "\ts_nop 7", "\tv_mov_b32_e32 v9, v1", "\ts_cbranch_scc1 .LBB0_1"]
    assert written_too_late(loop)
    assert not written_too_late(loop[:4] + ["\ts_nop 1"] + loop[4:])


def test_operands_are_written_in_time(tmp_path):
    """What the compiler takes for some instruction reads its operands as a matrix instruction
    does: two wait states have to lie between a vector instruction that writes one and the
    product (what comes from LDS is waited for, since the instruction names it)."""
    src = os.path.join(build.PKG, "csrc", "zero_matrix.hip")
    out = str(tmp_path / "zero_matrix.s")
    flags = [f for f in build.FLAGS if f != "-shared"]
    subprocess.run([build.HIPCC, *flags, "-S", "--cuda-device-only", "-o", out, src], check=True, capture_output=True)
    kernels, lines = 0, None
    for line in open(out):
        if re.match(r"_ZN\S+:", line):
            lines = [] if "matrix_product_kernel" in line else None
        elif lines is not None and line.startswith(".Lfunc_end"):
            assert any("v_mfma_" in ln for ln in lines)
            assert not written_too_late(lines)
            kernels, lines = kernels + 1, None
        elif lines is not None:
            lines.append(line)
    assert kernels == 28

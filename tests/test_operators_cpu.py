"""The operators' host side without a GPU: the plan of row moves, sizes and refused arguments."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_layer_kda_b200", "csrc")


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("rows") / "librows.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-x", "c++",
                           os.path.join(CSRC, "rows_plan.cu"), os.path.join(ROOT, "tests", "rows_shim.cpp"),
                           "-I" + CSRC, "-o", out])
    return ctypes.CDLL(out)


def plan(shim, dst, src, in_place=True):
    n = len(dst)
    A = ctypes.c_int * max(1, n)
    steps, first = (ctypes.c_int * (3 * n + 3))(), (ctypes.c_int * (n + 2))()
    c = shim.kda_test_rows_plan(A(*dst), A(*src), n, int(in_place), steps, first)
    if c < 0:
        return None
    total = first[c] if n else 0
    pairs = [(steps[2 * i], steps[2 * i + 1]) for i in range(total)]
    return [pairs[first[i]:first[i + 1]] for i in range(c)]


def apply(chains, pool, source):
    """The chains one after another in the given order, as a thread makes them; source may be pool."""
    for chain in chains:
        saved = None
        for s, d in chain:
            x = saved if s == -2 else 0 if s == -1 else source[s]
            if d == -3:
                saved = x
            else:
                pool[d] = x


def check(shim, dst, src, rows, rng, in_place=True):
    chains = plan(shim, dst, src, in_place)
    old = [100 + i for i in range(rows)]
    want = list(old) if in_place else [0] * rows
    for d, s in zip(dst, src):
        want[d] = old[s] if s >= 0 else 0
    for _ in range(3):   # the chains run in any order
        pool = list(old) if in_place else [0] * rows
        apply(chains, pool, pool if in_place else old)
        assert pool == want, (dst, src)
        rng.shuffle(chains)
    steps = sum(len(c) for c in chains)
    assert steps <= len(dst) + len(dst) // 2     # the table's size
    assert all(chains) and len(chains) <= max(1, len(dst))


def test_plan_of_row_moves(shim):
    rng = random.Random(5)
    check(shim, [], [], 4, rng)
    check(shim, [0, 1], [1, 0], 4, rng)
    check(shim, [3, 1, 2], [3, 2, 1], 4, rng)
    check(shim, [0, 1, 2, 3], [1, 2, 3, 0], 5, rng)
    for _ in range(3000):
        rows = rng.randint(1, 12)
        n = rng.randint(1, rows)
        dst = rng.sample(range(rows), n)
        check(shim, dst, [rng.randint(-1, rows - 1) for _ in dst], rows, rng)
        check(shim, dst, [rng.randint(-1, rows - 1) for _ in dst], rows, rng, in_place=False)
    for rows in (1024,):
        p = list(range(rows))
        rng.shuffle(p)
        check(shim, list(range(rows)), p, rows, rng)
        check(shim, list(range(rows)), [i ^ 1 for i in range(rows)], rows, rng)   # the most steps
        check(shim, list(range(1, rows)), [0] * (rows - 1), rows, rng)
    assert plan(shim, [1, 1], [0, 2]) is None


def test_plan_reads_a_forked_row_once(shim):
    """The copies of one row follow one another, so that the kernel keeps the row in registers."""
    chains = plan(shim, [4, 9, 5, 8, 6, 7], [0, 1, 0, 1, 0, 1])
    assert len(chains) == 2
    assert all(len({s for s, _ in c}) == 1 and len(c) == 3 for c in chains)


@pytest.fixture(scope="module")
def lib():
    from linear_attention_layer_kda_b200 import binding, build
    build.build()
    return binding.load()


def desc(**over):
    from linear_attention_layer_kda_b200 import binding as B
    d = B.kda_scan_desc()
    kw = dict(num_heads=2, head_dk=128, head_dv=64, dtype=B.KDA_DTYPE_BF16, nseq=2, rows=200)
    kw.update(over)
    for n, x in kw.items():
        if n == "reserved":
            d.reserved[0] = x
        else:
            setattr(d, n, x)
    return d


BAD_DESC = [(dict(num_heads=0), "S"), (dict(num_heads=513), "S"), (dict(head_dk=96), "S"), (dict(head_dv=256), "S"),
            (dict(dtype=2), "I"), (dict(nseq=0), "S"), (dict(nseq=65536), "S"), (dict(rows=-2), "S"),
            (dict(rows=2 ** 31), "S"), (dict(reserved=1), "I"), (dict(ld_q=255), "I"), (dict(ld_v=129), "I"),
            (dict(ld_b=1), "I"), (dict(ld_z=2 ** 31), "I"), (dict(rows=2 ** 31 - 2, num_heads=512), "S")]


def test_scan_workspace_and_bad_shapes(lib):
    from linear_attention_layer_kda_b200 import binding as B
    assert B.kda_scan_workspace_bytes(desc(), False, False) > 0
    assert B.kda_scan_workspace_bytes(desc(), True, True) > B.kda_scan_workspace_bytes(desc(), True, False)
    assert B.kda_scan_workspace_bytes(desc(rows=2), False, False) == 0      # token by token
    assert B.kda_scan_workspace_bytes(desc(rows=0), False, False) == 0
    code = {"S": B.KDA_ERR_UNSUPPORTED_SHAPE, "I": B.KDA_ERR_INVALID_ARG}
    for over, want in BAD_DESC:
        with pytest.raises(B.KdaError) as ei:
            B.kda_scan_workspace_bytes(desc(**over), False, False)
        assert ei.value.status == code[want], over
    with pytest.raises(B.KdaError):
        B.kda_scan_workspace_bytes(desc(rows=201), False, False)            # not one length
    assert B.kda_scan_workspace_bytes(desc(rows=201), True, False) > 0
    n = ctypes.c_size_t(7)
    assert lib.kda_scan_workspace_bytes(None, 0, 0, ctypes.byref(n)) == B.KDA_ERR_INVALID_ARG
    assert lib.kda_scan_workspace_bytes(ctypes.byref(desc()), 0, 0, None) == B.KDA_ERR_INVALID_ARG
    for rows, hidden in ((-1, 128), (4, 0), (4, 100), (4, 65536 + 128), (2 ** 31, 128)):
        with pytest.raises(B.KdaError) as ei:
            B.kda_residual_norm_workspace_bytes(rows, hidden)
        assert ei.value.status == B.KDA_ERR_UNSUPPORTED_SHAPE


# addresses that no call reaches: on a machine without a GPU a call that passes the checks stops at the device
A = [1 << 40 | i << 32 for i in range(1, 24)]


def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the accepted calls would run")


def test_scan_arguments_without_a_gpu(lib):
    no_gpu()
    from linear_attention_layer_kda_b200 import binding as B
    big = 1 << 30

    def forward(d=None, **over):
        kw = dict(q=A[0], k=A[1], v=A[2], z=A[3], b=A[4], cu_seqlens=None, state0=A[5], o=A[6], state_out=A[7],
                  workspace=A[8], workspace_bytes=big, stream=None)
        kw.update(over)
        with pytest.raises(B.KdaError) as ei:
            B.kda_scan_forward(d or desc(), **kw)
        return ei.value.status

    def backward(d=None, **over):
        kw = dict(q=A[0], k=A[1], v=A[2], z=A[3], b=A[4], cu_seqlens=None, state0=A[5], go=A[6], dstate_out=A[7],
                  dq=A[8], dk=A[9], dv=A[10], dz=A[11], db=A[12], dstate0=A[13], workspace=A[14],
                  workspace_bytes=big, stream=None)
        kw.update(over)
        with pytest.raises(B.KdaError) as ei:
            B.kda_scan_backward(d or desc(), **kw)
        return ei.value.status

    OK, BAD = B.KDA_ERR_NO_DEVICE, B.KDA_ERR_INVALID_ARG
    assert forward() == OK and backward() == OK
    assert forward(state0=None, cu_seqlens=A[9]) == OK
    assert forward(state_out=A[5]) == OK and backward(dstate0=A[7]) == OK       # in place
    assert backward(state0=None, dstate_out=None, dstate0=None) == OK
    assert forward(desc(rows=0), q=None, k=None, v=None, z=None, b=None, o=None, workspace=None) == OK
    for name in ("q", "k", "v", "z", "b", "o", "state_out", "workspace"):
        assert forward(**{name: None}) == BAD, name
    for name in ("q", "k", "v", "z", "b", "go", "dq", "dk", "dv", "dz", "db", "workspace"):
        assert backward(**{name: None}) == BAD, name
    for name in ("q", "k", "v", "z", "state0", "o", "state_out", "workspace"):
        assert forward(**{name: A[20] + 8}) == BAD, name
    for name in ("go", "dstate_out", "dq", "dk", "dv", "dz", "dstate0", "workspace"):
        assert backward(**{name: A[20] + 8}) == BAD, name
    assert forward(b=A[4] + 1) == BAD and forward(b=A[4] + 2) == OK and backward(db=A[12] + 1) == BAD
    assert forward(cu_seqlens=A[9] + 2) == BAD
    need = B.kda_scan_workspace_bytes(desc(), False, False)
    assert forward(workspace_bytes=need) == OK and forward(workspace_bytes=need - 1) == BAD
    need = B.kda_scan_workspace_bytes(desc(), False, True)
    assert backward(workspace_bytes=need) == OK and backward(workspace_bytes=need - 1) == BAD
    # overlaps
    assert forward(o=A[2]) == BAD and forward(o=A[2] + 16) == BAD and forward(state_out=A[5] + 16) == BAD
    assert forward(state_out=A[6]) == BAD and forward(workspace=A[3]) == BAD
    assert forward(cu_seqlens=A[9], o=A[9] + 256 - 256) == BAD
    assert backward(dq=A[0]) == BAD and backward(dk=A[8]) == BAD and backward(dv=A[6]) == BAD
    assert backward(dstate0=A[5]) == BAD and backward(dstate0=A[7] + 16) == BAD
    # columns of one projection: inputs may interleave, and an output may not lie between their columns
    wide = desc(ld_q=1024, ld_k=1024)
    assert forward(wide, k=A[0] + 512) == OK and forward(wide, o=A[0] + 1024) == BAD


def test_norm_arguments_without_a_gpu(lib):
    no_gpu()
    from linear_attention_layer_kda_b200 import binding as B

    def norm(**over):
        kw = dict(rows=4, hidden=256, x=A[0], x_dtype=1, residual=A[1], residual_dtype=1, weight=A[2], eps=1e-6,
                  residual_out=A[3], y=A[4], y8=A[5], scale=A[6], rstd=A[7], stream=None)
        kw.update(over)
        with pytest.raises(B.KdaError) as ei:
            B.kda_residual_norm(**kw)
        return ei.value.status

    def grad(**over):
        kw = dict(rows=4, hidden=256, dy=A[0], residual=A[1], residual_dtype=1, weight=A[2], rstd=A[3], dresidual=A[4],
                  dresidual_out=A[5], dweight=A[6], workspace=A[7], workspace_bytes=1 << 30, stream=None)
        kw.update(over)
        with pytest.raises(B.KdaError) as ei:
            B.kda_residual_norm_backward(**kw)
        return ei.value.status

    OK, BAD, SHAPE = B.KDA_ERR_NO_DEVICE, B.KDA_ERR_INVALID_ARG, B.KDA_ERR_UNSUPPORTED_SHAPE
    assert norm() == OK and grad() == OK
    assert norm(residual_out=A[1]) == OK and norm(residual_out=A[0]) == OK and norm(residual=None, y=None) == OK
    assert norm(y8=None, scale=None, rstd=None) == OK
    assert norm(residual_out=A[0], x_dtype=0) == BAD            # another type's bytes
    assert norm(y8=None) == BAD and norm(scale=None) == BAD and norm(weight=None) == BAD and norm(x=None) == BAD
    assert norm(residual_out=None) == BAD and norm(eps=-1e-9) == BAD and norm(eps=float("nan")) == BAD
    assert norm(hidden=200) == SHAPE and norm(rows=-1) == SHAPE and norm(x_dtype=3) == BAD
    for name in ("x", "residual", "weight", "residual_out", "y"):
        assert norm(**{name: A[20] + 8}) == BAD, name
    assert norm(y8=A[5] + 8) == OK and norm(y8=A[5] + 4) == BAD
    assert norm(y=A[0]) == BAD and norm(y=A[3]) == BAD and norm(y8=A[2]) == BAD and norm(residual_out=A[1] + 16) == BAD
    assert grad(dresidual=None) == OK
    assert grad(dresidual_out=A[4]) == OK and grad(dresidual_out=A[0]) == OK
    for name in ("dy", "residual", "weight", "rstd", "dresidual_out", "dweight"):
        assert grad(**{name: None}) == BAD, name


def test_rows_arguments_without_a_gpu(lib):
    no_gpu()
    from linear_attention_layer_kda_b200 import binding as B

    def rows(dst, src, **over):
        kw = dict(dst_pool=A[0], dst_rows=8, src_pool=A[0], src_rows=8, row_bytes=64, stream=None)
        kw.update(over)
        with pytest.raises(B.KdaError) as ei:
            B.kda_state_rows(dst=dst, src=src, **kw)
        return ei.value.status

    OK, BAD, SHAPE = B.KDA_ERR_NO_DEVICE, B.KDA_ERR_INVALID_ARG, B.KDA_ERR_UNSUPPORTED_SHAPE
    assert rows([0, 1], [1, 0]) == OK and rows([0], [-1]) == OK
    assert rows([0], [2], src_pool=A[1], src_rows=3) == OK and rows([0], [3], src_pool=A[1], src_rows=3) == BAD
    assert rows([8], [0]) == BAD and rows([-1], [0]) == BAD and rows([0], [8]) == BAD and rows([0], [-2]) == BAD
    assert rows([0, 0], [1, 2]) == BAD and rows(list(range(1025)), [0] * 1025, dst_rows=2000) == BAD
    assert rows([0], [1], row_bytes=0) == SHAPE and rows([0], [1], row_bytes=24) == SHAPE
    assert rows([0], [1], row_bytes=1 << 41) == SHAPE
    assert rows([0], [1], src_pool=A[0] + 64) == BAD and rows([0], [1], dst_pool=None) == BAD
    assert rows([0], [1], dst_pool=A[0] + 8, src_pool=A[0] + 8) == BAD
    with pytest.raises(ValueError, match="same length"):
        B.kda_state_rows(A[0], 8, A[0], 8, 64, [0, 1], [1], None)


def test_operators_refuse_cpu_tensors():
    import torch
    from linear_attention_layer_kda_b200 import operators as K
    t = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        K.scan_forward(t, t, t, t, t[:, :, 0])
    with pytest.raises(ValueError, match="CUDA"):
        K.scan_backward(t, t, t, t, t[:, :, 0], t)
    with pytest.raises(ValueError, match="CUDA"):
        K.residual_norm(t[0], t[0], t[0, 0])
    with pytest.raises(ValueError, match="CUDA"):
        K.state_rows(t, [0], [1])

"""CPU-side checks of libhqq_layers.so: it exports exactly what include/hqq_layers.h declares,
the header compiles as C and C++, workspace sizes, and every invalid argument is refused on the
host before any HIP call (no GPU is needed; no compute call is made here)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hqq_layers.h")

NBITS, GROUP, SHAPE, PTR, DTYPE, ACT, WORKSPACE = -1, -3, -4, -5, -8, -10, -11
# fake, 16-byte aligned, never dereferenced: every call below fails validation first
A, MIS, MIS4 = 0x1000, 0x1008, 0x1002


@pytest.fixture(scope="module")
def w():
    import weight_quantization_group_amd as w

    if not os.path.exists(w.LAYERS_LIB_PATH):
        pytest.fail(f"{w.LAYERS_LIB_PATH} is not built (run __graft_entry__.build())")
    w.load_layers_library()
    return w


@pytest.fixture(scope="module")
def lib(w):
    return w.load_layers_library()


def test_exports_exactly_the_header(w):
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"^HQQ_API (?:int|int64_t|const char \*)\s*(hqq_\w+)\s*\(", text, re.M)))
    assert declared == sorted(w.LAYERS_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", w.LAYERS_LIB_PATH], capture_output=True, text=True).stdout
    assert sorted(line.split()[-1] for line in out.splitlines() if " T " in line) == declared


@pytest.mark.parametrize("lang,compiler", [("c", "gcc"), ("c++", "g++")])
def test_header_compiles_cleanly(lang, compiler, tmp_path):
    if shutil.which(compiler) is None:
        pytest.skip(f"{compiler} not installed")
    src = tmp_path / ("use." + ("c" if lang == "c" else "cpp"))
    src.write_text('#include "hqq_layers.h"\nint main(void) { return hqq_linear_gated_workspace(1, 32, 1, 4, 32) < 0; }\n')
    r = subprocess.run([compiler, "-fsyntax-only", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_strerror(w):
    text = open(HEADER).read()
    for name, code in (("HQQ_EINVAL_ACT", ACT), ("HQQ_EWORKSPACE", WORKSPACE)):
        assert int(re.search(rf"#define {name} \((-\d+)\)", text).group(1)) == code
    for code in (0, NBITS, GROUP, SHAPE, PTR, -7, DTYPE, ACT, WORKSPACE):
        assert w.hqq_layers_strerror(code) != "unknown status"
    assert w.hqq_layers_strerror(12345) == "unknown status"


SIZES = [
    (dict(nbits=3), NBITS), (dict(nbits=16), NBITS),
    (dict(M=0), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(K=0), SHAPE), (dict(K=48), SHAPE),
    (dict(K=1 << 18), SHAPE), (dict(N=0), SHAPE), (dict(N=-3), SHAPE), (dict(N=1 << 40), SHAPE),
    (dict(N=(1 << 22) + 1), SHAPE),
    (dict(N=1 << 20, K=4096, gs=256), SHAPE),               # the codes take 2^31 bytes
    (dict(N=1 << 20, K=4096, gs=8, nbits=1), SHAPE),        # the meta does
    (dict(gs=48), GROUP), (dict(gs=4), GROUP), (dict(gs=512, K=512), GROUP), (dict(K=96, gs=64), GROUP),
]


def weight(w, packed=A, scale=A, zero=A):
    from weight_quantization_group_amd.layers import HqqWeight
    return HqqWeight(packed, scale, zero)


def gated(w, lib, X=A, gate=A, up=A, Y=A, M=4, K=128, N=40, nbits=4, gs=64, dtype=0, act=0, ws=A, size=1 << 40):
    g = ctypes.byref(weight(w, gate)) if gate else None
    u = ctypes.byref(weight(w, up)) if up else None
    return lib.hqq_linear_gated(X, M, K, g, u, N, nbits, gs, dtype, act, Y, ws, size, None)


def gated_backward(w, lib, dY=A, X=A, gate=A, up=A, dX=A, M=4, K=128, N=40, nbits=4, gs=64, dtype=0, act=0, ws=A,
                   size=1 << 40):
    g = ctypes.byref(weight(w, gate)) if gate else None
    u = ctypes.byref(weight(w, scale=up)) if up else None
    return lib.hqq_linear_gated_backward(dY, X, M, K, g, u, N, nbits, gs, dtype, act, dX, ws, size, None)


def batch_backward(w, lib, dY=A, packed=A, scale=A, zero=A, dX=A, count=2, M=4, K=128, N=40, nbits=4, gs=64, dtype=0,
                   ws=A, size=1 << 40, array=True):
    from weight_quantization_group_amd.layers import HqqLinearGrad
    arr = (HqqLinearGrad * 32)(*[HqqLinearGrad(A, A, A, 40, A)] * 32)
    arr[1] = HqqLinearGrad(packed, scale, zero, N, dY)      # the second one is the bad one
    return lib.hqq_linear_batch_backward(arr if array else None, count, M, K, nbits, gs, dtype, dX, ws, size, None)


def loss(w, lib, X=A, head=A, targets=A, loss=A, lse=A, M=4, K=128, N=40, nbits=4, gs=64, dtype=0, ws=A,
         size=1 << 40):
    h = ctypes.byref(weight(w, zero=head)) if head else None
    return lib.hqq_linear_cross_entropy(X, M, K, h, N, nbits, gs, dtype, targets, loss, lse, ws, size, None)


def loss_backward(w, lib, dloss=A, X=A, head=A, targets=A, lse=A, dX=A, M=4, K=128, N=40, nbits=4, gs=64, dtype=0,
                  ws=A, size=1 << 40):
    h = ctypes.byref(weight(w, head)) if head else None
    return lib.hqq_linear_cross_entropy_backward(dloss, X, M, K, h, N, nbits, gs, dtype, targets, lse, dX, ws, size, None)


CALLS = [gated, gated_backward, batch_backward, loss, loss_backward]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw,code", SIZES + [(dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
                                             (dict(ws=MIS), PTR), (dict(ws=None), PTR), (dict(size=-1), PTR),
                                             (dict(M=400, size=0), WORKSPACE), (dict(M=400, ws=None, size=0), WORKSPACE)])
def test_rejects(w, lib, call, kw, code):
    assert call(w, lib, **kw) == code


@pytest.mark.parametrize("call,names", [
    (gated, ["X", "gate", "up", "Y"]), (gated_backward, ["dY", "X", "gate", "up", "dX"]),
    (batch_backward, ["dY", "packed", "scale", "zero", "dX"]), (loss, ["X", "head"]),
    (loss_backward, ["X", "head", "dX"])], ids=lambda v: getattr(v, "__name__", ""))
def test_rejects_pointers(w, lib, call, names):
    for name in names:
        assert call(w, lib, **{name: None}) == PTR, name
        assert call(w, lib, **{name: MIS}) == PTR, name


def test_rejects_row_arrays(w, lib):
    """targets need 8-byte alignment, the fp32 rows 4."""
    for call, names in ((loss, ["targets", "loss", "lse"]), (loss_backward, ["targets", "lse", "dloss"])):
        for name in names:
            assert call(w, lib, **{name: None}) == PTR
            assert call(w, lib, **{name: MIS4}) == PTR
        assert call(w, lib, targets=0x1004) == PTR


def test_rejects_overlapping_outputs(w, lib):
    """An output that shares bytes with an input, the other output or the workspace."""
    far = [0x10000000 * i for i in range(1, 7)]
    M, K, N = 4, 128, 40
    need = w.hqq_linear_gated_backward_workspace(M, K, N, 4, 64)
    x, y, ws = far[0], far[1], far[2]
    assert gated(w, lib, X=x, Y=x + 2 * M * K - 16, ws=ws) == PTR
    assert gated(w, lib, X=x, Y=x - 2 * M * N + 16, ws=ws) == PTR
    for dX in (x, y, x + 2 * M * K - 16, y - 2 * M * K + 16, ws + need - 16):
        assert gated_backward(w, lib, dY=y, X=x, dX=dX, ws=ws) == PTR
    for dX in (A, y, y + 2 * M * N - 16):                  # A: the first weight's dY
        assert batch_backward(w, lib, dY=y, dX=dX, ws=ws) == PTR
    t = far[3]
    for out in (dict(loss=x, lse=y), dict(loss=y, lse=t + 8 * M - 4), dict(loss=y, lse=y + 4 * M - 4), dict(loss=ws, lse=y)):
        assert loss(w, lib, X=x, targets=t, ws=ws, **out) == PTR
    for dX in (x, t, far[4], far[5]):
        assert loss_backward(w, lib, X=x, targets=t, dloss=far[4], lse=far[5], dX=dX, ws=ws) == PTR


def test_rejects_activation_and_counts(w, lib):
    for call in (gated, gated_backward):
        assert call(w, lib, act=3) == ACT and call(w, lib, act=-1) == ACT
    assert batch_backward(w, lib, count=0) == SHAPE
    assert batch_backward(w, lib, count=17) == SHAPE
    assert batch_backward(w, lib, count=-1) == SHAPE
    assert batch_backward(w, lib, array=False) == PTR


def test_workspace_sizes(w):
    """One byte less than stated is refused; invalid sizes raise; sizes stay far below the logits'
    for long batches over large vocabularies."""
    sizes = (37, 1056, 2753, 2, 32)
    assert w.hqq_linear_gated_workspace(1, 1056, 2753, 2, 32) == 0       # straight from the codes
    for call, fn in ((gated, w.hqq_linear_gated_workspace), (gated_backward, w.hqq_linear_gated_backward_workspace),
                     (loss, w.hqq_linear_cross_entropy_workspace),
                     (loss_backward, w.hqq_linear_cross_entropy_backward_workspace)):
        need = fn(*sizes)
        if need:
            assert call(w, w.load_layers_library(), M=37, K=1056, N=2753, nbits=2, gs=32, size=need - 1) == WORKSPACE
        with pytest.raises(w.LayersError):
            fn(37, 1056, 2753, 3, 32)
    assert w.hqq_linear_batch_backward_workspace(500, 128, [40, 7], 4, 64) > 0
    with pytest.raises(w.LayersError):
        w.hqq_linear_batch_backward_workspace(5, 128, [], 4, 64)
    with pytest.raises(w.LayersError):
        w.hqq_linear_batch_backward_workspace(5, 128, [40] * 17, 4, 64)
    M, K, N = 65536, 4096, 128000
    logits = 2 * M * N
    assert w.hqq_linear_cross_entropy_workspace(M, K, N, 4, 64) < logits / 16
    assert w.hqq_linear_cross_entropy_backward_workspace(M, K, N, 4, 64) < logits / 16


def test_forced_route_keeps_to_its_rows(w, monkeypatch):
    """HQQ_LAYERS_PATH=codes holds up to 256 rows; beyond, the tiled route's workspace is asked for."""
    def need(M):
        return w.hqq_linear_gated_workspace(M, 1056, 2753, 2, 32)

    monkeypatch.setenv("HQQ_LAYERS_PATH", "codes")
    assert need(256) == 0 and need(1) == 0
    codes = need(257), need(1 << 20)
    monkeypatch.setenv("HQQ_LAYERS_PATH", "tiled")
    assert need(1) > 0 and codes == (need(257), need(1 << 20))


def test_workspace_holds_no_sums_that_one_launch_keeps(w):
    """A product that is not split takes no room for partial sums: W_hat alone, rows apart by K + 64."""
    K = N = 4096
    assert w.hqq_linear_batch_backward_workspace(4096, K, [N], 4, 64) == N * (K + 64) * 2


def test_binding_refuses_host_tensors(w):
    import torch

    X = torch.zeros(4, 128, dtype=torch.float16)
    q = (torch.zeros(40, 16, dtype=torch.int32), torch.zeros(40, 2), torch.zeros(40, 2))
    t = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: w.hqq_linear_gated(X, q, q, 40, 4, 64), lambda: w.hqq_linear_gated_backward(X, X, q, q, 40, 4, 64),
                 lambda: w.hqq_linear_backward(X, *q, 128, 4, 64),
                 lambda: w.hqq_linear_cross_entropy(X, t, *q, 40, 4, 64),
                 lambda: w.hqq_linear_cross_entropy_backward(t.float(), X, t, t.float(), *q, 40, 4, 64)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        w.hqq_linear_batch_backward([], [], 128, 4, 64)


def test_batch_width_limit(w, lib):
    """Every width may be within its limit and their sum beyond the batch's."""
    from weight_quantization_group_amd.layers import HqqLinearGrad
    N = 1 << 22
    arr = (HqqLinearGrad * 3)(*[HqqLinearGrad(A, A, A, N, A)] * 3)
    assert lib.hqq_linear_batch_backward(arr, 3, 1, 32, 1, 32, 0, A, A, 1 << 40, None) == SHAPE
    assert lib.hqq_linear_batch_backward(arr, 2, 400, 32, 1, 32, 0, A, A, 0, None) == WORKSPACE


def test_binding_checks_the_shape_of_a_tensor_given_twice(w):
    """The tensor that sets a call's dtype and device has to fit like any other: the first gradient
    of a batch, or X given again as the gradient of an output of another width."""
    import torch
    from weight_quantization_group_amd.layers import _matrix

    t = torch.zeros(4, 5, dtype=torch.float16)
    for rows, cols in ((4, 500), (4, 4), (5, 5)):
        with pytest.raises(ValueError):
            _matrix(t, "dYs", rows, cols, t)


@pytest.mark.parametrize("route", ["codes", "tiled"])
def test_rejects_writes_over_weights_and_inputs(w, lib, monkeypatch, route):
    """Outputs over a weight's codes, scales or zeros, and a workspace over any input: refused."""
    monkeypatch.setenv("HQQ_LAYERS_PATH", route)
    from weight_quantization_group_amd.layers import HqqLinearGrad
    x, y, o, p, s, z, t, ws = [0x10000000 * i for i in range(1, 9)]
    M, K, N, fmt = 40, 128, 40, (4, 64)
    codes, meta = N * K // 2, N * (K // 64) * 4
    big = 1 << 40
    first, other = weight(w, 0x7000000, 0x8000000, 0x9000000), weight(w, p, s, z)
    f, g = ctypes.byref(first), ctypes.byref(other)
    grads = (HqqLinearGrad * 2)(HqqLinearGrad(0x7000000, 0x8000000, 0x9000000, N, y + 4096 * 16), HqqLinearGrad(p, s, z, N, y))
    sizes = (M, K, N, *fmt)

    def gated_call(out, work):
        return lib.hqq_linear_gated(x, M, K, f, g, N, *fmt, 0, 0, out, work, big, None)

    def gated_grad(out, work):
        return lib.hqq_linear_gated_backward(y, x, M, K, g, f, N, *fmt, 0, 0, out, work, big, None)

    def batch(out, work):
        return lib.hqq_linear_batch_backward(grads, 2, M, K, *fmt, 0, out, work, big, None)

    def loss_call(out, work):
        return lib.hqq_linear_cross_entropy(x, M, K, g, N, *fmt, 0, t, o, out, work, big, None)

    def loss_grad(out, work):
        return lib.hqq_linear_cross_entropy_backward(t + 4096, x, M, K, g, N, *fmt, 0, t, t + 8192, out, work, big, None)

    def last(base, size):
        return base + (size - 1) // 16 * 16

    calls = {gated_call: (w.hqq_linear_gated_workspace(*sizes), {x: 2 * M * K}),
             gated_grad: (w.hqq_linear_gated_backward_workspace(*sizes), {x: 2 * M * K, y: 2 * M * N}),
             batch: (w.hqq_linear_batch_backward_workspace(M, K, [N, N], *fmt), {y: 2 * M * N, y + 4096 * 16: 2 * M * N}),
             loss_call: (w.hqq_linear_cross_entropy_workspace(*sizes), {x: 2 * M * K, t: 8 * M}),
             loss_grad: (w.hqq_linear_cross_entropy_backward_workspace(*sizes),
                         {x: 2 * M * K, t: 8 * M, t + 4096: 4 * M, t + 8192: 4 * M})}
    for call, (need, inputs) in calls.items():
        for base, size in ((p, codes), (s, meta), (z, meta)):
            assert call(base, ws) == PTR and call(last(base, size), ws) == PTR, call.__name__
        for base, size in {**inputs, p: codes, s: meta, z: meta, o: 2 * M * N}.items():
            if need and (base != o or call in (gated_call, gated_grad, batch)):
                out = o if call is not loss_call else o + 4096
                assert call(out, base) == PTR and call(out, last(base, size)) == PTR, call.__name__
                assert call(out, base - (need - 16) // 256 * 256) == PTR, call.__name__


@pytest.mark.parametrize("name,K,N,gs,most", [
    # large enough that the rows alone decide: up to `most` rows straight from the codes
    ("gated", 2048, 10240, 64, 64), ("gated_backward", 2048, 10240, 64, 64), ("gated_backward", 2048, 10240, 32, 32),
    ("batch_backward", 2048, 20480, 64, 64), ("batch_backward", 2048, 20480, 32, 32),
    ("cross_entropy", 2048, 20480, 64, 64), ("cross_entropy_backward", 2048, 20480, 64, 32),
    # shallow
    ("gated_backward", 1024, 20480, 64, 32), ("cross_entropy", 1024, 20480, 64, 32),
    # more than 200 million weights
    ("gated", 8192, 14336, 64, 96), ("cross_entropy", 8192, 28672, 64, 96), ("cross_entropy_backward", 8192, 28672, 64, 64),
    ("batch_backward", 8192, 28672, 32, 64),
    # small: blocks of 32 rows times the weights
    ("gated", 512, 4000, 64, 160), ("gated_backward", 512, 4000, 64, 64), ("batch_backward", 512, 4000, 64, 64),
    ("cross_entropy", 512, 4000, 64, 160), ("cross_entropy_backward", 512, 4000, 64, 128), ("gated", 512, 1100, 64, 256),
])
def test_route_limits(w, monkeypatch, name, K, N, gs, most):
    """The rows up to which each operator runs straight from the codes by itself, seen by the workspace
    that it asks for beside those of the two forced routes."""
    def need(M):
        if name == "batch_backward":
            return w.hqq_linear_batch_backward_workspace(M, K, [N], 4, gs)
        return getattr(w, f"hqq_linear_{name}_workspace")(M, K, N, 4, gs)

    def forced(route, M):
        monkeypatch.setenv("HQQ_LAYERS_PATH", route)
        n = need(M)
        monkeypatch.delenv("HQQ_LAYERS_PATH")
        return n

    for M in (1, most, most + 1):
        codes, tiled = forced("codes", M), forced("tiled", M)
        if M <= 256:
            assert codes != tiled
        assert need(M) == (codes if M <= most else tiled), M

"""CPU-side checks of libhqq_cache.so: it exports exactly what include/hqq_cache.h declares, the
header compiles as C and C++, workspace sizes, and every invalid argument is refused on the host
before any HIP call (no GPU is needed; no compute call is made here)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hqq_cache.h")

NBITS, GROUP, SHAPE, PTR, PARAM, DTYPE, WORKSPACE = -1, -3, -4, -5, -6, -8, -11
# fake, 16-byte aligned, never dereferenced: every call below fails validation first
KP, KS, KZ, VP, VS, VZ, X, Y, S, O, P, T, L, W = [0x100000000 * i for i in range(1, 15)]


@pytest.fixture(scope="module")
def w():
    import weight_quantization_group_amd as w

    if not os.path.exists(w.CACHE_LIB_PATH):
        pytest.fail(f"{w.CACHE_LIB_PATH} is not built (run __graft_entry__.build())")
    w.load_cache_library()
    return w


@pytest.fixture(scope="module")
def lib(w):
    return w.load_cache_library()


def test_exports_exactly_the_header(w):
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"^HQQ_API (?:int|int64_t|const char \*)\s*(hqq_\w+)\s*\(", text, re.M)))
    assert declared == sorted(w.CACHE_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", w.CACHE_LIB_PATH], capture_output=True, text=True).stdout
    assert sorted(line.split()[-1] for line in out.splitlines() if " T " in line) == declared


@pytest.mark.parametrize("lang,compiler", [("c", "gcc"), ("c++", "g++")])
def test_header_compiles_cleanly(lang, compiler, tmp_path):
    if shutil.which(compiler) is None:
        pytest.skip(f"{compiler} not installed")
    src = tmp_path / ("use." + ("c" if lang == "c" else "cpp"))
    src.write_text('#include "hqq_cache.h"\n#include "hqq_layers.h"\n'
                   'int main(void) { return hqq_cache_attention_workspace(0, 1, 1, 1) < 0; }\n')
    r = subprocess.run([compiler, "-fsyntax-only", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_strerror(w):
    for code in (0, NBITS, GROUP, SHAPE, PTR, PARAM, -7, DTYPE, WORKSPACE):
        assert w.hqq_cache_strerror(code) != "unknown status"
    assert w.hqq_cache_strerror(12345) == "unknown status"


def cache(pages=10, page_size=16, heads=2, dim=128, nbits=4, gs=64, kp=KP, ks=KS, kz=KZ, vp=VP, vs=VS, vz=VZ):
    from weight_quantization_group_amd.cache import HqqCache, HqqCacheSide
    return HqqCache(HqqCacheSide(kp, ks, kz), HqqCacheSide(vp, vs, vz), pages, page_size, heads, dim, nbits, gs)


def write(lib, k=X, v=Y, tokens=4, slots=S, dtype=0, k_hat=None, v_hat=None, token=256, head=128, k_strides=None,
          v_strides=None, c=None, **kw):
    c = None if c == "none" else ctypes.byref(cache(**kw))
    return lib.hqq_cache_write(c, k, *(k_strides or (token, head)), v, *(v_strides or (token, head)), tokens, slots, dtype,
                               k_hat, v_hat, None)


def read(lib, k=X, v=Y, tokens=4, slots=S, dtype=0, c=None, **kw):
    return lib.hqq_cache_read(None if c == "none" else ctypes.byref(cache(**kw)), slots, tokens, dtype, k, v, None)


def attention(lib, q=X, batch=3, q_heads=4, table=T, width=80, lengths=L, scale=0.1, window=0, dtype=0, out=O, lse=P,
              ws=W, size=1 << 32, token=512, head=128, c=None, **kw):
    c = None if c == "none" else ctypes.byref(cache(**kw))
    return lib.hqq_cache_attention(c, q, token, head, batch, q_heads, table, width, lengths, scale, window, dtype,
                                   out, lse, ws, size, None)


LAYOUTS = [
    (dict(nbits=1), NBITS), (dict(nbits=3), NBITS), (dict(nbits=16), NBITS),
    (dict(dim=0), SHAPE), (dict(dim=80, gs=16), SHAPE), (dict(dim=32, gs=32), SHAPE), (dict(dim=512, gs=256), SHAPE),
    (dict(dim=-128), SHAPE),
    (dict(gs=0), GROUP), (dict(gs=16), GROUP), (dict(gs=48, dim=96), GROUP), (dict(gs=-64), GROUP), (dict(gs=256), GROUP),
    (dict(gs=32, dim=192), GROUP), (dict(gs=32, dim=256), GROUP), (dict(gs=64, dim=96), GROUP),
    (dict(page_size=0), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=2048), SHAPE),
    (dict(page_size=-16), SHAPE), (dict(pages=0), SHAPE), (dict(pages=-1), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(pages=1 << 62), SHAPE), (dict(pages=1 << 28, heads=1024, page_size=1024), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(heads=-2), SHAPE),
    (dict(c="none"), PTR), (dict(kp=None), PTR), (dict(ks=KS + 8), PTR), (dict(kz=None), PTR), (dict(vp=VP + 4), PTR),
    (dict(vs=None), PTR), (dict(vz=VZ + 8), PTR), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
]


@pytest.mark.parametrize("call", [write, read, attention], ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw,code", LAYOUTS)
def test_rejects_layouts(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 25) + 1), SHAPE), (dict(tokens=1 << 62), SHAPE),
    (dict(k=None), PTR), (dict(v=None), PTR), (dict(k=X + 2), PTR), (dict(v=Y + 8), PTR), (dict(slots=None), PTR),
    (dict(slots=S + 4), PTR), (dict(k_hat=O), PTR), (dict(v_hat=O), PTR), (dict(k_hat=O + 8, v_hat=P), PTR),
    (dict(token=4), SHAPE), (dict(token=-256), SHAPE), (dict(head=12), SHAPE), (dict(head=-8), SHAPE),
    (dict(token=1 << 62), SHAPE), (dict(head=1 << 40), SHAPE),
    (dict(k_strides=(260, 128)), SHAPE), (dict(v_strides=(256, 130)), SHAPE),
])
def test_write_rejects(lib, kw, code):
    assert write(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 25) + 1), SHAPE), (dict(k=None), PTR), (dict(v=None), PTR),
    (dict(k=X + 8), PTR), (dict(slots=None), PTR), (dict(slots=S + 4), PTR), (dict(v=X), PTR), (dict(v=X + 2032), PTR),
    (dict(k=KP), PTR), (dict(k=VZ), PTR), (dict(v=S), PTR),
])
def test_read_rejects(lib, kw, code):
    assert read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), SHAPE), (dict(batch=(1 << 15) + 1), SHAPE), (dict(q_heads=0), SHAPE), (dict(q_heads=3), SHAPE),
    (dict(q_heads=-2), SHAPE), (dict(q_heads=(1 << 16) + 2), SHAPE), (dict(batch=1 << 15, q_heads=1 << 14), SHAPE),
    (dict(width=0), SHAPE), (dict(width=-1), SHAPE), (dict(width=(1 << 26) + 1), SHAPE), (dict(batch=1 << 8, width=(1 << 25) + 1), SHAPE), (dict(width=1 << 62), SHAPE),
    (dict(scale=0.0), PARAM), (dict(scale=-1.0), PARAM), (dict(scale=float("nan")), PARAM),
    (dict(scale=float("inf")), PARAM), (dict(scale=3e38), PARAM), (dict(window=-1), PARAM),
    (dict(q=None), PTR), (dict(q=X + 2), PTR), (dict(q=X + 8), PTR), (dict(token=12), SHAPE), (dict(head=-8), SHAPE),
    (dict(table=None), PTR), (dict(table=T + 2), PTR), (dict(lengths=None), PTR), (dict(lengths=L + 1), PTR),
    (dict(out=None), PTR), (dict(out=O + 8), PTR), (dict(lse=P + 2), PTR), (dict(ws=None), PTR), (dict(ws=W + 8), PTR),
    (dict(size=-1), PTR), (dict(size=0), WORKSPACE), (dict(ws=None, size=0), WORKSPACE), (dict(size=4096), WORKSPACE),
])
def test_attention_rejects(lib, kw, code):
    assert attention(lib, **kw) == code


def test_a_call_of_nothing_needs_no_pointers(lib):
    assert write(lib, k=None, v=None, tokens=0, slots=None) == 0
    assert read(lib, k=None, v=None, tokens=0, slots=None) == 0
    assert attention(lib, q=None, batch=0, table=None, lengths=None, out=None, lse=None, ws=None, size=0) == 0
    # but a cache and a format
    assert write(lib, tokens=0, nbits=3) == NBITS and read(lib, tokens=0, kp=None) == PTR
    assert attention(lib, batch=0, q_heads=3) == SHAPE


def test_workspace(w, lib):
    """None where no sequence can exceed 768 tokens; else dim sums and two statistics per query head and
    segment: as many segments as runs (the chip's workgroups per key-value head) and sequences."""
    def need(batch, q_heads, width, **kw):
        return lib.hqq_cache_attention_workspace(ctypes.byref(cache(**kw)), batch, q_heads, width)

    assert need(3, 4, 48) == 0 and need(3, 4, 49) > 0 and need(0, 4, 49) == 0
    sizes = {need(b, 4, 100) for b in (1, 2, 3)}
    assert len(sizes) == 3 and max(sizes) - min(sizes) <= 2 * (4 * 128 * 4 + 4 * 8) + 512
    segments = (need(3, 4, 100) // (4 * 128 * 4 + 4 * 8))
    assert 256 // 2 + 3 <= segments <= 4 * 256 * 8 + 3
    for kw, code in LAYOUTS[:29]:
        assert need(3, 4, 9, **kw) == code
    assert lib.hqq_cache_attention_workspace(None, 3, 4, 9) == PTR
    assert need(3, 5, 9) == SHAPE and need(-1, 4, 9) == SHAPE and need(3, 4, 0) == SHAPE
    n = need(3, 4, 100)
    assert attention(lib, width=100, size=n - 1) == WORKSPACE
    # a cache's arrays are not needed to ask
    assert need(3, 4, 100, kp=None, vz=None) == n


def last(base, size):
    return base + (size - 1) // 16 * 16


def test_rejects_writes_over_what_is_read(lib):
    """Outputs over the cache, an input or one another: refused, at their first and last bytes."""
    n = 10 * 2 * 16
    arrays = [(KP, n * 64), (KS, n * 8), (KZ, n * 8), (VP, n * 64), (VS, n * 8), (VZ, n * 8)]
    row = 4 * 2 * 128 * 2
    for base, size in arrays + [(X, row), (Y, row), (S, 32)]:
        for at in (base, last(base, size), base - row + 16):
            assert write(lib, k_hat=at, v_hat=P) == PTR and write(lib, k_hat=P, v_hat=at) == PTR
    assert write(lib, k_hat=O, v_hat=last(O, row)) == PTR
    # a strided input reaches as far as its last row
    far = 3 * 4096 + 128
    assert write(lib, token=4096, k_hat=X + 2 * far, v_hat=P) == PTR
    assert write(lib, token=4096, head=256, k_hat=X + 2 * (far + 256) - 16, v_hat=P) == PTR
    for base, size in arrays:                      # tokens cut from the cache's own arrays
        assert write(lib, k=last(base, size)) == PTR and write(lib, v=base) == PTR
        assert write(lib, slots=base) == PTR
    for one, other in [("kp", "ks"), ("kp", "vp"), ("kz", "vz"), ("ks", "vs")]:      # one array for two
        at = dict(kp=KP, ks=KS, kz=KZ, vp=VP, vs=VS, vz=VZ)[one]
        assert write(lib, **{other: at}) == PTR
    for base, size in arrays + [(S, 32)]:
        for at in (base, last(base, size), base - row + 16):
            assert read(lib, k=at) == PTR and read(lib, v=at) == PTR
    q_row, table, ws = 3 * 4 * 128 * 2, 3 * 80 * 4, lib.hqq_cache_attention_workspace(ctypes.byref(cache()), 3, 4, 80)
    inputs = arrays + [(X, q_row), (T, table), (L, 12)]
    for base, size in inputs:
        for at in (base, last(base, size)):
            assert attention(lib, out=at) == PTR and attention(lib, lse=at) == PTR and attention(lib, ws=at) == PTR
        assert attention(lib, out=base - q_row + 16) == PTR
        assert attention(lib, ws=base - ws // 16 * 16 + 16) == PTR
    assert attention(lib, lse=O + q_row - 4) == PTR and attention(lib, ws=O) == PTR and attention(lib, ws=P) == PTR


def test_binding_refuses(w):
    import torch

    host = (torch.zeros(4, 2, 16, 16, dtype=torch.int32), torch.ones(4, 2, 16, 2), torch.zeros(4, 2, 16, 2))
    with pytest.raises(TypeError):
        w.QuantizedCache(host, host, 4, 64)
    with pytest.raises(TypeError):
        w.QuantizedCache.empty(4, 16, 2, 128, 4, 64, device="cpu")
    for bad in (dict(nbits=3), dict(group_size=0), dict(group_size=-64), dict(group_size=48)):
        with pytest.raises(ValueError):
            w.QuantizedCache.empty(4, 16, 2, 128, **{**dict(nbits=4, group_size=64, device="cpu"), **bad})


def test_imports_on_a_torch_without_a_gpu_runtime():
    """The package, its host-side checks and workspace sizes need none of torch's device functions."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:
    delattr(torch._C, name)
import weight_quantization_group_amd as w
for name in w.CACHE_EXPORTS:
    assert callable(getattr(w, name)), name
try:
    w.QuantizedCache.empty(4, 16, 2, 128, 4, 64, device='cpu')
    raise SystemExit('not refused')
except TypeError:
    pass
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr


def test_workspace_of_large_batches(w, lib):
    """A run has at most two parts of split sequences, however many sequences there are: beyond as many as runs,
    the workspace grows by the plan's number per sequence alone, and the largest admitted sizes have one that
    fits the card."""
    def need(batch, q_heads, width, **kw):
        return lib.hqq_cache_attention_workspace(ctypes.byref(cache(**kw)), batch, q_heads, width)

    for heads, q_heads, dim in ((8, 64, 128), (32, 32, 128), (1, 1, 64), (40, 680, 64), (2, 8192, 256)):
        kw = dict(heads=heads, dim=dim, gs=64)
        rows = q_heads * (dim * 4 + 8)
        workers = 4 * 256 * 2 // heads                          # more runs per key-value head than there are
        top = need(1 << 15, q_heads, 100, **kw)
        assert 2 * rows <= top <= 2 * workers * rows + 4 * (1 << 15) + 2048
        batch = 1 << 12
        assert need(2 * batch, q_heads, 100, **kw) - need(batch, q_heads, 100, **kw) == 4 * batch
    assert need(4096, 64, 100, heads=8) < 5 << 20               # 64 runs of 8 heads
    assert need(1 << 15, 1 << 13, 1 << 18, heads=1, dim=256) < 64 << 20


def test_runs_are_for_the_workgroups_that_fit(w, lib):
    """As many runs as the chip holds workgroups at a time: two a CU, but one where a workgroup takes more than
    half of a CU's shared memory (8 bits of 256 dims in groups of 64)."""
    def segments(gs, heads, dim=256, nbits=8):
        n = lib.hqq_cache_attention_workspace(ctypes.byref(cache(heads=heads, dim=dim, gs=gs, nbits=nbits)), 1, heads, 100)
        return n // (heads * (dim * 4 + 8))

    for heads in (1, 2, 4, 16):
        assert segments(64, heads) == 256 // heads + 1
        assert segments(128, heads) == segments(256, heads) == segments(64, heads, nbits=4) == 512 // heads + 1

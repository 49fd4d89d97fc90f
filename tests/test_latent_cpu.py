"""Host-side checks of the latent-attention entry points and wrappers: sizes
and refusals, all before any CUDA call."""

import ctypes
import os
import shutil
import subprocess
import sys

import pytest
import torch

from chunked_gated_delta_kda_gb300 import binding, latent

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-pointer validation cases run on CPU-only hosts")


def host_block():
    buf = (ctypes.c_uint8 * 4096)()
    return buf, ctypes.addressof(buf) + (-ctypes.addressof(buf) % 256)


def caller(fn, defaults):
    def call(**kw):
        assert set(kw) <= set(defaults), kw
        return fn(*{**defaults, **kw}.values())
    return call


def test_workspace_sizes():
    lib = binding.load_library()
    r256 = lambda b: (b + 255) // 256 * 256  # noqa: E731

    def bwd(slots, rows, H):   # header, two tables of 64 a tile slot and head, 64 floats a key and head
        return 256 + r256(slots * H * 128 * 4) + rows * H * 64 * 4

    assert lib.kda_latent_bwd_workspace_bytes(2, 2048, 2048, 8, 2) == bwd(64, 4096, 8)
    assert lib.kda_latent_bwd_workspace_bytes(1, 9192, 9192, 32, 6) == bwd(9192 // 64 + 6, 9192, 32)
    assert lib.kda_latent_bwd_workspace_bytes(1, 0, 0, 1, 1) > 0
    for bad in ((0, 1, 1, 1, 1), (1, -1, 1, 1, 1), (1, 1, -1, 1, 1), (1, 1, 1, 0, 1), (1, 1, 1, 1, 0),
                (1, 1, 1, 65536, 1), (1 << 16, 1 << 16, 1, 1, 1)):
        assert lib.kda_latent_bwd_workspace_bytes(*bad) == 0

    def dec(n, rows):          # header, 152 error words, offsets, two parts a CTA
        return 256 + 768 + r256((n + 1) * 8) + r256(304 * rows * 4) + 304 * rows * 512 * 4

    assert lib.kda_latent_decode_workspace_bytes(1, 1, 16) == dec(1, 16)
    assert lib.kda_latent_decode_workspace_bytes(256, 1, 32) == dec(256, 32)
    assert lib.kda_latent_decode_workspace_bytes(3, 4, 128) == dec(3, 64)
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (65536, 1, 1), (65535, 65535, 2)):
        assert lib.kda_latent_decode_workspace_bytes(*bad) == 0


def test_status_string():
    assert b"page" in binding.load_library().kda_status_str(8)


@cpu_only
def test_fwd_refusals():
    keep, p = host_block()
    call = caller(binding.load_library().kda_latent_fwd, dict(
        q=p, kv=p, pe=p, stride=64, scale=0.0, cu_q=None, cu_k=None, o=p, lse=p, B=1, Tq=8, Tk=8, H=1, N=1, flags=0,
        ws=None, stream=None))
    for kw in (dict(q=None), dict(kv=None), dict(pe=None), dict(o=None), dict(q=p + 8), dict(kv=p + 2), dict(pe=p + 4),
               dict(o=p + 8), dict(lse=p + 2), dict(ws=p + 64), dict(stride=63), dict(stride=56), dict(stride=68),
               dict(B=0), dict(Tq=-1), dict(Tk=-1), dict(H=0), dict(N=0), dict(N=2), dict(H=65536), dict(cu_q=p),
               dict(cu_k=p), dict(cu_q=p, cu_k=p, B=2, N=2), dict(cu_q=p + 2, cu_k=p), dict(flags=1), dict(flags=512)):
        assert call(**kw) == 1, kw


@cpu_only
def test_bwd_refusals():
    keep, p = host_block()
    lib = binding.load_library()
    need = lib.kda_latent_bwd_workspace_bytes(1, 8, 8, 1, 1)
    call = caller(lib.kda_latent_bwd, dict(
        q=p, kv=p, pe=p, stride=64, o=p, lse=p, do=p, scale=0.0, cu_q=None, cu_k=None, dq=p, dkv=p, dpe=p, B=1, Tq=8,
        Tk=8, H=1, N=1, flags=0, ws=p, wsb=need, stream=None))
    for kw in (dict(q=None), dict(o=None), dict(lse=None), dict(do=None), dict(dq=None), dict(dkv=None), dict(dpe=None),
               dict(ws=None), dict(wsb=need - 1), dict(ws=p + 16), dict(o=p + 8), dict(do=p + 8), dict(dq=p + 8),
               dict(dkv=p + 8), dict(dpe=p + 8), dict(N=2), dict(stride=65), dict(flags=2)):
        assert call(**kw) == 1, kw


@cpu_only
def test_decode_refusals():
    keep, p = host_block()
    lib = binding.load_library()
    need = lib.kda_latent_decode_workspace_bytes(2, 1, 4)
    call = caller(lib.kda_latent_decode, dict(
        q=p, cache=p, pages=4, page=64, table=p, width=2, lens=p, scale=0.0, o=p, lse=p, N=2, S=1, H=4, flags=0, ws=p,
        wsb=need, stream=None))
    for kw in (dict(q=None), dict(cache=None), dict(table=None), dict(lens=None), dict(o=None), dict(ws=None),
               dict(pages=0), dict(width=0), dict(page=0), dict(page=8), dict(page=48), dict(page=96), dict(page=-64),
               dict(pages=1 << 26), dict(width=1 << 26), dict(N=0), dict(S=0), dict(H=0), dict(flags=256),
               dict(wsb=need - 1), dict(q=p + 8), dict(cache=p + 8), dict(table=p + 2), dict(lens=p + 1), dict(o=p + 8),
               dict(ws=p + 128)):
        assert call(**kw) == 1, kw


@cpu_only
def test_append_refusals():
    keep, p = host_block()
    call = caller(binding.load_library().kda_latent_append, dict(
        rows=p, stride=576, slots=p, weight=None, eps=1e-6, cache=p, num=64, T=1, flags=0, ws=None, stream=None))
    for kw in (dict(rows=None), dict(slots=None), dict(cache=None), dict(stride=575), dict(stride=580), dict(T=-1),
               dict(num=-1), dict(flags=256), dict(rows=p + 8), dict(slots=p + 4), dict(weight=p + 8), dict(cache=p + 2),
               dict(weight=p, eps=-1.0), dict(weight=p, eps=float("nan")), dict(ws=p + 4)):
        assert call(**kw) == 1, kw


@cpu_only
def test_tables_refusals():
    keep, p = host_block()
    call = caller(binding.load_library().kda_block_tables, dict(
        lens=p, new=p, table=p, width=2, free=p, num_free=1, head=p, page=16, slots=p, tokens=1, cu=p, out=p, head_out=p,
        N=1, ws=None, stream=None))
    for kw in (dict(lens=None), dict(new=None), dict(table=None), dict(free=None), dict(head=None), dict(slots=None),
               dict(cu=None), dict(out=None), dict(head_out=None), dict(N=0), dict(width=-1), dict(num_free=-1),
               dict(tokens=-1), dict(page=0), dict(page=24), dict(slots=p + 4), dict(lens=p + 2), dict(ws=p + 32)):
        assert call(**kw) == 1, kw


def test_wrappers_refuse_what_the_kernels_do_not_take():
    """CPU tensors, types, shapes: a clear error and no fallback."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d)  # noqa: E731
    i32 = torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        latent.latent_fwd(z(1, 4, 2, 192), z(1, 4, 2, 256), z(1, 4, 64))
    with pytest.raises(TypeError, match="bfloat16 or"):
        latent.latent_fwd(z(1, 4, 2, 192, d=torch.float32), z(1, 4, 2, 256), z(1, 4, 64))
    with pytest.raises(TypeError, match="torch.Tensor"):
        latent.latent_decode([1], z(1, 16, 576), z(1, 1, d=i32), z(1, d=i32))
    with pytest.raises(ValueError, match="CUDA"):
        latent.latent_decode(z(1, 1, 1, 576), z(1, 16, 576), z(1, 1, d=i32), z(1, d=i32))
    with pytest.raises(TypeError, match="rows must be"):
        latent.latent_append(z(1, 576, d=i32), z(1, d=torch.int64), z(1, 16, 576))
    with pytest.raises(ValueError, match="CUDA"):
        latent.latent_append(z(1, 576), z(1, d=torch.int64), z(1, 16, 576))
    with pytest.raises(ValueError, match="CUDA"):
        latent.block_tables(z(1, d=i32), z(1, d=i32), z(1, 1, d=i32), z(1, d=i32), z(1, d=i32), 16, 1)
    with pytest.raises(TypeError, match="seq_lens"):
        latent.block_tables(z(1, d=torch.int64), z(1, d=i32), z(1, 1, d=i32), z(1, d=i32), z(1, d=i32), 16, 1)


def test_wrappers_name_what_is_not_a_tensor():
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d)  # noqa: E731
    i32 = torch.int32
    for args in ((z(1, 1, 1, 576), None, z(1, 1, d=i32), z(1, d=i32)), (z(1, 1, 1, 576), z(1, 16, 576), [[0]], z(1, d=i32))):
        with pytest.raises((TypeError, ValueError), match="must be"):
            latent.latent_decode(*args)
    for bad in range(5):
        args = [z(1, d=i32), z(1, d=i32), z(1, 1, d=i32), z(1, d=i32), z(1, d=i32)]
        args[bad] = [0]
        with pytest.raises((TypeError, ValueError), match="must be"):
            latent.block_tables(*args, 16, 1)


def test_workspaces_and_scales_are_checked_before_the_launch():
    """A workspace elsewhere would be written through a host pointer; a scale that is not above zero would be taken
    for the default."""
    host = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="on cuda:0"):
        latent._status_workspace(host, 0)
    with pytest.raises(ValueError, match="on cuda:1"):
        latent._scratch(host, 256, 1, host.device)
    with pytest.raises(TypeError, match="workspace"):
        latent._scratch(4096, 256, 0, host.device)
    assert latent._status_workspace(None, 0) is None
    assert latent._scale(None) == -1.0 and latent._scale(0.25) == 0.25 and latent._scale(1) == 1.0
    for bad in (0.0, -0.5, float("nan"), float("inf"), 1e-50):
        with pytest.raises(ValueError, match="scale"):
            latent._scale(bad)


def test_fwd_workspace_sizes():
    """Records and 256 parts of 256 rows where packed sequences have 8192 keys or more; the status header elsewhere."""
    lib = binding.load_library()
    shared = 256 + 896 * 16 + 256 * 256 * 130 * 4
    assert lib.kda_latent_fwd_workspace_bytes(1, 1642, 16231, 16, 4) == shared
    assert lib.kda_latent_fwd_workspace_bytes(1, 64, 8192, 1, 30) == shared
    for sizes in ((1, 1642, 8191, 16, 4), (1, 9000, 9000, 8, 1), (2, 9000, 9000, 8, 2), (1, 1642, 16231, 129, 4),
                  (1, 8, 16384, 8, 2), (1, 200000, 200000, 8, 9), (1, 600, 600000, 1, 600), (1, 0, 0, 1, 1)):
        assert lib.kda_latent_fwd_workspace_bytes(*sizes) == 256, sizes
    assert lib.kda_latent_fwd_workspace_bytes(0, 1, 1, 1, 1) == 0


@cpu_only
def test_fwd_with_a_workspace_refusals():
    keep, p = host_block()
    call = caller(binding.load_library().kda_latent_fwd_ws, dict(
        q=p, kv=p, pe=p, stride=64, scale=0.0, cu_q=None, cu_k=None, o=p, lse=p, B=1, Tq=8, Tk=8, H=1, N=1, flags=0,
        ws=p, wsb=256, stream=None))
    for kw in (dict(q=None), dict(o=None), dict(wsb=255), dict(wsb=0), dict(ws=p + 64), dict(N=2), dict(flags=1)):
        assert call(**kw) == 1, kw


# A runtime whose n-th launch fails, in front of the real one: no GPU is needed, nothing runs.
FAKE_RUNTIME = r"""
static int count = 0, last = 0, fail_at = 0;
void fake_begin(int at) { count = last = 0; fail_at = at; }
int fake_launches(void) { return count; }
static int launched(void) { return ++count == fail_at ? (last = 719) : 0; }
int __cudaLaunchKernel(void) { return launched(); }
int cudaLaunchKernel(void) { return launched(); }
int cudaLaunchKernelExC(void) { return launched(); }
int __cudaGetKernel(void) { return 0; }
int cudaFuncSetAttribute(void) { return 0; }
int cudaMemsetAsync(void) { return 0; }
int cudaGetLastError(void) { int e = last; last = 0; return e; }
static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char* name, void** f, unsigned version, unsigned long long flags, int* found) {
    *f = (void*)encode; *found = 0; return 0;
}
"""
FAKE_CALLS = r"""
import ctypes
from chunked_gated_delta_kda_gb300 import binding
lib = binding.load_library()
buf = (ctypes.c_uint8 * 4096)()
p = ctypes.addressof(buf) + (-ctypes.addressof(buf) % 256)
big = 1 << 40
calls = dict(
    fwd=lambda: lib.kda_latent_fwd(p, p, p, 64, 0.0, None, None, p, p, 1, 64, 64, 2, 1, 0, None, None),
    fwd_shared=lambda: lib.kda_latent_fwd_ws(p, p, p, 64, 0.0, p, p, p, p, 1, 64, 8192, 1, 30, 0, p, big, None),
    bwd=lambda: lib.kda_latent_bwd(p, p, p, 64, p, p, p, 0.0, None, None, p, p, p, 1, 64, 64, 2, 1, 0, p, big, None),
    bwd_fp16=lambda: lib.kda_latent_bwd(p, p, p, 64, p, p, p, 0.0, None, None, p, p, p, 1, 64, 64, 2, 1, 128, p, big, None),
    decode=lambda: lib.kda_latent_decode(p, p, 4, 64, p, 2, p, 0.0, p, p, 2, 1, 16, 0, p, big, None),
    append=lambda: lib.kda_latent_append(p, 576, p, None, 1e-6, p, 64, 5, 0, None, None),
    fwd_huge=lambda: lib.kda_latent_fwd(p, p, p, 64, 0.0, p, p, p, p, 1, 512, 512, 65535, 65535, 0, None, None),
    bwd_huge=lambda: lib.kda_latent_bwd(p, p, p, 64, p, p, p, 0.0, p, p, p, p, p, 1, 512, 512, 65535, 65535, 0, p, 1 << 50, None),
    tables=lambda: lib.kda_block_tables(p, p, p, 2, p, 1, p, 16, p, 1, p, p, p, 1, None, None))
fake = ctypes.CDLL(None)
for name, call in calls.items():
    for at in range(5):
        fake.fake_begin(at)
        print(name, at, call(), fake.fake_launches())
"""


@pytest.fixture(scope="module")
def fake_launches(tmp_path_factory):
    """{(call, launch that fails): (status, launches tried)}"""
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    at = tmp_path_factory.mktemp("fake")
    (at / "fake.c").write_text(FAKE_RUNTIME)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(at / "fake.so"), str(at / "fake.c")], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FAKE_CALLS], env=dict(os.environ, LD_PRELOAD=str(at / "fake.so"), PYTHONPATH=root),
                         cwd=root, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-1000:]
    return {(name, int(at)): (int(rc), int(n)) for name, at, rc, n in (line.split() for line in out.stdout.splitlines())}


@pytest.mark.parametrize("call,launches", [("fwd", 1), ("fwd_shared", 3), ("bwd", 4), ("bwd_fp16", 4), ("decode", 2),
                                           ("append", 1), ("tables", 1)])
def test_a_failed_launch_ends_the_call(fake_launches, call, launches):
    """What follows reads what the failed one would have written (work items among it): it is not launched, and the
    call says so."""
    assert fake_launches[call, 0] == (0, launches)
    for at in range(1, launches + 1):
        assert fake_launches[call, at] == (3, at), at


def test_sizes_that_do_not_fit_the_c_entries_are_refused():
    """2^32 + 16 would arrive as 16."""
    z = lambda *s, d=torch.int32: torch.zeros(1, dtype=d).expand(s)  # noqa: E731
    big = 2 ** 32 + 16
    good = dict(seq_lens=z(1), new_lens=z(1), block_table=z(1, 1), free_pages=z(1), free_head=z(1), page_size=16, num_tokens=1)
    for name, value in (("page_size", big), ("page_size", 16 - 2 ** 32), ("page_size", 16.5), ("num_tokens", big), ("num_tokens", 2 ** 31),
                        ("block_table", z(1, big)), ("free_pages", z(big))):
        with pytest.raises(ValueError, match=name):
            latent.block_tables(**{**good, name: value})
    with pytest.raises(ValueError, match="seq_lens"):
        latent.block_tables(**{**good, "seq_lens": z(big), "new_lens": z(big), "block_table": z(big, 1)})
    with pytest.raises(ValueError, match="CUDA"):
        latent.block_tables(**good)
    latent._check_int("width", 2 ** 31 - 1)
    with pytest.raises(ValueError, match="width"):
        latent._check_int("width", 2 ** 31)


@pytest.mark.parametrize("Tq,Tk,N", [(1, 1, 65535), (512, 1, 65535), (1, 512, 65535), (512, 512, 32768)])
def test_more_tiles_and_heads_than_a_grid_are_refused(fake_launches, Tq, Tk, N):
    """512 rows in 65535 sequences with 65535 heads came out as a grid of 2^32 and some CTAs, cut to the some."""
    lib = binding.load_library()
    assert lib.kda_latent_fwd_workspace_bytes(1, Tq, Tk, 65535, N) == 0
    assert lib.kda_latent_bwd_workspace_bytes(1, Tq, Tk, 65535, N) == 0
    assert lib.kda_latent_bwd_workspace_bytes(1, 1, 1, 65535, 32767) > 0
    assert fake_launches["fwd_huge", 0] == fake_launches["bwd_huge", 0] == (1, 0)

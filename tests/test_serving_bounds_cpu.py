"""Serving entry points on the host, without a GPU: what a call sets and leaves
behind in the runtime, and what the sources have to say for it."""

import ctypes
import glob
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

from test_serving_cpu import caller, cpu_only, host_block

from chunked_gated_delta_kda_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A runtime whose n-th launch fails, in front of the real one; like the real one it keeps the last error until that is read.
RUNTIME = r"""
static int count = 0, last = 0, fail_at = 0, smem = 0;
void fake_begin(int at, int before) { count = smem = 0; fail_at = at; last = before; }
int fake_last(void) { return last; }
int fake_smem(void) { return smem; }
static int launched(void) { return ++count == fail_at ? (last = 719) : 0; }
int __cudaLaunchKernel(void) { return launched(); }
int cudaLaunchKernel(void) { return launched(); }
int cudaLaunchKernelExC(void) { return launched(); }
int __cudaGetKernel(void) { return 0; }
int cudaFuncSetAttribute(const void* f, int attr, int value) { smem = value; return 0; }
int cudaMemsetAsync(void) { return 0; }
int cudaGetLastError(void) { int e = last; last = 0; return e; }
static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char* name, void** f, unsigned version, unsigned long long flags, int* found) {
    *f = (void*)encode; *found = 0; return 0;
}
"""
CALLS = r"""
import ctypes
from chunked_gated_delta_kda_gb300 import binding, build
lib = binding.load_library()
buf = (ctypes.c_uint8 * 4096)()
p = ctypes.addressof(buf) + (-ctypes.addressof(buf) % 256)
big = 1 << 50
pair, pools = (ctypes.c_longlong * 2)(64, 16), (ctypes.c_void_p * 70)(*[p] * 70)
chunk = lambda T, keys, H, N: lib.kda_latent_chunk(p, p, 4, 64, p, 2, p, p, 0.0, p, keys, p, p, T, H, N, 0, p, big, None)
compact = lambda pages: lib.kda_page_compact(p, 2, p, p, pages, p, 4, p, 16, p, p, p, p, p, p, 2, None, None)
calls = dict(
    chunk=lambda: chunk(64, 300, 2, 1),
    chunk_shared=lambda: chunk(64, 8192, 1, 30),
    fork=lambda: lib.kda_page_fork(p, 2, p, p, p, None, p, 4, p, 4, p, 16, p, p, p, p, 2, 1, None, None),
    fork_many=lambda: lib.kda_page_fork(p, 2, p, p, p, None, p, 4, p, 4, p, 16, p, p, p, p, 2, 300, None, None),
    copy=lambda: lib.kda_page_copy(pools, 70, 4, 32, p, None, 1, None, None),
    free=lambda: lib.kda_page_free(p, 2, p, p, p, 4, p, 4, p, 16, p, p, p, 2, None, None),
    free_many=lambda: lib.kda_page_free(p, 1000, p, p, p, 4, p, 4, p, 16, p, p, p, 2000, None, None),
    compact=lambda: compact(4),
    compact_large=lambda: compact(1 << 21),
    verify=lambda: lib.kda_verify_drafts(p, p, pair, p, pair, p, p, p, 2, 3, 16, 512, None, None))
fake = ctypes.CDLL(None)
for name, call in calls.items():
    for at, before in ((0, 0), (0, 700), (1, 0), (2, 0), (3, 0)):
        fake.fake_begin(at, before)
        print(name, at, before, call(), fake.fake_last())
for pages in (1, 512, 8192, 1 << 20):
    fake.fake_begin(0, 0)
    compact(pages)
    print("smem", pages, 0, 0, fake.fake_smem())
"""


@pytest.fixture(scope="module")
def left_behind(tmp_path_factory):
    """{(call, launch that fails, error there before): (status, error there afterwards)}"""
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    at = tmp_path_factory.mktemp("fake")
    (at / "fake.c").write_text(RUNTIME)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(at / "fake.so"), str(at / "fake.c")], check=True)
    out = subprocess.run([sys.executable, "-c", CALLS], env=dict(os.environ, LD_PRELOAD=str(at / "fake.so"), PYTHONPATH=ROOT),
                         cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-1000:]
    return {(name, int(at), int(b)): (int(rc), int(e)) for name, at, b, rc, e in (line.split() for line in out.stdout.splitlines())}


def test_compaction_sets_its_kernels_shared_memory_alike_for_every_pool(left_behind):
    """The limit is the function's, not the call's: another thread's smaller pool must not lower it between the setting
    and the launch."""
    set_to = {left_behind["smem", pages, 0][1] for pages in (1, 512, 8192, 1 << 20)}
    assert len(set_to) == 1 and set_to.pop() >= (1 << 20) // 8


@pytest.mark.parametrize("call,launches", [("chunk", 3), ("chunk_shared", 3), ("fork", 1), ("fork_many", 1), ("copy", 2), ("free", 1),
                                           ("free_many", 3), ("compact", 1), ("compact_large", 2), ("verify", 1)])
def test_a_failed_launch_is_told_once(left_behind, call, launches):
    """A call does not report an error that was there before it, nor leave its own for the thread's next call."""
    assert left_behind[call, 0, 0] == (0, 0)
    assert left_behind[call, 0, 700][0] == 0
    for at in range(1, launches + 1):
        assert left_behind[call, at, 0] == (3, 0), at


def source(name):
    with open(os.path.join(ROOT, "chunked_gated_delta_kda_gb300", "csrc", name)) as f:
        return f.read()


def test_memory_is_read_behind_the_wait_for_the_kernel_before():
    """A wait that the compiler may move loads over is none."""
    waits = 0
    for path in glob.glob(os.path.join(ROOT, "chunked_gated_delta_kda_gb300", "csrc", "*.cu*")):
        for line in source(os.path.basename(path)).splitlines():
            if "griddepcontrol.wait" in line:
                waits += 1
                assert re.search(r'asm volatile\(".*griddepcontrol\.wait;.*" ::: "memory"\)', line), (path, line)
    assert waits > 10


def test_the_expansion_lets_the_next_kernel_begin_behind_its_own_wait():
    """latent_share_kernel, launched behind the expansion, reads the plan that the expansion waits for, without a wait."""
    text = source("kda_latent_chunk.cu")
    kernel = text[text.index("latent_expand_kernel("):]
    assert kernel.index("griddepcontrol.wait") < kernel.index("griddepcontrol.launch_dependents")
    share = source("kda_latent_fwd.cu")
    share = share[share.index("latent_share_kernel("):]
    assert share.index("p.cu_k") < share.index("griddepcontrol.wait")


@cpu_only
def test_sizes_that_an_index_could_step_out_of_are_refused():
    """The pages' kernels walk rows, columns and pages in steps of up to 155648 with 32-bit numbers."""
    keep, p = host_block()
    lib = binding.load_library()
    shared = dict(table=p, width=2, lens=p, refs=p, pages=4, free=p, free_n=4, head=p, page=16)
    last = dict(N=2, ws=p, stream=None)
    fork = caller(lib.kda_page_fork, dict(
        table=p, width=2, lens=p, parents=p, children=p, fork_lens=None, refs=p, pages=4, free=p, free_n=4, head=p, page=16, lens_out=p,
        refs_out=p, head_out=p, pairs=p, N=2, F=1, ws=p, stream=None))
    free = caller(lib.kda_page_free, dict(
        table=p, width=2, lens=p, keep=p, refs=p, pages=4, free=p, free_n=4, head=p, page=16, lens_out=p, refs_out=p, head_out=p, **last))
    compact = caller(lib.kda_page_compact, dict(
        **shared, table_out=p, refs_out=p, free_out=p, pairs=p, count=p, moved=p, **last))
    for big in (2 ** 30 + 1, 2 ** 31 - 1):
        for call in (fork, free, compact):
            for name in ("N", "width", "pages", "free_n"):
                assert call(**{name: big}) == 1, (name, big)
        assert fork(F=big) == 1


@cpu_only
def test_more_drafts_than_an_index_could_step_over_are_refused():
    keep, p = host_block()
    pair = (ctypes.c_longlong * 2)(64, 16)
    call = caller(binding.load_library().kda_verify_drafts, dict(
        tokens=p, draft=p, ds=pair, target=p, ts=pair, uniform=p, out=p, accepted=p, N=2, S=3, V=16, flags=512, ws=None, stream=None))
    for S in (2 ** 30 + 1, 2 ** 31 - 2):
        assert call(S=S) == 1


def test_the_library_is_built_without_torchs_headers(tmp_path, monkeypatch):
    """A module that does not compile says so, and the library it would have called is there all the same."""
    tiny = tmp_path / "tiny.cu"
    tiny.write_text('extern "C" int tiny() { return 5; }\n')
    monkeypatch.setattr(build, "OUT", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(build, "sources", lambda: [str(tiny)])
    monkeypatch.setattr(build, "_marshal_commands", lambda: (["false"], ["false", "-shared", "-o", str(tmp_path / "x")]))
    with pytest.raises(RuntimeError, match="kda_marshal"):
        build.build()
    assert ctypes.CDLL(str(tmp_path / "libkda.so")).tiny() == 5


def test_the_module_of_another_torch_is_not_taken(tmp_path, monkeypatch):
    """It is compiled against torch's C++ and Python's C interfaces."""
    monkeypatch.setattr(build, "OUT", str(tmp_path))
    here = build.marshal()
    open(here, "w").close()
    assert build.marshal_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0")
        assert build.marshal() != here and not build.marshal_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-0.so")
        assert not build.marshal_up_to_date()
    assert build.marshal_up_to_date()

"""Host-side checks of the chunk, draft and page entry points and wrappers:
sizes and refusals, all before any CUDA call."""

import ctypes
import os
import shutil
import subprocess
import sys

import pytest
import torch

from test_latent_cpu import FAKE_RUNTIME

from chunked_gated_delta_kda_gb300 import binding, drafts, latent, pages

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
    shared = 896 * 16 + 256 * 256 * 130 * 4
    rows = lambda keys, H, low: keys * H * 512 + r256(keys * 128) + low * H * 256  # noqa: E731
    assert lib.kda_latent_chunk_workspace_bytes(37, 237, 8, 1) == 256 + 3 * 256 + rows(237, 8, 237)
    assert lib.kda_latent_chunk_workspace_bytes(1642, 16231, 16, 4) == 256 + r256(shared) + 3 * 256 + rows(16231, 16, 8192)
    assert lib.kda_latent_chunk_workspace_bytes(0, 0, 1, 1) == 256 + 3 * 256
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 65536, 1), (1, 1, 1, 65536),
                (1 << 30, 1, 65535, 1), (1, 1, 65535, 65535)):
        assert lib.kda_latent_chunk_workspace_bytes(*bad) == 0, bad
    assert lib.kda_latent_chunk_workspace_bytes(8, 100000, 1, 2) == 256 + 3 * 256 + rows(100000, 1, 4096)


def test_status_string():
    lib = binding.load_library()
    assert b"token" in lib.kda_status_str(9) and "token" in str(binding.KdaError(9, "x"))


@cpu_only
def test_chunk_refusals():
    keep, p = host_block()
    lib = binding.load_library()
    need = lib.kda_latent_chunk_workspace_bytes(8, 64, 2, 2)
    call = caller(lib.kda_latent_chunk, dict(
        q=p, cache=p, pages=4, page=64, table=p, width=2, lens=p, w=p, scale=0.0, cu=p, keys=64, o=p, lse=p, T=8, H=2, N=2,
        flags=0, ws=p, wsb=need, stream=None))
    for kw in (dict(q=None), dict(cache=None), dict(table=None), dict(lens=None), dict(w=None), dict(cu=None), dict(o=None),
               dict(ws=None), dict(wsb=need - 1), dict(pages=0), dict(width=0), dict(page=0), dict(page=8), dict(page=48),
               dict(page=96), dict(page=-64), dict(pages=1 << 26), dict(width=1 << 26), dict(keys=-1), dict(T=-1), dict(H=0),
               dict(N=0), dict(H=65536), dict(N=65536), dict(flags=256), dict(flags=512), dict(q=p + 8), dict(cache=p + 8),
               dict(w=p + 8), dict(o=p + 8), dict(table=p + 2), dict(lens=p + 2), dict(cu=p + 1), dict(lse=p + 2),
               dict(ws=p + 128)):
        assert call(**kw) == 1, kw


@cpu_only
def test_page_refusals():
    keep, p = host_block()
    lib = binding.load_library()
    shared = (dict(refs=None), dict(lens=None), dict(head=None), dict(table=None), dict(refs_out=None), dict(refs_out=p + 8),
              dict(width=-1), dict(pages=0), dict(free_n=-1), dict(free=None), dict(page=0), dict(page=-16),
              dict(N=0), dict(ws=p + 16), dict(table=p + 2), dict(lens=p + 1), dict(refs=p + 2), dict(free=p + 2),
              dict(head=p + 2), dict(refs_out=p + 2))
    fork = caller(lib.kda_page_fork, dict(
        table=p, width=2, lens=p, parents=p, children=p, fork_lens=None, refs=p, pages=4, free=p, free_n=4, head=p, page=16, lens_out=p,
        refs_out=p, head_out=p, pairs=p, N=2, F=1, ws=p, stream=None))
    for kw in shared + (dict(parents=None), dict(children=None), dict(pairs=None), dict(lens_out=None), dict(head_out=None),
                        dict(F=-1), dict(parents=p + 2), dict(fork_lens=p + 2), dict(pairs=p + 2)):
        assert fork(**kw) == 1, kw
    free = caller(lib.kda_page_free, dict(
        table=p, width=2, lens=p, keep=p, refs=p, pages=4, free=p, free_n=4, head=p, page=16, lens_out=p, refs_out=p,
        head_out=p, N=2, ws=p, stream=None))
    for kw in shared + (dict(keep=None), dict(lens_out=None), dict(head_out=None), dict(keep=p + 2)):
        assert free(**kw) == 1, kw
    compact = caller(lib.kda_page_compact, dict(
        table=p, width=2, lens=p, refs=p, pages=4, free=p, free_n=4, head=p, page=16, table_out=p, refs_out=p, free_out=p,
        pairs=p, count=p, moved=p, N=2, ws=p, stream=None))
    for kw in shared + (dict(table_out=None), dict(free_out=None), dict(pairs=None), dict(count=None), dict(moved=None),
                        dict(moved=p + 4), dict(table_out=p + 1)):
        assert compact(**kw) == 1, kw
    at = (ctypes.c_void_p * 2)(p, p)
    copy = caller(lib.kda_page_copy, dict(pools=at, n=2, pages=4, bytes=32, pairs=p, count=None, F=1, ws=None, stream=None))
    for kw in (dict(pools=None), dict(n=0), dict(pages=0), dict(bytes=0), dict(bytes=24), dict(bytes=-16), dict(pairs=None),
               dict(F=-1), dict(pairs=p + 2), dict(count=p + 2), dict(ws=p + 16),
               dict(pools=(ctypes.c_void_p * 2)(p, None)), dict(pools=(ctypes.c_void_p * 2)(p, p + 8))):
        assert copy(**kw) == 1, kw


@cpu_only
def test_draft_refusals():
    keep, p = host_block()
    pair = (ctypes.c_longlong * 2)(64, 16)
    call = caller(binding.load_library().kda_verify_drafts, dict(
        tokens=p, draft=p, ds=pair, target=p, ts=pair, uniform=p, out=p, accepted=p, N=2, S=3, V=16, flags=512, ws=None,
        stream=None))
    for kw in (dict(tokens=None), dict(ds=None), dict(target=None), dict(ts=None), dict(uniform=None), dict(out=None),
               dict(accepted=None), dict(N=0), dict(S=-1), dict(V=0), dict(S=2 ** 31 - 1), dict(N=2 ** 24 + 1), dict(V=2 ** 30 + 1),
               dict(flags=1), dict(flags=512 + 128), dict(tokens=p + 4), dict(draft=p + 2), dict(target=p + 2),
               dict(uniform=p + 2), dict(out=p + 4), dict(accepted=p + 2), dict(ws=p + 16),
               dict(ts=(ctypes.c_longlong * 2)(-1, 16)), dict(ds=(ctypes.c_longlong * 2)(64, 1 << 40))):
        assert call(**kw) == 1, kw


def z(*s, d=torch.int32):
    return torch.zeros(s, dtype=d)


def big(*s, d=torch.int32):
    return torch.zeros(1, dtype=d).expand(s)


def test_wrappers_refuse_what_the_kernels_do_not_take():
    """CPU tensors, types, shapes: a clear error and no fallback."""
    bf, f32, i64 = torch.bfloat16, torch.float32, torch.int64
    chunk = dict(q=z(4, 2, 192, d=bf), cache=z(3, 16, 576, d=bf), block_table=z(1, 2), seq_lens=z(1), w_up=z(2, 256, 512, d=bf),
                 cu_seqlens_q=z(2), num_keys=4)
    fork = dict(block_table=z(2, 3), seq_lens=z(2), parents=z(1), children=z(1), refs=z(4), free_pages=z(4), free_head=z(1),
                page_size=16)
    free = {k: v for k, v in fork.items() if k not in ("parents", "children")}
    free["keep_lens"] = z(2)
    compact = {k: v for k, v in free.items() if k != "keep_lens"}
    verify = dict(draft_tokens=z(2, 3, d=i64), target_probs=z(2, 4, 9, d=f32), uniform=z(2, 4, d=f32), draft_probs=z(2, 3, 9, d=f32))
    copy = dict(pools=z(4, 8), pairs=z(1, 2))
    for fn, good, bad in (
            (latent.latent_chunk, chunk, [("q", z(4, 2, 192, d=f32)), ("q", z(4, 2, 128, d=bf)), ("cache", z(3, 16, 512, d=bf)),
                                          ("w_up", z(1, 256, 512, d=bf)), ("w_up", z(2, 256, 512, d=torch.float16)),
                                          ("block_table", z(1, 2, d=i64)), ("seq_lens", z(2)), ("cu_seqlens_q", z(1)),
                                          ("num_keys", -1), ("num_keys", 2 ** 32 + 4), ("num_keys", 4.5), ("q", None), ("w_up", 3)]),
            (pages.page_fork, fork, [("parents", z(2)), ("children", z(1, d=i64)), ("refs", z(4, d=i64)), ("free_head", z(2)),
                                     ("page_size", 0), ("page_size", 2 ** 32 + 16), ("page_size", 16.5), ("block_table", z(3, 3)),
                                     ("seq_lens", None), ("refs", big(2 ** 32 + 4)), ("parents", [0]), ("fork_lens", z(2)), ("fork_lens", z(1, d=i64))]),
            (pages.page_free, free, [("keep_lens", z(3)), ("keep_lens", None), ("free_pages", z(2, 2)), ("page_size", -1),
                                     ("block_table", big(2, 2 ** 32))]),
            (pages.page_compact, compact, [("refs", z(2, 2)), ("free_pages", z(4, d=f32)), ("page_size", 0), ("free_head", 0)]),
            (pages.page_copy, copy, [("pairs", z(2)), ("pairs", z(1, 2, d=i64)), ("pools", []), ("pools", [3]), ("pools", None)]),
            (drafts.verify_drafts, verify, [("draft_tokens", z(2, 3)), ("draft_tokens", z(3, 3, d=i64)), ("target_probs", z(2, 3, 9, d=f32)),
                                            ("target_probs", z(2, 4, 9, d=torch.float64)), ("uniform", z(2, 3, d=f32)),
                                            ("uniform", z(2, 4, d=bf)), ("draft_probs", z(2, 3, 8, d=f32)),
                                            ("draft_probs", z(2, 3, 9, d=bf)), ("draft_tokens", None), ("target_probs", 1)])):
        with pytest.raises(ValueError, match="CUDA"):
            fn(**good)
        for name, value in bad:
            with pytest.raises((TypeError, ValueError)) as e:
                fn(**{**good, name: value})
            assert "must" in str(e.value), (fn.__name__, name, e.value)


FAKE_CALLS = r"""
import ctypes
from chunked_gated_delta_kda_gb300 import binding
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
    chunk_no_rows=lambda: chunk(64, 0, 2, 1),
    chunk_nothing=lambda: chunk(0, 300, 2, 1),
    fork=lambda: lib.kda_page_fork(p, 2, p, p, p, None, p, 4, p, 4, p, 16, p, p, p, p, 2, 1, None, None),
    copy=lambda: lib.kda_page_copy(pools, 70, 4, 32, p, None, 1, None, None),
    free=lambda: lib.kda_page_free(p, 2, p, p, p, 4, p, 4, p, 16, p, p, p, 2, None, None),
    free_many=lambda: lib.kda_page_free(p, 1000, p, p, p, 4, p, 4, p, 16, p, p, p, 2000, None, None),
    compact=lambda: compact(4),
    compact_large=lambda: compact(1 << 21),
    verify=lambda: lib.kda_verify_drafts(p, p, pair, p, pair, p, p, p, 2, 3, 16, 512, None, None))
fake = ctypes.CDLL(None)
for name, call in calls.items():
    for at in range(7):
        fake.fake_begin(at)
        print(name, at, call(), fake.fake_launches())
"""


@pytest.fixture(scope="module")
def fake_launches(tmp_path_factory):
    """{(call, launch that fails): (status, launches tried)}, with a runtime whose n-th launch fails in front of the real
    one: no GPU is needed, nothing runs."""
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


@pytest.mark.parametrize("call,launches", [("chunk", 3), ("chunk_shared", 5), ("chunk_no_rows", 2), ("chunk_nothing", 1), ("fork", 1),
                                           ("copy", 2), ("free", 1), ("free_many", 3), ("compact", 1), ("compact_large", 2),
                                           ("verify", 1)])
def test_a_failed_launch_ends_the_call(fake_launches, call, launches):
    """What follows reads what the failed one would have written: it is not launched, and the call says so."""
    assert fake_launches[call, 0] == (0, launches)
    for at in range(1, launches + 1):
        assert fake_launches[call, at] == (3, at), at

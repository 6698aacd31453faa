"""What a bounded wait that runs out leaves behind in chunk and cross attention:
zeros in the rows that depend on it, never attention over the keys that were in
time, and the other rows as ever.

The library is built once more with one met wait counted as run out (one warp, one
step of one CTA) and a limit of 0.1 s: every copy lands, no wait is skipped, and
the warps that then wait for that one come back by their own limits."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import oracle
import serving_util as U
from gpu_util import assert_parity, require_gpu, to_f64, upload
from paged_kv_cache_376_b200 import _lib, build

pytestmark = pytest.mark.gpu

HQ, HKV = 8, 2
# kernel 0 is launched without a workspace on a grid of (KV heads, sequences, row
# blocks); 1 has its CTAs by (range, KV head); 2 takes units as they come
GIVE_UP = """
#define TV_WAIT_LIMIT_NS 100000000ull
#define TV_GIVE_UP(kernel, warp, step)                                     \\
  ((kernel) == 0   ? blockIdx.x == 1 && blockIdx.y == 1 && (warp) == 2 &&  \\
                       (step) == 3                                         \\
   : (kernel) == 1 ? blockIdx.x == 20 && (warp) == 1 && (step) >= 6        \\
                   : blockIdx.x == 3 && (warp) == 9 && (step) == 5)
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    require_gpu()
    tmp = tmp_path_factory.mktemp("tv")
    path = str(tmp / "libtv_give_up.so")
    (tmp / "give_up.h").write_text(GIVE_UP)
    subprocess.run(
        [build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-t", "0",
         "-Xcompiler", "-fPIC", "-shared", "-I", build.INCLUDE, "-I",
         build.CSRC, "-include", str(tmp / "give_up.h"), "-o", path,
         *build.sources()], check=True)
    lib = ctypes.CDLL(path)
    for name in ("tv_paged_chunk", "tv_paged_cross_attention",
                 "tv_chunk_workspace_size"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = _lib.SIGNATURES[name]
    return lib


def _call(lib, wl, causal, workspace):
    """The output and its distance to the oracle's, in bounds, per row and
    head; the error word has to say that a wait ran out."""
    db = upload(wl)
    b, maxq = len(wl.context_lens), int(np.diff(wl.query_start_loc).max())
    ws, size = None, 0
    if workspace:
        n = ctypes.c_size_t(0)
        assert lib.tv_chunk_workspace_size(b, maxq, HQ, HKV, 64,
                                           ctypes.byref(n)) == 0
        # what an earlier call left there must not come out
        ws = torch.full((n.value,), 63, dtype=torch.uint8, device="cuda")
        ws[:65536] = 0
        size = n.value
    out = torch.full_like(db.q, 7.0)
    fn = lib.tv_paged_chunk if causal else lib.tv_paged_cross_attention
    kp = db.k_pool
    assert fn(out.data_ptr(), db.q.data_ptr(), db.q.shape[0],
              db.query_start_loc.data_ptr(), kp.data_ptr(),
              db.v_pool.data_ptr(), db.block_tables.data_ptr(),
              db.block_tables.shape[1], db.context_lens.data_ptr(), b, maxq,
              HQ, HKV, 64, kp.shape[1], kp.shape[0], wl.scale,
              None if ws is None else ws.data_ptr(), size, db.err.data_ptr(),
              torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert int(db.err.item()) == _lib.DEVERR_TIMEOUT
    fn = oracle.paged_prefill if causal else oracle.paged_cross
    ref = fn(wl.q, wl.query_start_loc, wl.k_pool, wl.v_pool, wl.block_tables,
             wl.context_lens, wl.scale)
    zero = ~to_f64(out).any(2)
    assert_parity(np.where(zero[..., None], ref, to_f64(out)), ref,
                  "rows that are not zero")
    return zero


def _workload(lens, rows, seed):
    return U.cross_workload(lens, rows, seed, num_q_heads=HQ,
                            num_kv_heads=HKV)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows", [1, 4, 8])
def test_without_a_workspace(lib, rows, causal):
    wl = _workload([600, 900, 300], [rows] * 3, 901)
    zero = _call(lib, wl, causal, False)
    want = np.zeros_like(zero)
    want[rows:2 * rows, HQ // HKV:] = True      # sequence 1, KV head 1
    np.testing.assert_array_equal(zero, want)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows", [1, 8])
@pytest.mark.parametrize("lens", [[20000, 900, 9000], [700] * 90],
                         ids=["few", "many"])
def test_balanced(lib, lens, rows, causal):
    """KV head 0 of the CTA's range: whole sequences of it, and those of which
    it has a part."""
    wl = _workload(lens, [rows] * len(lens), 902)
    zero = _call(lib, wl, causal, True)
    assert zero.any()
    assert not zero[:, HQ // HKV:].any()
    per_seq = zero[:, :HQ // HKV].reshape(len(lens), -1)
    assert (per_seq.all(1) == per_seq.any(1)).all()
    assert not per_seq.all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,rows", [
    ([3000, 400, 900], [70, 2, 300]),           # cut along the keys
    ([500] * 120 + [90], [130] * 120 + [1]),    # many units a CTA
], ids=["cut", "many"])
def test_tiles(lib, lens, rows, causal):
    """Units are taken as they come, so every sequence of the tile kernel is
    zero; those of the streaming kernel are not."""
    wl = _workload(lens, rows, 903)
    zero = _call(lib, wl, causal, True)
    tiles = np.repeat(np.asarray(rows) * HQ // HKV > 32, rows)
    np.testing.assert_array_equal(zero, np.repeat(tiles[:, None], HQ, 1))

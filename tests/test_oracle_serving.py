"""The oracles of the serving operators, pinned without a GPU, and the
refusals of their entry points (which return before any launch)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import serving_util as U
from oracle.pool import PagePool, pages_for
from paged_kv_cache_376_b200 import _lib, build
from paged_kv_cache_376_b200 import workloads as W


# ---- oracles ------------------------------------------------------------------

def test_mrope_with_one_axis_is_rope():
    rows = W._normal_bf16(5, 3, (40, 4, 64))
    tab = U.rope_table(128)
    pos = np.arange(40, dtype=np.int32)[None] * 3
    for axes in (1, 3):
        a, bad = oracle.mrope(rows, np.repeat(pos, axes, 0),
                              U.pair_axes(axes, True), tab)
        b, _ = oracle.rope(rows, pos[0], tab)
        assert bad == 0 and np.array_equal(a, b)


def test_mrope_turns_each_pair_by_its_own_axis():
    """Against the rotation in 64 bits: half a bf16 step (2^-8 relative to the
    result) plus the binary32 steps (two products and a sum, and the table:
    4 x 2^-24 of the operands)."""
    t, axes = 50, 3
    rows = W._normal_bf16(6, 3, (t, 2, 64))
    tab = U.rope_table(4096)
    pos = U.multi_axis_positions(t, axes, 4096, 1)
    for inter in (False, True):
        axis = U.pair_axes(axes, inter)
        got, bad = oracle.mrope(rows, pos, axis, tab)
        assert bad == 0
        ang = pos[axis].T * (500000.0 ** (-np.arange(32) / 32.0))
        x = W.bf16_to_f64(rows)
        z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(1j * ang)[:, None]
        ref = np.concatenate([z.real, z.imag], -1)
        size = np.tile(np.abs(x[..., :32]) + np.abs(x[..., 32:]), 2)
        err = np.abs(W.bf16_to_f64(got) - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * size).all()


def test_mrope_leaves_tokens_with_a_bad_position_whole():
    rows = W._normal_bf16(7, 3, (6, 2, 64))
    tab = U.rope_table(16)
    pos = np.full((2, 6), 3, np.int32)
    pos[0, 1], pos[1, 4] = -1, 16
    axis = U.pair_axes(2, True)
    got, bad = oracle.mrope(rows, pos, axis, tab)
    assert bad == 2
    assert np.array_equal(got[[1, 4]], rows[[1, 4]])
    assert not np.array_equal(got[0], rows[0])
    # an axis that no pair uses is not looked at
    got, bad = oracle.mrope(rows, pos, np.zeros(32, np.int32), tab)
    assert bad == 1
    # an axis that is none: no token turns
    axis[5] = 2
    got, bad = oracle.mrope(rows, pos, axis, tab)
    assert bad == 6 and np.array_equal(got, rows)


@pytest.mark.parametrize("page_size", [16, 32])
def test_cross_oracle_is_full_attention(page_size):
    wl = U.cross_workload([50, 0, 7], [4, 3, 9], 11, page_size=page_size)
    ref = oracle.paged_cross(wl.q, wl.query_start_loc, wl.k_pool, wl.v_pool,
                             wl.block_tables, wl.context_lens, wl.scale)
    q = torch.from_numpy(W.bf16_to_f64(wl.q))
    for s, n in enumerate(wl.context_lens):
        lo, hi = wl.query_start_loc[s], wl.query_start_loc[s + 1]
        if n == 0:
            assert not ref[lo:hi].any()
            continue
        slot = W._slots(wl.block_tables, s, np.arange(n), page_size)
        k, v = (torch.from_numpy(W.bf16_to_f64(
            p.reshape(-1, 8, 64)[slot])).repeat_interleave(4, 1)
            for p in (wl.k_pool, wl.v_pool))
        o = torch.nn.functional.scaled_dot_product_attention(
            q[lo:hi].transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1),
            scale=wl.scale).transpose(0, 1)
        assert np.abs(ref[lo:hi] - o.numpy()).max() < 1e-12


def _check_pool(pool, bt, ctx):
    """Counts are the rows that hold a page; the stack holds the others."""
    held = np.zeros(pool.num_pages, int)
    for s in range(len(ctx)):
        n = pages_for(ctx[s], pool.ps)
        np.add.at(held, bt[s, :n], 1)
        assert (bt[s, n:] == -1).all()
    assert np.array_equal(held, pool.ref)
    assert sorted(pool.stack) == list(np.flatnonzero(held == 0))


@pytest.mark.parametrize("seed", range(6))
def test_truncate_and_compact_models(seed):
    """Random truncations and compactions keep every sequence's tokens: the
    rows gathered through its table are a prefix of what they were."""
    rng = np.random.default_rng(seed)
    ps = 16 if seed % 2 else 32
    bt, ctx = U.random_pool(seed, 90, 9, ps)
    pool = PagePool(90, bt, ctx, page_size=ps)
    kp = rng.integers(0, 1 << 16, (90, ps, 1, 2)).astype(np.uint16)
    vp = kp[:, ::-1].copy()

    def tokens(s):
        pos = np.arange(ctx[s])
        return kp[bt[s, pos // ps], pos % ps].copy()

    for step in range(6):
        _check_pool(pool, bt, ctx)
        before = [tokens(s) for s in range(9)]
        if step % 2 == 0:
            new = [int(rng.integers(0, c + 1)) for c in ctx]
            new[step] = int(ctx[step]) + 1            # refused: unchanged
            pool.truncate(bt, ctx, new)
            new[step] = len(before[step])
            assert list(ctx) == new
        else:
            top = pool.top
            moves = pool.compact(bt, ctx, kp, vp)
            assert pool.top == top
            assert all(b < 90 - top <= a for a, b in moves)
            assert pool.stack == list(range(89, 90 - top - 1, -1))
        for s in range(9):
            assert np.array_equal(tokens(s), before[s][:ctx[s]])
    _check_pool(pool, bt, ctx)


# ---- refusals -------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
FAR = ctypes.c_void_p(0x10000000)


def _chunk(lib, name, **kw):
    a = dict(out=FAR, q=P, rows=8, qsl=P, k=P, v=P, bt=P, mb=4, ctx=P, b=1,
             maxq=8, hq=32, hkv=8, d=64, ps=16, np=10, scale=0.125, ws=None,
             ws_bytes=0)
    a.update(kw)
    return getattr(lib, name)(
        a["out"], a["q"], a["rows"], a["qsl"], a["k"], a["v"], a["bt"],
        a["mb"], a["ctx"], a["b"], a["maxq"], a["hq"], a["hkv"], a["d"],
        a["ps"], a["np"], a["scale"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("name", ["tv_paged_chunk",
                                  "tv_paged_cross_attention"])
def test_chunk_refusals(lib, name):
    for kw in (dict(d=128), dict(ps=8), dict(hq=12), dict(hq=128),
               dict(b=65536), dict(np=1 << 28), dict(mb=1 << 28),
               dict(maxq=1 << 19), dict(rows=1 << 31)):
        assert _chunk(lib, name, **kw) == 2, kw
    for kw in (dict(b=-1), dict(rows=-1), dict(maxq=-1), dict(mb=0),
               dict(np=0), dict(scale=float("nan")), dict(scale=0.0),
               dict(scale=-0.1), dict(scale=float("inf")), dict(q=None),
               dict(out=None), dict(qsl=None), dict(k=None), dict(v=None),
               dict(bt=None), dict(ctx=None), dict(q=ODD), dict(out=ODD),
               dict(k=ODD), dict(v=ODD), dict(ws=ODD, ws_bytes=1 << 30),
               dict(out=P), dict(out=ctypes.c_void_p(0x10000 + 4096 * 8 - 16)),
               dict(q=ctypes.c_void_p(0x10000000 + 16))):
        assert _chunk(lib, name, **kw) == 1, kw
    for kw in (dict(b=0), dict(rows=0), dict(maxq=0)):
        assert _chunk(lib, name, **kw) == 0, kw


def test_chunk_workspace_size_refusals(lib):
    n = ctypes.c_size_t(0)
    r = ctypes.byref(n)
    assert lib.tv_chunk_workspace_size(4, 8, 32, 8, 128, r) == 2
    assert lib.tv_chunk_workspace_size(4, 8, 12, 8, 64, r) == 2
    assert lib.tv_chunk_workspace_size(-1, 8, 32, 8, 64, r) == 1
    assert lib.tv_chunk_workspace_size(4, -8, 32, 8, 64, r) == 1
    assert lib.tv_chunk_workspace_size(4, 8, 32, 8, 64, None) == 1


def test_mrope_refusals(lib):
    def call(**kw):
        a = dict(qo=FAR, q=P, qs=2048, k=P, ks=512, v=P, vs=512, slots=P, pos=P,
                 axes=3, axis=P, t=4, kp=P, vp=P, np=10, hq=32, hkv=8, d=64,
                 ps=16, tab=P, npos=8)
        a.update(kw)
        return lib.tv_kv_append_mrope(
            a["qo"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
            a["slots"], a["pos"], a["axes"], a["axis"], a["t"], a["kp"],
            a["vp"], a["np"], a["hq"], a["hkv"], a["d"], a["ps"], a["tab"],
            a["npos"], None, None)

    for kw in (dict(d=128), dict(ps=24)):
        assert call(**kw) == 2, kw
    for kw in (dict(t=-1), dict(np=0), dict(hkv=0), dict(axes=0),
               dict(q=None), dict(qo=None), dict(hq=0), dict(k=None),
               dict(v=None), dict(slots=None), dict(pos=None),
               dict(axis=None), dict(kp=None), dict(vp=None), dict(tab=None),
               dict(npos=0), dict(q=ODD), dict(qo=ODD), dict(k=ODD),
               dict(v=ODD), dict(kp=ODD), dict(vp=ODD), dict(tab=ODD),
               dict(qs=2047), dict(qs=2052), dict(ks=504), dict(ks=516),
               dict(vs=504), dict(vs=517), dict(ks=0),
               dict(q=FAR, qs=2056), dict(k=FAR), dict(v=FAR),
               dict(q=ctypes.c_void_p(0x10000010))):
        assert call(**kw) == 1, kw
    assert call(t=0) == 0


def test_pool_edit_refusals(lib):
    t = lib.tv_pool_truncate
    assert t(P, 10, P, 4, P, P, 1025, None, None) == 2
    assert t(P, 1 << 30, P, 4, P, P, 4, None, None) == 2
    assert t(None, 10, P, 4, P, P, 4, None, None) == 1
    assert t(P, 10, P, 4, P, None, 4, None, None) == 1
    assert t(P, 10, None, 4, P, P, 4, None, None) == 1
    assert t(P, 0, P, 4, P, P, 4, None, None) == 1
    assert t(P, 10, P, 4, P, P, 0, None, None) == 0

    def compact(**kw):
        a = dict(st=P, np=10, bt=P, mb=4, ctx=P, b=4, src=P, dst=P, cap=5,
                 n=P, k=P, v=P, hkv=8, d=64, ps=16)
        a.update(kw)
        return lib.tv_pool_compact(
            a["st"], a["np"], a["bt"], a["mb"], a["ctx"], a["b"], a["src"],
            a["dst"], a["cap"], a["n"], a["k"], a["v"], a["hkv"], a["d"],
            a["ps"], None, None)

    for kw in (dict(b=1025), dict(d=32), dict(ps=64), dict(np=1 << 30)):
        assert compact(**kw) == 2, kw
    for kw in (dict(st=None), dict(src=None), dict(dst=None), dict(n=None),
               dict(cap=4), dict(k=None), dict(v=None), dict(k=ODD),
               dict(v=ODD), dict(hkv=0)):
        assert compact(**kw) == 1, kw

    def copy(**kw):
        a = dict(k=P, v=P, np=10, src=P, dst=P, cap=5, n=None, hkv=8, d=64,
                 ps=16)
        a.update(kw)
        return lib.tv_page_copy(a["k"], a["v"], a["np"], a["src"], a["dst"],
                                a["cap"], a["n"], a["hkv"], a["d"], a["ps"],
                                None, None)

    for kw in (dict(d=32), dict(ps=64), dict(np=1 << 28), dict(cap=1 << 31),
               dict(hkv=1 << 20)):
        assert copy(**kw) == 2, kw
    for kw in (dict(k=None), dict(v=None), dict(src=None), dict(dst=None),
               dict(cap=-1), dict(k=ODD), dict(hkv=0), dict(np=0)):
        assert copy(**kw) == 1, kw
    assert copy(cap=0) == 0


def test_bindings_refuse_host_tensors_and_shapes():
    q = torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 16, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (
            lambda: _lib.tv_paged_chunk(q, q, i, pool, pool, i, i, 1.0, 1),
            lambda: _lib.tv_paged_cross_attention(q, q, i, pool, pool, i, i,
                                                  1.0, 1),
            lambda: _lib.tv_kv_append_mrope(q, q, q, q, i, i, i, pool, pool,
                                            q),
            lambda: _lib.tv_page_copy(pool, pool, i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="go together"):
        _lib.tv_kv_append_mrope(None, q, q, q, i, i, i, pool, pool, q)


def test_one_device_refuses_mixed_devices():
    class T:
        def __init__(self, index):
            self.index = index
            self.device = torch.device("cuda", index)

        def get_device(self):
            return self.index

    with pytest.raises(ValueError, match="in one call"):
        _lib._one_device((T(0), None, T(1)), None)
    with pytest.raises(ValueError, match="stream on"):
        _lib._one_device((T(0),), T(1))

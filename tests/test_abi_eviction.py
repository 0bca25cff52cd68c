"""CPU-only checks of the cache-eviction entry points: struct layouts, and the host-side
refusals (fake addresses; every request below is refused before anything is launched)."""
import ctypes as C
import math

import pytest

import sparse_top_kv_validate_gb300 as sa
from test_abi import _c_layout, host_lib, lib  # noqa: F401  (fixtures)
from test_abi_serving import _set

K31 = 1 << 31


@pytest.mark.parametrize("cname,py", [("sa_weights_params", sa.WeightsParams), ("sa_select_params", sa.SelectParams),
                                      ("sa_compact_params", sa.CompactParams)])
def test_struct_layout_matches_header(cname, py):
    fields = [f for f, _ in py._fields_]
    size, offs = _c_layout(cname, fields)
    assert C.sizeof(py) == size
    assert [getattr(py, f).offset for f in fields] == offs


def test_packed_parameters_fill_the_structs(lib):            # noqa: F811
    for packer, py in ((sa._WEIGHTS, sa.WeightsParams), (sa._SELECT, sa.SelectParams), (sa._COMPACT, sa.CompactParams)):
        assert packer.size == C.sizeof(py)


def _weights():
    return _set(sa.WeightsParams(), q=0x1000000, k=0x2000000, weights=0x3000000, block_table=0x4000000, q_start=0x5000000,
                k_start=0x5001000, dtype=sa.BF16, accumulate=1, B=2, Tq=20, Tk=50, Hq=8, Hkv=2, D=128, page_tokens=16,
                max_pages=4, num_pages=8, q_strides=[1024, 128], k_strides=[256, 128], workspace=0x6000000,
                workspace_bytes=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(weights=None), -1), (dict(block_table=None), -1), (dict(q_start=None), -1),
    (dict(dtype=7), -3), (dict(dtype=sa.FP8_E4M3_PAGE), -3), (dict(reserved_=1), -7),
    (dict(B=0), -2), (dict(Tq=-1), -2), (dict(Hq=0), -2), (dict(Hkv=0), -2), (dict(Hkv=3), -2), (dict(D=0), -2),
    (dict(page_tokens=0), -2), (dict(max_pages=0), -2), (dict(num_pages=0), -2), (dict(k_start=None), -2),
    (dict(scale=math.nan), -2), (dict(scale=math.inf), -2), (dict(q_strides=[-1024, 128]), -2),
    (dict(D=258), -7), (dict(D=130), -7), (dict(Tq=1 << 30), -7), (dict(B=1 << 24), -7), (dict(Hq=1 << 17), -7),
    (dict(page_tokens=K31), -7), (dict(page_tokens=1 << 16, max_pages=1 << 15), -7),
    (dict(q=0x1000001), -4), (dict(weights=0x3000002), -4), (dict(q_start=0x5000002), -4), (dict(workspace=0x6000010), -4),
    (dict(weights=0x1000000), -6), (dict(weights=0x2000000 + 64), -6), (dict(weights=0x4000000), -6),
    (dict(weights=0x5001000), -6), (dict(weights=0x6000000), -6),
    (dict(workspace=None), -5), (dict(workspace_bytes=256), -5)])
def test_weights_refusals(host_lib, change, status):         # noqa: F811
    assert host_lib.attn_weights_packed(C.byref(_set(_weights(), **change)), None) == status


def test_weights_without_queries_or_keys_do_nothing(host_lib):  # noqa: F811
    for change in (dict(Tq=0), dict(Tk=0), dict(Tq=0, workspace=None, workspace_bytes=0)):
        assert host_lib.attn_weights_packed(C.byref(_set(_weights(), **change)), None) == 0
    p = _weights()
    tc = host_lib.attn_weights_packed_workspace(C.byref(p))
    p.weights = None                                         # a size query needs no output
    assert host_lib.attn_weights_packed_workspace(C.byref(p)) == tc > 0
    assert host_lib.attn_weights_packed_workspace(C.byref(_set(_weights(), dtype=sa.F32))) == 20 * 8 * 4
    assert host_lib.attn_weights_packed_workspace(C.byref(_set(_weights(), D=0))) == 0


def _select():
    return _set(sa.SelectParams(), weights=0x1000000, block_table=0x2000000, ctx_len=0x3000000, keep=0x4000000,
                new_len=0x5000000, B=2, Hkv=2, page_tokens=16, max_pages=4, num_pages=8, budget=32, sink=4, recent=8)


@pytest.mark.parametrize("change,status", [
    (dict(weights=None), -1), (dict(block_table=None), -1), (dict(ctx_len=None), -1), (dict(keep=None), -1),
    (dict(B=0), -2), (dict(Hkv=0), -2), (dict(page_tokens=0), -2), (dict(max_pages=-1), -2), (dict(num_pages=0), -2),
    (dict(budget=0), -2), (dict(sink=-1), -2), (dict(recent=-1), -2), (dict(sink=25, recent=8), -2),
    (dict(sink=1 << 62, recent=1 << 62), -2),
    (dict(max_pages=(1 << 18) + 1), -7), (dict(page_tokens=K31), -7), (dict(budget=K31), -7), (dict(B=1 << 30), -7),
    (dict(num_pages=(1 << 31) - 1, Hkv=(1 << 20) - 1, page_tokens=1 << 22, max_pages=1), -7),
    (dict(weights=0x1000002), -4), (dict(keep=0x4000001), -4), (dict(new_len=0x5000002), -4), (dict(ctx_len=0x3000001), -4),
    (dict(keep=0x1000000), -6), (dict(keep=0x2000010), -6), (dict(keep=0x3000000), -6), (dict(new_len=0x3000000), -6),
    (dict(new_len=0x4000000), -6), (dict(new_len=0x1000000), -6), (dict(new_len=0x2000000), -6)])
def test_select_refusals(host_lib, change, status):          # noqa: F811
    assert host_lib.paged_kv_select(C.byref(_set(_select(), **change)), None) == status


def _compact():
    return _set(sa.CompactParams(), k_pool=0x10000000, v_pool=0x20000000, weights=0x30000000, block_table=0x40000000,
                ctx_len=0x41000000, keep=0x42000000, dtype=sa.BF16, pool_format=sa.FP8_E4M3_PAGE, B=2, Hkv=2, D=128,
                page_tokens=16, max_pages=4, num_pages=8, width=32)


@pytest.mark.parametrize("change,status", [
    (dict(k_pool=None), -1), (dict(v_pool=None), -1), (dict(block_table=None), -1), (dict(ctx_len=None), -1), (dict(keep=None), -1),
    (dict(pool_format=5), -3), (dict(pool_format=0, dtype=9), -3),
    (dict(B=0), -2), (dict(Hkv=0), -2), (dict(D=0), -2), (dict(width=0), -2), (dict(page_tokens=-1), -2),
    (dict(D=96), -7), (dict(page_tokens=24), -7), (dict(pool_format=0, D=1025), -7), (dict(width=K31), -7),
    (dict(num_pages=1 << 30, Hkv=4), -7), (dict(max_pages=1 << 28), -7),
    (dict(k_pool=0x10000008), -4), (dict(pool_format=0, v_pool=0x20000001), -4), (dict(weights=0x30000002), -4),
    (dict(keep=0x42000002), -4),
    (dict(v_pool=0x10000000), -6), (dict(weights=0x10000100), -6), (dict(keep=0x20000000), -6), (dict(ctx_len=0x30000000), -6),
    (dict(block_table=0x10000010), -6)])
def test_compact_refusals(host_lib, change, status):         # noqa: F811
    assert host_lib.paged_kv_compact(C.byref(_set(_compact(), **change)), None) == status


def _decode():
    return _set(sa.PagedParams(), q=0x1000000, k_pool=0x10000000, v_pool=0x20000000, block_table=0x2000000, ctx_len=0x3000000,
                y=0x4000000, dtype=sa.BF16, B=2, Hq=8, Hkv=2, D=128, page_tokens=16, max_pages=4, num_pages=8,
                pool_format=sa.FP8_E4M3_PAGE, workspace=0x6000000, workspace_bytes=1 << 24)


@pytest.mark.parametrize("change,weights,status", [
    (dict(), None, -1), (dict(q=None), 0x30000000, -1), (dict(), 0x30000002, -4), (dict(options=1, pool_format=0), 0x30000000, -7),
    (dict(max_pages=1 << 27), 0x30000000, -7), (dict(B=4096, max_pages=1 << 26), 0x30000000, -7),
    (dict(), 0x10000000, -6), (dict(), 0x20000400, -6), (dict(), 0x1000000, -6), (dict(), 0x4000000, -6), (dict(), 0x2000000, -6),
    (dict(), 0x3000000, -6), (dict(), 0x6000000, -6), (dict(workspace=None), 0x30000000, -5),
    (dict(workspace_bytes=4096), 0x30000000, -5), (dict(pool_format=0, workspace_bytes=4096), 0x30000000, -5)])
def test_decode_weights_refusals(host_lib, change, weights, status):  # noqa: F811
    assert host_lib.paged_attn_decode_weights(C.byref(_set(_decode(), **change)), weights, None) == status


def test_decode_weights_workspace_holds_the_scores(host_lib):  # noqa: F811
    for fmt in (0, sa.FP8_E4M3_PAGE):
        p = _set(_decode(), pool_format=fmt)
        own = host_lib.paged_attn_decode_workspace(C.byref(p))
        assert host_lib.paged_attn_decode_weights_workspace(C.byref(p)) >= own + 2 * 8 * 64 * 4
    assert host_lib.paged_attn_decode_weights_workspace(C.byref(_set(_decode(), options=1, pool_format=0))) == 0

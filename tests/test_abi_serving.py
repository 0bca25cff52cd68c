"""CPU-only checks of the serving-step entry points: struct layouts, and the
host-side refusals (fake addresses; every request below is refused before
anything is launched)."""
import ctypes as C

import pytest

import sparse_top_kv_validate_gb300 as sa
from test_abi import _c_layout, host_lib, lib  # noqa: F401  (fixtures)


@pytest.mark.parametrize("cname,py", [("sa_rope", sa.RopeTable), ("sa_rope_config", sa._RopeConfig),
                                      ("sa_rotary_params", sa.RotaryParams),
                                      ("sa_kv_pages_params", sa.KvPagesParams),
                                      ("sa_packed_params", sa.PackedParams),
                                      ("sa_paged_params", sa.PagedParams)])
def test_struct_layout_matches_header(cname, py):
    fields = [f for f, _ in py._fields_]
    size, offs = _c_layout(cname, fields)
    assert C.sizeof(py) == size
    assert [getattr(py, f).offset for f in fields] == offs


def _rope(R=64):
    return sa.rope_table(R)


def _set(p, **kw):
    for k, v in kw.items():
        if isinstance(v, (list, tuple)):
            getattr(p, k)[:] = v
        else:
            setattr(p, k, v)
    return p


def _rotary(keep):
    p = sa.RotaryParams()
    keep.append(_rope())
    return _set(p, q=0x100000, k=0x200000, q_out=0x300000, k_out=0x400000, positions=0x500000,
                rope=C.addressof(keep[-1]), dtype=sa.BF16, B=1, S=10, Hq=8, Hk=2, D=128,
                q_strides=[0, 1024, 128], k_strides=[0, 256, 128], q_out_strides=[0, 1024, 128],
                k_out_strides=[0, 256, 128])


@pytest.mark.parametrize("change,status", [
    (dict(q=None), -1), (dict(positions=None), -1), (dict(rope=None), -1), (dict(k_out=None), -1),
    (dict(dtype=9), -3), (dict(B=0), -2), (dict(Hq=0), -2), (dict(S=-1), -2), (dict(D=0), -2),
    (dict(D=32), -2),                                    # rotary_dim 64 beyond the head
    (dict(q_strides=[0, -1024, 128]), -2),
    (dict(q_out_strides=[0, 0, 128]), -2),               # rows on top of one another
    (dict(q_out_strides=[0, 1024, 64]), -2),
    (dict(q=0x100001), -4), (dict(positions=0x500002), -4),
    (dict(q_out=0x100000 + 256), -6), (dict(k_out=0x100000), -6), (dict(k_out=0x300000), -6),
    (dict(positions=0x300000), -6),
    (dict(S=1 << 31), -7), (dict(D=512, q_strides=[0, 4096, 512], k_strides=[0, 1024, 512],
                                 q_out_strides=[0, 4096, 512], k_out_strides=[0, 1024, 512]), -7)])
def test_rotary_refusals(host_lib, change, status):      # noqa: F811
    keep = []
    assert host_lib.rotary_embed(C.byref(_set(_rotary(keep), **change)), None) == status


def test_rotary_takes_interleaved_views_in_place_and_empty_calls(host_lib):  # noqa: F811
    keep = []
    # q and k are heads of one buffer, rotated in place: no overlap is found, and S = 0
    # launches nothing
    p = _set(_rotary(keep), S=0, k=0x100000 + 8 * 256, q_out=0x100000, k_out=0x100000 + 8 * 256,
             q_strides=[0, 1536, 128], k_strides=[0, 1536, 128], q_out_strides=[0, 1536, 128],
             k_out_strides=[0, 1536, 128])
    assert host_lib.rotary_embed(C.byref(p), None) == 0
    # the same views one head further into each other
    p = _set(p, S=10, k=0x100000 + 7 * 256, k_out=0x100000 + 7 * 256)
    assert host_lib.rotary_embed(C.byref(p), None) == -6


def _pages():
    p = sa.KvPagesParams()
    return _set(p, k=0x100000, v=0x200000, k_pool=0x10000000, v_pool=0x20000000, block_table=0x300000,
                ctx_len=0x400000, seq_start=0x500000, dtype=sa.BF16, pool_format=sa.FP8_E4M3_PAGE, T=20,
                B=2, Hkv=2, D=128, page_tokens=16, max_pages=4, num_pages=8, k_strides=[256, 128],
                v_strides=[256, 128])


@pytest.mark.parametrize("change,status", [
    (dict(k=None), -1), (dict(v_pool=None), -1), (dict(ctx_len=None), -1), (dict(block_table=None), -1),
    (dict(dtype=3), -3), (dict(pool_format=2), -3), (dict(B=0), -2), (dict(T=-1), -2), (dict(page_tokens=0), -2),
    (dict(seq_start=None), -2), (dict(k_strides=[-256, 128]), -2),
    (dict(D=96), -7), (dict(page_tokens=8), -7), (dict(max_pages=1 << 28), -7), (dict(pool_format=0, D=2000), -7),
    (dict(k_pool=0x10000008), -4), (dict(k=0x100001), -4),
    (dict(v_pool=0x10000000 + 4096), -6), (dict(k=0x10000000), -6)])
def test_page_write_and_read_refusals(host_lib, change, status):  # noqa: F811
    for fn in (host_lib.paged_kv_write, host_lib.paged_kv_read):
        assert fn(C.byref(_set(_pages(), **change)), None) == status


def test_page_read_refuses_a_rotation_and_one_output_for_both(host_lib):  # noqa: F811
    rope = _rope()
    p = _set(_pages(), rope=C.addressof(rope))
    assert host_lib.paged_kv_read(C.byref(p), None) == -7
    p = _set(_pages(), v=0x100000)
    assert host_lib.paged_kv_read(C.byref(p), None) == -6
    rope.reserved_ = 1
    p = _set(_pages(), rope=C.addressof(rope))
    assert host_lib.paged_kv_write(C.byref(p), None) == -2
    p = _set(_pages(), rope=C.addressof(_rope(256)))
    assert host_lib.paged_kv_write(C.byref(p), None) == -2


def _fp8_decode():
    p = sa.PagedParams()
    return _set(p, q=0x100000, y=0x200000, k_pool=0x10000000, v_pool=0x20000000, block_table=0x300000,
                ctx_len=0x400000, dtype=sa.F16, pool_format=sa.FP8_E4M3_PAGE, B=2, Hq=8, Hkv=2, D=128,
                page_tokens=16, max_pages=4, num_pages=8)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=sa.F32), -3), (dict(pool_format=7), -3), (dict(D=96), -7), (dict(page_tokens=24), -7),
    (dict(options=sa.OPT_ROW_COPIES), -7), (dict(B=8193), -7), (dict(k_new=0x700000), -1),
    (dict(k_pool=0x10000004), -4), (dict(y=0x200002), -4), (dict(y=0x20000000 + 64), -6),
    (dict(max_pages=1 << 27), -7), (dict(Hq=7), -2)])
def test_fp8_page_decode_refusals(host_lib, change, status):  # noqa: F811
    assert host_lib.paged_attn_decode(C.byref(_set(_fp8_decode(), **change)), None) == status


@pytest.mark.parametrize("change", [dict(q=0x100008), dict(y=0x200008), dict(k_new=0x700001, v_new=0x800000)])
def test_fp8_page_decode_wants_aligned_rows(host_lib, change):  # noqa: F811
    assert host_lib.paged_attn_decode(C.byref(_set(_fp8_decode(), **change)), None) == -4


def test_fp8_page_decode_needs_its_workspace(host_lib):  # noqa: F811
    p = _fp8_decode()
    need = host_lib.paged_attn_decode_workspace(C.byref(p))
    assert need > 0
    assert host_lib.paged_attn_decode(C.byref(p), None) == -5
    _set(p, workspace=0x40000000, workspace_bytes=need - 1)
    assert host_lib.paged_attn_decode(C.byref(p), None) == -5
    _set(p, workspace=0x40000010, workspace_bytes=need)
    assert host_lib.paged_attn_decode(C.byref(p), None) == -4


def _packed():
    p = sa.PackedParams()
    return _set(p, q=0x1000000, k=0x2000000, v=0x3000000, y=0x4000000, q_start=0x500000, k_start=0x600000,
                dtype=sa.BF16, causal=1, B=2, Tq=20, Tk=30, Hq=8, Hkv=2, D=128, q_strides=[1024, 128],
                k_strides=[256, 128], v_strides=[256, 128], y_strides=[1024, 128])


@pytest.mark.parametrize("change,status", [
    (dict(q=None), -1), (dict(y=None), -1), (dict(q_start=None), -1), (dict(dtype=8), -3), (dict(B=0), -2),
    (dict(Hq=9), -2), (dict(Tq=-1), -2), (dict(k_start=None), -2), (dict(softcap=-1.0), -2),
    (dict(scale=float("inf")), -2), (dict(y_strides=[0, 128]), -2), (dict(k_strides=[-256, 128]), -2),
    (dict(D=258), -7), (dict(D=66), -7), (dict(Tq=1 << 30), -7), (dict(q=0x1000001), -4), (dict(y=0x1000000), -6),
    (dict(y=0x2000000 + 512), -6)])
def test_packed_prefill_refusals(host_lib, change, status):  # noqa: F811
    assert host_lib.attn_prefill_packed(C.byref(_set(_packed(), **change)), None) == status


def test_packed_prefill_without_queries_launches_nothing(host_lib):  # noqa: F811
    assert host_lib.attn_prefill_packed(C.byref(_set(_packed(), Tq=0)), None) == 0


@pytest.mark.parametrize("packed,py", [(sa._ROTARY, sa.RotaryParams), (sa._KV_PAGES, sa.KvPagesParams),
                                       (sa._PACKED, sa.PackedParams), (sa._PAGED, sa.PagedParams)])
def test_packed_parameters_are_the_structures(packed, py):
    """Field for field: every value packed comes out of the structure's field."""
    def flat(p):
        for name, _ in py._fields_:
            x = getattr(p, name)
            yield from x if isinstance(x, C.Array) else (x,)

    values = list(range(1, 1 + len(list(flat(py())))))
    p = py.from_buffer_copy(packed.pack(*values))
    assert packed.size == C.sizeof(py) and list(flat(p)) == values


@pytest.mark.parametrize("T", [(1 << 31) - 8, (1 << 31) - 256])
def test_token_counts_near_2_to_the_31_are_refused(host_lib, T):  # noqa: F811
    """The kernels round the tokens up to blocks in 32 bits."""
    keep = []
    p = _set(_rotary(keep), S=T, k=None, k_out=None, q_out=1 << 44)
    assert host_lib.rotary_embed(C.byref(p), None) == -7
    p = _set(p, S=T // 2 + 1, B=2, q_strides=[T * 1024, 1024, 128], q_out_strides=[T * 1024, 1024, 128])
    assert host_lib.rotary_embed(C.byref(p), None) == -7
    p = _set(_pages(), T=T, k=1 << 44, v=1 << 46)
    for fn in (host_lib.paged_kv_write, host_lib.paged_kv_read):
        assert fn(C.byref(p), None) == -7


def test_sizes_whose_products_leave_64_bits_are_refused(host_lib):  # noqa: F811
    big = dict(num_pages=(1 << 31) - 1, Hkv=1 << 19, page_tokens=(1 << 31) - 16, max_pages=1, k_strides=[1 << 26, 128],
               v_strides=[1 << 26, 128])
    for fmt in (sa.FP8_E4M3_PAGE, 0):
        p = _set(_pages(), pool_format=fmt, **big)
        for fn in (host_lib.paged_kv_write, host_lib.paged_kv_read):
            assert fn(C.byref(p), None) == -7
        p = _set(_fp8_decode(), pool_format=fmt, num_pages=1 << 40, Hkv=1 << 20, Hq=1 << 20, page_tokens=16)
        assert host_lib.paged_attn_decode(C.byref(p), None) == -7
    keep = []
    p = _set(_rotary(keep), S=1 << 30, k=None, k_out=None, q_out=1 << 44, q_strides=[0, (1 << 40) - 128, 128])
    assert host_lib.rotary_embed(C.byref(p), None) == -2
    p = _set(_packed(), Tq=(1 << 30) - 1, q_strides=[(1 << 40) - 128, 128])
    assert host_lib.attn_prefill_packed(C.byref(p), None) == -2


def test_fused_views_of_several_batches_do_not_overlap(host_lib):  # noqa: F811
    """q and k as heads of one [B, Hq + 2 Hk, S, D] or [B, S, Hq + 2 Hk, D] buffer, rotated in
    place; without a device the launch itself is what fails."""
    keep = []
    B, S, D, heads = 3, 10, 128, 12
    for token, head in ((D, S * D), (heads * D, D)):
        st = [heads * S * D, token, head]
        k = 0x100000 + 8 * head * 2
        p = _set(_rotary(keep), B=B, S=S, k=k, q_out=0x100000, k_out=k, q_strides=st, k_strides=st, q_out_strides=st,
                 k_out_strides=st)
        assert host_lib.rotary_embed(C.byref(p), None) not in (0, -6)
        for shift in (1, -1):                             # a head into each other, in every batch
            x = k + shift * head * 2
            assert host_lib.rotary_embed(C.byref(_set(p, k=x, k_out=x)), None) == (-6 if shift < 0 else -8)
        # the next batch's queries: a batch stride too short for the heads
        short = [10 * S * D - 128, token, head]
        p = _set(p, k=k, k_out=k, q_strides=short, k_strides=short, q_out_strides=short, k_out_strides=short)
        assert host_lib.rotary_embed(C.byref(p), None) in (-6, -2)


def test_threads_do_not_share_the_kept_scratch(monkeypatch):
    """A call is several launches; two threads' launches on one stream may alternate."""
    import threading

    import torch
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(sa, "new_workspace", lambda n, device: torch.empty(n, dtype=torch.uint8))
    device, got = torch.device("cuda", 0), {}

    def work(name):
        got[name] = [sa._stream_workspace(n, device, 7, None)[0] for n in (1 << 21, 1 << 10)]
        got[name].append(sa._kept_workspace(device, 7))
        barrier.wait()

    barrier = threading.Barrier(2)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for mine in got.values():                            # kept within a thread
        assert mine[0] is mine[1] and mine[0] is mine[2]
    assert got[0][0].data_ptr() != got[1][0].data_ptr()


def test_a_stream_or_a_workspace_of_another_device_is_refused():
    """Stand-ins for what a second device would give: the checks read nothing else."""
    import types

    import torch
    device, other = torch.device("cuda", 0), torch.device("cuda", 1)
    with pytest.raises(ValueError):
        with sa._launching(device, types.SimpleNamespace(device=other, cuda_stream=5)):
            pass

    class Elsewhere(torch.Tensor):
        device, is_cuda = other, True

    with pytest.raises(ValueError):
        sa._stream_workspace(16, device, 5, torch.empty(16, dtype=torch.uint8).as_subclass(Elsewhere))


@pytest.mark.parametrize("name,params", [("paged_attn_decode", sa.PagedParams), ("rotary_embed", sa.RotaryParams),
                                         ("paged_kv_write", sa.KvPagesParams), ("paged_kv_read", sa.KvPagesParams),
                                         ("attn_prefill_packed", sa.PackedParams)])
def test_entries_check_the_structure_they_are_given(lib, name, params):  # noqa: F811
    fn = getattr(lib, name)
    assert fn(None, None) == -1
    for wrong in (C.byref(sa.PrefillParams()), bytes(C.sizeof(params)), 0x1000):
        with pytest.raises(C.ArgumentError):
            fn(wrong, None)


def test_callers_that_never_set_the_field_before_pool_format(host_lib):  # noqa: F811
    """The field was padding: what an older caller left there changes nothing."""
    assert host_lib.sa_version() >= 200
    need = host_lib.paged_attn_decode_workspace(C.byref(_set(_fp8_decode(), pool_format=0)))
    assert need > 0
    for rubbish in (0x40490FDB, -1, 256, 0x7FFFFFFF, -(1 << 31)):
        p = _set(_fp8_decode(), pool_format=rubbish)
        assert host_lib.paged_attn_decode_workspace(C.byref(p)) == need
        assert host_lib.paged_attn_decode(C.byref(p), None) == -5
    for fmt in (1, 2, 3, 5, 255):
        assert host_lib.paged_attn_decode(C.byref(_set(_fp8_decode(), pool_format=fmt)), None) == -3

"""Refusals of the rotary append and of the 4-bit operators: every bad argument is reported before any launch
(no GPU needed)."""
import ctypes

import pytest
import torch

BIG = 1 << 44


@pytest.fixture(scope="module")
def ta():
    import tree_masked_speculative_gb300 as m
    return m


def _b(ta, code, nbytes=BIG, ptr=0x10000, reserved=0):
    return ta.Buf(ptr, nbytes, code, reserved)


def _call(ta, fn, p, bufs):
    before = ta.ta_launch_count()
    st = fn(ctypes.byref(p) if p is not None else None, *[ctypes.byref(b) if b is not None else None for b in bufs], None)
    assert ta.ta_launch_count() == before
    return st, ta.ta_last_error()


def _refused(ta, fn, p, names, codes, buf, change, want, frag):
    bufs = {n: _b(ta, codes.get(n, ta.TA_F16)) for n in names}
    if buf is not None:
        c = dict(change or {})
        bufs[buf] = None if change is None else _b(ta, getattr(ta, c.pop("code")) if "code" in c else bufs[buf].dtype, **c)
    st, msg = _call(ta, fn, p, bufs.values())
    assert st == want and frag in msg, msg


def test_struct_sizes(ta):
    assert ctypes.sizeof(ta.RotaryAppendParams) == 40 + 11 * 8
    assert ctypes.sizeof(ta.QuantAppendParams) == 40 + 14 * 8
    assert ctypes.sizeof(ta.PagedQuantParams) == 56 + 10 * 8


def test_null_params(ta):
    for fn, n in ((ta.lib.paged_rotary_append, 9), (ta.lib.paged_quant_append, 11), (ta.lib.paged_quant_read, 7),
                  (ta.lib.paged_quant_attn_fwd, 11)):
        st, msg = _call(ta, fn, None, [None] * n)
        assert st == 1 and "NULL" in msg
    assert ta.lib.paged_quant_attn_workspace_bytes(None) == 2 ** 64 - 1


ROTARY = dict(tokens=10, n_heads=4, n_kv_heads=2, head_dim=128, page_size=16, n_pages=5, rotary_dim=64, max_positions=100)
ROTARY_BUFS = ["q", "k_new", "v_new", "slot_map", "positions", "table", "q_out", "k_cache", "v_cache"]
SIZES = [
    (dict(n_kv_heads=0), None, None, 1, "n_kv_heads"),
    (dict(n_pages=0), None, None, 1, "n_pages"),
    (dict(head_dim=96), None, None, 1, "head_dim"),
    (dict(page_size=48), None, None, 1, "page_size"),
    (dict(n_heads=65536), None, None, 4, "index range"),
    (dict(tokens=2 ** 30, n_heads=1, n_kv_heads=1), None, None, 4, "index range"),
    (dict(rotary_dim=8), None, None, 1, "rotary_dim"),
    (dict(rotary_dim=144), None, None, 1, "rotary_dim"),
    (dict(interleaved=2), None, None, 1, "interleaved"),
    (dict(max_positions=2 ** 31), None, None, 4, "max_positions"),
    (dict(q_token_stride=260), None, None, 1, "q_token_stride"),
    (dict(q_out_head_stride=4), None, None, 1, "q_out_head_stride"),
    (dict(k_head_stride=1 << 38), None, None, 4, "k_head_stride"),
    (dict(n_heads=0), None, None, 1, "absent"),
    ({}, "q", None, 1, "q"),
    ({}, "q", dict(code="TA_BF16"), 1, "q dtype"),
    ({}, "q_out", dict(nbytes=10 * 512 * 2 - 1), 2, "q_out"),
    (dict(q_out_token_stride=1024), None, None, 1, "its strides"),
    ({}, "k_new", dict(code="TA_F32"), 1, "k_new dtype"),
    ({}, "k_new", dict(nbytes=10 * 256 * 2 - 1), 2, "k_new"),
    ({}, "v_new", dict(ptr=0x10008), 1, "aligned"),
    ({}, "slot_map", dict(code="TA_I32"), 1, "slot_map dtype"),
    ({}, "slot_map", dict(nbytes=79), 2, "slot_map"),
    ({}, "positions", dict(code="TA_I64"), 1, "positions dtype"),
    ({}, "positions", None, 1, "positions"),
    ({}, "positions", dict(nbytes=39), 2, "positions"),
    ({}, "table", None, 1, "table"),
    ({}, "table", dict(code="TA_F16"), 1, "table dtype"),
    ({}, "table", dict(nbytes=100 * 64 * 4 - 1), 2, "table"),
    ({}, "table", dict(ptr=0x10004), 1, "aligned"),
]


def _rot_codes(ta):
    return dict(slot_map=ta.TA_I64, positions=ta.TA_I32, table=ta.TA_F32, k_codes=ta.TA_U32, v_codes=ta.TA_U32,
                cu=ta.TA_I32, kv_lens=ta.TA_I32, parents=ta.TA_I32, tmp=ta.TA_F32)


@pytest.mark.parametrize("kw,buf,change,want,frag", SIZES + [
    (dict(rotary_dim=0), None, None, 1, "rotary_dim"),
    (dict(reserved=1), None, None, 1, "reserved"),
    (dict(page_stride=4), None, None, 1, "page_stride"),
    (dict(n_pages=2 ** 31 - 1, page_stride=2 ** 37), None, None, 3, "overflow"),
    ({}, "k_cache", dict(code="TA_BF16"), 1, "k_cache dtype"),
    ({}, "v_cache", dict(nbytes=5 * 16 * 256 * 2 - 1), 2, "v_cache"),
    ({}, "v_cache", None, 1, "v_cache"),
])
def test_rotary_append_rejections(ta, kw, buf, change, want, frag):
    _refused(ta, ta.lib.paged_rotary_append, ta.RotaryAppendParams(**{**ROTARY, **kw}), ROTARY_BUFS, _rot_codes(ta), buf,
             change, want, frag)


QUANT = dict(ROTARY, group_size=64)
QUANT_BUFS = ROTARY_BUFS[:7] + ["k_codes", "k_affine", "v_codes", "v_affine"]
PAGES = [
    (dict(group_size=16), None, None, 1, "group_size"),
    (dict(group_size=128), None, None, 1, "group_size"),
    (dict(codes_token_stride=18), None, None, 1, "codes"),
    (dict(affine_token_stride=6), None, None, 1, "affine"),
    (dict(affine_page_stride=1 << 30), None, None, 4, "stride"),

    ({}, "k_codes", dict(code="TA_I32"), 1, "k_codes dtype"),
    ({}, "v_codes", dict(nbytes=5 * 16 * 2 * 64 - 1), 2, "v_codes"),
    ({}, "v_codes", dict(ptr=0x10004), 1, "aligned"),
    ({}, "k_affine", dict(code="TA_BF16"), 1, "k_affine dtype"),
    ({}, "k_affine", dict(nbytes=5 * 16 * 2 * 8 - 1), 2, "k_affine"),
    ({}, "v_affine", None, 1, "v_affine"),
]


@pytest.mark.parametrize("kw,buf,change,want,frag", SIZES + PAGES + [(dict(rotary_dim=0), None, None, 1, "without a rotation")])
def test_quant_append_rejections(ta, kw, buf, change, want, frag):
    _refused(ta, ta.lib.paged_quant_append, ta.QuantAppendParams(**{**QUANT, **kw}), QUANT_BUFS, _rot_codes(ta), buf,
             change, want, frag)


READ = dict(tokens=10, n_kv_heads=2, head_dim=128, page_size=16, n_pages=5, group_size=64)
READ_BUFS = ["slot_map", "k_codes", "k_affine", "v_codes", "v_affine", "k", "v"]


@pytest.mark.parametrize("kw,buf,change,want,frag", PAGES + [
    (dict(n_heads=1), None, None, 1, "must be 0"),
    (dict(rotary_dim=16), None, None, 1, "must be 0"),
    (dict(tokens=2 ** 30), None, None, 4, "index range"),
    ({}, "k", dict(code="TA_F32"), 1, "k dtype"),
    ({}, "v", dict(code="TA_BF16"), 1, "v dtype"),
    ({}, "v", dict(nbytes=10 * 256 * 2 - 1), 2, "v"),
    ({}, "slot_map", dict(nbytes=79), 2, "slot_map"),
    (dict(v_token_stride=12), None, None, 1, "v_token_stride"),
])
def test_quant_read_rejections(ta, kw, buf, change, want, frag):
    _refused(ta, ta.lib.paged_quant_read, ta.QuantAppendParams(**{**READ, **kw}), READ_BUFS, _rot_codes(ta), buf, change,
             want, frag)


ATTEND = dict(batch=3, n_heads=8, n_kv_heads=2, head_dim=128, tokens=12, max_q_len=4, page_size=16, n_pages=5, max_pages=4,
              group_size=64, scale=0.1)
ATTEND_BUFS = ["q", "k_codes", "k_affine", "v_codes", "v_affine", "table", "cu", "kv_lens", "parents", "tmp", "out"]


@pytest.mark.parametrize("kw,buf,change,want,frag", PAGES + [
    (dict(batch=0), None, None, 1, "batch"),
    (dict(batch=65536), None, None, 4, "index range"),
    (dict(n_heads=9), None, None, 1, "divisible"),
    (dict(n_heads=258), None, None, 4, "128 query heads"),
    (dict(head_dim=512), None, None, 1, "head_dim"),
    (dict(max_q_len=0), None, None, 1, "max_q_len"),
    (dict(page_size=8), None, None, 1, "page_size"),
    (dict(n_pages=0), None, None, 1, "n_pages"),
    (dict(max_pages=1 << 27), None, None, 4, "index range"),
    (dict(window=1 << 31), None, None, 4, "index range"),
    (dict(kernel=4), None, None, 1, "kernel"),
    (dict(scale=float("nan")), None, None, 1, "scale"),
    (dict(reserved=7), None, None, 1, "reserved"),
    (dict(window=5), None, None, 1, "window must be 0 with parents"),
    (dict(max_q_len=257), None, None, 4, "max_q_len <= 256"),
    (dict(q_head_stride=132), None, None, 1, "q_head_stride"),
    ({}, "q", dict(code="TA_F32"), 1, "q dtype"),
    ({}, "q", dict(nbytes=12 * 1024 * 2 - 1), 2, "q"),
    ({}, "table", dict(nbytes=47), 2, "table"),
    ({}, "cu", dict(nbytes=12), 2, "cu"),
    ({}, "kv_lens", None, 1, "kv_lens"),
    ({}, "parents", dict(nbytes=44), 2, "parents"),
    ({}, "tmp", dict(nbytes=8), 2, "tmp"),
    ({}, "out", dict(code="TA_BF16"), 1, "out dtype"),
])
def test_attention_rejections(ta, kw, buf, change, want, frag):
    _refused(ta, ta.lib.paged_quant_attn_fwd, ta.PagedQuantParams(**{**ATTEND, **kw}), ATTEND_BUFS,
             dict(_rot_codes(ta), table=ta.TA_I32), buf,
             change, want, frag)


def test_nothing_to_do_launches_nothing(ta):
    for fn, p, n in ((ta.lib.paged_rotary_append, ta.RotaryAppendParams(**{**ROTARY, "tokens": 0}), 9),
                     (ta.lib.paged_quant_append, ta.QuantAppendParams(**{**QUANT, "tokens": 0}), 11),
                     (ta.lib.paged_quant_read, ta.QuantAppendParams(**{**READ, "tokens": 0}), 7),
                     (ta.lib.paged_quant_attn_fwd, ta.PagedQuantParams(**{**ATTEND, "tokens": 0}), 11)):
        assert _call(ta, fn, p, [None] * n)[0] == 0


@pytest.mark.parametrize("kw,status,frag", [(dict(head_dim=80), 1, "head_dim"), (dict(group_size=8), 1, "group_size"),
                                            (dict(n_heads=258), 4, "128 query heads")])
def test_a_refused_workspace_names_the_status(ta, kw, status, frag):
    with pytest.raises(ta.TreeAttentionError, match=frag) as e:
        ta._workspace(ta.PagedQuantParams(**{**ATTEND, **kw}), torch.device("cuda"))
    assert e.value.status == status


def test_python_refuses_host_tensors_and_shapes(ta):
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    slot, pos, table = torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 64)
    cache = ta.paged_quant_cache(3, 2, 16, 64, group_size=32, dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_append_rotary(x, x, x, x[None], x[None], slot, pos, table)
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_quant_append(x, x, cache, slot)
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_quant_read(cache, slot)
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_quant_attention(x, cache, pos[None], pos, pos, scale=1.0, max_q_len=1)
    for kw in (dict(group_size=48), dict(group_size=128), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            ta.paged_quant_cache(3, 2, 16, 64, **{**dict(group_size=32, dtype=torch.float16, device="cpu"), **kw})


def test_new_rows_refusals(ta):
    """What both appends check of their rows, on host tensors."""
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    slot, pos, table = torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 64)
    good = dict(q=x, k_new=x, v_new=x, slot_map=slot, positions=pos, rotary=table, q_out=None, hk=2, d=64, dev=-1)
    assert ta._new_rows(**good)[:4] == (4, 2, 64, 8)
    for kw, frag in ((dict(k_new=x[:3]), "k_new"), (dict(hk=3), "k_new"), (dict(slot_map=slot[:3]), "slot_map"),
                     (dict(q=x[:3]), "q must"), (dict(q=x[:, :0]), "q must"), (dict(q_out=x[:3]), "q_out"),
                     (dict(q=None, q_out=x), "q_out without q"), (dict(positions=None), "positions"),
                     (dict(positions=pos[:3]), "positions"), (dict(rotary=table[0]), "rotary"),
                     (dict(rotary=None), "rotary table"), (dict(rotary=None, positions=None), "rotary table")):
        with pytest.raises(ValueError, match=frag):
            ta._new_rows(**{**good, **kw})


def test_cache_refusals(ta):
    """What the 4-bit operators check of a cache, on host tensors."""
    c = ta.paged_quant_cache(3, 2, 16, 128, group_size=32, dtype=torch.float16, device="cpu")
    assert ta._quant_cache(c, -1)[:5] == (3, 2, 16, 128, 32)
    nhd = [torch.zeros(3, 16, 2, *x.shape[3:], dtype=x.dtype).transpose(1, 2) for x in c]
    got = ta._quant_cache(nhd, -1)
    assert got[:5] == (3, 2, 16, 128, 32) and got[5] == (16 * 2 * 16, 16, 32, 16 * 2 * 8, 8, 16)
    for parts, frag in (((c[0].long(), *c[1:]), "int32"), ((c[0][:2], *c[1:]), "one shape"),
                        ((c[0], c[1][:2], c[2], c[3][:2]), "a cache is"), ((c[0], c[1][..., 0], c[2], c[3][..., 0]), "a cache is"),
                        ((c[0], c[1].transpose(3, 4).contiguous().transpose(3, 4), c[2], c[3]), "contiguous"),
                        ((nhd[0], c[1], c[2], c[3]), "same strides")):
        with pytest.raises(ValueError, match=frag):
            ta._quant_cache(parts, -1)


def test_rotary_table_angles(ta):
    t = ta.rotary_table(100001, 32, device="cpu")
    import math
    for p, i in ((0, 0), (1, 3), (99999, 0), (100000, 15), (54321, 7)):
        a = p * 10000.0 ** (-2 * i / 32)
        assert abs(t[p, i] - math.cos(a)) < 1e-7 and abs(t[p, 16 + i] - math.sin(a)) < 1e-7


@pytest.mark.parametrize("h,hk,d,new,kernel,scale,tensor_cores", [
    (32, 8, 128, 4, 0, 0.1, False), (32, 8, 128, 5, 0, 0.1, True), (17, 1, 64, 1, 0, 0.1, True), (16, 1, 64, 1, 0, 0.0, False),
    (8, 1, 256, 1, 0, 0.1, False), (9, 1, 256, 1, 0, 0.1, True), (32, 8, 128, 1, 2, 0.1, True), (32, 8, 128, 5, 3, 0.1, True),
    (32, 8, 128, 5, 1, 0.1, False), (32, 8, 128, 5, 2, -0.1, False)])
def test_kernel_choice(ta, h, hk, d, new, kernel, scale, tensor_cores):
    """Up to 16 rows a KV head (8 with head_dim 256) stay off the tensor-core kernel, as a negative scale does."""
    p = ta.PagedQuantParams(**{**ATTEND, "tokens": 0, "n_heads": h, "n_kv_heads": hk, "head_dim": d, "max_q_len": new,
                               "kernel": kernel, "scale": scale})
    fn = lambda *a: ta.lib.ta_test_paged_quant_attn_fwd_wait_limit(1, *a)
    st, msg = _call(ta, fn, p, [None] * 11)
    assert st == (0 if tensor_cores else 4)
    assert tensor_cores or "tensor-core kernel only" in msg

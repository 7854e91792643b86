"""Refusals of the serving entry points: every bad argument is reported before
any launch (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def ta():
    import tree_masked_speculative_gb300 as m
    return m


BIG = 1 << 44


def _b(ta, code, nbytes=BIG, ptr=0x10000, reserved=0):
    return ta.Buf(ptr, nbytes, code, reserved)


def _call(ta, fn, p, bufs):
    before = ta.ta_launch_count()
    st = fn(ctypes.byref(p) if p is not None else None, *[ctypes.byref(b) if b is not None else None for b in bufs], None)
    assert ta.ta_launch_count() == before
    return st, ta.ta_last_error()


def test_struct_sizes(ta):
    assert ctypes.sizeof(ta.PlanParams) == 24
    assert ctypes.sizeof(ta.AppendParams) == 24 + 7 * 8
    assert ctypes.sizeof(ta.PagedParams) == 48 + 7 * 8
    assert ctypes.sizeof(ta.PromptParams) == 32 + 8 * 8


PLAN = dict(batch=4, page_size=16, max_pages=8, capacity=64, max_tokens=100)
PLAN_BUFS = ["keep", "fresh", "held", "table", "stack", "n_free", "held_out", "n_free_out", "cu", "kv_lens",
             "slot_map", "positions", "status"]


@pytest.mark.parametrize("kw,buf,change,want,frag", [
    (dict(batch=0), None, None, 1, "batch"),
    (dict(batch=16385), None, None, 4, "batch"),
    (dict(page_size=24), None, None, 1, "page_size"),
    (dict(page_size=8), None, None, 1, "page_size"),
    (dict(max_pages=0), None, None, 1, "max_pages"),
    (dict(max_pages=1 << 30), None, None, 4, "index range"),
    (dict(reserved=1), None, None, 1, "reserved"),
    ({}, "table", dict(nbytes=4 * 8 * 4 - 1), 2, "table"),
    ({}, "cu", dict(nbytes=16), 2, "cu"),
    ({}, "slot_map", dict(nbytes=799), 2, "slot_map"),
    ({}, "slot_map", dict(ptr=0x10004), 1, "aligned"),
    ({}, "slot_map", dict(code="TA_I32"), 1, "slot_map dtype"),
    ({}, "keep", dict(code="TA_I64"), 1, "keep dtype"),
    ({}, "status", None, 1, "status"),
    ({}, "positions", dict(reserved=3), 1, "reserved"),
])
def test_plan_rejections(ta, kw, buf, change, want, frag):
    p = ta.PlanParams(**{**PLAN, **kw})
    bufs = {n: _b(ta, ta.TA_I64 if n == "slot_map" else ta.TA_I32) for n in PLAN_BUFS}
    if buf is not None:
        if change is None:
            bufs[buf] = None
        else:
            c = dict(change)
            code = getattr(ta, c.pop("code")) if "code" in c else bufs[buf].dtype
            bufs[buf] = _b(ta, code, **c)
    st, msg = _call(ta, ta.lib.paged_plan_build, p, bufs.values())
    assert st == want and frag in msg, msg


def test_null_params(ta):
    for fn, n in ((ta.lib.paged_plan_build, 13), (ta.lib.paged_kv_append, 5), (ta.lib.paged_attn_fwd, 9),
                  (ta.lib.prompt_attn_fwd, 6)):
        st, msg = _call(ta, fn, None, [None] * n)
        assert st == 1 and "NULL" in msg
    assert ta.lib.paged_attn_workspace_bytes(None) == 2 ** 64 - 1
    assert ta.lib.prompt_attn_workspace_bytes(None) == 2 ** 64 - 1


APPEND = dict(tokens=10, n_kv_heads=2, head_dim=128, page_size=16, n_pages=5)


@pytest.mark.parametrize("kw,buf,change,want,frag", [
    (dict(n_kv_heads=0), None, None, 1, "n_kv_heads"),
    (dict(n_pages=0), None, None, 1, "n_pages"),
    (dict(head_dim=96), None, None, 1, "head_dim"),
    (dict(page_size=48), None, None, 1, "page_size"),
    (dict(k_token_stride=260), None, None, 1, "k_token_stride"),
    (dict(page_stride=1 << 38), None, None, 4, "page_stride"),
    (dict(n_pages=2 ** 31 - 1, page_stride=2 ** 37), None, None, 3, "overflow"),
    ({}, 0, dict(code="TA_F32"), 1, "k_new dtype"),
    ({}, 1, dict(code="TA_BF16"), 1, "v_new dtype"),
    ({}, 2, dict(code="TA_BF16"), 1, "k_cache dtype"),
    ({}, 2, dict(ptr=0x10008), 1, "aligned"),
    ({}, 0, dict(nbytes=10 * 256 * 2 - 1), 2, "k_new"),
    ({}, 3, dict(nbytes=5 * 16 * 256 * 2 - 1), 2, "v_cache"),
    ({}, 4, dict(code="TA_I32"), 1, "slot_map dtype"),
    ({}, 4, dict(nbytes=79), 2, "slot_map"),
    ({}, 4, None, 1, "slot_map"),
])
def test_append_rejections(ta, kw, buf, change, want, frag):
    p = ta.AppendParams(**{**APPEND, **kw})
    bufs = [_b(ta, ta.TA_F16) for _ in range(4)] + [_b(ta, ta.TA_I64)]
    if buf is not None:
        c = dict(change or {})
        bufs[buf] = None if change is None else _b(ta, getattr(ta, c.pop("code")) if "code" in c else bufs[buf].dtype, **c)
    st, msg = _call(ta, ta.lib.paged_kv_append, p, bufs)
    assert st == want and frag in msg, msg


def test_nothing_to_do_launches_nothing(ta):
    none = [None] * 9
    assert _call(ta, ta.lib.paged_kv_append, ta.AppendParams(**{**APPEND, "tokens": 0}), none[:5])[0] == 0
    assert _call(ta, ta.lib.paged_attn_fwd, ta.PagedParams(**{**PAGED, "tokens": 0}), none)[0] == 0
    assert _call(ta, ta.lib.prompt_attn_fwd, ta.PromptParams(**{**PROMPT, "tokens": 0}), none[:6])[0] == 0


PAGED = dict(batch=3, n_heads=8, n_kv_heads=2, head_dim=128, tokens=12, max_q_len=4, page_size=16, n_pages=9,
             max_pages=4, scale=0.1)
PAGED_BUFS = ["q", "k_cache", "v_cache", "table", "cu", "kv_lens", "parents", "tmp", "out"]


@pytest.mark.parametrize("kw,buf,change,want,frag", [
    (dict(batch=0), None, None, 1, "batch"),
    (dict(batch=65536), None, None, 4, "index range"),
    (dict(n_heads=9), None, None, 1, "divisible"),
    (dict(n_heads=258), None, None, 4, "128 query heads"),
    (dict(head_dim=512), None, None, 1, "head_dim"),
    (dict(head_dim=80), None, None, 1, "head_dim"),
    (dict(max_q_len=0), None, None, 1, "max_q_len"),
    (dict(page_size=0), None, None, 1, "page_size"),
    (dict(page_size=512), None, None, 1, "page_size"),
    (dict(n_pages=0), None, None, 1, "n_pages"),
    (dict(max_pages=0), None, None, 1, "max_pages"),
    (dict(max_pages=1 << 27), None, None, 4, "index range"),
    (dict(window=1 << 31), None, None, 4, "index range"),
    (dict(tokens=2 ** 30), None, None, 4, "index range"),
    (dict(n_heads=2, tokens=2 ** 23, max_q_len=2 ** 23, max_pages=2 ** 22, head_dim=64), None, None, 4, "tokens x keys"),
    (dict(kernel=4), None, None, 1, "kernel"),
    (dict(scale=float("nan")), None, None, 1, "scale"),
    (dict(scale=float("inf")), None, None, 1, "scale"),
    (dict(window=5), None, None, 1, "window must be 0 with parents"),
    (dict(max_q_len=257), None, None, 4, "max_q_len <= 256"),
    (dict(q_head_stride=132), None, None, 1, "q_head_stride"),
    (dict(token_stride=4), None, None, 1, "token_stride"),
    (dict(head_stride=1 << 40), None, None, 4, "head_stride"),
    ({}, "q", dict(code="TA_F32"), 1, "q dtype"),
    ({}, "q", dict(nbytes=12 * 1024 * 2 - 1), 2, "q"),
    ({}, "q", dict(ptr=0x10002), 1, "aligned"),
    ({}, "k_cache", dict(code="TA_BF16"), 1, "k_cache dtype"),
    ({}, "v_cache", dict(nbytes=9 * 16 * 256 * 2 - 2), 2, "v_cache"),
    ({}, "table", dict(nbytes=47), 2, "table"),
    ({}, "table", dict(code="TA_I64"), 1, "table dtype"),
    ({}, "cu", dict(nbytes=12), 2, "cu"),
    ({}, "kv_lens", None, 1, "kv_lens"),
    ({}, "parents", dict(nbytes=44), 2, "parents"),
    ({}, "parents", dict(code="TA_I64"), 1, "parents dtype"),
    ({}, "tmp", dict(nbytes=8), 2, "tmp"),
    ({}, "tmp", dict(code="TA_F16"), 1, "tmp dtype"),
    ({}, "out", dict(code="TA_F32"), 1, "out dtype"),
    ({}, "out", None, 1, "out"),
    ({}, "out", dict(reserved=1), 1, "reserved"),
])
def test_paged_rejections(ta, kw, buf, change, want, frag):
    p = ta.PagedParams(**{**PAGED, **kw})
    codes = dict(table=ta.TA_I32, cu=ta.TA_I32, kv_lens=ta.TA_I32, parents=ta.TA_I32, tmp=ta.TA_F32)
    bufs = {n: _b(ta, codes.get(n, ta.TA_F16)) for n in PAGED_BUFS}
    if buf is not None:
        c = dict(change or {})
        bufs[buf] = None if change is None else _b(ta, getattr(ta, c.pop("code")) if "code" in c else bufs[buf].dtype, **c)
    st, msg = _call(ta, ta.lib.paged_attn_fwd, p, bufs.values())
    assert st == want and frag in msg, msg


PROMPT = dict(batch=3, n_heads=8, n_kv_heads=2, head_dim=128, tokens=12, scale=0.1)
PROMPT_BUFS = ["q", "k", "v", "cu", "tmp", "out"]


@pytest.mark.parametrize("kw,buf,change,want,frag", [
    (dict(n_kv_heads=0), None, None, 1, "n_kv_heads"),
    (dict(n_heads=7), None, None, 1, "divisible"),
    (dict(head_dim=32), None, None, 1, "head_dim"),
    (dict(window=2 ** 32 - 1), None, None, 4, "index range"),
    (dict(n_heads=2, tokens=2 ** 23, head_dim=64), None, None, 4, "tokens x keys"),
    (dict(n_heads=128, n_kv_heads=1, tokens=2 ** 21), None, None, 4, "tokens x keys"),
    (dict(kernel=9), None, None, 1, "kernel"),
    (dict(v_token_stride=12), None, None, 1, "v_token_stride"),
    (dict(k_head_stride=1 << 39), None, None, 4, "k_head_stride"),
    ({}, "k", dict(code="TA_BF16"), 1, "k dtype"),
    ({}, "v", dict(nbytes=12 * 256 * 2 - 1), 2, "v"),
    ({}, "v", dict(ptr=0x10001), 1, "aligned"),
    ({}, "cu", dict(code="TA_F32"), 1, "cu dtype"),
    ({}, "tmp", None, 1, "tmp"),
    ({}, "out", dict(nbytes=0), 2, "out"),
])
def test_prompt_rejections(ta, kw, buf, change, want, frag):
    p = ta.PromptParams(**{**PROMPT, **kw})
    codes = dict(cu=ta.TA_I32, tmp=ta.TA_F32)
    bufs = {n: _b(ta, codes.get(n, ta.TA_F16)) for n in PROMPT_BUFS}
    if buf is not None:
        c = dict(change or {})
        bufs[buf] = None if change is None else _b(ta, getattr(ta, c.pop("code")) if "code" in c else bufs[buf].dtype, **c)
    st, msg = _call(ta, ta.lib.prompt_attn_fwd, p, bufs.values())
    assert st == want and frag in msg, msg


def test_python_refuses_host_tensors(ta):
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        ta.prompt_attention(x, x, x, torch.tensor([0, 4], dtype=torch.int32), scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_append(x, x, x[None], x[None], torch.zeros(4, dtype=torch.int64))


def test_work_counted_within_32_bits_is_taken(ta):
    # a window, another family and a smaller request leave the range alone: the next check speaks
    for kw in (dict(window=4096), dict(kernel=1), dict(tokens=2 ** 22)):
        p = ta.PromptParams(**{**PROMPT, **dict(n_heads=2, tokens=2 ** 23, head_dim=64), **kw})
        st, msg = _call(ta, ta.lib.prompt_attn_fwd, p, [None] * 6)
        assert st == 1 and "q dtype" in msg, msg


def test_a_stream_of_another_device_is_refused(ta, monkeypatch):
    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

    made = []
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: made.append((handle, device)))
    mine = Stream(1)
    assert ta._as_stream(mine, 1) is mine
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        ta._as_stream(Stream(0), 1)
    ta._as_stream(0x1234, 1)
    assert made == [(0x1234, 1)]


def test_stream_handles_of_the_default_stream(ta, monkeypatch):
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle, device))
    for handle in (0, 1):
        assert ta._as_stream(handle, 1) == ("default", 1)
    assert ta._as_stream(0x1230, 1) == ("external", 0x1230, 1)


@pytest.mark.parametrize("kw,status,frag", [(dict(head_dim=80), 1, "head_dim"), (dict(batch=65536), 4, "index range"),
                                            (dict(n_heads=258), 4, "128 query heads"), ({}, 5, "no CUDA device"),
                                            (dict(tokens=0), 5, "no CUDA device")])
def test_a_refused_workspace_names_the_status(ta, kw, status, frag):
    if status == 5 and torch.cuda.is_available():
        pytest.skip("a device is visible")
    for p in (ta.PagedParams(**{**PAGED, **kw}), ta.PromptParams(**{**PROMPT, **kw})):
        before = ta.ta_launch_count()
        with pytest.raises(ta.TreeAttentionError, match=frag) as e:
            ta._workspace(p, torch.device("cuda"))
        assert e.value.status == status and ta.ta_launch_count() == before


def test_the_wait_limit_hook_takes_the_tensor_core_kernel_alone(ta):
    f16, i32 = _b(ta, ta.TA_F16), _b(ta, ta.TA_I32)
    bufs = [ctypes.byref(b) for b in (f16, f16, f16, i32, i32, i32)] + [None, ctypes.byref(_b(ta, ta.TA_F32)), ctypes.byref(f16)]
    for kernel in (0, 1, 3):                    # 16 rows a KV head: the warp-MMA kernel, or the CUDA cores
        p, before = ta.PagedParams(**{**PAGED, "kernel": kernel}), ta.ta_launch_count()
        assert ta.lib.ta_test_paged_attn_fwd_wait_limit(0, ctypes.byref(p), *bufs, None) == 4
        assert "tensor-core kernel only" in ta.ta_last_error() and ta.ta_launch_count() == before
    assert ta.lib.ta_test_paged_attn_fwd_wait_limit(0, None, *bufs, None) == 1


@pytest.mark.parametrize("d,rows,batch,hk,auto,asked", [
    (64, 16, 4, 2, True, True), (64, 17, 4, 2, False, False), (128, 16, 300, 90, True, True), (128, 17, 4, 2, False, False),
    (256, 8, 4, 2, True, True), (256, 1, 3, 3, False, True), (256, 9, 4, 2, False, False)])
def test_the_kernel_choice(ta, d, rows, batch, hk, auto, asked):
    """The warp-MMA kernel by itself and when asked for; else the tensor-core kernel (the one that
    the hook takes: there the next check, of tmp, speaks)."""
    f16, i32 = _b(ta, ta.TA_F16), _b(ta, ta.TA_I32)
    bufs = [ctypes.byref(b) for b in (f16, f16, f16, i32, i32, i32)] + [None, None, ctypes.byref(f16)]
    for kernel, mma in ((0, auto), (3, asked)):
        p = ta.PagedParams(**{**PAGED, "head_dim": d, "n_heads": hk, "n_kv_heads": hk, "max_q_len": rows, "batch": batch,
                              "kernel": kernel})
        st = ta.lib.ta_test_paged_attn_fwd_wait_limit(0, ctypes.byref(p), *bufs, None)
        assert (st, "tensor-core kernel only" in ta.ta_last_error()) == ((4, True) if mma else (1, False))


@pytest.mark.parametrize("at,value", [(0, -1), (0, 2 ** 32), (11, 1e300), (11, "x"), (12, -8)])
def test_values_that_no_field_holds_are_refused(ta, at, value):
    """A negative or too large size, a scale past f32: ValueError before the call."""
    values = [1, 8, 2, 128, 4, 4, 0, 16, 9, 4, 0, 0.1] + [0] * 7 + [0, 0, 0, 0] * 9
    values[at] = value
    before = ta.ta_launch_count()
    with pytest.raises(ValueError, match="out of range"):
        ta._paged_entry(0, *values)
    assert ta.ta_launch_count() == before

"""What the Python names of include/bitq_lm.h do with tensors that do not hold what the call reads (no GPU needed: every
refusal comes before the library is called, and what passes ends at its device check)."""
import pytest
import torch

import bit_plane_gemv_amd as bq

GPU = torch.cuda.is_available()
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731


def buffer(n):
    """n bytes at a multiple of 256."""
    b = torch.zeros(n + 256, dtype=torch.uint8)
    at = -b.data_ptr() % 256
    return b[at:at + n]


def passes(call):
    """The arguments are taken; there is no device here."""
    if GPU:
        pytest.skip("addresses of host memory")
    with pytest.raises(bq.BitqError) as e:
        call()
    assert e.value.status in (bq.E_DEVICE, bq.E_UNSUPPORTED), bq.last_error()


KV = bq.kvdesc(2, 64, 16, 10)
CACHE = buffer(bq.kv_cache_size(KV))


def plan(**k):
    d = bq.kv_plan_desc(3, 16, 4, 10, 20)
    a = dict(old_len=i32(3), new_len=i32(3), ring=i32(10), state=i32(4), table=i32(3, 4))
    a.update(k)
    return lambda: bq.kv_plan(d, *a.values(), buffer(bq.kv_plan_size(d)), stream=0)


def write(T=5, **k):
    a = dict(k=torch.zeros(T, 2, 64), v=torch.zeros(T, 2, 64), x_dtype=bq.DT_F32, slots=i32(T), cache=CACHE)
    a.update(k)
    return lambda: bq.kv_write(KV, **a, stream=0)


def attn(R=3, **k):
    d = bq.attn_desc(KV, 4, R, 4, 40, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    a = dict(q=torch.zeros(R, 4, 64), cache=CACHE, table=i32(R, 4), lens=i32(R), out=torch.zeros(R, 4, 64), ws=None)
    a.update(k)
    return lambda: bq.paged_attn(d, **a, stream=0)


@pytest.mark.parametrize("dtype", [torch.int64, torch.int16, torch.float32, torch.bool])
@pytest.mark.parametrize("name", ["old_len", "new_len", "ring", "state", "table"])
def test_plan_takes_int32_only(name, dtype):
    with pytest.raises(TypeError, match=name):
        plan(**{name: torch.zeros(12, dtype=dtype)})()


@pytest.mark.parametrize("name,bad", [("old_len", i32(2)), ("new_len", i32(6)[::2]), ("ring", i32(9)), ("state", i32(1)),
                                      ("table", i32(2, 4)), ("table", i32(4, 3).t()), ("table", i32(3, 5)[:, :4])])
def test_plan_takes_as_many_as_the_descriptor_says(name, bad):
    with pytest.raises(ValueError, match=name):
        plan(**{name: bad})()


def test_plan_takes_views_that_hold_them():
    passes(plan())
    passes(plan(state=buffer(8), table=i32(12), old_len=i32(8)[2:5]))
    d = bq.kv_plan_desc(3, 16, 4, 10, 20)
    passes(plan(old_len=bq.kv_plan_views(d, buffer(bq.kv_plan_size(d)))["len"], table=i32(3, 4)[:, :3]))
    passes(plan(ring=1 << 20, state=1 << 21))                       # addresses


@pytest.mark.parametrize("slots", [torch.zeros(5, dtype=torch.int64), torch.zeros(5)])
def test_write_takes_int32_slots_only(slots):
    with pytest.raises(TypeError, match="slots"):
        write(slots=slots)()


def test_write_takes_slots_in_a_row():
    passes(write())
    with pytest.raises(ValueError, match="slots"):
        write(slots=i32(10)[::2])()
    with pytest.raises(ValueError, match="slots"):
        write(slots=i32(4), tokens=5)()


@pytest.mark.parametrize("name", ["table", "lens"])
def test_attention_takes_int32_only(name):
    passes(attn())
    for dtype in (torch.int64, torch.float32):
        with pytest.raises(TypeError, match=name):
            attn(**{name: torch.zeros((3, 4) if name == "table" else 3, dtype=dtype)})()


@pytest.mark.parametrize("name,bad", [("lens", i32(2)), ("lens", i32(6)[::2]), ("table", i32(11)), ("table", i32(4, 3).t()),
                                      ("table", i32(3, 6)[:, :4])])
def test_attention_takes_as_many_as_the_descriptor_says(name, bad):
    with pytest.raises(ValueError, match=name):
        attn(**{name: bad})()


f32 = lambda *s: torch.zeros(s)  # noqa: E731


@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("bad,error", [
    (f32(4, 2, 64), ValueError),                              # fewer rows than slots: they would be read past the end
    (f32(5, 2, 63), ValueError), (f32(5, 64, 2).transpose(1, 2), ValueError), (f32(5, 2, 128)[..., ::2], ValueError),
    (f32(2, 5, 64).transpose(0, 1), ValueError),              # heads outermost
    (f32(5, 2, 64).to(torch.bfloat16), TypeError), (f32(5, 2, 64).double(), TypeError), (f32(5, 2, 64).half(), TypeError),
])
def test_write_takes_the_rows_it_reads(name, bad, error):
    with pytest.raises(error, match=name):
        write(**{name: bad})()


def test_write_reads_a_row_for_every_slot_of_the_list():
    """A plan's list holds the most tokens of a step, padded with -1: k and v with fewer rows are refused, unless `tokens`
    says how many slots to take."""
    p = bq.kv_plan_views(bq.kv_plan_desc(3, 16, 4, 10, 20), buffer(bq.kv_plan_size(bq.kv_plan_desc(3, 16, 4, 10, 20))))
    with pytest.raises(ValueError, match="k has shape"):
        write(slots=p["slot"])()
    passes(write(slots=p["slot"], tokens=5))
    passes(write(T=20, slots=p["slot"]))


def test_write_takes_views_that_hold_the_rows():
    passes(write(k=f32(5, 4, 64)[:, :2], v=f32(5, 4, 64)[:, 2:]))
    passes(write(k=f32(5, 128), v=f32(9, 3, 2, 64)[:, 1]))
    passes(write(k=f32(5, 2, 64).to(torch.bfloat16), v=torch.zeros(5, 2, 64, dtype=torch.int16), x_dtype=bq.DT_BF16))
    passes(write(k=f32(2000), v=f32(2000), k_stride=130, v_stride=128))
    passes(write(k=1 << 20, v=1 << 21, k_stride=130, v_stride=128))


@pytest.mark.parametrize("name,bad,error", [
    ("q", f32(2, 4, 64), ValueError), ("q", f32(4, 3, 64).transpose(0, 1), ValueError), ("q", f32(3, 64, 4).transpose(1, 2), ValueError),
    ("q", f32(3, 4, 63), ValueError), ("q", f32(3, 4, 64).to(torch.bfloat16), TypeError), ("q", f32(3, 4, 64).half(), TypeError),
    ("out", f32(3, 4, 63), ValueError), ("out", f32(4, 3, 64).transpose(0, 1), ValueError),
    ("out", torch.zeros(3, 4, 64, dtype=torch.bfloat16), TypeError), ("lse", f32(3, 3), ValueError),
    ("lse", torch.zeros(3, 4, dtype=torch.bfloat16), TypeError),
])
def test_attention_takes_what_the_descriptor_says(name, bad, error):
    with pytest.raises(error, match=name):
        attn(**{name: bad})()


def test_attention_takes_views_that_hold_the_rows():
    passes(attn(q=f32(3, 8, 64)[:, :4], out=f32(3, 256), lse=f32(12)))
    passes(attn(q=f32(3, 300), out=f32(4, 4, 64)))
    passes(attn(q=1 << 20, q_stride=256, table=1 << 21, lens=1 << 22, out=1 << 23))


def test_a_single_row_has_any_stride():
    """The stride of a dimension of size 1 is arbitrary: a transposed or expanded single row is still one row."""
    one = f32(2, 1, 64).transpose(0, 1)
    assert one.stride(0) == 64
    passes(write(T=1, k=one, v=one))
    passes(write(T=1, k=f32(2, 64).expand(1, 2, 64)))
    d = bq.attn_desc(KV, 4, 1, 4, 40, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    passes(lambda: bq.paged_attn(d, f32(4, 1, 64).transpose(0, 1), CACHE, i32(1, 4), i32(1), f32(1, 4, 64), None, stream=0))


def test_names_of_the_older_calls_are_untouched():
    """The binding's own abbreviations do not hide each other (a launch shape needs ctypes integers)."""
    grid, block = bq.ctx_launch_shape(bq.wdesc("rabit", 11008, 4096), 1, bq.DT_BF16, 0)
    assert grid > 0 and block > 0

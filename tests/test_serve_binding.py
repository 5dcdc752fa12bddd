"""What the Python names of the operators that serve prompts and shared pages do with tensors that do not hold what the call
reads (no GPU needed: what passes ends at the library's device check)."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
from test_lm_binding import CACHE, KV, buffer, f32, i32, passes


def prompt(**k):
    d = bq.prompt_desc(KV, 4, 3, 7, 4, 40, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    a = dict(q=f32(7, 4, 64), cache=CACHE, table=i32(3, 4), start=i32(4), lens=i32(3), out=f32(7, 4, 64),
             ws=buffer(max(256, bq.prompt_attn_workspace(d))))
    a.update(k)
    return lambda: bq.prompt_attn(d, **a, stream=0)


def shared(**k):
    d = bq.shared_desc(bq.attn_desc(KV, 4, 3, 4, 40, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32), 2, 30)
    a = dict(q=f32(3, 4, 64), cache=CACHE, table=i32(3, 4), lens=i32(3), start=i32(3), prefix=i32(2), out=f32(3, 4, 64),
             ws=buffer(bq.shared_attn_workspace(d)))
    a.update(k)
    return lambda: bq.shared_attn(d, **a, stream=0)


def pages(fn, **k):
    d = bq.kv_pages_desc(3, 16, 4, 10, 10)
    a = dict(src=i32(3), keep=i32(3), lens=i32(3), ring=i32(10), state=i32(4), table=i32(3, 4), table_out=i32(3, 4))
    if fn is bq.kv_compact:
        a = dict(lens=i32(3), table=i32(3, 4), table_out=i32(3, 4), ring=i32(10))
    a.update(k)
    return lambda: fn(d, *a.values(), buffer(bq.kv_pages_size(d)), buffer(bq.kv_pages_workspace(d)), stream=0)


def rope(**k):
    d = bq.rope_desc(5, 4, 2, 64, x_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    a = dict(q=f32(5, 4, 64), k=f32(5, 2, 64), q_w=f32(64), k_w=f32(64), table=torch.from_numpy(bq.rope_table(64)), pos=i32(5),
             q_out=f32(5, 4, 64), k_out=f32(5, 2, 64))
    a.update(k)
    return lambda: bq.qk_rope(d, **a, stream=0)


CALLS = [("prompt", prompt, ["table", "start", "lens"]), ("shared", shared, ["table", "lens", "start", "prefix"]),
         ("fork", lambda **k: pages(bq.kv_fork, **k), ["src", "keep", "lens", "ring", "state", "table", "table_out"]),
         ("compact", lambda **k: pages(bq.kv_compact, **k), ["lens", "ring", "table", "table_out"]), ("rope", rope, ["pos"])]


@pytest.mark.parametrize("make,name", [pytest.param(m, n, id=f"{c}-{n}") for c, m, names in CALLS for n in names])
def test_whole_numbers_are_int32_and_as_many_as_the_descriptor_says(make, name):
    passes(make())
    for dtype in (torch.int64, torch.int16, torch.float32, torch.bool):
        with pytest.raises(TypeError, match=name):
            make(**{name: torch.zeros((3, 4) if "table" in name else 16, dtype=dtype)})()
    for bad in (i32(1), i32(12)[::2]):
        with pytest.raises(ValueError, match=name):
            make(**{name: bad})()


@pytest.mark.parametrize("make,rows", [(prompt, 7), (shared, 3)], ids=["prompt", "shared"])
def test_attention_takes_the_rows_it_reads(make, rows):
    for name, bad, error in (("q", f32(rows - 1, 4, 64), ValueError), ("q", f32(rows, 4, 63), ValueError),
                             ("q", f32(4, rows, 64).transpose(0, 1), ValueError), ("q", f32(rows, 4, 64).half(), TypeError),
                             ("out", f32(rows, 4, 63), ValueError), ("out", f32(rows, 4, 64).bfloat16(), TypeError),
                             ("lse", f32(rows, 3), ValueError), ("lse", f32(rows, 4).double(), TypeError)):
        with pytest.raises(error, match=name):
            make(**{name: bad})()
    passes(make(q=f32(rows, 8, 64)[:, :4], lse=f32(rows, 4)))
    passes(make(q=f32(rows + 3, 400), out=f32(rows * 256)))
    if make is shared:                               # (a prompt this short is not split)
        with pytest.raises(bq.BitqError) as e:
            make(ws=None)()
        assert e.value.status == bq.E_ARG


def test_rope_takes_the_rows_it_reads():
    for name, bad, error in (("q", f32(4, 4, 64), ValueError), ("k", f32(5, 2, 63), ValueError), ("q", f32(5, 4, 64).bfloat16(), TypeError),
                             ("q_out", f32(5, 4, 64).bfloat16(), TypeError), ("k_out", f32(2, 5, 64).transpose(0, 1), ValueError),
                             ("q_w", f32(63), ValueError), ("k_w", f32(64).double(), TypeError), ("table", f32(32), TypeError),
                             ("table", torch.zeros(31, dtype=torch.int64), ValueError), ("table", torch.zeros(64, dtype=torch.int64)[::2], ValueError)):
        with pytest.raises(error, match=name):
            rope(**{name: bad})()
    qkv = f32(5, 8, 64)
    passes(rope(q=qkv[:, :4], k=qkv[:, 4:6], q_out=qkv[:, :4], k_out=qkv[:, 4:6]))
    passes(rope(q_w=None, k_w=None, table=torch.from_numpy(bq.rope_table(64).view(np.int64))))
    passes(rope(q=1 << 20, k=1 << 21, q_out=1 << 22, k_out=1 << 23, strides=(256, 128, 256, 128)))
    d = bq.rope_desc(5, 4, 0, 64, x_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    passes(lambda: bq.qk_rope(d, f32(5, 4, 64), None, None, None, torch.from_numpy(bq.rope_table(64)), i32(5), f32(5, 4, 64), None, stream=0))


def test_copy_takes_lists_of_int32():
    passes(lambda: bq.kv_copy(KV, i32(5), i32(5), CACHE, stream=0))
    passes(lambda: bq.kv_copy(KV, i32(9), i32(5), CACHE, stream=0))
    for a, b, moves, error, name in ((torch.zeros(5), i32(5), None, TypeError, "frm"), (i32(4), i32(5), None, ValueError, "frm"),
                                     (i32(5), i32(4), 5, ValueError, "to"), (i32(5), i32(10)[::2], None, ValueError, "to")):
        with pytest.raises(error, match=name):
            bq.kv_copy(KV, a, b, CACHE, moves=moves, stream=0)

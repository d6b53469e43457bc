"""What the calls for pages, rotary positions and prompt attention refuse, at
the C entry points and in the Python layer (no GPU: nothing is launched)."""
import ctypes
import os
import subprocess

import pytest
import torch

import draft_token_verification_sv_gb300 as sv
from draft_token_verification_sv_gb300 import build as _build

from test_kv_arguments import Stand, _ints, fake_streams  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def N():
    _build.build()
    from draft_token_verification_sv_gb300 import _native
    _native.lib()
    return _native


ELSE = ctypes.c_void_p(0x20000000)
A, ODD, OFF4 = ctypes.c_void_p(0x10000000), ctypes.c_void_p(0x10000001), ctypes.c_void_p(0x10000004)


def test_struct_layout_matches_c(N, tmp_path):
    names = {"sv_kv_assign_desc": N.KvAssignDesc, "sv_rope_desc": N.RopeDesc, "sv_prompt_attention_desc": N.PromptAttentionDesc}
    lines = [f'printf("%zu\\n", sizeof({c}));' + "".join(f'printf("%zu\\n", offsetof({c}, {f[0]}));' for f in t._fields_) for c, t in names.items()]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spec_verify.h"\nint main(void) {' + "\n".join(lines)
                    + 'printf("%d %d\\n", SV_ROW_NO_PAGE, SV_MAX_ROPE_AXES); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    want = [x for t in names.values() for x in [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]]
    assert [int(x) for x in got] == want + [N.SV_ROW_NO_PAGE, N.SV_MAX_ROPE_AXES]


# ---- pages ----

def _assign(N, ptr=None, **kw):
    d = N.KvAssignDesc(4, 16, 100, 8, 3, 12, 10)
    for k, v in kw.items():
        setattr(d, k, v)
    at = dict(free=0x1000000, count=0x2000000, table=0x3000000, held=0x4000000, ctx=0x5000000, start=None, parents=None, slots=0x6000000,
              positions=0x7000000, status=0x8000000)
    at.update(ptr or {})
    return N.lib().sv_kv_assign(ctypes.byref(d), *(ctypes.c_void_p(at[n]) for n in at), None)


@pytest.mark.parametrize("field,value", [("batch", -1), ("batch", 65536), ("page_size", 8), ("page_size", 48), ("page_size", 256), ("num_pages", 0),
                                         ("max_pages", 0), ("max_pages", 1 << 27), ("max_new", -1), ("max_new", 4), ("total_new", 13), ("total_new", -1),
                                         ("table_stride", 7), ("table_stride", 1 << 40)])
def test_assign_refuses_descriptors(N, field, value):
    assert _assign(N, **{field: value}) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("name", ["free", "count", "table", "held", "ctx", "start", "parents", "slots", "positions", "status"])
def test_assign_refuses_pointers(N, name):
    assert _assign(N, {name: 0x9000002}) == N.SV_ERR_INVALID_ARGUMENT
    if name == "slots":
        assert _assign(N, {name: 0x9000004}) == N.SV_ERR_INVALID_ARGUMENT
    if name in ("free", "count", "table", "held", "ctx"):
        assert _assign(N, {name: None}) == N.SV_ERR_INVALID_ARGUMENT


# bytes of each: 4 sequences, 100 pages, rows of 8 entries 10 apart, 12 tokens
SIZES = dict(free=400, count=4, table=152, held=16, slots=96, positions=48, status=16, ctx=16, start=20, parents=48)


@pytest.mark.parametrize("written", ["free", "count", "table", "held", "slots", "positions", "status"])
@pytest.mark.parametrize("other", sorted(SIZES))
def test_assign_refuses_shared_memory(N, written, other):
    if written == other:
        pytest.skip("one array")
    at = 0xa000000
    for place in (at, at - SIZES[other] // 8 * 8 + (8 if SIZES[other] > 8 else 0), at + SIZES[written] // 8 * 8 - (8 if SIZES[written] > 8 else 0)):
        assert _assign(N, {written: at, other: place}) == N.SV_ERR_INVALID_ARGUMENT, hex(place)


def test_assign_without_sequences(N):
    assert _assign(N, batch=0, total_new=0) == N.SV_OK


def _pool(n=20, **kw):
    return dict(free=_ints(n, **kw), count=_ints(1, **kw))


def _assign_py(**kw):
    args = dict(pool=_pool(), page_table=_ints(4, 5), held=_ints(4, address=2 << 20), ctx_lens=_ints(4, address=3 << 20), page_size=16, max_new=3,
                out=(Stand((4, 3), torch.int64), _ints(4, 3)))
    args.update(kw)
    return lambda: sv.kv_assign(**args)


@pytest.mark.parametrize("bad", [
    dict(pool=dict(free=Stand((20,), torch.int64), count=_ints(1))), dict(pool=dict(free=_ints(4, 5), count=_ints(1))),
    dict(pool=dict(free=_ints(20, strides=(2,)), count=_ints(1))), dict(pool=dict(free=_ints(20), count=_ints(2))),
    dict(held=_ints(3)), dict(held=Stand((4,), torch.int64)), dict(ctx_lens=_ints(5)), dict(page_table=_ints(4, 5, strides=(4, 1))),
    dict(page_table=_ints(4, 5, strides=(10, 2))), dict(page_table=_ints(20)), dict(out=(_ints(4, 3), _ints(4, 3))),
    dict(out=(Stand((4, 3), torch.int64), _ints(12))), dict(max_new=4), dict(max_new=-1), dict(max_new=2 ** 31, new_start=_ints(5)),
    dict(new_start=_ints(4)), dict(parents=_ints(11)), dict(row_status=_ints(5)), dict(held=_ints(4, device="cuda:1")),
    dict(held=_ints(4, device="cpu")), dict(page_size=2 ** 31), dict(new_start=_ints(5), out=None), dict(new_start=_ints(5), total=11), dict(total=11),
], ids=lambda d: "-".join(d))
def test_assign_refuses_tensors(N, bad):
    with pytest.raises(ValueError):
        _assign_py(**bad)()


@pytest.mark.parametrize("page", [0, 7, 256])
def test_assign_refuses_page_sizes(N, page, monkeypatch):
    monkeypatch.setattr(sv.kvcache, "_current_device", lambda: 0)
    monkeypatch.setattr(sv.kvcache, "_raw_stream", lambda index: 0)
    with pytest.raises(sv.SVError, match="invalid argument"):
        _assign_py(page_size=page)()


# ---- rotary positions ----

def _rope(N, ptr=None, axis=None, **kw):
    d = N.RopeDesc(5, 4, 2, 64, 64, 1, 0, N.SV_BF16, 5, 256, 64, 128, 64, 256, 64, 128, 64)
    for k, v in kw.items():
        setattr(d, k, v)
    if axis:
        d.axis[axis[0]] = axis[1]
    at = dict(q=A, k=OFF4, positions=A, freq=A, q_out=A, k_out=OFF4)
    at.update(ptr or {})
    return N.lib().sv_rope(ctypes.byref(d), at["q"], at["k"], at["positions"], at["freq"], at["q_out"], at["k_out"], None)


@pytest.mark.parametrize("field,value", [("rows", -1), ("heads", 0), ("heads", 1 << 18), ("kv_heads", -1), ("head_dim", 8), ("head_dim", 72),
                                         ("head_dim", 272), ("rotary_dim", 0), ("rotary_dim", 63), ("rotary_dim", 66), ("axes", 0), ("axes", 5),
                                         ("adjacent", 2), ("dtype", 2), ("q_row_stride", 63), ("q_head_stride", 0), ("k_row_stride", -64),
                                         ("k_head_stride", 1 << 40), ("q_out_row_stride", 63), ("q_out_head_stride", 1), ("k_out_row_stride", 0),
                                         ("k_out_head_stride", 63)])
def test_rope_refuses_descriptors(N, field, value):
    assert _rope(N, **{field: value}) == N.SV_ERR_INVALID_ARGUMENT


def test_rope_refuses_axes(N):
    assert _rope(N, axis=(31, 1)) == N.SV_ERR_INVALID_ARGUMENT
    assert _rope(N, axes=2, position_stride=4) == N.SV_ERR_INVALID_ARGUMENT
    assert _rope(N, rows=0) == N.SV_OK


@pytest.mark.parametrize("name", ["q", "k", "positions", "freq", "q_out", "k_out"])
def test_rope_refuses_pointers(N, name):
    assert _rope(N, {name: None}) == N.SV_ERR_INVALID_ARGUMENT
    assert _rope(N, {name: ODD}) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("ptr,kw", [
    (dict(q_out=OFF4), {}), (dict(k_out=A), {}), (dict(q_out=ELSE, k_out=ELSE), {}), ({}, dict(q_out_row_stride=264)), ({}, dict(q_out_head_stride=72)),
    ({}, dict(k_out_row_stride=136)), ({}, dict(k_out_head_stride=72)), (dict(k_out=A), dict(kv_heads=1, rows=1)),
])
def test_rope_refuses_results_in_another_input_s_place(N, ptr, kw):
    assert _rope(N, ptr, **kw) == N.SV_ERR_INVALID_ARGUMENT


def _rope_py(**kw):
    args = dict(q=Stand((7, 4, 64)), k=Stand((7, 2, 64)), positions=_ints(7), inv_freq=Stand((32,)), out=(Stand((7, 4, 64)), Stand((7, 2, 64))))
    args.update(kw)
    return lambda: sv.rope(**args)


@pytest.mark.parametrize("bad,error", [
    (dict(positions=_ints(6)), ValueError), (dict(positions=_ints(2, 7)), ValueError), (dict(positions=_ints(2, 7), sections=(16,)), ValueError),
    (dict(positions=_ints(2, 7), sections=(16, 15)), ValueError), (dict(positions=_ints(2, 7), sections=(33, -1)), ValueError),
    (dict(positions=_ints(5, 7), sections=(8, 8, 8, 4, 4)), ValueError), (dict(positions=Stand((7,), torch.int64)), ValueError),
    (dict(positions=_ints(7, strides=(2,))), ValueError), (dict(sections=(16, 16)), ValueError), (dict(inv_freq=Stand((33,))), ValueError),
    (dict(inv_freq=Stand((0,))), ValueError), (dict(inv_freq=Stand((32,), torch.float64)), ValueError),
    (dict(inv_freq=Stand((32,), strides=(2,))), ValueError), (dict(q=Stand((7, 64))), ValueError), (dict(q=Stand((7, 4, 64), torch.float16)), TypeError),
    (dict(k=Stand((6, 2, 64))), ValueError), (dict(k=Stand((7, 2, 32))), ValueError), (dict(k=Stand((7, 2, 64), torch.bfloat16)), ValueError),
    (dict(out=(Stand((7, 4, 32)), Stand((7, 2, 64)))), ValueError), (dict(out=(Stand((7, 4, 64)), None)), ValueError),
    (dict(out=(None, Stand((7, 2, 64)))), ValueError), (dict(out=(Stand((7, 4, 64)), Stand((7, 3, 64)))), ValueError), (dict(q=Stand((7, 4, 64), strides=(256, 1, 4))), ValueError),
    (dict(positions=_ints(7, device="cuda:1")), ValueError), (dict(positions=_ints(7, device="cpu")), ValueError),
], ids=lambda d: "-".join(d) if isinstance(d, dict) else "")
def test_rope_refuses_tensors(N, bad, error):
    bad = dict(bad)
    if "q" in bad and "out" not in bad:
        bad["out"] = (bad["q"], Stand((7, 2, 64), bad["q"].dtype))
    if bad.get("q") is not None and bad["q"].dtype == torch.float16:
        bad["k"] = Stand((7, 2, 64), torch.float16)
    with pytest.raises(error):
        _rope_py(**bad)()


# ---- prompt attention ----

def _prompt_desc(N, **kw):
    d = N.PromptAttentionDesc(4, 8, 2, 64, 3, 12, N.SV_BF16, 0.125, 0, 0, 512, 64, 128, 64, 128, 64, 512, 64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _prompt(N, ptr=None, **kw):
    at = dict(q=A, k=A, v=A, start=None, out=OFF4, lse=None, status=None)
    at.update(ptr or {})
    return N.lib().sv_prompt_attention(ctypes.byref(_prompt_desc(N, **kw)), *(at[n] for n in at), None)


@pytest.mark.parametrize("field,value", [("batch", -1), ("batch", 65536), ("kv_heads", 0), ("kv_heads", 1025), ("kv_heads", 3), ("heads", 0),
                                         ("heads", 258), ("head_dim", 8), ("head_dim", 72), ("head_dim", 272), ("max_new", -1), ("total_new", 13),
                                         ("total_new", -1), ("dtype", 3), ("scale", float("nan")), ("scale", float("inf")), ("window", -1),
                                         ("sinks", -1), ("q_row_stride", 63), ("q_head_stride", 0), ("k_row_stride", -1), ("k_head_stride", 1 << 40),
                                         ("v_row_stride", 63), ("v_head_stride", 63), ("out_row_stride", 63), ("out_head_stride", 0)])
def test_prompt_attention_refuses_descriptors(N, field, value):
    assert _prompt(N, **{field: value}) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("name", ["q", "k", "v", "out"])
def test_prompt_attention_refuses_pointers(N, name):
    assert _prompt(N, {name: None}) == N.SV_ERR_INVALID_ARGUMENT
    assert _prompt(N, {name: ODD}) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("name", ["start", "lse", "status"])
def test_prompt_attention_refuses_words_off_their_boundary(N, name):
    assert _prompt(N, {name: ctypes.c_void_p(0x10000002)}) == N.SV_ERR_INVALID_ARGUMENT


def test_prompt_attention_without_sequences_and_with_too_many_rows(N):
    assert _prompt(N, batch=0, total_new=0) == N.SV_OK
    # rows times heads of a kv head pass 32 bits
    assert _prompt(N, {"start": A}, max_new=1 << 30, total_new=12) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_prompt_attention_refuses_results_in_an_input_s_place(N, name):
    assert _prompt(N, {name: OFF4}) == N.SV_ERR_INVALID_ARGUMENT


def test_prompt_attention_refuses_more_rows_than_items_are_counted_for(N):
    assert _prompt(N, {"start": A}, total_new=1 << 28) == N.SV_ERR_INVALID_ARGUMENT


def _prompt_py(**kw):
    rows = lambda h, t=torch.float32: Stand((12, h, 64), t)
    args = dict(q=rows(8), k=rows(2), v=rows(2), new_start=_ints(5), max_new=3, out=rows(8))
    args.update(kw)
    return lambda: sv.prompt_attention(**args)


@pytest.mark.parametrize("bad,error", [
    (dict(max_new=None), ValueError), (dict(max_new=2 ** 31), ValueError), (dict(new_start=None), ValueError), (dict(new_start=Stand((5,), torch.int64)), ValueError),
    (dict(new_start=_ints(0)), ValueError), (dict(k=Stand((11, 2, 64))), ValueError), (dict(k=Stand((12, 3, 64))), ValueError),
    (dict(v=Stand((12, 2, 32))), ValueError), (dict(k=Stand((12, 2, 64), torch.bfloat16)), ValueError), (dict(out=Stand((12, 8, 32))), ValueError),
    (dict(out=Stand((12, 8, 64), torch.bfloat16)), ValueError), (dict(window=2 ** 31), ValueError), (dict(sinks=-2 ** 31 - 1), ValueError),
    (dict(row_status=_ints(5)), ValueError), (dict(q=Stand((12, 8, 64), strides=(512, 1, 8))), ValueError),
    (dict(q=Stand((12, 8, 64), device="cuda:1"), out=Stand((12, 8, 64), device="cuda:1")), ValueError),
    (dict(new_start=_ints(5, device="cpu")), ValueError),
    (dict(q=Stand((12, 8, 64), torch.float16), k=Stand((12, 2, 64), torch.float16), v=Stand((12, 2, 64), torch.float16),
          out=Stand((12, 8, 64), torch.float16)), TypeError),
    (dict(q=Stand((4, 3, 8, 64)), out=Stand((4, 3, 8, 64)), new_start=None, max_new=None), ValueError),
    (dict(q=Stand((4, 3, 8, 64)), k=Stand((4, 3, 2, 64)), v=Stand((4, 3, 2, 64)), out=Stand((4, 3, 8, 64)), new_start=None, max_new=4), ValueError),
], ids=lambda d: "-".join(d) if isinstance(d, dict) else "")
def test_prompt_attention_refuses_tensors(N, bad, error):
    with pytest.raises(error):
        _prompt_py(**bad)()


# ---- streams ----

CALLS = {
    "assign": lambda **kw: sv.kv_assign(_pool(), _ints(4, 5), _ints(4), _ints(4), 16, max_new=3, **kw),
    "rope": lambda **kw: sv.rope(Stand((7, 4, 64)), Stand((7, 2, 64)), _ints(7), Stand((32,)), **kw),
    "prompt": lambda **kw: sv.prompt_attention(Stand((4, 3, 8, 64)), Stand((4, 3, 2, 64)), Stand((4, 3, 2, 64)), lse=True, **kw),
}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_results_belong_to_the_stream_they_are_made_on(N, call, fake_streams):  # noqa: F811
    Fake, made = fake_streams
    CALLS[call](stream=Fake("side"))
    assert made == [("side", ["main"])] * 2
    other = Fake("other")
    other.device_index = 1
    with pytest.raises(ValueError, match="another GPU"):
        CALLS[call](stream=other)

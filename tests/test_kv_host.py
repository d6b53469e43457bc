"""Refusals of the cache and attention entry points (no GPU): descriptors and
pointers that are wrong are rejected before anything is launched, and the
Python layer rejects tensors it cannot pass on."""
import ctypes

import pytest

A = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100008)  # 8-byte aligned only
MIS = ctypes.c_void_p(0x100001)


@pytest.fixture(scope="module")
def N():
    from draft_token_verification_sv_gb300 import build as b
    b.build()
    from draft_token_verification_sv_gb300 import _native
    _native.lib()
    return _native


def _kv(N, **kw):
    d = N.KvDesc(4, 2, 64, 16, 100, 8, 2 * 16 * 64, 16 * 64, 64, 8)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _rows(N, **kw):
    r = N.KvRowsDesc(3, 12, N.SV_BF16, 0, 128, 64, 128, 64)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _append(N, d, r, **p):
    a = dict(k=A, v=A, table=A, ctx=A, start=None, kc=A, vc=A, ks=A, vs=A, status=None)
    a.update(p)
    return N.lib().sv_kv_append(ctypes.byref(d) if d else None, ctypes.byref(r) if r else None, a["k"], a["v"], a["table"],
                                a["ctx"], a["start"], a["kc"], a["vc"], a["ks"], a["vs"], a["status"], None)


def _read(N, d, r, **p):
    a = dict(k=A, v=A, table=A, ctx=A, start=None, kc=A, vc=A, ks=A, vs=A, status=None)
    a.update(p)
    return N.lib().sv_kv_read(ctypes.byref(d) if d else None, ctypes.byref(r) if r else None, a["kc"], a["vc"], a["ks"], a["vs"],
                              a["table"], a["ctx"], a["start"], a["k"], a["v"], a["status"], None)


BAD_DESC = [dict(batch=-1), dict(batch=65536), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=0), dict(head_dim=72),
            dict(head_dim=272), dict(page_size=0), dict(page_size=48), dict(page_size=256), dict(num_pages=0),
            dict(max_pages=0), dict(max_pages=1 << 27), dict(page_stride=-16), dict(page_stride=1000), dict(head_stride=32),
            dict(token_stride=72), dict(token_stride=0), dict(table_stride=7), dict(table_stride=1 << 41)]


@pytest.mark.parametrize("bad", BAD_DESC, ids=lambda b: "-".join(f"{k}{v}" for k, v in b.items()))
def test_bad_cache_descriptor(N, bad):
    d = _kv(N, **bad)
    assert _append(N, d, _rows(N)) == N.SV_ERR_INVALID_ARGUMENT
    assert _read(N, d, _rows(N)) == N.SV_ERR_INVALID_ARGUMENT
    assert N.lib().sv_kv_commit(ctypes.byref(d), 8, 4, A, A, A, A, A, A, A, A, ctypes.c_void_p(0x200000), None,
                                None) == N.SV_ERR_INVALID_ARGUMENT
    a = _attention_desc(N, kv=d)
    assert N.lib().sv_kv_attention_workspace_size(ctypes.byref(a)) == 0
    assert _attend(N, a) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", [dict(max_new=-1), dict(total_new=-1), dict(total_new=11), dict(dtype=2), dict(reserved=1),
                                 dict(k_row_stride=63), dict(k_head_stride=0), dict(v_row_stride=-64),
                                 dict(v_head_stride=1 << 41)],
                         ids=lambda b: "-".join(f"{k}{v}" for k, v in b.items()))
def test_bad_rows(N, bad):
    assert _append(N, _kv(N), _rows(N, **bad)) == N.SV_ERR_INVALID_ARGUMENT
    assert _read(N, _kv(N), _rows(N, **bad)) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=MIS), dict(v=MIS), dict(table=None), dict(ctx=None),
                                 dict(kc=None), dict(vc=None), dict(kc=ODD), dict(vc=ODD), dict(ks=None), dict(vs=MIS)],
                         ids=lambda b: "-".join(b))
def test_bad_pointers(N, bad):
    assert _append(N, _kv(N), _rows(N), **bad) == N.SV_ERR_INVALID_ARGUMENT
    assert _read(N, _kv(N), _rows(N), **bad) == N.SV_ERR_INVALID_ARGUMENT


def test_null_descriptors_and_empty_batch(N):
    assert _append(N, None, _rows(N)) == N.SV_ERR_INVALID_ARGUMENT
    assert _append(N, _kv(N), None) == N.SV_ERR_INVALID_ARGUMENT
    assert _append(N, _kv(N, batch=0), _rows(N, total_new=0)) == N.SV_OK
    assert _read(N, _kv(N, batch=0), _rows(N, total_new=0)) == N.SV_OK
    assert _attend(N, _attention_desc(N, kv=_kv(N, batch=0), total_new=0)) == N.SV_OK


@pytest.mark.parametrize("nodes,path_len", [(0, 1), (1025, 1), (8, 0), (8, 66)])
def test_bad_commit_sizes(N, nodes, path_len):
    assert N.lib().sv_kv_commit(ctypes.byref(_kv(N)), nodes, path_len, A, A, A, A, A, A, A, A, ctypes.c_void_p(0x200000),
                                None, None) == N.SV_ERR_INVALID_ARGUMENT


def test_commit_refuses_missing_pointers_and_lengths_in_place(N):
    good = [A, A, A, A, A, A, A, A, ctypes.c_void_p(0x200000)]
    for i in range(len(good)):
        args = list(good)
        args[i] = None
        assert N.lib().sv_kv_commit(ctypes.byref(_kv(N)), 8, 4, *args, None, None) == N.SV_ERR_INVALID_ARGUMENT
    good[8] = good[1]
    assert N.lib().sv_kv_commit(ctypes.byref(_kv(N)), 8, 4, *good, None, None) == N.SV_ERR_INVALID_ARGUMENT


def _attention_desc(N, kv=None, **kw):
    a = N.KvAttentionDesc(kv or _kv(N), 8, 3, 12, N.SV_BF16, 0.125, 0, 0, 0, 512, 64, 512, 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _attend(N, a, ws=1 << 40, **p):
    x = dict(q=A, kc=A, vc=A, ks=A, vs=A, table=A, ctx=A, start=None, parents=None, out=A, lse=None, status=None, work=A)
    x.update(p)
    return N.lib().sv_kv_attention(ctypes.byref(a), x["q"], x["kc"], x["vc"], x["ks"], x["vs"], x["table"], x["ctx"], x["start"],
                                   x["parents"], x["out"], x["lse"], x["status"], x["work"], ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=7), dict(heads=2 * 129), dict(max_new=-1), dict(total_new=13),
                                 dict(dtype=5), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
                                 dict(sinks=-1), dict(reserved=3), dict(q_row_stride=0), dict(q_head_stride=48),
                                 dict(out_row_stride=63), dict(out_head_stride=-64)],
                         ids=lambda b: "-".join(f"{k}{v}" for k, v in b.items()))
def test_bad_attention_descriptor(N, bad):
    assert _attend(N, _attention_desc(N, **bad)) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=MIS), dict(out=None), dict(out=MIS), dict(kc=ODD), dict(vc=None),
                                 dict(ks=None), dict(vs=MIS), dict(table=None), dict(ctx=None), dict(work=None),
                                 dict(work=ODD)], ids=lambda b: "-".join(b))
def test_bad_attention_pointers(N, bad):
    assert _attend(N, _attention_desc(N), **bad) == N.SV_ERR_INVALID_ARGUMENT


def test_small_attention_workspace(N):
    a = _attention_desc(N)
    need = N.lib().sv_kv_attention_workspace_size(ctypes.byref(a))
    assert need > 0
    assert _attend(N, a, ws=need - 1) == N.SV_ERR_WORKSPACE_TOO_SMALL


def test_struct_layout_matches_c(N, tmp_path):
    import os
    import subprocess
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    prog = tmp_path / "layout.c"
    fields = {"sv_kv_desc": (N.KvDesc, ["max_pages", "page_stride", "table_stride"]),
              "sv_kv_rows_desc": (N.KvRowsDesc, ["dtype", "k_row_stride", "v_head_stride"]),
              "sv_kv_attention_desc": (N.KvAttentionDesc, ["heads", "scale", "sinks", "q_row_stride", "out_head_stride"])}
    body = "".join(f'printf("%zu ", sizeof({s}));' + "".join(f'printf("%zu ", offsetof({s}, {f}));' for f in fs)
                   for s, (_, fs) in fields.items())
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spec_verify.h"\nint main(void) {' + body +
                    'printf("%d %d %d %d %d", SV_ROW_BAD_PAGE, SV_ROW_BAD_LENGTH, SV_ROW_NOT_FINITE, SV_ROW_BAD_PATH, '
                    "SV_MAX_HEAD_DIM); return 0;}\n")
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(prog), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()
    want = []
    for _, (c, fs) in fields.items():
        want += [ctypes.sizeof(c)] + [getattr(c, f).offset for f in fs]
    want += [N.SV_ROW_BAD_PAGE, N.SV_ROW_BAD_LENGTH, N.SV_ROW_NOT_FINITE, N.SV_ROW_BAD_PATH, N.SV_MAX_HEAD_DIM]
    assert [int(x) for x in got] == want


def test_python_refuses_host_tensors(N):
    import torch

    import draft_token_verification_sv_gb300 as sv
    cache = sv.kv_cache(4, 2, 64, 16, device="cpu")
    assert cache["k"].shape == (4, 2, 16, 64) and cache["k_scale"].shape == (4, 2)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 1, 2, 64))
    for call in (lambda: sv.kv_append(cache, x, x, table, lens), lambda: sv.kv_read(cache, table, lens, 1),
                 lambda: sv.kv_attention(x, cache, table, lens),
                 lambda: sv.kv_commit(cache, table, lens, table, lens, 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()

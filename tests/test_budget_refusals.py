"""Calls of the budgeted-cache operators that are refused, and the statuses:
none of them touches a device (host checks come first)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def va():
    from speculative_decoding_verify_gqa_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gqa_gb300 as m
    m.lib()
    return m


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20     # addresses that are never read
INVALID, UNSUPPORTED = -1, -2


def _qkv(va, options=None, **kw):
    a = dict(q=A, qs=256, k=2 * A, ks=256, v=3 * A, vs=256, ai=64, kvp=64, ids=64, last=64, out=4 * A, kc=5 * A, vc=6 * A,
             batch=1, hq=2, h=2, d=128, page=16, pages=4, code=0, total=2)
    a.update(kw)
    o = va.QkvOptions()
    for n, x in (options or {}).items():
        setattr(o, n, x)
    return va.lib().paged_qkv_append(*a.values(), None if options == "null" else ctypes.byref(o), None, None)


@pytest.mark.parametrize("options, kw, status", [
    (dict(eps=-1.0), {}, INVALID), (dict(eps=float("nan")), {}, INVALID), (dict(weight_offset=float("inf")), {}, INVALID),
    (dict(weight_dtype=1), {}, UNSUPPORTED), (dict(kv_layout=2), {}, INVALID), (dict(interleaved=2), {}, INVALID),
    (dict(head_dim_v=96), {}, UNSUPPORTED), (dict(head_dim_v=-1), {}, INVALID),
    (dict(rotary_dim=16), {}, INVALID), (dict(positions=64), {}, INVALID), (dict(rotary_dim=-16), {}, INVALID),
    (dict(positions=64, rotary_dim=24, rope_theta=1e4), {}, UNSUPPORTED),
    (dict(positions=64, rotary_dim=144, rope_theta=1e4), {}, UNSUPPORTED),
    (dict(positions=64, rotary_dim=128, rope_theta=0.0), {}, INVALID),
    (dict(positions=64, rotary_dim=128, rope_theta=1e4, rope_scale=-1.0), {}, INVALID),
    ({}, dict(code=1), INVALID), (dict(k_scale=1.0, v_scale=0.0), dict(code=1), INVALID),
    ({}, dict(code=2), UNSUPPORTED), ({}, dict(d=96), UNSUPPORTED), ({}, dict(page=24), UNSUPPORTED),
    ({}, dict(hq=3), INVALID), ({}, dict(batch=-1), INVALID), ({}, dict(total=-1), INVALID), ({}, dict(batch=0), INVALID),
    ({}, dict(qs=248), INVALID), ({}, dict(ks=260), INVALID), ({}, dict(vs=128), INVALID),
    ({}, dict(q=A + 8), INVALID), ({}, dict(vc=6 * A + 4), INVALID), ({}, dict(kc=0), INVALID), ({}, dict(pages=0), INVALID),
    ({}, dict(out=A + 512), INVALID), ({}, dict(out=2 * A), INVALID), ({}, dict(out=3 * A + 16), INVALID),
    (dict(q_weight=A + 1), {}, INVALID), (dict(k_weight=A + 2, weight_dtype=2), {}, INVALID),
    ({}, dict(out=A, qs=512), INVALID), ({}, dict(total=1 << 31), UNSUPPORTED), ({}, dict(qs=1 << 40), UNSUPPORTED),
])
def test_qkv_append_refuses(va, options, kw, status):
    assert _qkv(va, options, **kw) == status


def test_qkv_append_more(va):
    assert _qkv(va, "null" and None, total=0) == 0
    a = va.QkvOptions()
    a.reserved[3] = 1
    assert va.lib().paged_qkv_append(*([0] * 13), 0, 2, 2, 128, 16, 4, 0, 0, ctypes.byref(a), None, None) == INVALID
    assert va.lib().paged_qkv_append(*([0] * 13), 0, 2, 2, 128, 16, 4, 0, 0, None, None, None) == INVALID
    bad = np.array([1.0, np.inf] * 32)
    assert _qkv(va, dict(positions=64, rotary_dim=128, inv_freq=bad.ctypes.data)) == INVALID


def _weights(va, **kw):
    a = dict(q=A, k=A, kvp=64, ids=64, last=64, qo=64, mask=0, mi=0, acc=0, path=0, lse=64, w=64, total=2, batch=1, hq=4,
             h=2, d=128, page=16, pages=4, code=0, layout=0, ml=0, scale=0.0, ks=1.0, decay=1.0)
    a.update(kw)
    return va.lib().verify_attn_key_weights(*a.values(), None, 1, None)


@pytest.mark.parametrize("kw, status", [
    (dict(batch=-1), INVALID), (dict(total=-1), INVALID), (dict(hq=5), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(page=3), UNSUPPORTED), (dict(code=2), UNSUPPORTED), (dict(layout=7), INVALID), (dict(ml=3), INVALID),
    (dict(mask=64), INVALID), (dict(mi=64), INVALID), (dict(acc=64), INVALID), (dict(path=64), INVALID),
    (dict(mask=64, mi=64, acc=64, path=64), INVALID), (dict(ks=0.0), INVALID), (dict(ks=float("inf")), INVALID),
    (dict(scale=1e38, ks=1e38), INVALID), (dict(decay=-0.5), INVALID), (dict(decay=float("nan")), INVALID),
    (dict(q=0), INVALID), (dict(lse=0), INVALID), (dict(w=0), INVALID), (dict(lse=66), INVALID), (dict(w=A + 2), INVALID), (dict(k=A + 8), INVALID), (dict(q=A + 2), INVALID),
    (dict(pages=0), INVALID), (dict(total=1 << 31), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(batch=0), 0),
])
def test_key_weights_refuses(va, kw, status):
    assert _weights(va, **kw) == status


def _evict(va, **kw):
    a = dict(w=A, keep=64, kvp=64, ids=64, last=64, k=16 * A, v=32 * A, layers=1, batch=1, h=2, d=128, dv=0, page=16, pages=4,
             code=0, layout=0, most=64, sinks=0, recent=0)
    a.update(kw)
    return va.lib().paged_kv_evict(*a.values(), None, None, 1, None)


@pytest.mark.parametrize("kw, status", [
    (dict(layers=0), INVALID), (dict(batch=-1), INVALID), (dict(most=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(d=32), UNSUPPORTED), (dict(dv=96), UNSUPPORTED), (dict(dv=-1), INVALID),
    (dict(page=48), UNSUPPORTED), (dict(code=2), UNSUPPORTED), (dict(layout=2), INVALID),
    (dict(most=(1 << 19) + 1), UNSUPPORTED), (dict(batch=1 << 28, layers=64), UNSUPPORTED), (dict(w=0), INVALID),
    (dict(keep=0), INVALID), (dict(ids=0), INVALID), (dict(k=16 * A + 8), INVALID), (dict(w=A + 2), INVALID),
    (dict(pages=0), INVALID), (dict(v=16 * A + 16), INVALID), (dict(w=16 * A + 64), INVALID), (dict(w=32 * A), INVALID),
    (dict(pages=1 << 27, page=16), UNSUPPORTED), (dict(batch=0), 0),
])
def test_evict_refuses(va, kw, status):
    assert _evict(va, **kw) == status


def test_binding_wants_the_current_device(va):
    x = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        va.paged_qkv_append(x[:, 0], x[:, 0], x[:, 0], i, i, i, i, x, x)
    with pytest.raises(ValueError, match="current CUDA device"):
        va.verify_attn_key_weights(x[:, 0], x, i, i, i, i, i, i)
    with pytest.raises(ValueError, match="current CUDA device"):
        va.paged_kv_evict(x[..., 0].float(), i, i, i, i, x, x)


def test_options_layout(va, tmp_path):
    """The binding's structure is the header's, field by field."""
    names = [n for n, _ in va.QkvOptions._fields_]
    src = tmp_path / "o.c"
    src.write_text('#include <stdio.h>\n#include "verify_attn.h"\nint main(void) {\n%s  printf("%%zu\\n", sizeof(va_qkv_options_t));\n}\n'
                   % "".join('  printf("%%zu\\n", offsetof(va_qkv_options_t, %s));\n' % n for n in names))
    exe = str(tmp_path / "o")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(va.QkvOptions, n).offset for n in names] + [ctypes.sizeof(va.QkvOptions)]


@pytest.mark.parametrize("kw", [dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-float("inf")),
                                dict(scale=3e38, ks=1.0), dict(scale=1.0, ks=3e38), dict(ks=float("nan"))])
def test_key_weights_refuse_the_attentions_refused_scales(va, kw):
    """Scales that verify_attn_run refuses: not finite, or with a product that is not, times log2(e)."""
    assert _weights(va, **kw) == INVALID


@pytest.mark.parametrize("at", [4000, 4012, 8000, 8016, 7996, 12012, 11988])
def test_evict_refuses_lengths_over_its_tables(va, at):
    """kv_len_out is written while other CTAs still read keep_len, kv_indptr and last_page_len."""
    base = 64 * A
    tables = [base + 4000, base + 8000, 64, base + 12000]     # of 4 requests: 16, 20 and 16 bytes, and the page ids
    assert va.lib().paged_kv_evict(A, *tables, 16 * A, 32 * A, 1, 4, 2, 128, 0, 16, 4, 0, 0, 64, 0, 0, base + at,
                                   None, 1, None) == INVALID


def test_qkv_append_refuses_null_options(va):
    """NULL options beside arguments that are valid otherwise, and with nothing to append."""
    for total in (2, 0):
        args = (A, 256, 2 * A, 256, 3 * A, 256, 64, 64, 64, 64, 4 * A, 5 * A, 6 * A, 1, 2, 2, 128, 16, 4, 0, total)
        assert va.lib().paged_qkv_append(*args, None, None, None) == INVALID

"""The cache's C ABI and binding without a GPU: the header's functions are
exported, the struct's mirror matches, bad arguments are refused before
anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import draft_token_verification_verify_b200 as sv
from cachelib import Pages
from draft_token_verification_verify_b200 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spec_cache.h")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sv.cache_lib()


def test_exports_what_the_header_declares(L):
    declared = set(re.findall(r"SV_API\s+[\w\s\*]+?\b(\w+)\s*\(", open(HEADER).read()))
    assert declared == {"spec_cache_attend", "spec_cache_attend_workspace_size", "spec_cache_append",
                        "spec_cache_read", "spec_cache_page_bytes"}
    out = subprocess.run(["nm", "-D", "--defined-only", _build.CACHE_LIB], check=True, capture_output=True,
                         text=True).stdout
    assert set(re.findall(r"\sT\s+(\w+)$", out, flags=re.M)) == declared


def test_struct_mirror(tmp_path):
    names = [f[0] for f in sv.SvCache._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spec_cache.h"\nint main(void) {\n'
                   'printf("%zu %d", sizeof(sv_cache_t), SV_DTYPE_F16);\n' +
                   "".join(f'printf(" %zu", offsetof(sv_cache_t, {n}));\n' for n in names) + "return 0; }\n")
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", str(exe),
                    str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(sv.SvCache), sv.SV_DTYPE_F16] + [getattr(sv.SvCache, n).offset for n in names]


def test_page_bytes(L):
    assert sv.spec_cache_page_bytes(8, 64, 128) == 8 * 64 * 136
    assert sv.spec_cache_page_bytes(1, 16, 64) == 16 * 72
    for bad in ((0, 64, 128), (1, 8, 128), (1, 48, 128), (1, 2048, 128), (1, 64, 96), (-1, 64, 128)):
        assert sv.spec_cache_page_bytes(*bad) == 0
    assert Pages(3, 2, 32, 128, torch.float16).bytes().shape == (3, 2, sv.spec_cache_page_bytes(1, 32, 128))


def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("placeholder device pointers: runs only without a GPU")


def _cache(**over):
    f = dict(pages=1 << 20, page_table=1 << 12, lens=1 << 12, num_pages=4, max_pages=4, page_size=64, kv_heads=2,
             head_dim=128, dtype=0)
    f.update(over)
    return sv.SvCache(*(f[n] for n, _ in sv.SvCache._fields_))


BAD_CACHES = [dict(pages=0), dict(pages=(1 << 20) + 8), dict(page_table=0), dict(lens=0), dict(lens=6),
              dict(num_pages=0), dict(max_pages=0), dict(page_size=48), dict(page_size=8), dict(page_size=2048),
              dict(kv_heads=0), dict(head_dim=0), dict(dtype=1 << 8), dict(dtype=7)]
UNSUPPORTED = [dict(head_dim=96), dict(head_dim=256), dict(max_pages=1 << 25)]

P = 1 << 16  # a placeholder device pointer


def attend(c, q=P, q_stride=512, k=P, v=P, kv_stride=256, parents=None, B=2, n=3, heads=4, scale=0.1, out=P, lse=None,
           ws=P, wb=1 << 30, opts=None, status=None):
    return sv.spec_cache_attend(q, q_stride, k, v, kv_stride, parents, c, B, n, heads, scale, out, lse, ws, wb, opts,
                                status, stream=0)


def append(c, k=P, v=P, stride=256, B=2, n=3, acc=None, nodes=None, ns=0, out=P):
    return sv.spec_cache_append(c, k, v, stride, B, n, acc, nodes, ns, out, stream=0)


def read(c, B=2, n=3, first=None, k=P, v=P):
    return sv.spec_cache_read(c, B, n, first, k, v, stream=0)


def test_refusals(L):
    _no_gpu()
    for call in (attend, append, read):
        for over in BAD_CACHES:
            assert call(_cache(**over)) == sv.SV_ERR_INVALID_ARG, (call, over)
        for over in UNSUPPORTED:
            assert call(_cache(**over)) == sv.SV_ERR_UNSUPPORTED, (call, over)
        assert call(_cache()) == sv.SV_ERR_UNSUPPORTED  # no device here: the arguments are fine
    c = _cache()
    for over in (dict(q=None), dict(q=P + 8), dict(q_stride=504), dict(q_stride=516), dict(k=None), dict(v=None),
                 dict(k=P + 2), dict(v=P + 4), dict(kv_stride=248), dict(kv_stride=257), dict(B=0), dict(n=0), dict(n=258),
                 dict(heads=3), dict(heads=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None),
                 dict(out=P + 8), dict(lse=P + 2), dict(ws=None), dict(ws=P + 4), dict(parents=P + 1),
                 dict(status=P + 2)):
        assert attend(c, **over) == sv.SV_ERR_INVALID_ARG, over
    assert attend(c, k=None, v=None, kv_stride=0) == sv.SV_ERR_UNSUPPORTED
    for name in ("top_p", "vocab_mask", "rep_ids"):
        o = sv.SvOptions()
        setattr(o, name, P)
        assert attend(c, opts=o) == sv.SV_ERR_UNSUPPORTED
    for over in (dict(k=None), dict(v=None), dict(k=P + 8), dict(stride=128), dict(stride=260), dict(B=0), dict(n=0),
                 dict(out=None), dict(out=P + 2), dict(acc=P + 1), dict(nodes=P + 2, ns=3), dict(nodes=P, ns=1),
                 dict(out=(1 << 12) + 4)):  # overlaps the lengths without being them
        assert append(c, **over) == sv.SV_ERR_INVALID_ARG, over
    assert append(c, out=1 << 12) == sv.SV_ERR_UNSUPPORTED  # in place
    for over in (dict(B=0), dict(n=0), dict(k=None, v=None), dict(k=P + 8), dict(v=P + 8), dict(first=P + 2)):
        assert read(c, **over) == sv.SV_ERR_INVALID_ARG, over
    assert sv.spec_cache_attend_workspace_size(2, 3, 4, 2, 128) == 0  # no device


def test_append_refuses_lengths_over_its_inputs(L):
    """New lengths written over the counts or nodes that other CTAs still read."""
    _no_gpu()
    c = _cache()
    for over in (dict(acc=P), dict(acc=P + 4), dict(acc=P - 4), dict(nodes=P, ns=3), dict(nodes=P - 20, ns=3),
                 dict(acc=1 << 12, out=1 << 12)):
        assert append(c, **over) == sv.SV_ERR_INVALID_ARG, over
    for over in (dict(acc=P + 8), dict(acc=P - 8), dict(nodes=P - 24, ns=3), dict(nodes=P + 8, ns=3)):
        assert append(c, **over) == sv.SV_ERR_UNSUPPORTED, over  # side by side: the arguments are fine


def test_kv_cache_refusals():
    ok = torch.zeros((3, 2, 64 * 136), dtype=torch.uint8)
    c = sv.KvCache(ok, 128)
    assert (c.num_pages, c.kv_heads, c.page_size, c.dtype) == (3, 2, 64, torch.bfloat16)
    for args, err in (((ok.float(), 128), TypeError), ((ok, 128, torch.float32), TypeError), ((ok, 96), ValueError),
                      ((ok, 64), ValueError), ((ok[:, :, :-1], 128), ValueError), ((ok[0], 128), ValueError),
                      ((ok[:, :1], 128), ValueError), ((ok[:0], 128), ValueError),
                      ((torch.zeros((1, 1, 48 * 136), dtype=torch.uint8), 128), ValueError)):
        with pytest.raises(err):
            sv.KvCache(*args)


def test_tensor_calls_refuse(L):
    """The binding's own checks, on CPU tensors that no call ever takes."""
    c = sv.KvCache.empty(4, 2, 64, 128, device="cpu")
    table, lens = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 3, 2, 128), dtype=torch.bfloat16)
    for call in (lambda: sv.cache_attend(x, c, table, lens), lambda: sv.cache_append(c, table, lens, x, x),
                 lambda: sv.cache_read(c, table, lens, 3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_token_strides():
    from draft_token_verification_verify_b200.cache import _tokens

    c = sv.KvCache.empty(4, 2, 64, 128, device="cpu")
    rows = torch.zeros((2, 3, 8, 128), dtype=torch.bfloat16)
    assert _tokens(rows, "x", c)[1] == 8 * 128 and _tokens(rows[:, :, 4:6], "x", c, 2)[1] == 8 * 128
    assert _tokens(rows[:, :1], "x", c)[1] == 3 * 8 * 128 and _tokens(rows[:1, :1, :2], "x", c)[1] == 2 * 128
    for bad, err in ((rows.float(), TypeError), (rows[..., :64], ValueError), (rows[:, :2], ValueError),
                     (rows[:, :, ::2], ValueError), (rows[:, :, :, 1:], ValueError), (rows.transpose(0, 1), ValueError),
                     (rows[:0], ValueError), (rows[0], ValueError), (None, TypeError)):
        with pytest.raises(err):
            _tokens(bad, "x", c)
    wide = torch.zeros((2, 3, 8 * 128 + 4), dtype=torch.bfloat16)[:, :, :1024].unflatten(2, (8, 128))
    with pytest.raises(ValueError, match="16-byte"):
        _tokens(wide, "x", c)

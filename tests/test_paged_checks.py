"""Refusals of the paged-cache entry points, on the CPU: the C ABI's status
codes before anything is launched, and the binding's checks before any pointer
reaches the library."""

import ctypes

import pytest
import torch

from exact_io_aware_bwd_b200 import binding
from exact_io_aware_bwd_b200.build import build

FAKE = 1 << 20  # a 16-byte-aligned non-null pointer value; never dereferenced
INVALID, UNSUPPORTED, MISALIGNED = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


SIZES = dict(B=2, Hq=4, Hkv=2, N=3, d=64, P=16, max_pages=8, num_pages=20, dtype=0)


def sizes(kw):
    s = dict(SIZES, **{k: v for k, v in kw.items() if k in SIZES})
    return [s[k] for k in ("B", "Hq", "Hkv", "N", "d", "P", "max_pages", "num_pages")], s["dtype"]


def pointers(n, kw):
    p = [FAKE] * n
    for i, value in kw.get("ptr", {}).items():
        p[i] = value
    return [ctypes.c_void_p(x) for x in p]


def append(lib, **kw):
    s, dtype = sizes(kw)
    p = pointers(11, kw)
    strides = kw.get("strides")
    strides = None if strides is None else (ctypes.c_int64 * 9)(*strides)
    return lib.fa_append_paged(*p[:3], strides, *p[3:], *s, kw.get("rot", 64), kw.get("inter", 0), dtype, None)


def paged(lib, **kw):
    s, dtype = sizes(kw)
    p = pointers(9, kw)
    need = binding.fa_fwd_paged_workspace_bytes(*s[:7])
    return lib.fa_fwd_paged(*p[:8], *s, kw.get("scale", 0.125), dtype, p[8], kw.get("ws", need), None)


def prefix(lib, **kw):
    s, dtype = sizes(kw)
    p = pointers(8, kw)
    pre = kw.get("prefix", 32)
    need = binding.fa_decode_prefix_workspace_bytes(*s[:7], pre)
    return lib.fa_decode_prefix(*p[:7], *s, pre, kw.get("scale", 0.125), dtype, p[7], kw.get("ws", need), None)


COMMON = [
    (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(B=-1), INVALID), (dict(N=-1), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(P=8), UNSUPPORTED), (dict(P=48), UNSUPPORTED), (dict(P=256), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED), (dict(num_pages=1 << 30), UNSUPPORTED),
]


@pytest.mark.parametrize("call", [append, paged, prefix], ids=["append", "fwd_paged", "decode_prefix"])
@pytest.mark.parametrize("kw,status", COMMON, ids=[str(c[0]) for c in COMMON])
def test_sizes_are_refused(lib, call, kw, status):
    assert call(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rot=-16), INVALID), (dict(rot=80), INVALID), (dict(rot=24), UNSUPPORTED), (dict(inter=2), INVALID),
    (dict(ptr={0: 0}), INVALID),       # q_out without q
    (dict(ptr={3: 0}), INVALID),       # q without q_out
    (dict(ptr={1: 0}), INVALID), (dict(ptr={2: 0}), INVALID), (dict(ptr={5: 0}), INVALID), (dict(ptr={6: 0}), INVALID),
    (dict(ptr={7: 0}), INVALID), (dict(ptr={8: 0}), INVALID), (dict(ptr={10: 0}), INVALID),
    (dict(ptr={1: FAKE + 8}), MISALIGNED), (dict(ptr={4: FAKE + 2}), MISALIGNED), (dict(ptr={8: FAKE + 2}), MISALIGNED),
    (dict(strides=[8] * 8 + [4]), MISALIGNED), (dict(strides=[12] + [8] * 8), MISALIGNED),
    (dict(B=1 << 20, Hq=1024, Hkv=1024, N=2), UNSUPPORTED),
])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(ptr={0: 0}), INVALID), (dict(ptr={3: 0}), INVALID), (dict(ptr={6: 0}), INVALID), (dict(ptr={7: 0}), INVALID),
    (dict(ptr={0: FAKE + 4}), MISALIGNED), (dict(ptr={5: FAKE + 1}), MISALIGNED),
    (dict(B=1 << 16, Hq=1 << 8, N=1 << 8), UNSUPPORTED),
])
def test_fwd_paged_refusals(lib, kw, status):
    assert paged(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(scale=-1.0), INVALID), (dict(N=0), INVALID), (dict(prefix=-16), INVALID), (dict(prefix=24), INVALID),
    (dict(prefix=16 * 9), INVALID), (dict(Hq=34), UNSUPPORTED), (dict(Hq=8, N=9), UNSUPPORTED),
    (dict(ptr={1: 0}), INVALID), (dict(ptr={5: 0}), INVALID), (dict(ptr={2: FAKE + 8}), MISALIGNED),
])
def test_decode_prefix_refusals(lib, kw, status):
    assert prefix(lib, **kw) == status


def test_a_small_workspace_is_refused(lib):
    # sizes whose passes are split along the keys
    kw = dict(B=1, Hq=4, Hkv=2, N=1, d=128, max_pages=4096, num_pages=5000)
    assert paged(lib, **kw, ws=15) == INVALID and paged(lib, **kw, ptr={8: 0}) == INVALID
    assert prefix(lib, **kw, prefix=4096, ws=15) == INVALID and prefix(lib, **kw, prefix=4096, ptr={7: 0}) == INVALID


def test_empty_problems_are_no_ops(lib):
    none = {i: 0 for i in range(11)}
    assert append(lib, B=0, ptr=none) == binding.FA_OK and append(lib, N=0, ptr=none) == binding.FA_OK
    none = {i: 0 for i in range(9)}
    assert paged(lib, B=0, ptr=none) == binding.FA_OK and paged(lib, N=0, ptr=none) == binding.FA_OK
    assert prefix(lib, B=0, ptr={i: 0 for i in range(8)}) == binding.FA_OK


# --------------------------------------------------------------- the binding

def tensors(B=2, Hq=4, Hkv=2, N=3, d=64, P=16, pages=5, dtype=torch.bfloat16):
    z = lambda *s: torch.zeros(s, dtype=dtype)
    return dict(q=z(B, Hq, N, d), k=z(B, Hkv, N, d), v=z(B, Hkv, N, d), q_out=z(B, Hq, N, d), k_out=None,
                k_cache=z(pages, Hkv, P, d), v_cache=z(pages, Hkv, P, d),
                block_table=torch.zeros((B, 2), dtype=torch.int32), seq_lens=torch.zeros(B, dtype=torch.int32),
                new_lens=None, inv_freq=torch.zeros(d // 2))


def do_append(t):
    binding.fa_append_paged(*[t[n] for n in ("q", "k", "v", "q_out", "k_out", "k_cache", "v_cache", "block_table",
                                             "seq_lens", "new_lens", "inv_freq")])


def do_attention(t):
    o, lse = torch.zeros_like(t["q"]), torch.zeros(t["q"].shape[:3])
    args = [t[n] for n in ("q", "k_cache", "v_cache", "block_table", "seq_lens")]
    ws = torch.zeros(1024, dtype=torch.uint8)
    if t.get("which") == "paged":
        binding.fa_fwd_paged(*args, t["new_lens"], t.get("o", o), t.get("lse", lse), 0.125, ws)
    else:
        binding.fa_decode_prefix(*args, t.get("o", o), t.get("lse", lse), 0.125, 0, ws)


@pytest.mark.parametrize("change,error,match", [
    (dict(), ValueError, "CUDA device"),
    (dict(q=None), ValueError, "come together"),
    (dict(k=torch.zeros((2, 3, 3, 64), dtype=torch.bfloat16)), ValueError, "v has shape|heads"),
    (dict(v=torch.zeros((2, 2, 4, 64), dtype=torch.bfloat16)), ValueError, "v has shape"),
    (dict(v=torch.zeros((2, 2, 3, 64), dtype=torch.float16)), TypeError, "v has dtype"),
    (dict(k=torch.zeros((2, 2, 64, 3), dtype=torch.bfloat16).transpose(2, 3)), ValueError, "rows of k"),
    (dict(k=torch.zeros((2, 2, 3, 64))), TypeError, "dtype"),
    (dict(k_cache=torch.zeros((5, 2, 16, 128), dtype=torch.bfloat16)), ValueError, "k_cache has shape"),
    (dict(v_cache=torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)), ValueError, "v_cache has shape"),
    (dict(block_table=torch.zeros((2, 2))), TypeError, "block_table"),
    (dict(block_table=torch.zeros((3, 2), dtype=torch.int32)), ValueError, "block_table"),
    (dict(block_table=torch.zeros(4, dtype=torch.int32)), ValueError, "2-D"),
    (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError, "seq_lens"),
    (dict(new_lens=torch.zeros(3, dtype=torch.int32)), ValueError, "new_lens"),
    (dict(inv_freq=torch.zeros((2, 16))), ValueError, "1-D"),
], ids=lambda x: str(list(x)) if isinstance(x, dict) else None)
def test_append_binding_checks(change, error, match):
    with pytest.raises(error, match=match):
        do_append(dict(tensors(), **change))


@pytest.mark.parametrize("which", ["paged", "prefix"])
@pytest.mark.parametrize("change,error,match", [
    (dict(), ValueError, "CUDA device"),
    (dict(q=torch.zeros((2, 4, 64), dtype=torch.bfloat16)), ValueError, "4-D"),
    (dict(q=torch.zeros((2, 4, 3, 64))), TypeError, "q has dtype"),
    (dict(k_cache=torch.zeros((5, 2, 16, 128), dtype=torch.bfloat16)), ValueError, "k_cache has shape"),
    (dict(o=torch.zeros((2, 4, 3, 64))), (TypeError, ValueError), None),
    (dict(block_table=None), TypeError, "block_table"),
])
def test_attention_binding_checks(which, change, error, match):
    with pytest.raises(error, match=match):
        do_attention(dict(tensors(), which=which, **change))

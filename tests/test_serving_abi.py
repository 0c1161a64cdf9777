"""Refusals of the serving-step operators on the host (no GPU): page plan,
paged K/V attention, e4m3 rows and linear layer.  Every bad argument is answered before
any CUDA call.  Fake addresses: nothing is dereferenced."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from test_attn_abi import FakeHandle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    BLD.build()
    return B.load()


_at = [0x5000000]


def fake():
    _at[0] += 0x1000
    return _at[0]


# in the order of the structs' fields
PLAN = dict(new=fake(), ended=0, lens=fake(), table=fake(), free=fake(), count=fake(), lens_out=fake(), count_out=fake(), cu=fake(),
            slots=fake(), pos=fake(), n=2, T=16, ts=4, page=16, nb=8)
KV = dict(qn=fake(), qp=fake(), cu=0, lens=fake(), table=fake(), k=fake(), v=fake(), e=fake(), ks=0, vs=0, es=0, out=fake(), lse=fake(),
          k_bs=16 * 16 * 128, k_hs=16 * 128, v_bs=16 * 16 * 128, v_hs=16 * 128, e_bs=16 * 64, n=2, T=2, ts=4, page=16, nb=8, k_rs=128,
          v_rs=128, e_rs=64, qn_t=16 * 128, qn_h=128, qp_t=16 * 64, qp_h=64)
ROWS = dict(x=fake(), gamma=0, q=fake(), scale=fake(), T=4, K=256, xs=256, qs=256, dtype=0, eps=1e-6)
LINEAR = dict(x=fake(), gamma=0, xq=0, xsc=0, out=fake(), T=4, xs=256, qs=0, os=264, eps=1e-6)
STRUCTS = dict(mla_fp8_linear_args=B._FP8_LINEAR_ARGS, mla_page_plan_args=B._PLAN_ARGS, mla_attn_paged_kv_args=B._PAGED_KV_ARGS, mla_fp8_quant_args=B._FP8_ROWS_ARGS)
BASES = dict(mla_fp8_linear_args=LINEAR, mla_page_plan_args=PLAN, mla_attn_paged_kv_args=KV, mla_fp8_quant_args=ROWS)


def packed(struct, base, **over):
    args = dict(base)
    args.update(over)
    return struct.pack(*args.values())


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(n=(1 << 30) + 1), 1), (dict(T=-1), 1), (dict(T=17), 3), (dict(page=0), 1), (dict(nb=0), 1), (dict(ts=-1), 1),
    (dict(page=1 << 16, nb=1 << 16), 1), (dict(new=0), 1), (dict(lens=0), 1), (dict(table=0), 1), (dict(free=0), 1),
    (dict(count=0), 1), (dict(lens_out=0), 1), (dict(count_out=0), 1), (dict(cu=0), 1), (dict(slots=0), 1), (dict(pos=0), 1),
    (dict(page=1, nb=(1 << 31) - 65535), 1), (dict(T=(1 << 31) - 65535), 1),
    (dict(new=0x5000008), 4), (dict(ended=0x5000004), 4), (dict(cu=0x5000004), 4), (dict(slots=0x5000008), 4),
])
def test_plan_refusals(L, over, code):
    assert L.mla_page_plan(FakeHandle().ptr, packed(B._PLAN_ARGS, PLAN, **over), None) == code, over


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(n=(1 << 30) + 1, cu=fake()), 1), (dict(T=-2), 1), (dict(T=17, n=17), 3), (dict(T=3), 1), (dict(page=0), 1), (dict(nb=-1), 1), (dict(ts=-1), 1),
    (dict(page=1 << 16, nb=1 << 15), 1), (dict(qn=0), 1), (dict(qp=0), 1), (dict(lens=0), 1), (dict(table=0), 1), (dict(k=0), 1),
    (dict(v=0), 1), (dict(e=0), 1), (dict(out=0), 1), (dict(ks=fake()), 1), (dict(vs=fake()), 1), (dict(ks=fake(), es=fake()), 1),
    (dict(qn_t=120), 1), (dict(qn_h=100), 1), (dict(qp_t=63), 1), (dict(qp_h=0), 1), (dict(k_bs=0), 1), (dict(k_hs=130), 1),
    (dict(k_rs=127), 1), (dict(v_bs=-2048), 1), (dict(v_hs=64), 1), (dict(v_rs=0), 1), (dict(e_bs=60), 1), (dict(e_rs=56), 1),
    (dict(ks=fake(), vs=fake(), es=fake(), e_rs=72), 1),  # (int8: 16 elements are 16 bytes)
    (dict(qn=0x5000008), 4), (dict(k=0x5000008), 4), (dict(ks=0x5000008, vs=fake(), es=fake()), 4), (dict(lse=0x5000004), 4),
    (dict(n=0), 0), (dict(T=0, qn=0), 0),
])
def test_paged_kv_refusals(L, over, code):
    assert L.mla_attn_paged_kv_run(FakeHandle().ptr, packed(B._PAGED_KV_ARGS, KV, **over), None) == code, over


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(K=0), 1), (dict(K=-16), 1), (dict(K=264), 2), (dict(dtype=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(x=0), 1), (dict(q=0), 1), (dict(scale=0), 1), (dict(xs=255), 1), (dict(xs=248), 1), (dict(xs=260), 1), (dict(qs=264), 1),
    (dict(qs=240), 1), (dict(x=0x5000008), 4), (dict(gamma=0x5000002), 4), (dict(q=0x5000004), 4), (dict(scale=0x5000008), 4),
    (dict(T=0, x=0), 0), (dict(T=(1 << 31) - 65535), 2), (dict(K=(1 << 31) - 65520, xs=(1 << 31) - 65520, qs=(1 << 31) - 65520), 2),
])
def test_fp8_rows_refusals(L, over, code):
    assert L.mla_fp8_quant_rows(packed(B._FP8_ROWS_ARGS, ROWS, **over), None) == code, over


def linear_cfg(**over):
    c = dict(in_features=256, out_features=264, dtype=B.MLA_F16, max_tokens=16, spin_budget_ns=0)
    c.update(over)
    return B.Fp8LinearConfig(**c)


@pytest.mark.parametrize("over,w,s,code", [
    (dict(in_features=0), 16, 16, 1), (dict(out_features=-8), 16, 16, 1), (dict(max_tokens=0), 16, 16, 1), (dict(dtype=2), 16, 16, 1),
    (dict(), 0, 16, 1), (dict(), 16, 0, 1), (dict(in_features=264), 16, 16, 2), (dict(out_features=260), 16, 16, 2),
    (dict(in_features=(1 << 31) - 65520), 16, 16, 2), (dict(out_features=65535 * 128 + 8), 16, 16, 2),
    (dict(max_tokens=(1 << 31) - 65535), 16, 16, 2),
    (dict(), 24, 16, 4), (dict(), 16, 20, 4),
])
def test_linear_create_refusals(L, over, w, s, code):
    h = P()
    assert L.mla_fp8_linear_create(ctypes.byref(linear_cfg(**over)), w or None, s or None, ctypes.byref(h)) == code
    assert not h.value


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(T=17), 3), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(out=0), 1), (dict(os=256), 1), (dict(os=268), 1),
    (dict(x=0), 1), (dict(xq=fake()), 1), (dict(xsc=fake()), 1), (dict(xs=248), 1), (dict(xs=260), 1),
    (dict(x=0, xq=fake(), qs=256), 1), (dict(x=0, xsc=fake(), qs=256), 1), (dict(x=0, xq=fake(), xsc=fake(), qs=264), 1),
    (dict(x=0, xq=fake(), xsc=fake(), qs=240), 1), (dict(x=0, xq=fake(), xsc=fake(), qs=256, gamma=fake()), 1),
    (dict(x=0x5000008), 4), (dict(gamma=0x5000008), 4), (dict(out=0x5000004), 4), (dict(x=0, xq=0x5000008, xsc=fake(), qs=256), 4),
    (dict(x=0, xq=fake(), xsc=0x5000004, qs=256), 4), (dict(T=0, x=0, out=0), 0),
])
def test_linear_refusals(L, over, code):
    mem = (ctypes.c_char * 1024)()  # a handle struct built on the host: the checks read its configuration only
    c = linear_cfg()
    ctypes.memmove(mem, ctypes.byref(c), ctypes.sizeof(c))
    assert L.mla_fp8_linear_run(ctypes.cast(mem, P), packed(B._FP8_LINEAR_ARGS, LINEAR, **over), None) == code, over


def test_linear_config_layout_matches_the_header(tmp_path):
    src = open(os.path.join(ROOT, "include", "mla_prolog.h")).read()
    body = re.search(r"typedef struct mla_fp8_linear_config \{(.*?)\} mla_fp8_linear_config;", src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = [re.match(r"\s*(.*?)\s+(\w+)$", f.strip()).groups() for f in body.split(";") if f.strip()]
    of = {"int": ctypes.c_int, "unsigned long long": ctypes.c_ulonglong}
    assert [(n, of[t]) for t, n in fields] == list(B.Fp8LinearConfig._fields_)


def test_null_arguments(L):
    h = FakeHandle().ptr
    assert L.mla_page_plan(None, packed(B._PLAN_ARGS, PLAN), None) == 1 and L.mla_page_plan(h, None, None) == 1
    assert L.mla_attn_paged_kv_run(None, packed(B._PAGED_KV_ARGS, KV), None) == 1 and L.mla_attn_paged_kv_run(h, None, None) == 1
    assert L.mla_fp8_quant_rows(None, None) == 1
    out = P()
    assert L.mla_fp8_linear_create(None, 16, 16, ctypes.byref(out)) == 1
    assert L.mla_fp8_linear_create(ctypes.byref(linear_cfg()), 16, 16, None) == 1
    assert L.mla_fp8_linear_destroy(None) == 1 and L.mla_fp8_linear_status(None, None) == 1
    assert L.mla_fp8_linear_last_launches(None) == -1 and L.mla_fp8_linear_run(None, packed(B._FP8_LINEAR_ARGS, LINEAR), None) == 1
    assert b"page" in L.mla_status_string(12)


@pytest.mark.parametrize("name", list(STRUCTS))
def test_argument_structs_match_the_header(name, tmp_path):
    """The binding packs the header's fields in their order and kinds, to the C compiler's size."""
    src = open(os.path.join(ROOT, "include", "mla_prolog.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    kinds = ""
    for line in body.split(";"):
        line = line.strip()
        if line:
            kind = "Q" if "*" in line else "q" if line.startswith("long long") else "f" if line.startswith("float") else "i"
            kinds += kind * (line.count(",") + 1)
    flat = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([a-zA-Z])", STRUCTS[name].format.lstrip("@")) if c != "x")
    assert flat == kinds
    assert len(BASES[name]) == len(kinds)
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/usr/local/cuda/include"):
        pytest.skip("gcc or the CUDA headers are missing")
    prog = tmp_path / "size.c"
    prog.write_text('#include <stdio.h>\n#include "mla_prolog.h"\nint main(void) { printf("%%zu\\n", sizeof(%s)); return 0; }\n' % name)
    exe = tmp_path / "size"
    subprocess.run([gcc, str(prog), "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", "-o", str(exe)],
                   check=True, capture_output=True)
    assert int(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout) == STRUCTS[name].size


def test_binding_rejects_host_tensors():
    """No CPU fallback: tensors that are not on a CUDA device raise before the library is called."""
    a = B.MLAAttention.__new__(B.MLAAttention)
    a.h, a.device, a.dtype, a.heads, a.kv_heads = None, 0, torch.float16, 4, 4
    a.rank, a.rope, a.nope, a.vdim = 512, 64, 128, 128
    i = torch.zeros(2, dtype=torch.int32)
    q, c = torch.zeros(2, 4, 128, dtype=torch.float16), torch.zeros(1, 4, 2, 128, dtype=torch.float16)
    with pytest.raises(TypeError):
        a.run_paged_kv(q, q[..., :64], i, i[None], c, c, c[:, :1, :, :64], q)
    with pytest.raises(TypeError):
        a.plan_pages(i, i, i[None], i, i[:1], 16, i, i, i)
    x = torch.zeros(2, 256, dtype=torch.float16)
    with pytest.raises(TypeError):
        B.mla_fp8_quant_rows(x, x.to(torch.float8_e4m3fn), torch.zeros(2, 2))
    with pytest.raises(TypeError):
        B.MLAFp8Linear(x.to(torch.float8_e4m3fn), torch.zeros(1, 2), "fp16", 4)
    with pytest.raises(TypeError):
        B.mla_fp8_quant_rows(x.float(), x.to(torch.float8_e4m3fn), torch.zeros(2, 2))

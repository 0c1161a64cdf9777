"""Refusals of the attention entry points on the host (no GPU): every bad
argument is answered before any CUDA call, and the binding checks shapes,
types and devices.  Fake addresses: nothing is dereferenced."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    BLD.build()
    return B.load()


def cfg(**over):
    c = dict(num_heads=16, num_kv_heads=0, kv_lora_rank=512, rope_dim=64, nope_dim=128, v_dim=128, dtype=B.MLA_F16,
             eps=1e-6, scale=0.0, max_tokens=16, max_pos=4096, spin_budget_ns=0)
    c.update(over)
    return B.AttnConfig(**c)


@pytest.mark.parametrize("over,code", [
    (dict(num_heads=0), 1), (dict(num_kv_heads=-1), 1), (dict(max_tokens=0), 1), (dict(max_pos=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(dtype=2), 1), (dict(kv_lora_rank=256), 2), (dict(rope_dim=32), 2), (dict(nope_dim=64), 2), (dict(v_dim=64), 2),
    (dict(num_kv_heads=3), 2), (dict(num_kv_heads=32), 2), (dict(num_heads=1025), 2),
    (dict(num_heads=1024, max_tokens=1 << 20), 2),
])
def test_create_rejects_bad_config(L, over, code):
    h = P()
    assert L.mla_attn_create(ctypes.byref(cfg(**over)), ctypes.byref(h)) == code
    assert not h.value


def test_null_handles(L):
    h = P()
    assert L.mla_attn_create(None, ctypes.byref(h)) == 1
    assert L.mla_attn_create(ctypes.byref(cfg()), None) == 1
    assert L.mla_attn_destroy(None) == 1
    assert L.mla_attn_status(None, None) == 1
    assert L.mla_attn_last_launches(None) == -1
    h = FakeHandle()
    for fn, base in ((L.mla_latent_append, APPEND), (L.mla_attn_paged_run, PAGED), (L.mla_attn_prompt_run, PROMPT)):
        assert fn(None, packed(fn, base), None) == 1
        assert fn(h.ptr, None, None) == 1


_at = [0x100000]


def fake():
    _at[0] += 0x1000
    return P(_at[0])


# in the order of the structs' fields
APPEND = dict(ckv=fake(), kpe=fake(), q=fake(), pos=fake(), gamma=fake(), cos=fake(), sin=fake(), slots=fake(), lat=fake(),
              kc=fake(), qo=fake(), T=2, page=16, nb=4, ckv_s=576, kpe_s=576, q_t=16 * 192, q_h=192, lat_s=512, kc_s=64,
              qo_t=1024, qo_h=64)
PAGED = dict(ql=fake(), qp=fake(), cu=None, lens=fake(), table=fake(), lat=fake(), kc=fake(), out=fake(), lse=fake(), n=2, T=2,
             ts=4, page=16, nb=8, ql_t=8192, ql_h=512, qp_t=1024, qp_h=64, lat_s=512, kc_s=64)
PROMPT = dict(qn=fake(), qp=fake(), kn=fake(), kp=fake(), v=fake(), o=fake(), lse=fake(), cu=None, b=1, s=4, n=0, causal=1,
              qn_b=8192, qn_h=512, qn_t=128, qp_b=4096, qp_h=256, qp_t=64, kn_b=8192, kn_h=512, kn_t=128, kp_b=256, kp_t=64,
              v_b=8192, v_h=512, v_t=128, o_b=8192, o_h=512, o_t=128)
STRUCTS = dict(mla_latent_append_args=B._APPEND_ARGS, mla_attn_paged_args=B._PAGED_ARGS, mla_attn_prompt_args=B._PROMPT_ARGS)


def packed(fn, base, **over):
    args = dict(base)
    args.update(over)
    st = {"mla_latent_append": B._APPEND_ARGS, "mla_attn_paged_run": B._PAGED_ARGS, "mla_attn_prompt_run": B._PROMPT_ARGS}[fn.__name__]
    return st.pack(*[(x.value if isinstance(x, P) else 0 if x is None else x) for x in args.values()])


class FakeHandle:
    """A handle struct built on the host: the checks read its configuration only."""

    def __init__(self, **over):
        self.c = cfg(**over)
        if not self.c.num_kv_heads:
            self.c.num_kv_heads = self.c.num_heads
        self.mem = (ctypes.c_char * 1024)()
        ctypes.memmove(self.mem, ctypes.byref(self.c), ctypes.sizeof(self.c))
        self.ptr = ctypes.cast(self.mem, P)


def refuse(fn, base, code, **over):
    h = FakeHandle()
    assert fn(h.ptr, packed(fn, base, **over), None) == code, over


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(T=17), 3), (dict(page=0), 1), (dict(nb=0), 1), (dict(page=1 << 16, nb=1 << 16), 1),
    (dict(ckv=None), 1), (dict(kpe=None), 1), (dict(slots=None), 1), (dict(lat=None), 1), (dict(kc=None), 1),
    (dict(cos=None), 1), (dict(sin=None), 1), (dict(pos=None), 1), (dict(qo=None), 1), (dict(cos=None, sin=None), 1),
    (dict(ckv_s=504), 1), (dict(ckv_s=580), 1), (dict(kpe_s=56), 1), (dict(lat_s=0), 1), (dict(lat_s=516), 1),
    (dict(kc_s=60), 1), (dict(q_t=0), 1), (dict(q_h=60), 1), (dict(qo_t=4), 1), (dict(qo_h=0), 1), (dict(ckv_s=-576), 1),
    (dict(qo=APPEND["q"]), 1),
    (dict(ckv=P(0x100008)), 4), (dict(gamma=P(0x100004)), 4), (dict(qo=P(0x100002)), 4), (dict(slots=P(0x100004)), 4),
    (dict(T=0, ckv=None, lat=None), 0),
])
def test_append_refusals(L, over, code):
    refuse(L.mla_latent_append, APPEND, code, **over)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(T=-1), 1), (dict(T=17, n=17), 3), (dict(T=3), 1), (dict(page=0), 1), (dict(nb=-1), 1),
    (dict(page=1 << 16, nb=1 << 15), 1), (dict(ts=-1), 1), (dict(ql=None), 1), (dict(qp=None), 1), (dict(lens=None), 1),
    (dict(table=None), 1), (dict(lat=None), 1), (dict(kc=None), 1), (dict(out=None), 1),
    (dict(ql_t=511), 1), (dict(ql_h=256), 1), (dict(qp_t=60), 1), (dict(qp_h=8), 1), (dict(lat_s=511), 1), (dict(kc_s=0), 1),
    (dict(ql=P(0x100008)), 4), (dict(table=P(0x100004)), 4), (dict(cu=P(0x100004)), 4), (dict(lse=P(0x100008)), 4),
    (dict(n=0), 0), (dict(T=0, ql=None), 0),
])
def test_paged_refusals(L, over, code):
    refuse(L.mla_attn_paged_run, PAGED, code, **over)


@pytest.mark.parametrize("over,code", [
    (dict(b=-1), 1), (dict(s=-1), 1), (dict(s=17), 3), (dict(b=5), 3), (dict(causal=2), 1), (dict(b=2, cu=fake(), n=1), 1),
    (dict(cu=fake(), n=-1), 1), (dict(qn=None), 1), (dict(qp=None), 1), (dict(kn=None), 1), (dict(kp=None), 1),
    (dict(v=None), 1), (dict(o=None), 1), (dict(qn_t=120), 1), (dict(qn_h=100), 1), (dict(kn_t=129), 1), (dict(kp_t=32), 1),
    (dict(v_h=-512), 1), (dict(o_t=127), 1), (dict(b=2, qn_b=0), 1), (dict(b=2, kp_b=63), 1),
    (dict(qn=P(0x100008)), 4), (dict(o=P(0x100002)), 4), (dict(cu=P(0x100004), n=1), 4), (dict(lse=P(0x100004)), 4),
    (dict(b=0), 0), (dict(s=0, qn=None), 0), (dict(cu=fake(), n=0), 0),
])
def test_prompt_refusals(L, over, code):
    refuse(L.mla_attn_prompt_run, PROMPT, code, **over)


def test_attn_config_layout_matches_the_header(tmp_path):
    src = open(os.path.join(ROOT, "include", "mla_prolog.h")).read()
    body = re.search(r"typedef struct mla_attn_config \{(.*?)\} mla_attn_config;", src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = [re.match(r"\s*(.*?)\s+(\w+)$", f.strip()).groups() for f in body.split(";") if f.strip()]
    ctypes_of = {"int": ctypes.c_int, "float": ctypes.c_float, "unsigned long long": ctypes.c_ulonglong}
    assert [(n, ctypes_of[t]) for t, n in fields] == list(B.AttnConfig._fields_)
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/usr/local/cuda/include"):
        pytest.skip("gcc or the CUDA headers are missing")
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mla_prolog.h"\nint main(void) {\n'
                    + '  printf("%zu\\n", sizeof(mla_attn_config));\n'
                    + "".join(f'  printf("%zu\\n", offsetof(mla_attn_config, {n}));\n' for _, n in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, str(prog), "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", "-o", str(exe)],
                   check=True, capture_output=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [ctypes.sizeof(B.AttnConfig)] + [getattr(B.AttnConfig, n).offset for _, n in fields]


def test_binding_rejects_host_tensors():
    """No CPU fallback: tensors that are not on the handle's device raise before the library is called."""
    a = B.MLAAttention.__new__(B.MLAAttention)
    a.cfg = dict(kv_lora_rank=512, rope_dim=64, nope_dim=128, v_dim=128, num_heads=4, max_pos=8)
    a.h, a.device, a.dtype, a.heads, a.kv_heads = None, 0, torch.float16, 4, 4
    a.rank, a.rope, a.nope, a.vdim, a.table_numel = 512, 64, 128, 128, 512
    x = torch.zeros(2, 576, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(2, 4, 512, dtype=torch.float16)
    with pytest.raises(TypeError):
        a.append_latent(x[:, :512], x[:, 512:], i, None, None, None, i, c, c[..., :64])
    with pytest.raises(TypeError):
        a.run_paged(c, c[..., :64], i, i[None], c, c[..., :64], c)
    with pytest.raises(TypeError):
        a.run_prompt(c[None, ..., :128], c[None, ..., :64], c[None, ..., :128], c[None, :, :1, :64], c[None, ..., :128], c[None])


@pytest.mark.parametrize("name", list(STRUCTS))
def test_argument_structs_match_the_header(name, tmp_path):
    """The binding packs pointers, then ints, in the header's order, to the C compiler's size."""
    src = open(os.path.join(ROOT, "include", "mla_prolog.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    kinds = []
    for line in body.split(";"):
        line = line.strip()
        if not line:
            continue
        kinds += ["Q"] if "*" in line else ["i"] * (line.count(",") + 1)
    assert kinds == sorted(kinds), "pointers come first"
    assert STRUCTS[name].format == "@%dQ%di4x" % (kinds.count("Q"), kinds.count("i"))
    base = dict(mla_latent_append_args=APPEND, mla_attn_paged_args=PAGED, mla_attn_prompt_args=PROMPT)[name]
    assert len(base) == len(kinds)
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/usr/local/cuda/include"):
        pytest.skip("gcc or the CUDA headers are missing")
    prog = tmp_path / "size.c"
    prog.write_text('#include <stdio.h>\n#include "mla_prolog.h"\nint main(void) { printf("%%zu\\n", sizeof(%s)); return 0; }\n' % name)
    exe = tmp_path / "size"
    subprocess.run([gcc, str(prog), "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", "-o", str(exe)],
                   check=True, capture_output=True)
    assert int(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout) == STRUCTS[name].size

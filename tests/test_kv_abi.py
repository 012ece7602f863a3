"""The cache operators' C ABI without a GPU: struct layouts, and arguments
refused on the host (fake pointers, never dereferenced)."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from speculative_decoding_verification_04_gb300 import kv_cache  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


def lib():
    return kv_cache._library()


def cache(**kw):
    c = sv.SVKvCache()
    v = dict(k=FAKE, v=FAKE, page_table=FAKE, max_pages=4, format=0, layers=1, num_pages=16, n_kv_heads=2, page_size=16, head_dim=64)
    v.update(kw)
    for n, x in v.items():
        setattr(c, n, x)
    return c


def tokens(**kw):
    t = sv.SVKvTokens()
    v = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=256, k_stride=128, v_stride=128, q_out=FAKE * 2, dtype=1, n_heads=4, B=2, S=3, rows=6, eps=1e-6)
    v.update(kw)
    for n, x in v.items():
        setattr(t, n, x)
    return t


def append(c=None, t=None, kv=FAKE):
    c, t = c or cache(), t or tokens()
    return lib().spec_kv_append(ctypes.addressof(c), ctypes.addressof(t), kv, None, None)


def attention(c=None, kv=FAKE, q=FAKE, stride=256, dtype=1, heads=4, B=2, N=3, scale=0.1, out=FAKE, ws=FAKE, nbytes=1 << 30, parent=None):
    c = c or cache()
    return lib().spec_tree_attention(ctypes.addressof(c), kv, None, parent, q, stride, dtype, heads, B, N, scale, out, None, ws, nbytes, None)


def commit(c=None, kv=FAKE, path=FAKE, length=FAKE, B=2, N=3, out=FAKE):
    c = c or cache()
    return lib().spec_kv_commit(ctypes.addressof(c), kv, path, length, B, N, out, None, None)


def read(c=None, start=FAKE, bounds=FAKE, B=2, rows=5, dtype=1, k=FAKE, v=FAKE):
    c = c or cache()
    return lib().spec_kv_read(ctypes.addressof(c), start, bounds, B, rows, dtype, k, v, None, None)


@pytest.mark.parametrize("call", [append, attention, commit, read])
def test_cache_descriptions_are_checked(call):
    for bad in (dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(page_table=0), dict(page_table=FAKE + 2), dict(max_pages=0), dict(format=2),
                dict(layers=0), dict(num_pages=0), dict(n_kv_heads=0), dict(k_scale=FAKE), dict(format=1), dict(format=1, k_scale=FAKE),
                dict(format=1, k_scale=FAKE, v_scale=FAKE + 2)):
        assert call(c=cache(**bad)) == sv.SV_ERR_INVALID_ARG, bad
    for bad in (dict(head_dim=48), dict(head_dim=72), dict(head_dim=272), dict(page_size=4), dict(page_size=24), dict(page_size=2048),
                dict(num_pages=1 << 27, page_size=16), dict(max_pages=1 << 28, page_size=16)):
        assert call(c=cache(**bad)) == sv.SV_ERR_UNSUPPORTED, bad


def test_append_arguments():
    assert append(t=tokens(B=0, S=0, rows=0)) == sv.SV_OK
    for bad in (dict(dtype=2), dict(B=-1), dict(S=-1), dict(rows=5), dict(k=0), dict(v=0), dict(q_out=0), dict(n_heads=0), dict(q=FAKE + 8),
                dict(k=FAKE + 4), dict(q_stride=260), dict(k_stride=4), dict(v_stride=1), dict(q_norm=FAKE + 2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(cos_sin=FAKE, rotary_dim=0, max_positions=9), dict(cos_sin=FAKE, rotary_dim=80, max_positions=9),
                dict(cos_sin=FAKE, rotary_dim=24, max_positions=9), dict(cos_sin=FAKE, rotary_dim=32, max_positions=0), dict(cos_sin=FAKE + 4, rotary_dim=32, max_positions=9),
                dict(row_start=FAKE, parent=FAKE), dict(row_start=FAKE, n_new=FAKE), dict(parent=FAKE, S=33, rows=66), dict(parent=FAKE + 1),
                dict(q_out=FAKE, q_stride=512)):
        assert append(t=tokens(**bad)) == sv.SV_ERR_INVALID_ARG, bad
    assert append(kv=None) == sv.SV_ERR_INVALID_ARG
    assert append(t=tokens(n_heads=1 << 17)) == sv.SV_ERR_UNSUPPORTED


def test_attention_arguments():
    assert attention(B=0) == sv.SV_OK
    for bad in (dict(B=-1), dict(N=0), dict(N=33), dict(heads=0), dict(heads=3), dict(dtype=7), dict(scale=float("nan")), dict(scale=float("inf")), dict(kv=None),
                dict(q=None), dict(q=FAKE + 8), dict(stride=257), dict(out=None), dict(out=FAKE + 2), dict(kv=FAKE + 2), dict(parent=FAKE + 2)):
        assert attention(**bad) == sv.SV_ERR_INVALID_ARG, bad
    assert attention(dtype=0) == sv.SV_ERR_UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(nbytes=8)):
        assert attention(**bad) == sv.SV_ERR_NO_MEMORY, bad


def test_attention_workspace_sizes():
    f = sv.sv_attention_workspace_size
    assert f(1, 1, 1, 64) >= 256
    assert f(32, 64, 8, 256) >= f(1, 64, 8, 256)
    for bad in ((0, 8, 8, 64), (33, 8, 8, 64), (4, 7, 2, 64), (4, 0, 0, 64), (4, 8, 8, 40), (4, 8, 8, 512)):
        assert f(*bad) == 0, bad


def test_commit_and_read_arguments():
    assert commit(B=0) == sv.SV_OK and read(rows=0) == sv.SV_OK
    for bad in (dict(B=-1), dict(N=0), dict(N=33), dict(kv=None), dict(path=None), dict(length=None), dict(out=None), dict(out=FAKE + 2)):
        assert commit(**bad) == sv.SV_ERR_INVALID_ARG, bad
    assert commit(c=cache(layers=70000)) == sv.SV_ERR_UNSUPPORTED
    for bad in (dict(B=0), dict(B=-1), dict(rows=-1), dict(dtype=4), dict(start=None), dict(bounds=None), dict(k=None), dict(v=None), dict(k=FAKE + 4), dict(bounds=FAKE + 1)):
        assert read(**bad) == sv.SV_ERR_INVALID_ARG, bad


def test_structs_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if gcc is None or not os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
        pytest.skip("needs gcc and the CUDA headers")
    structs = {"sv_kv_cache": sv.SVKvCache, "sv_kv_tokens": sv.SVKvTokens}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "specverify.h"', "int main(void) {"]
    for name, s in structs.items():
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in s._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = str(tmp_path / "layout")
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), "-I", inc, str(tmp_path / "layout.c"), "-o", exe], check=True)
    for line in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n"):
        if line.strip():
            name, field, value = line.split()
            s = structs[name]
            assert int(value) == (ctypes.sizeof(s) if field == "size" else getattr(s, field).offset), line


def test_binding_refuses_cpu_tensors():
    import torch
    c = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.spec_tree_attention(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), c, c, t, n)
    with pytest.raises(ValueError):
        sv.spec_kv_append(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), c, c, t, n)
    with pytest.raises(ValueError):
        sv.spec_kv_commit(c, c, t, n, torch.zeros(1, 4, dtype=torch.int32), n)
    with pytest.raises(ValueError):
        sv.spec_kv_read(c, c, t, n, torch.zeros(2, dtype=torch.int32), 0)

"""The filters' and the pages' C ABI and binding without a GPU: struct layout,
and arguments refused on the host (fake pointers, never dereferenced)."""
import ctypes
import os
import shutil
import subprocess
import types

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from speculative_decoding_verification_04_gb300 import filters, kv_cache, pages  # noqa: E402
from test_kv_devices import T  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000
I32, I64, F32, BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16


def sample(x=FAKE, dtype=1, u=FAKE, t=FAKE, k=None, p=None, m=None, B=2, V=100, tok=FAKE, prob=None, kept=None):
    return filters._library().spec_sample_filtered(x, dtype, u, t, k, p, m, B, V, tok, prob, kept, None)


def rows(x=FAKE, dtype=1, t=FAKE, k=None, p=None, m=None, B=2, S=3, n=None, V=100, out=FAKE, kept=None):
    return filters._library().spec_filter_logits(x, dtype, t, k, p, m, B, S, n, V, out, kept, None)


def pool(**kw):
    v = dict(page_table=FAKE, held=FAKE, free_pages=FAKE, free_count=FAKE, B=2, max_pages=4, page_size=16, capacity=9)
    v.update(kw)
    return sv.SVKvPool(**v)


def reserve(kv=FAKE, n=None, starts=None, S=3, rows=6, held=FAKE, free=FAKE, slots=None, errors=None, **kw):
    p = pool(**kw)
    return pages._library().spec_kv_reserve(ctypes.addressof(p), kv, n, starts, S, rows, held, free, slots, errors, None)


def release(kv=FAKE, held=FAKE, free=FAKE, errors=None, **kw):
    p = pool(**kw)
    return pages._library().spec_kv_release(ctypes.addressof(p), kv, held, free, errors, None)


def test_sample_arguments():
    assert sample(B=0) == sv.SV_OK
    for bad in (dict(x=None), dict(dtype=2), dict(dtype=-1), dict(u=None), dict(t=None), dict(B=-1), dict(V=0), dict(tok=None), dict(x=FAKE + 1), dict(x=FAKE + 2, dtype=0),
                dict(u=FAKE + 2), dict(t=FAKE + 1), dict(k=FAKE + 2), dict(p=FAKE + 2), dict(m=FAKE + 3), dict(tok=FAKE + 2), dict(prob=FAKE + 1), dict(kept=FAKE + 2)):
        assert sample(**bad) == sv.SV_ERR_INVALID_ARG, bad
    for dtype in (0, 1):
        assert sample(dtype=dtype, V=sv.sv_max_vocab(dtype) + 1) == sv.SV_ERR_UNSUPPORTED
    assert sample(B=1 << 30) == sv.SV_ERR_UNSUPPORTED


def test_filter_arguments():
    assert rows(B=0) == sv.SV_OK
    for bad in (dict(x=None), dict(dtype=2), dict(t=None), dict(B=-1), dict(S=0), dict(V=0), dict(out=None), dict(out=FAKE + 1), dict(n=FAKE + 2), dict(kept=FAKE + 2),
                dict(out=FAKE + 2), dict(out=FAKE + 2 * 3 * 100 * 2 - 2), dict(out=FAKE - 2), dict(out=FAKE - 2 * 3 * 100 * 2 + 2)):
        assert rows(**bad) == sv.SV_ERR_INVALID_ARG, bad
    assert rows(V=sv.sv_max_vocab(1) + 1) == sv.SV_ERR_UNSUPPORTED
    assert rows(B=1 << 20, S=1 << 10) == sv.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [reserve, release])
def test_pools_are_checked(call):
    assert call(B=0, **({"rows": 0} if call is reserve else {})) == sv.SV_OK
    for bad in (dict(page_table=0), dict(held=None), dict(free_pages=0), dict(free_count=0), dict(kv=None), dict(free=None), dict(B=-1), dict(max_pages=0),
                dict(capacity=-1), dict(page_table=FAKE + 2), dict(kv=FAKE + 1), dict(held=FAKE + 2), dict(free=FAKE + 2), dict(errors=FAKE + 2)):
        assert call(**bad) == sv.SV_ERR_INVALID_ARG, bad
    for bad in (dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(max_pages=1 << 28)):
        assert call(**bad) == sv.SV_ERR_UNSUPPORTED, bad


def test_reserve_arguments():
    for bad in (dict(rows=5), dict(S=-1, rows=-2), dict(starts=FAKE, n=FAKE), dict(starts=FAKE, rows=-1), dict(n=FAKE + 2), dict(starts=FAKE + 2), dict(slots=FAKE + 4)):
        assert reserve(**bad) == sv.SV_ERR_INVALID_ARG, bad


def test_struct_matches_the_header(tmp_path):
    gcc = shutil.which("gcc")
    inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if gcc is None or not os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
        pytest.skip("needs gcc and the CUDA headers")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "specverify.h"', "int main(void) {", '  printf("size %zu\\n", sizeof(sv_kv_pool));']
    lines += [f'  printf("{f} %zu\\n", offsetof(sv_kv_pool, {f}));' for f, _ in sv.SVKvPool._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = str(tmp_path / "layout")
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), "-I", inc, str(tmp_path / "layout.c"), "-o", exe], check=True)
    for line in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n"):
        if line.strip():
            field, value = line.split()
            assert int(value) == (ctypes.sizeof(sv.SVKvPool) if field == "size" else getattr(sv.SVKvPool, field).offset), line


@pytest.fixture
def calls(monkeypatch):
    """Device 0 is current; what would be launched is counted."""
    made = []
    record = lambda name: lambda *args: (made.append(name), 0)[1]  # noqa: E731
    monkeypatch.setattr(pages, "_lib", types.SimpleNamespace(**{n: record(n) for n in ("spec_kv_reserve", "spec_kv_release")}))
    monkeypatch.setattr(filters, "_lib", types.SimpleNamespace(**{n: record(n) for n in ("spec_sample_filtered", "spec_filter_logits")}))
    monkeypatch.setattr(kv_cache, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(kv_cache, "_current_raw_stream", lambda dev: 0)
    return made


POOL = dict(page_table=((3, 4), I32), kv_len=((3,), I32), held=((3,), I32), free_pages=((9,), I32), free_count=((1,), I32))
OUTS = dict(held_out=((3,), I32), free_count_out=((1,), I32), errors=((1,), I32))
FILTERS = dict(temperature=((3,), F32), top_k=((3,), I32), top_p=((3,), F32), min_p=((3,), F32))
CALLS = {
    "reserve": (sv.spec_kv_reserve, dict(POOL, **OUTS, n_new=((3,), I32), slots=((3, 5), I64)), dict(page_size=8, S=5)),
    "reserve packed": (sv.spec_kv_reserve, dict(POOL, **OUTS, row_start=((4,), I32), slots=((11,), I64)), dict(page_size=8)),
    "release": (sv.spec_kv_release, dict(POOL, **OUTS), dict(page_size=8)),
    "sample": (sv.spec_sample_filtered, dict(FILTERS, logits=((3, 50), BF16), uniforms=((3,), F32), out_tokens=((3,), I32), out_prob=((3,), F32), out_kept=((3,), I32)), {}),
    "filter": (sv.spec_filter_logits, dict(FILTERS, logits=((3, 2, 50), F32), n_rows=((3,), I32), out=((3, 2, 50), F32), out_kept=((3, 2), I32)), {}),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_type_or_shape(name, calls):
    f, spec, extra = CALLS[name]
    make = lambda **other: {n: other.get(n) or T(*v, 0) for n, v in spec.items()}  # noqa: E731
    f(**make(), **extra)
    assert len(calls) == 1
    for n, (shape, dtype) in spec.items():
        with pytest.raises(ValueError):
            f(**make(**{n: T(shape, dtype, 1)}), **extra)
        with pytest.raises((TypeError, ValueError)):
            f(**make(**{n: T(shape, torch.int8, 0)}), **extra)
        if n not in ("free_pages", "logits", "errors", "page_table") and not (name == "reserve packed" and n == "slots"):
            with pytest.raises(ValueError):
                f(**make(**{n: T((*shape[:-1], shape[-1] + 1), dtype, 0)}), **extra)
    with pytest.raises(ValueError):
        f(**{n: T(*v, 1) for n, v in spec.items()}, **extra)
    stream = lambda dev: types.SimpleNamespace(cuda_stream=77, device_index=dev)  # noqa: E731
    with pytest.raises(ValueError):
        f(**make(), **extra, stream=stream(1))
    assert len(calls) == 1
    f(**make(), **extra, stream=stream(0))
    assert len(calls) == 2


def test_reserve_wants_tokens_or_starts(calls):
    made = {n: T(*v, 0) for n, v in POOL.items()}
    for bad in (dict(), dict(S=-1), dict(S=1 << 31), dict(S=3, row_start=T((4,), I32, 0)), dict(n_new=T((3,), I32, 0), row_start=T((4,), I32, 0)),
                dict(row_start=T((4,), I32, 0), slots=T((3, 5), I64, 0))):
        with pytest.raises(ValueError):
            sv.spec_kv_reserve(**made, page_size=8, **bad)
    assert calls == []


def test_cpu_tensors_are_refused():
    z = torch.zeros
    with pytest.raises(ValueError):
        sv.spec_sample_filtered(z(2, 9), z(2), z(2))
    with pytest.raises(ValueError):
        sv.spec_filter_logits(z(2, 9), z(2))
    with pytest.raises(ValueError):
        sv.spec_kv_reserve(z(2, 3, dtype=I32), z(2, dtype=I32), z(2, dtype=I32), z(4, dtype=I32), z(1, dtype=I32), 8, S=1)
    with pytest.raises(ValueError):
        sv.spec_kv_release(z(2, 3, dtype=I32), z(2, dtype=I32), z(2, dtype=I32), z(4, dtype=I32), z(1, dtype=I32), 8)

"""The cache operators take tensors and streams of the current device alone:
the library launches there.  Stand-ins for tensors of two devices; the library
itself is a stand-in too, so nothing is launched."""
import types

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from speculative_decoding_verification_04_gb300 import kv_cache  # noqa: E402


class T:
    """What the binding asks of a contiguous tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, dev):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.insert(0, n)
            n *= s
        return tuple(out)


@pytest.fixture
def calls(monkeypatch):
    """The device that is current is 0; what would be launched is counted."""
    made = []
    record = lambda name: lambda *args: (made.append(name), 0)[1]  # noqa: E731
    lib = types.SimpleNamespace(**{n: record(n) for n in ("spec_kv_append", "spec_tree_attention_ex", "spec_kv_commit", "spec_kv_read")})
    monkeypatch.setattr(kv_cache, "_lib", lib)
    monkeypatch.setattr(kv_cache, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(kv_cache, "_current_raw_stream", lambda dev: 0)
    return made


I32, BF16, F32, E4M3 = torch.int32, torch.bfloat16, torch.float32, torch.float8_e4m3fn
CACHE = dict(k_cache=((4, 2, 8, 64), E4M3), v_cache=((4, 2, 8, 64), E4M3), k_scale=((4, 2, 8), F32), v_scale=((4, 2, 8), F32), page_table=((3, 2), I32))
CALLS = {
    sv.spec_kv_append: dict(CACHE, k=((3, 5, 2, 64), BF16), v=((3, 5, 2, 64), BF16), q=((3, 5, 4, 64), BF16), kv_len=((3,), I32), n_new=((3,), I32),
                            q_norm=((64,), BF16), k_norm=((64,), BF16), cos_sin=((9, 32), F32), parent=((3, 5), I32), q_out=((3, 5, 4, 64), BF16), errors=((1,), I32)),
    sv.spec_tree_attention: dict(CACHE, q=((3, 5, 4, 64), BF16), kv_len=((3,), I32), n_nodes=((3,), I32), parent=((3, 5), I32), out=((3, 5, 4, 64), BF16),
                                 workspace=((1 << 20,), torch.uint8), errors=((1,), I32)),
    sv.spec_kv_commit: dict(CACHE, kv_len=((3,), I32), out_path=((3, 5), I32), out_len=((3,), I32), kv_len_out=((3,), I32), errors=((1,), I32)),
    sv.spec_kv_read: dict(CACHE, start=((3,), I32), row_start=((4,), I32), k_out=((9, 2, 64), BF16), v_out=((9, 2, 64), BF16), errors=((1,), I32)),
}


@pytest.mark.parametrize("f", CALLS, ids=lambda f: f.__name__)
def test_one_tensor_on_another_device(f, calls):
    extra = {"rows": 9} if f is sv.spec_kv_read else {}
    make = lambda other=(): {n: T(*spec, 1 if n in other else 0) for n, spec in CALLS[f].items()}  # noqa: E731
    f(**make(), **extra)
    assert len(calls) == 1
    for n in CALLS[f]:
        with pytest.raises(ValueError):
            f(**make({n}), **extra)
    with pytest.raises(ValueError):          # all of them, but another device is current
        f(**make(set(CALLS[f])), **extra)
    stream = lambda dev: types.SimpleNamespace(cuda_stream=77, device_index=dev)  # noqa: E731
    with pytest.raises(ValueError):
        f(**make(), **extra, stream=stream(1))
    assert len(calls) == 1
    f(**make(), **extra, stream=stream(0))
    assert len(calls) == 2


def test_packed_starts_on_another_device(calls):
    made = {n: T(*spec, 0) for n, spec in CALLS[sv.spec_kv_append].items() if n in CACHE or n == "kv_len"}
    rows = {n: T((7, 2, 64), BF16, 0) for n in ("k", "v")}
    sv.spec_kv_append(**made, **rows, row_start=T((4,), I32, 0))
    with pytest.raises(ValueError):
        sv.spec_kv_append(**made, **rows, row_start=T((4,), I32, 1))
    assert calls == ["spec_kv_append"]


def test_streams_name_their_device():
    assert hasattr(torch.cuda.Stream, "device_index")

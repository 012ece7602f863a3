"""What the cache operators refuse on the host (fake pointers, never
dereferenced)."""
import pytest

pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from speculative_decoding_verification_04_gb300 import kv_cache  # noqa: E402
from test_kv_abi import FAKE, cache  # noqa: E402


def test_attention_waits_that_do_not_exist():
    import ctypes
    call = lambda bits, B=2: kv_cache._library().spec_tree_attention_ex(  # noqa: E731
        ctypes.addressof(c), FAKE, None, None, FAKE, 256, 1, 4, B, 3, 0.1, FAKE, None, FAKE, 1 << 30, bits, None)
    c = cache()
    for bits in (1 << sv.SV_ATTENTION_WAITS, 1 << 31, (1 << 32) - 1):
        assert call(bits) == sv.SV_ERR_INVALID_ARG
    assert call((1 << sv.SV_ATTENTION_WAITS) - 1, B=0) == sv.SV_OK


LIMIT = (1 << 31) - (1 << 16)   # positions of a page table's row


@pytest.mark.parametrize("page", [8, 64, 1024])
def test_positions_of_a_sequence(page):
    import ctypes
    lib = kv_cache._library()
    for pages, want in ((LIMIT // page, sv.SV_OK), (LIMIT // page + 1, sv.SV_ERR_UNSUPPORTED)):
        c, t = cache(page_size=page, max_pages=pages), sv.SVKvTokens()   # (no tokens)
        at = ctypes.addressof(c)
        assert lib.spec_kv_append(at, ctypes.addressof(t), FAKE, None, None) == want
        assert lib.spec_tree_attention(at, FAKE, None, None, FAKE, 256, 1, 4, 0, 3, 0.1, FAKE, None, FAKE, 1 << 30, None) == want
        assert lib.spec_kv_commit(at, FAKE, FAKE, FAKE, 0, 3, FAKE, None, None) == want
        assert lib.spec_kv_read(at, FAKE, FAKE, 2, 0, 1, FAKE, FAKE, None, None) == want

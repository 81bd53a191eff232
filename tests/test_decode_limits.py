"""Sizes whose launches would pass 2^32 threads are refused before anything
runs (CPU: every call returns from the library's checks)."""
import ctypes

import lora_serving_build_amd as lsb
from lora_serving_build_amd import decode as D
from test_decode_abi import FAKE, UNS, WS, _attention, _cache, _expect


def test_q4_weights():
    most = (1 << 27) - 16                       # 2^23 - 1 tiles of 16 outputs
    assert lsb.lora_q4_packed_bytes(most, 128, 128, False) > 0
    assert lsb.lora_q4_packed_bytes(most + 1, 128, 128, False) == 0
    assert lsb.lora_q4_packed_bytes(1 << 18, 127 * 1024, 128, False) > 0
    assert lsb.lora_q4_packed_bytes(1 << 18, 128 * 1024, 128, False) == 0  # 2^24 blocks
    w = D._CQ4Weight()
    call = lambda n, k: lsb.lib().lora_q4_pack(FAKE, 1 << 30, FAKE, 1 << 24, None, 0, n, k, 128, 0, FAKE, 0,  # noqa: E731
                                               ctypes.addressof(w), None)
    _expect(call(most + 1, 128), UNS, "too large")
    _expect(call(most, 128), WS, "needed")
    big = D._CQ4Weight(most + 1, 128, 128, 0, 0, FAKE)
    _expect(lsb.lib().lora_q4_matmul(FAKE, 128, ctypes.addressof(big), 1, FAKE, 1 << 28, 0, None, 0, None), UNS, "too large")


def test_append_and_compact():
    lib, c = lsb.lib(), _cache()
    r = ctypes.addressof(c)
    _expect(lib.lora_pages_append(r, 0, 1, FAKE, 128, 64, FAKE, 128, 64, 2, 64, FAKE, FAKE, 1, 1 << 24, None), UNS, "T 16777216")
    for seqs, code, text in ((1 << 24, UNS, "rows of the table"), ((1 << 24) - 1, WS, "needed")):
        c = _cache(max_seqs=seqs)
        _expect(lib.lora_pages_compact(ctypes.addressof(c), FAKE, FAKE, 0, None), code, text)


def test_attention_of_very_many_sequences():
    call = lambda **a: _attention(lsb.lib(), ws_bytes=0, mask=None, **a)  # noqa: E731
    short = dict(heads=16, kv_heads=16, max_pages=1, ld_table=1)
    _expect(call(T=1 << 20, B=1 << 20, **short), UNS, "row tiles")       # 512 threads for each line
    _expect(call(T=1 << 18, B=1 << 18, **short), WS, "needed")
    parts = dict(heads=16, kv_heads=16, max_pages=70, ld_table=70)
    _expect(call(T=1 << 20, B=1 << 20, **parts), UNS, "row tiles")       # 256 threads for each in the join
    _expect(call(T=15 << 16, B=1000, **parts), WS, "needed")

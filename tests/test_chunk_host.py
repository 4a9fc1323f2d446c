"""Host checks of the chunk-attention, read-back and 4-bit slot-append calls: every refusal comes before any device work, so no
GPU is needed."""
import ctypes

import pytest

from decode_attention_mfa_gb300 import build as mfa_build
from decode_attention_mfa_gb300 import capi


@pytest.fixture(scope="module")
def lib():
    mfa_build.build()
    return capi.load()


@pytest.fixture(scope="module")
def mem():
    buf = (ctypes.c_uint8 * 16384)()
    return buf, (ctypes.addressof(buf) + 255) & ~255


def refused(fn, good, bad, status=1):
    for key, value in bad:
        assert fn(*dict(good, **{key: value}).values()) == status, (key, value)


@pytest.mark.parametrize("kv", ["", "_fp8", "_fp4"])
def test_chunk_attention_refusals(lib, mem, kv):
    p = mem[1]
    good = dict(q=p, kc=p + 512, vc=p + 1024)
    good.update(dict(k_scale=p + 4096, v_scale=p + 4352) if kv else {})
    good.update(table=p + 1536, lens=p + 2048, starts=p + 2304, out=p + 3584, lse=p + 3840, scale=1 / 16, batch=4, tokens=16,
                max_pages=2, num_pages=8, ws=p + 5120, n=1 << 30, stream=None)
    fn = getattr(lib, "mfa_chunk_attention" + kv)
    pointers = [k for k in good if k in ("q", "kc", "vc", "k_scale", "v_scale", "table", "lens", "starts", "out", "lse")]
    bad = [(k, None) for k in pointers] + [(k, good[k] + 2) for k in pointers]
    bad += [(k, good[k] + 8) for k in pointers if k in ("q", "kc", "vc", "k_scale", "v_scale", "out")]
    bad += [(k, good[k] + 16) for k in ("kc", "vc") if kv == "_fp4"]
    bad += [("batch", 0), ("batch", capi.MAX_BATCH + 1), ("tokens", -1), ("tokens", 2 ** 24 + 1), ("max_pages", 0), ("max_pages", 2 ** 26),
            ("max_pages", 2 ** 24 + 1), ("num_pages", 0)]
    refused(fn, good, bad)
    # every position of the line of work fits 31 bits
    refused(fn, dict(good, tokens=2 ** 24), [("max_pages", 1100)])
    refused(fn, good, [("ws", None), ("ws", p + 8)], 4)
    with pytest.raises(capi.MFAError):
        getattr(capi, "mfa_chunk_attention" + kv)(*dict(good, batch=0, stream=0).values())


def test_chunk_workspace_refusals(lib):
    for args in ((0, 1), (capi.MAX_BATCH + 1, 1), (4, -1), (4, 2 ** 24 + 1)):
        assert lib.mfa_chunk_workspace_bytes(*args) == 0
        with pytest.raises(capi.MFAError):
            capi.mfa_chunk_workspace_bytes(*args)


@pytest.mark.parametrize("kv", ["", "_fp8", "_fp4"])
def test_read_refusals(lib, mem, kv):
    p = mem[1]
    good = dict(kc=p, vc=p + 512)
    good.update(dict(k_scale=p + 4096, v_scale=p + 4352) if kv else {})
    good.update(table=p + 1536, first=p + 2048, starts=p + 2304, k=p + 3584, v=p + 3840, ks=256, vs=256, batch=4, rows=16, max_pages=2,
                num_pages=8, ws=p + 5120, stream=None)
    fn = getattr(lib, "mfa_kv_read" + kv)
    pointers = [k for k in good if k in ("kc", "vc", "k_scale", "v_scale", "table", "starts", "k", "v")]
    bad = [(k, None) for k in pointers] + [(k, good[k] + 2) for k in pointers + ["first"]]
    bad += [(k, good[k] + 8) for k in ("kc", "vc", "k", "v")]
    bad += [("ks", 255), ("vs", 260), ("ks", 0), ("vs", -256), ("batch", 0), ("batch", capi.MAX_BATCH + 1), ("rows", -1), ("max_pages", 0),
            ("num_pages", 0)]
    refused(fn, good, bad)
    refused(fn, good, [("ws", None), ("ws", p + 8)], 4)
    with pytest.raises(capi.MFAError):
        getattr(capi, "mfa_kv_read" + kv)(*dict(good, rows=-1, stream=0).values())


def test_append_slots_fp4_refusals(lib, mem):
    p = mem[1]
    good = dict(k=p, v=p + 512, ks=256, vs=256, slots=p + 1024, rows=1, kc=p + 2048, vc=p + 2560, k_scale=p + 4096, v_scale=p + 4352,
                pages=1, ws=p + 4608, stream=None)
    bad = [(k, None) for k in ("k", "v", "slots", "kc", "vc", "k_scale", "v_scale")]
    bad += [(k, good[k] + 8) for k in ("k", "v", "kc", "vc")] + [(k, good[k] + 2) for k in ("slots", "k_scale", "v_scale")]
    bad += [("ks", 257), ("vs", 4), ("ks", -256), ("rows", -1), ("pages", 0)]
    refused(lib.mfa_kv_append_slots_fp4, good, bad)
    refused(lib.mfa_kv_append_slots_fp4, good, [("ws", None), ("ws", p + 64)], 4)

"""Host checks of the page-table, slot-append and shared-prefix calls: every refusal comes before any device work, so no GPU
is needed."""
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
    buf = (ctypes.c_uint8 * 8192)()
    return buf, (ctypes.addressof(buf) + 255) & ~255


def test_reserve_refusals(lib, mem):
    p = mem[1]
    good = dict(n_new=p, lens=p + 256, table=p + 512, free=p + 768, n=p + 1024, batch=4, max_pages=2, pages=8, most=16,
                starts=p + 1280, slots=p + 1536, lens_out=p + 1792, n_out=p + 2048, ws=p + 2304, stream=None)
    bad = [(k, None) for k in ("n_new", "lens", "table", "free", "n", "starts", "slots", "lens_out", "n_out")]
    bad += [(k, good[k] + 2) for k in ("n_new", "lens", "table", "free", "n", "starts", "lens_out", "n_out")]
    bad += [("slots", good["slots"] + 4), ("batch", 0), ("batch", capi.MAX_BATCH + 1), ("max_pages", 0), ("pages", 0),
            ("most", -1), ("max_pages", 2 ** 26), ("lens_out", good["lens"] + 4), ("lens_out", good["lens"] - 12)]
    for key, value in bad:
        assert lib.mfa_reserve_pages(*dict(good, **{key: value}).values()) == 1, (key, value)
    for ws in (None, p + 8):
        assert lib.mfa_reserve_pages(*dict(good, ws=ws).values()) == 4
    with pytest.raises(capi.MFAError):
        capi.mfa_reserve_pages(*dict(good, batch=0, stream=0).values())


def test_release_refusals(lib, mem):
    p = mem[1]
    good = dict(done=p, keep=p + 256, lens=p + 512, table=p + 768, free=p + 1024, n=p + 1280, batch=4, max_pages=2, pages=8,
                lens_out=p + 1536, n_out=p + 1792, ws=p + 2048, stream=None)
    bad = [(k, None) for k in ("done", "lens", "table", "free", "n", "lens_out", "n_out")]
    bad += [(k, good[k] + 1) for k in ("done", "keep", "lens", "table", "free", "n", "lens_out", "n_out")]
    bad += [("batch", 0), ("batch", capi.MAX_BATCH + 1), ("max_pages", 0), ("pages", -1), ("lens_out", good["lens"] + 8)]
    for key, value in bad:
        assert lib.mfa_release_pages(*dict(good, **{key: value}).values()) == 1, (key, value)
    assert lib.mfa_release_pages(*dict(good, ws=None).values()) == 4


@pytest.mark.parametrize("fp8", [False, True])
def test_append_slots_refusals(lib, mem, fp8):
    p = mem[1]
    good = dict(k=p, v=p + 512, ks=256, vs=256, slots=p + 1024, rows=1, kc=p + 2048, vc=p + 2560)
    good.update(dict(k_scale=p + 4096, v_scale=p + 4352) if fp8 else {}, pages=1, ws=p + 4608, stream=None)
    fn = lib.mfa_kv_append_slots_fp8 if fp8 else lib.mfa_kv_append_slots
    bad = [(k, None) for k in good if k in ("k", "v", "slots", "kc", "vc", "k_scale", "v_scale")]
    bad += [(k, good[k] + 8) for k in ("k", "v", "kc", "vc")] + [("slots", good["slots"] + 4)]
    bad += [(k, good[k] + 2) for k in good if k in ("k_scale", "v_scale")]
    bad += [("ks", 257), ("vs", 4), ("ks", -256), ("rows", -1), ("pages", 0)]
    for key, value in bad:
        assert fn(*dict(good, **{key: value}).values()) == 1, (key, value)
    for ws in (None, p + 64):
        assert fn(*dict(good, ws=ws).values()) == 4


@pytest.mark.parametrize("fp8", [False, True])
def test_prefix_attention_refusals(lib, mem, fp8):
    p = mem[1]
    good = dict(q=p, kc=p + 512, vc=p + 1024)
    good.update(dict(k_scale=p + 4096, v_scale=p + 4352) if fp8 else {})
    good.update(table=p + 1536, lens=p + 2048, starts=p + 2304, pages=p + 2560, n_groups=2, out=p + 3584, lse=p + 3840,
                scale=1 / 16, batch=4, max_pages=2, num_pages=8, prefix_hint=64, suffix_hint=64, ws=p + 5120, n=1 << 30,
                stream=None)
    fn = lib.mfa_decode_attention_prefix_fp8 if fp8 else lib.mfa_decode_attention_prefix
    pointers = [k for k in good if k in ("q", "kc", "vc", "k_scale", "v_scale", "table", "lens", "starts", "pages", "out", "lse")]
    bad = [(k, None) for k in pointers] + [(k, good[k] + 2) for k in pointers]
    bad += [(k, good[k] + 8) for k in pointers if k in ("q", "kc", "vc", "k_scale", "v_scale", "out")]
    bad += [("n_groups", 0), ("n_groups", 5), ("n_groups", -1), ("batch", 0), ("batch", capi.MAX_BATCH + 1), ("batch", 1),
            ("max_pages", 0), ("max_pages", 2 ** 30), ("max_pages", 2 ** 26), ("num_pages", 0), ("prefix_hint", -1),
            ("suffix_hint", -1)]
    for key, value in bad:
        assert fn(*dict(good, **{key: value}).values()) == 1, (key, value)
    for ws in (None, p + 8):
        assert fn(*dict(good, ws=ws).values()) == 4
    call = capi.mfa_decode_attention_prefix_fp8 if fp8 else capi.mfa_decode_attention_prefix
    with pytest.raises(capi.MFAError):
        call(*dict(good, n_groups=0, stream=0).values())


def test_prefix_workspace_refusals(lib):
    for args in ((0, 1, 0, 0), (capi.MAX_BATCH + 1, 1, 0, 0), (4, 0, 0, 0), (4, 5, 0, 0), (4, 1, -1, 0), (4, 1, 0, -1)):
        assert lib.mfa_decode_prefix_workspace_bytes(*args) == 0
        with pytest.raises(capi.MFAError):
            capi.mfa_decode_prefix_workspace_bytes(*args)

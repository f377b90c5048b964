"""Host-side refusals of the 4-bit cache's entry points: nothing is launched, so no GPU is needed."""
import ctypes
import math
import os

import pytest
import torch

import attention_guided_kv_gb300 as K

INV, UNS = K.KVSEL_ERR_INVALID_ARG, K.KVSEL_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from attention_guided_kv_gb300 import _build
        _build.build()
    return K.lib()


def _kv(**kw):
    d = dict(k_codes=16, v_codes=16, k_scales=16, v_scales=16, num_pages=10, num_kv_heads=8, num_q_heads=64, head_dim=128,
             page_size=16)
    d.update(kw)
    return K.PagedKV4(**d)


BAD_KV = [(dict(k_codes=None), INV), (dict(v_scales=None), INV), (dict(k_scales=8), INV), (dict(v_codes=24), INV),
          (dict(num_pages=0), INV), (dict(num_kv_heads=0), INV), (dict(head_dim=64), UNS), (dict(page_size=8), UNS),
          (dict(page_size=48), UNS), (dict(page_size=512), UNS), (dict(num_pages=1 << 24), UNS)]


def _append(lib, kv=None, **over):
    a = dict(bt=16, max_pages=4, seq=16, batch=2, off=16, total=3, k=16, v=16, pos=None, nxt=None, cum=None, max_len=0,
             ws=256, ws_bytes=1 << 20)
    a.update(over)
    return lib.kvsel_kv4_append(ctypes.byref(kv or _kv()), a["bt"], a["max_pages"], a["seq"], a["batch"], a["off"],
                                a["total"], a["k"], a["v"], a["pos"], a["nxt"], a["cum"], a["max_len"], a["ws"],
                                a["ws_bytes"], None)


def _read(lib, kv=None, **over):
    a = dict(bt=16, max_pages=4, seq=16, batch=2, off=16, total=3, start=None, k=16, v=16, ws=256, ws_bytes=256)
    a.update(over)
    return lib.kvsel_kv4_read(ctypes.byref(kv or _kv()), a["bt"], a["max_pages"], a["seq"], a["batch"], a["off"],
                              a["total"], a["start"], a["k"], a["v"], a["ws"], a["ws_bytes"], None)


def _decode(lib, kv=None, mod=None, **over):
    a = dict(bt=16, max_pages=4, seq=16, batch=2, q=16, kn=None, vn=None, pos=None, nxt=None, scale=0.1, out=16, odt=0,
             probs=None, cum=None, max_len=64, ws=256, ws_bytes=1 << 40)
    a.update(over)
    return lib.kvsel_kv4_decode_attn(ctypes.byref(kv or _kv()), a["bt"], a["max_pages"], a["seq"], a["batch"], a["q"],
                                     a["kn"], a["vn"], a["pos"], a["nxt"], a["scale"],
                                     ctypes.byref(mod) if mod is not None else None, a["out"], a["odt"], a["probs"],
                                     a["cum"], a["max_len"], a["ws"], a["ws_bytes"], None)


def _evict(lib, kv=None, **over):
    a = dict(bt=16, max_pages=4, seq=16, batch=2, cum=16, pos=None, max_len=64, budget=10, sink=4, window=4, compact=1,
             keep=None, freed=None, ws=256, ws_bytes=1 << 20)
    a.update(over)
    return lib.kvsel_kv4_evict(ctypes.byref(kv or _kv()), a["bt"], a["max_pages"], a["seq"], a["batch"], a["cum"],
                               a["pos"], a["max_len"], a["budget"], a["sink"], a["window"], a["compact"], a["keep"],
                               a["freed"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [_append, _read, _decode, _evict])
@pytest.mark.parametrize("bad,want", BAD_KV)
def test_descriptor(lib, call, bad, want):
    assert call(lib, _kv(**bad)) == want
    assert lib.kvsel_last_error_string()


def test_append(lib):
    for bad in (dict(bt=None), dict(seq=None), dict(off=None), dict(batch=0), dict(max_pages=0), dict(total=-1),
                dict(k=None), dict(v=None), dict(k=8), dict(v=24), dict(pos=16, max_len=64), dict(cum=16), dict(ws=None),
                dict(ws=128), dict(ws_bytes=256)):
        assert _append(lib, **bad) == INV, bad
    assert K.kvsel_kv4_append_workspace(_kv(), 2) == 512
    assert K.kvsel_kv4_append_workspace(_kv(), 0) == 0
    assert _append(lib, total=0, k=None, v=None) == K.KVSEL_OK      # nothing to do, nothing launched


def test_read(lib):
    for bad in (dict(bt=None), dict(seq=None), dict(off=None), dict(batch=0), dict(max_pages=0), dict(total=-1),
                dict(k=None), dict(v=8), dict(ws=None), dict(ws=16), dict(ws_bytes=255)):
        assert _read(lib, **bad) == INV, bad
    assert _read(lib, total=0, k=None, v=None) == K.KVSEL_OK


def test_decode(lib):
    for bad in (dict(bt=None), dict(seq=None), dict(q=None), dict(out=None), dict(batch=0), dict(batch=1025),
                dict(max_pages=0), dict(max_len=0), dict(kn=16), dict(vn=16), dict(kn=16, vn=16, pos=16), dict(odt=2),
                dict(q=8), dict(kn=8, vn=16), dict(ws=None), dict(ws=64)):
        assert _decode(lib, **bad) == INV, bad
    assert _decode(lib, _kv(num_q_heads=12)) == INV                # not a multiple of 8
    assert _decode(lib, _kv(num_q_heads=0)) == INV
    assert _decode(lib, _kv(num_q_heads=136)) == UNS               # 17 q heads per kv head
    assert _decode(lib, batch=1024, max_len=1 << 26) == UNS        # tiles beyond 32 bits
    for mod in (K.ScoreMod(softcap=-1.0), K.ScoreMod(softcap=math.nan), K.ScoreMod(softcap=math.inf),
                K.ScoreMod(window=-1), K.ScoreMod(window=4, n_sink=-1)):
        assert _decode(lib, mod=mod) == INV
    need = K.kvsel_kv4_decode_attn_workspace(_kv(), 2, 64, False, True)
    assert _decode(lib, cum=16, ws_bytes=need - 1) == INV
    assert b"workspace too small" in lib.kvsel_last_error_string()
    # scores are kept in the workspace only where the probabilities are not
    assert need - K.kvsel_kv4_decode_attn_workspace(_kv(), 2, 64, True, True) == 2 * 64 * 64 * 4
    assert K.kvsel_kv4_decode_attn_workspace(_kv(num_q_heads=136), 2, 64, True, True) == 0
    assert K.kvsel_kv4_decode_attn_workspace(_kv(), 1025, 64, True, True) == 0


def test_evict(lib):
    for bad in (dict(bt=None), dict(seq=None), dict(cum=None), dict(batch=0), dict(batch=65536), dict(max_pages=0),
                dict(max_len=0), dict(budget=0), dict(budget=7), dict(sink=-1), dict(window=-1), dict(ws=None),
                dict(ws=8), dict(ws_bytes=64)):
        assert _evict(lib, **bad) == INV, bad
    assert _evict(lib, batch=65535, budget=(1 << 31) - 1, sink=0, window=0, max_len=(1 << 31) - 1) == UNS
    need = K.kvsel_kv4_evict_workspace(_kv(), 2, 10)
    assert need >= 256 + 2 * 8 * 10 * 4
    assert _evict(lib, ws_bytes=need - 1) == INV
    assert K.kvsel_kv4_evict_workspace(_kv(), 0, 10) == 0


def test_binding_refuses_what_is_not_on_a_gpu():
    codes, scales = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 16, 4, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        K.paged_kv4(codes, codes, scales, scales, 4)


def test_prefill(lib):
    def st(kv=None, **over):
        a = dict(bt=16, max_pages=4, seq=16, batch=2, q=16, off=16, total=9, scale=0.1, cap=0.0, slopes=None, window=0,
                 prefix=None, doc=None, out=16, odt=0, lse=None, ws=256, ws_bytes=1 << 40)
        a.update(over)
        d = dict(k_pool=16, v_pool=16, num_pages=10, num_kv_heads=8, num_q_heads=64, head_dim=128, page_size=16)
        d.update(kv or {})
        return lib.kvsel_prefill_attn(ctypes.byref(K.PagedKV(**d)), a["bt"], a["max_pages"], a["seq"], a["batch"], a["q"],
                                      a["off"], a["total"], a["scale"], a["cap"], a["slopes"], a["window"], a["prefix"],
                                      a["doc"], a["out"], a["odt"], a["lse"], a["ws"], a["ws_bytes"], None)
    for bad, want in ((dict(k_pool=None), INV), (dict(v_pool=8), INV), (dict(num_q_heads=12), INV), (dict(num_pages=0), INV),
                      (dict(head_dim=64), UNS), (dict(page_size=48), UNS), (dict(num_q_heads=136), UNS),
                      (dict(num_pages=1 << 25), UNS)):
        assert st(bad) == want, bad
    for bad in (dict(bt=None), dict(seq=None), dict(off=None), dict(q=None), dict(out=None), dict(q=8), dict(out=24),
                dict(batch=0), dict(max_pages=0), dict(total=-1), dict(odt=3), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.nan), dict(window=-1),
                dict(cap=1e-38, scale=1.0), dict(ws=None), dict(ws=64)):
        assert st(**bad) == INV, bad
    assert st(total=1 << 26) == UNS                                # 2^26 x 64 rows
    kv = K.PagedKV(k_pool=16, v_pool=16, num_pages=10, num_kv_heads=8, num_q_heads=64, head_dim=128, page_size=16)
    assert st(ws_bytes=K.kvsel_prefill_attn_workspace(kv, 2, 9) - 1) == INV
    assert K.kvsel_prefill_attn_workspace(kv, 0, 9) == 0
    assert st(total=0, q=None, out=None) == K.KVSEL_OK


def test_evict_workspace_of_many_rows_does_not_wrap():
    """Six words a (sequence, kv head) at a budget of one, also where their number passes 2^31 (whole 256-byte blocks here)."""
    def size(batch):
        return K.kvsel_kv4_evict_workspace(_kv(), batch, 1)
    for batch in (72, 1 << 20, (1 << 31) - 8):
        assert size(batch) - size(64) == 24 * 8 * (batch - 64), batch

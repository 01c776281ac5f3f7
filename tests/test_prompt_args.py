"""Refusals of the prompt-side calls that need no GPU: every bad argument is
turned away on the host before any CUDA call."""
import pytest
import torch

from paged_kv_cache_228_gb300 import pa


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_cache_228_gb300 import build
    build.build()


BAD, UNSUP = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
P = 0x10000  # an aligned address that is never read


def _attention(fn, **kw):
    a = dict(q=P, k=P, v=P, ks=None, vs=None, kv=pa.PA_KV_BF16, tab=P, width=4, start=P, lens=P,
             B=2, T=5, hq=4, hkv=2, d=64, bs=16, nb=8, scale=0.125, out=P, ws=None, wsb=0,
             splits=0)
    a.update(kw)
    return getattr(pa.lib(), fn)(*a.values(), None)


@pytest.mark.parametrize("fn", ["pa_prefill", "pa_cross_attention"])
def test_attention_refusals(fn):
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(tab=None), dict(lens=None),
                dict(out=None), dict(B=-1), dict(T=-1), dict(hq=0), dict(hkv=0), dict(hq=3),
                dict(nb=0), dict(width=-1), dict(splits=-1), dict(splits=70000),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-float("inf")),
                dict(scale=3e38), dict(kv=pa.PA_KV_NVFP4), dict(kv=9), dict(start=None),
                dict(q=P + 8), dict(k=P + 2), dict(out=P + 4), dict(lens=P + 2),
                dict(start=P + 1), dict(tab=P + 3), dict(kv=pa.PA_KV_FP8_E4M3),
                dict(kv=pa.PA_KV_FP8_E4M3, ks=P)):
        assert _attention(fn, **bad) == BAD, bad
    for unsup in (dict(d=96), dict(d=256), dict(bs=4), dict(bs=24), dict(bs=512),
                  dict(hq=65 * 2), dict(width=1 << 28), dict(nb=(1 << 31) - 1),
                  dict(T=(1 << 31) - 8)):
        assert _attention(fn, **unsup) == UNSUP, unsup
    # nothing to do
    assert _attention(fn, B=0, T=0, q=None, out=None) == pa.PA_OK
    assert _attention(fn, T=0, q=None) == pa.PA_OK


def test_workspace_size_refusals():
    import ctypes
    n = ctypes.c_size_t(0)
    f = pa.lib().pa_attention_workspace_size
    assert f(1, 4, 2, 64, 0, None) == BAD
    assert f(-1, 4, 2, 64, 0, ctypes.byref(n)) == BAD
    assert f(1, 4, 3, 64, 0, ctypes.byref(n)) == BAD
    assert f(1, 4, 2, 64, -1, ctypes.byref(n)) == BAD
    assert f(1, 4, 2, 80, 0, ctypes.byref(n)) == UNSUP
    assert f(1, 130, 2, 64, 0, ctypes.byref(n)) == UNSUP


def _append(**kw):
    a = dict(lens=P, new=P, tab=P, width=4, free=P, nf=P, B=2, T=5, bs=16, nb=8, slots=P, start=P,
             out=P, nfo=P, done=P)
    a.update(kw)
    return pa.lib().pa_append_slots_device(*a.values(), None)


def _trim(**kw):
    a = dict(lens=P, new=P, tab=P, width=4, free=P, nf=P, B=2, bs=16, nb=8, out=P, nfo=P)
    a.update(kw)
    return pa.lib().pa_trim_slots_device(*a.values(), None)


def test_slot_refusals():
    for call in (_append, _trim):
        for bad in (dict(lens=None), dict(new=None), dict(tab=None), dict(free=None),
                    dict(nf=None), dict(out=None), dict(nfo=None), dict(B=-1), dict(bs=0),
                    dict(nb=0), dict(width=-1), dict(lens=P + 2), dict(nf=P + 1)):
            assert call(**bad) == BAD, bad
        assert call(width=1 << 28) == UNSUP
    for bad in (dict(T=-1), dict(slots=None), dict(start=None), dict(done=None),
                dict(slots=P + 4)):
        assert _append(**bad) == BAD, bad


def test_binding_refuses_what_the_library_cannot_see():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    ok = dict(q=q, k_cache=c, v_cache=c, block_tables=i(2, 4), q_start=i(3), seq_lens=i(2),
              scale=1.0, out=q.clone())
    for change, exc in ((dict(q=q.half()), TypeError), (dict(out=q[:4].clone()), ValueError),
                        (dict(q=q.transpose(0, 1)), ValueError), (dict(q_start=i(2)), ValueError),
                        (dict(block_tables=i(3, 4)), ValueError),
                        (dict(v_cache=c[:7].clone()), ValueError),
                        (dict(k_cache=c[..., :32].contiguous(), v_cache=c[..., :32].contiguous()),
                         ValueError),
                        (dict(k_scale=torch.ones(8, 2)), ValueError),
                        (dict(k_cache=c.to(torch.uint8), v_cache=c.to(torch.uint8)), ValueError),
                        (dict(seq_lens=i(2).long()), TypeError), ({}, ValueError)):
        for fn in (pa.pa_prefill, pa.pa_cross_attention):
            with pytest.raises(exc):   # the last: tensors on the CPU
                fn(**{**ok, **change})
    ok = dict(lens=i(2), n_new=i(2), block_tables=i(2, 4), free_ids=i(8), num_free=i(1),
              block_size=16, slot_mapping=torch.zeros(4, dtype=torch.int64), q_start=i(3),
              seq_lens=i(2), num_free_out=i(1), num_done=i(1))
    for change, exc in ((dict(n_new=i(3)), ValueError), (dict(q_start=i(2)), ValueError),
                        (dict(slot_mapping=i(4)), TypeError), (dict(num_free=i(2)), ValueError),
                        (dict(block_tables=i(3, 4)), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            pa.pa_append_slots_device(**{**ok, **change})
    ok = {k: ok[k] for k in ("lens", "block_tables", "free_ids", "num_free", "block_size",
                             "seq_lens", "num_free_out")}
    for change, exc in ((dict(new_lens=i(3)), ValueError), (dict(new_lens=i(2).long()), TypeError),
                        (dict(new_lens=i(2)), ValueError)):
        with pytest.raises(exc):
            pa.pa_trim_slots_device(**{**ok, **change})

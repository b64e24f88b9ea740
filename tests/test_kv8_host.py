"""Host checks of the paged int8 key/value cache: every refusal comes before any CUDA call."""
import ctypes

import pytest
import torch

import post_weight_quantization_rowwise_b200 as m

V = ctypes.c_void_p


def _cache(**kw):
    f = dict(k_codes=16, v_codes=16, k_scales=16, v_scales=16, n_pages=10, n_kv_heads=2, page_size=16, head_dim=64)
    f.update(kw)
    return m._Kv8CacheStruct(**f)


def _seqs(**kw):
    f = dict(block_tables=16, table_stride=4, table_width=4, seq_lens=16, cu_tokens=16, n_seqs=3)
    f.update(kw)
    return m._Kv8SeqsStruct(**f)


def _append(cache=None, seqs=None, **at):
    args = [ctypes.byref(cache or _cache()), ctypes.byref(seqs or _seqs()), 0, V(16), 128, 64, V(16), 128, 64, 5, None, None]
    for i, v in at.items():
        args[int(i[1:])] = v
    return m._lib.iqq_kv8_append(*args)


def _gather(cache=None, seqs=None, **at):
    args = [ctypes.byref(cache or _cache()), ctypes.byref(seqs or _seqs()), 0, V(16), V(16), 5, None, None]
    for i, v in at.items():
        args[int(i[1:])] = v
    return m._lib.iqq_kv8_gather(*args)


def _attend(cache=None, seqs=None, **at):
    args = [ctypes.byref(cache or _cache()), ctypes.byref(seqs or _seqs()), 1, V(16), 256, 64, 4, 5, V(16), None, 0.125,
            V(1 << 20), 1 << 40, None, None]
    for i, v in at.items():
        args[int(i[1:])] = v
    return m._lib.iqq_kv8_attention(*args)


@pytest.mark.parametrize("call", [_append, _gather, _attend])
def test_shared_refusals(call):
    assert call(_0=None) == 1 and call(_1=None) == 1
    for kw in (dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(head_dim=32), dict(head_dim=96),
               dict(n_kv_heads=0), dict(n_pages=-1), dict(n_pages=1 << 31), dict(n_kv_heads=1 << 17)):
        assert call(cache=_cache(**kw)) == 2, kw
    for kw in (dict(n_seqs=-1), dict(n_seqs=1 << 25), dict(table_width=-1), dict(table_stride=3), dict(table_width=1 << 31)):
        assert call(seqs=_seqs(**kw)) == 2, kw
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert call(cache=_cache(**{name: None})) == 1
        assert call(cache=_cache(**{name: 18})) == 3
    for name in ("block_tables", "seq_lens", "cu_tokens"):
        assert call(seqs=_seqs(**{name: None})) == 1
        assert call(seqs=_seqs(**{name: 18})) == 3
    assert call(seqs=_seqs(n_seqs=0)) == 0


def test_append_refusals():
    assert _append(_2=3) == 5 and _append(_9=-1) == 2 and _append(_9=0) == 0
    assert _append(_3=None) == 1 and _append(_6=None) == 1
    assert _append(_3=V(8)) == 3 and _append(_4=130) == 3 and _append(_5=66) == 3 and _append(_10=V(2)) == 3
    assert _append(_2=1, _7=132) == 3 and _append(_4=-128) == 2


def test_gather_refusals():
    assert _gather(_2=3) == 5 and _gather(_5=-1) == 2 and _gather(_5=0) == 0
    assert _gather(_3=None) == 1 and _gather(_4=V(8)) == 3 and _gather(_6=V(2)) == 3


def test_attention_refusals():
    assert _attend(_2=0) == 5 and _attend(_2=3) == 5
    assert _attend(_10=float("nan")) == 5 and _attend(_10=float("inf")) == 5
    assert _attend(_6=3) == 2 and _attend(_6=0) == 2 and _attend(_7=-1) == 2 and _attend(_7=0) == 0
    assert _attend(_3=None) == 1 and _attend(_8=None) == 1
    assert _attend(_3=V(8)) == 3 and _attend(_8=V(8)) == 3 and _attend(_4=260) == 3 and _attend(_5=68) == 3
    assert _attend(_9=V(2)) == 3 and _attend(_11=V(8)) == 3 and _attend(_13=V(2)) == 3
    for kw in (dict(n_pages=1 << 30, n_kv_heads=8), dict(n_pages=1 << 24, n_kv_heads=1, page_size=128, head_dim=128)):
        assert _attend(cache=_cache(**kw), _6=8) == 2, kw  # 2^31 rows of 128 bytes and more
    W = m._lib.iqq_kv8_attention_workspace_bytes
    long = _seqs(n_seqs=1, table_width=1 << 14, table_stride=1 << 14)
    need = W(ctypes.byref(_cache()), ctypes.byref(long), 4, 1)
    if need:
        assert _attend(seqs=long, _7=1, _12=need - 1) == 2 and _attend(seqs=long, _7=1, _11=None) == 1


def test_binding_refusals():
    z = torch.zeros
    with pytest.raises(ValueError):
        m.Kv8Cache(z(2, 1, 16, 64, dtype=torch.int8), z(2, 1, 16, 64, dtype=torch.int8), z(2, 1), z(2, 1))
    for n in ("Kv8Cache", "kv8_cache", "kv8_gather", "kv8_attention", "iqq_kv8_append", "iqq_kv8_gather", "iqq_kv8_attention"):
        assert n in m.__all__


@pytest.mark.skipif(torch.cuda.is_available(), reason="what calls say without a device")
def test_without_a_device_every_call_says_why():
    """The CUDA error of the call itself (no device, or no driver for it), each time; for tokens, prompts
    and the cache."""
    W = m._lib.iqq_last_cuda_error
    for _ in range(2):
        for call in (_append, _gather, _attend, lambda: _attend(_7=5000)):
            assert call() == 4 and W() in (35, 100), W()


def test_workspace_of_short_tables():
    """One sequence of few tiles: a CTA takes a tile up to 704 keys, beyond them the keys are shared out;
    more tiles or sequences up to 1024 keys.  A workspace that is too small, or none, is refused."""
    W = m._lib.iqq_kv8_attention_workspace_bytes

    def need(n_seqs, width, kv, heads):
        seqs = _seqs(n_seqs=n_seqs, table_width=width, table_stride=width)
        return W(ctypes.byref(_cache(n_kv_heads=kv, page_size=64, head_dim=128)), ctypes.byref(seqs), heads, n_seqs)

    for kv, heads in ((1, 8), (8, 32), (32, 32)):
        assert need(1, 11, kv, heads) == 0 and need(1, 12, kv, heads) > 0 and need(1, 16, kv, heads) > 0
    assert need(1, 16, 64, 64) == 0 and need(1, 17, 64, 64) > 0
    assert need(8, 16, 8, 32) == 0 and need(8, 17, 8, 32) > 0
    long = _seqs(n_seqs=1, table_width=1 << 14, table_stride=1 << 14)
    size = W(ctypes.byref(_cache()), ctypes.byref(long), 4, 1)
    assert size > 0
    assert _attend(seqs=long, _7=1, _12=size - 1) == 2 and _attend(seqs=long, _7=1, _11=None) == 1

"""The 8-bit arm and the page operators on the host (no GPU): layout sizes, refusals, the oracle against itself."""

import ctypes

import numpy as np
import pytest

from oracle import int8 as O8


@pytest.fixture(scope="module")
def L():
    from kv_cache_vector_head_gb300 import build

    build.build()
    from kv_cache_vector_head_gb300 import _lib

    return _lib


def params(L, d=128, hkv=2, g=4, window=32, **over):
    p = L.LayerParams()
    p.d, p.n_kv_heads, p.n_q_heads, p.page_size, p.window = d, hkv, hkv * g, 16, window
    p.key_bits = p.value_bits = 8
    p.key_qjl, p.kind, p.int8 = L.KEY_MSE, L.TQ_FWHT, 1
    for k, v in over.items():
        setattr(p, k, v)
    return p


def fake_cache(L, batch=2, max_pages=8):
    """A descriptor whose pointers are aligned but never read: every call below is refused before a launch."""
    c = L.Cache()
    c.page_pool = c.block_table = c.seq_len = c.n_compressed = c.win_k = c.win_v = 4096
    c.n_pages, c.max_pages_per_seq, c.batch = 64, max_pages, batch
    return c


def other(c, L, **over):
    o = L.Cache()
    for name, _ in L.Cache._fields_:
        setattr(o, name, getattr(c, name))
    for k, v in over.items():
        setattr(o, k, v)
    return o


@pytest.mark.parametrize("d", [128, 256])
def test_subblock_holds_bounds_scales_and_codes(L, d):
    assert L.subblock_bytes(params(L, d=d)) == 2 * d + 32 + 2 * 16 * d
    assert L.subblock_bytes(params(L, d=d, head_dim=d - 40)) == 2 * d + 32 + 2 * 16 * d
    x = np.random.default_rng(0).standard_normal((16, d))
    assert O8.pack_page(x, x).size == L.subblock_bytes(params(L, d=d))


@pytest.mark.parametrize("over,status", [
    (dict(key_bits=4), 1), (dict(value_bits=2), 1), (dict(key_qjl=1), 1), (dict(key_split=1), 1), (dict(key_norm_u8=1), 1),
    (dict(qjl_structured=1), 1), (dict(kivi=1), 1), (dict(window=0), 1), (dict(int8=2), 1), (dict(d=64), 2),
    (dict(n_q_heads=18), 2), (dict(head_dim=100), 1), (dict(head_dim=64), 1), (dict(page_size=32), 2),
])
def test_layers_that_do_not_combine_are_refused(L, over, status):
    p = params(L, **over)
    assert L.lib().tq_subblock_bytes(ctypes.byref(p)) == 0
    c = fake_cache(L)
    assert L.lib().tq_prefill_cache(ctypes.byref(p), ctypes.byref(c), 4096, 4096, 1, 64, None) == status


def test_eight_bits_need_the_arm(L):
    p = params(L, int8=0)
    assert L.lib().tq_subblock_bytes(ctypes.byref(p)) == 0


def call(L, name, *args):
    return getattr(L.lib(), name)(*args)


def test_refusals_of_the_calls(L):
    p, c = params(L), fake_cache(L)
    P, C = ctypes.byref(p), ctypes.byref(c)
    q4 = params(L, int8=0, key_bits=4, value_bits=4, k_rot=4096, v_rot=4096)
    Q4 = ctypes.byref(q4)
    big = 1 << 40
    bad, unsup, cap = L.TQ_ERR_INVALID_ARG, L.TQ_ERR_UNSUPPORTED, L.TQ_ERR_CAPACITY
    # flat quantize does not apply
    assert call(L, "tq_quantize_keys", P, 4096, 1, 16, 4096, None, 4096, None, None) == unsup
    assert call(L, "tq_quantize_values", P, 4096, 1, 16, 4096, 4096, None) == unsup
    # direct appends write whole pages; a decode step has one token a sequence; rows are 16-byte aligned
    assert call(L, "tq_append_page", P, C, 4096, 4096, 1, 17, 4096, None) == bad
    assert call(L, "tq_append_page", P, C, 4096, 4096, 1, 3, None, None) == bad
    assert call(L, "tq_append_page", P, C, 4100, 4096, 1, 16, 4096, None) == bad
    assert call(L, "tq_prefill_cache", P, C, 4096, 4096, 1, 16 * 8 + 32 + 16, None) == cap
    assert call(L, "tq_prefill_cache", P, C, 4096, 4096, 7, 64, None) == bad
    # read
    assert call(L, "tq_read_cache", Q4, C, 4096, 4096, 1, 0, 16, None) == unsup
    assert call(L, "tq_read_cache", P, C, 4096, 4096, 1, -1, 16, None) == bad
    assert call(L, "tq_read_cache", P, C, 4096, 4096, 1, 2**31 - 64, 16, None) == bad
    assert call(L, "tq_read_cache", P, C, 4096, 4104, 1, 0, 16, None) == bad
    assert call(L, "tq_read_cache", P, C, None, 4096, 1, 0, 16, None) == bad
    assert call(L, "tq_read_cache", P, C, None, None, 1, 0, 0, None) == L.TQ_OK
    # decode
    assert call(L, "tq_decode_attention", P, C, 4096, 1, 0.1, 4096, None, None, 4096, 0, 8192, 0, None) == cap
    assert call(L, "tq_decode_attention", P, C, 4096, 1, float("nan"), 4096, None, None, 4096, big, 8192, 0, None) == bad
    # select
    assert L.lib().tq_select_workspace_size(Q4, 2, 1024) == 0
    assert L.lib().tq_select_workspace_size(P, 0, 1024) == 0
    assert L.lib().tq_select_workspace_size(P, 2, 1024) >= 2 * 2 * 64 * 4
    sel = lambda P=P, C=C, q=4096, n=8, s=1, r=1, pages=4096, ws=4096, nb=big, ctx=1024: call(  # noqa: E731
        L, "tq_select_pages", P, C, q, 1, n, s, r, pages, 4096, ws, nb, ctx, None)
    assert sel(P=Q4) == unsup
    for kw in (dict(n=0), dict(s=-1), dict(r=-1), dict(n=3, s=2, r=2), dict(q=None), dict(pages=None), dict(ws=4100), dict(ctx=-1)):
        assert sel(**kw) == bad, kw
    assert sel(nb=16) == cap
    # decode over a list
    assert L.lib().tq_decode_pages_workspace_size(Q4, 2, 8, 0) == 0
    assert L.lib().tq_decode_pages_workspace_size(P, 2, 0, 0) == 0
    dec = lambda P=P, pages=4096, counts=4096, n=8, nb=big, ctx=1024, sp=0, scale=0.1: call(  # noqa: E731
        L, "tq_decode_attention_pages", P, C, 4096, 1, scale, pages, counts, n, 4096, None, 4096, nb, ctx, sp, None)
    assert dec(P=Q4) == unsup
    for kw in (dict(pages=None), dict(counts=None), dict(n=0), dict(ctx=-1), dict(sp=-1), dict(scale=float("nan"))):
        assert dec(**kw) == bad, kw
    assert dec(nb=0, n=512, sp=4) == cap
    # track
    assert call(L, "tq_track_pages", P, C, None, 4096, 4096, 1024, None) == bad
    assert call(L, "tq_track_pages", P, C, 4096, 4096, 4096, -1, None) == bad
    assert call(L, "tq_track_pages", P, C, 4096, 4096, 4096, 0, None) == L.TQ_OK
    # evict
    assert L.lib().tq_evict_workspace_size(P, 0, 8) == 0
    assert L.lib().tq_evict_workspace_size(P, 2, 8) == 2 * 8 * 8
    ev = lambda a=c, b=c, P=P, m=4096, n=4, s=1, r=1, ws=4096, nb=big: call(  # noqa: E731
        L, "tq_evict_pages", P, ctypes.byref(a), ctypes.byref(b), m, 4096, n, s, r, None, ws, nb, None)
    for kw in (dict(m=None), dict(n=0), dict(n=2, s=2), dict(ws=4100), dict(b=other(c, L, batch=1)), dict(b=other(c, L, max_pages_per_seq=9)),
               dict(b=other(c, L, page_pool=8192)), dict(b=other(c, L, seq_len=8192)), dict(b=other(c, L, win_k=8192)),
               dict(b=other(c, L, block_table=8192, seq_len=8192, n_compressed=8192, win_v=8192))):
        assert ev(**kw) == bad, kw
    assert ev(nb=8) == cap
    assert ev(P=ctypes.byref(params(L, window=12785))) == unsup


def test_bounds_that_round_up_past_32_bits_are_refused(L):
    p, c = params(L), fake_cache(L)
    P, C = ctypes.byref(p), ctypes.byref(c)
    big, bad = 1 << 60, L.TQ_ERR_INVALID_ARG
    lib = L.lib()
    for ctx in (2**31 - 1, 2**31 - 1023):
        assert lib.tq_decode_workspace_size(P, 1, ctx, 1) == 0
        assert lib.tq_prefill_workspace_size(P, 1, 1, ctx) == 0
        assert lib.tq_select_workspace_size(P, 1, ctx) == 0
        assert call(L, "tq_decode_attention", P, C, 4096, 1, 0.1, 4096, None, None, 4096, big, ctx, 0, None) == bad
        assert call(L, "tq_decode_attention_static", P, C, 4096, 1, 0.1, 4096, None, None, ctx, 1, None) == bad
        assert call(L, "tq_prefill_attention", P, C, 1, 4096, 1, 0.1, 4096, None, 4096, big, ctx, None) == bad
        assert call(L, "tq_select_pages", P, C, 4096, 1, 8, 1, 1, 4096, 4096, 4096, big, ctx, None) == bad
        assert call(L, "tq_decode_attention_pages", P, C, 4096, 1, 0.1, 4096, 4096, 8, 4096, None, 4096, big, ctx, 0, None) == bad
        assert call(L, "tq_track_pages", P, C, 4096, 4096, 4096, ctx, None) == bad
    assert lib.tq_decode_workspace_size(P, 1, 2**31 - 1024, 1) > 0 and lib.tq_select_workspace_size(P, 1, 2**31 - 1024) > 0


def test_a_layer_is_made_without_a_gpu_only_parameters(L):
    import kv_cache_vector_head_gb300 as tq

    layer = tq.TQLayer(128, 2, 8, 8, 8, tq.TQ_FWHT, window=16, key_qjl=tq.KEY_MSE, int8=True, device="cpu")
    assert layer.sub_bytes == 34 * 128 + 32 and layer.k_rot is None and layer.k_cb is None
    bits = tq.bits_per_channel(layer)
    assert abs(bits["kv_bits_per_channel"] - (34 * 128 + 32) * 8 / (2 * 16 * 128)) < 1e-12
    with pytest.raises(tq.TQError):
        tq.TQLayer(128, 2, 8, 8, 8, tq.TQ_FWHT, window=16, key_qjl=tq.KEY_QJL, int8=True, device="cpu")
    with pytest.raises(tq.TQError):
        tq.TQLayer(128, 2, 8, 8, 8, tq.TQ_FWHT, window=0, key_qjl=tq.KEY_MSE, int8=True, device="cpu")


# ------------------------------------------------------------------ the oracle

def test_oracle_codes_round_to_the_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, 128)).astype(np.float32).astype(np.float64)
    c, s = O8.quantize_page(x)
    assert np.abs(c).max() == 127
    assert np.abs(c * np.float64(s) - x).max() <= np.float64(s) / 2 * (1 + 2**-23)
    # ties to even: the scale is 1 where the largest magnitude is 127
    t = np.zeros((16, 128))
    t[0, :6] = [127, 0.5, 1.5, 2.5, -0.5, -1.5]
    c, s = O8.quantize_page(t)
    assert s == 1 and c[0, :6].tolist() == [127, 0, 2, 2, 0, -2]
    t[1, :3] = [np.nan, np.inf, -np.inf]
    c, s = O8.quantize_page(t)
    assert s == 1 and c[1, :3].tolist() == [0, 127, -127]
    assert O8.quantize_page(np.zeros((16, 128)))[1] == 0
    assert O8.quantize_page(np.full((16, 128), 1e-39))[1] == 0


def test_oracle_page_score_bounds_every_token():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((4, 128)), rng.standard_normal((64, 128))
    qc, _ = O8.quantize_page(q)
    sc = O8.page_scores(q, k, 64)
    for i in range(4):
        c, s = O8.quantize_page(k[16 * i:16 * i + 16])
        assert sc[i] >= np.float32((qc @ c.T).max()) * s


def test_oracle_choice():
    assert O8.choose([1, 5, 5, 2, 5], 2, 0, 0) == [1, 2]
    assert O8.choose([1, 5, 5, 2, 5], 3, 1, 1) == [0, 1, 4]
    assert O8.choose([np.nan, -1.0, np.nan, 0.0], 3, 0, 0) == [0, 1, 3]
    assert O8.choose([1, 2], 5, 1, 1) == [0, 1]

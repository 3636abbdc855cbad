"""The 8-bit arm on the GPU against its definition in float64 (oracle/int8.py).

Codes, scales, channel bounds, chosen pages, block tables and counters are compared exactly.  Outputs are float sums;
their tolerances count the roundings:
* a logit l = scale sum_j q_j k_j: the query has two f16 limbs (2^-22 of a row's largest entry), products are exact,
  at most 16 + 4 float additions follow (2^-23 of the partial sums each, which sum |q_j k_j| bounds), three factors:
  |dl| <= scale * max over tokens of sum_j |q_j| |k_j| * 2^-18 with d max|q| for sum |q| in the limb's part;
* exp2 of a difference: 2^-22 relative, and |l - m| log2(e) 2^-23 of its argument, under 2^-17 for the |l| < 64 used here;
  weights as two f16 limbs 2^-22, float sums of up to 2^12 of them 2^-12 2^-11 at worst in a serial order and 2^-20
  for the trees used: together under 2^-16 of max |v|.
"""

import ctypes
import math

import numpy as np
import pytest

from oracle import int8 as O8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    from kv_cache_vector_head_gb300 import build

    build.build()
    import kv_cache_vector_head_gb300 as tq

    return tq


def layer(tq, d=128, hkv=2, g=4, window=32, head_dim=None):
    return tq.TQLayer(d, hkv, hkv * g, 8, 8, tq.TQ_FWHT, window=window, key_qjl=tq.KEY_MSE, int8=True, head_dim=head_dim)


def data(shape, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * (1 + 3 * torch.rand(shape[-1], generator=g) ** 6) * spread
    return x.to(DT[dtype]).cuda()


def f64(x):
    return x.detach().cpu().double().numpy()


def pad(x, d):
    return np.pad(x, [(0, 0)] * (x.ndim - 1) + [(0, d - x.shape[-1])])


class Mirror:
    """What the cache holds, head by head: inputs in float64, and the ring's float16 rounding at a flush."""

    def __init__(self, L, k, v):
        self.L, self.k, self.v = L, f64(k), f64(v)  # [b, T, Hkv, dh]
        self.flushed_from_ring = [0] * len(self.k)  # tokens from this position on passed through the float16 window

    def values(self, b, h, T, first_flush):
        """(k, v) float64 [T, dh] held at length T; pages of positions >= first_flush were quantized from float16."""
        nc = O8.n_compressed(T, self.L.window)
        out = []
        for x in (self.k, self.v):
            y = x[b, :T, h].copy()
            y[first_flush:] = y[first_flush:].astype(np.float16).astype(np.float64)
            out.append(O8.held(y, nc))
        return out

    def raw(self, b, h, T, first_flush):
        out = []
        for x in (self.k, self.v):
            y = x[b, :T, h].copy()
            y[first_flush:] = y[first_flush:].astype(np.float16).astype(np.float64)
            out.append(y)
        return out


def page_bytes(pc, b, pg, h):
    L = pc.layer
    pool = pc.pool.reshape(pc.n_pages, L.n_kv_heads, L.sub_bytes)
    return pool[int(pc.block_table[b, pg]), h].cpu().numpy()


def check_attention(q, out, lse, k, v, scale, what, live=None):
    """One head; q, out [d], k, v [n, d] float64."""
    o, z, l = O8.attend(q, k, v, scale)
    if len(k) == 0:
        assert (out == 0).all() and lse == -np.inf, what
        return
    prod = scale * (np.abs(k).sum(1) * np.abs(q).max()).max()
    dl = prod * 2.0**-18
    tol = (2 * dl + 2.0**-16) * np.abs(v).max()
    assert np.abs(out - o).max() <= tol, (what, np.abs(out - o).max(), tol)
    assert abs(lse - z) <= dl + 2.0**-18 * max(1, abs(z)), (what, lse, z)


def decode(tq, pc, q, T, n_splits=0, scores=False, scale=None):
    L = pc.layer
    scale = L.head_dim**-0.5 if scale is None else scale
    ws = torch.empty(tq.decode_workspace_size(L.params, pc.batch, T, n_splits), dtype=torch.uint8, device="cuda")
    out = torch.full((pc.batch, L.n_q_heads, L.head_dim), float("nan"), device="cuda")
    lse = torch.full((pc.batch, L.n_q_heads), float("nan"), device="cuda")
    sc = torch.full((pc.batch, L.n_q_heads, T), float("nan"), device="cuda") if scores else None
    tq.decode_attention(L.params, pc.cache, q, scale, out, lse, sc, ws, T, n_splits)
    return out, lse, sc


# ---------------------------------------------------------------------------------------------- pages

@pytest.mark.parametrize("d,head_dim,dtype,window,T,hkv", [
    (128, None, "bf16", 32, 100, 2), (128, None, "f32", 1, 17, 3), (128, 80, "f16", 16, 64, 1), (256, None, "f32", 5, 85, 2),
    (256, 200, "bf16", 7, 40, 2), (128, 120, "f32", 3, 51, 1), (128, None, "f16", 40, 33, 2), (256, None, "f16", 16, 48, 1),
])
def test_prefilled_pages_are_exact(tq, d, head_dim, dtype, window, T, hkv):
    L = layer(tq, d, hkv, 2, window, head_dim)
    k, v = data((2, T, hkv, L.head_dim), dtype, 1), data((2, T, hkv, L.head_dim), dtype, 2)
    pc = tq.PagedCache(L, 2, T)
    pc.prefill(k, v)
    nc = O8.n_compressed(T, window)
    assert pc.seq_len.tolist() == [T] * 2 and pc.n_compressed.tolist() == [nc] * 2
    kk, vv = pad(f64(k), d), pad(f64(v), d)
    for b in range(2):
        for h in range(hkv):
            for pg in range(nc // 16):
                want = O8.pack_page(kk[b, 16 * pg:16 * pg + 16, h], vv[b, 16 * pg:16 * pg + 16, h])
                assert np.array_equal(page_bytes(pc, b, pg, h), want), (b, h, pg)
            for ring, x in ((pc.win_k, kk), (pc.win_v, vv)):
                for p in range(nc, T):
                    got = ring[b, h, p % (window + 16)].cpu().numpy()
                    assert np.array_equal(got, x[b, p, h].astype(np.float16)), (b, h, p)
    assert tq.check_device_error() == 0


def test_steps_flush_the_window_into_the_same_pages(tq):
    L = layer(tq, 128, 3, 2, 19)
    T = 19 + 16 * 3 + 5
    k, v = data((2, T, 3, 128), "bf16", 3), data((2, T, 3, 128), "bf16", 4)
    pc = tq.PagedCache(L, 2, T)
    for t in range(T):
        pc.append(k[:, t].contiguous(), v[:, t].contiguous())
    nc = O8.n_compressed(T, 19)
    assert pc.seq_len.tolist() == [T] * 2 and pc.n_compressed.tolist() == [nc] * 2
    h16 = lambda x: f64(x.half())  # noqa: E731 (pages are quantized from the float16 window)
    for b in range(2):
        for h in range(3):
            for pg in range(nc // 16):
                want = O8.pack_page(h16(k)[b, 16 * pg:16 * pg + 16, h], h16(v)[b, 16 * pg:16 * pg + 16, h])
                assert np.array_equal(page_bytes(pc, b, pg, h), want), (b, h, pg)
    assert tq.check_device_error() == 0


def test_step_without_a_page_to_flush_into_keeps_the_window(tq):
    L = layer(tq, 128, 1, 1, 16)
    pc = tq.PagedCache(L, 2, 16)  # one page a sequence
    k = data((2, 64, 1, 128), "f16", 5)
    for t in range(47):
        pc.append(k[:, t].contiguous(), k[:, t].contiguous())
    assert pc.n_compressed.tolist() == [16, 16] and tq.check_device_error() == 0
    before = pc.win_k.clone()
    pc.append(k[:, 47].contiguous(), k[:, 47].contiguous())  # would need a second page
    assert tq.check_device_error() == 0x2
    assert pc.seq_len.tolist() == [47, 47] and pc.n_compressed.tolist() == [16, 16] and torch.equal(before, pc.win_k)
    pc.block_table[1, 0] = 99  # a page outside the pool, found at the flush that needs it
    pc.seq_len.fill_(31)
    pc.n_compressed.fill_(0)
    pc.append(k[:, 31].contiguous(), k[:, 31].contiguous())
    assert tq.check_device_error() == 0x1
    assert pc.seq_len.tolist() == [32, 31] and pc.n_compressed.tolist() == [16, 0]


def test_direct_slots(tq):
    L = layer(tq, 128, 2, 2, 8)
    pc = tq.PagedCache(L, 1, 16 * 6)
    k, v = data((80, 2, 128), "bf16", 6), data((80, 2, 128), "bf16", 7)
    pc.pool.fill_(255)
    slots = torch.cat([torch.arange(16) + 16 * 4, torch.full((16,), -1), torch.arange(16) + 16, torch.arange(16) + 16 * 3 + 1,
                       torch.arange(16) + 16 * 6]).cuda()
    tq.append_page(L.params, pc.cache, k, v, 80, slots)
    assert tq.check_device_error() == 0x4  # the fourth group is out of order, the fifth outside the pool
    pool = pc.pool.reshape(6, 2, -1).cpu().numpy()
    kk, vv = f64(k), f64(v)
    for h in range(2):
        assert np.array_equal(pool[4, h], O8.pack_page(kk[:16, h], vv[:16, h]))
        assert np.array_equal(pool[1, h], O8.pack_page(kk[32:48, h], vv[32:48, h]))
    for page in (0, 2, 3, 5):
        assert (pool[page] == 255).all()


def test_extreme_pages_are_exact(tq):
    """Zero pages, magnitudes from 1e-44 to 3e38, exact half steps, and what is not finite."""
    L = layer(tq, 128, 1, 1, 1)
    n = 16 * 9 + 1
    g = torch.Generator().manual_seed(8)
    x = torch.randn((1, n, 1, 128), generator=g)
    x[0, 16:32] = 0
    x[0, 32:48] *= 1e-38
    x[0, 48:64] = 1e-44
    x[0, 64:80] *= 3e37
    x[0, 80:96] = torch.randint(-127, 127, (16, 1, 128), generator=g) + 0.5  # scale 1: every entry but one a half step
    x[0, 80, 0, 0] = 127
    x[0, 96, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, 2.0])
    x[0, 112:128] = math.nan
    x[0, 128:144] = math.inf
    x = x.cuda()
    pc = tq.PagedCache(L, 1, n)
    pc.prefill(x, x)
    for pg in range(9):
        y = f64(x)[0, 16 * pg:16 * pg + 16, 0]
        assert np.array_equal(page_bytes(pc, 0, pg, 0), O8.pack_page(y, y)), pg


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,head_dim,window,T,first,n", [(128, None, 20, 90, 0, 90), (256, 136, 3, 70, 13, 40), (128, 72, 16, 50, 45, 30)])
def test_read_gives_what_pages_and_window_stand_for(tq, dtype, d, head_dim, window, T, first, n):
    L = layer(tq, d, 2, 2, window, head_dim)
    k, v = data((2, T, 2, L.head_dim), "bf16", 9), data((2, T, 2, L.head_dim), "bf16", 10)
    pc = tq.PagedCache(L, 2, T)
    pc.prefill(k, v)
    ko, vo = (torch.full((2, n, 2, L.head_dim), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    tq.read_cache(L.params, pc.cache, ko, vo, first, n)
    m = Mirror(L, k, v)
    for b in range(2):
        for h in range(2):
            for got, want in zip((ko, vo), m.values(b, h, T, T)):
                want = torch.from_numpy(want[first:first + n].astype(np.float32)).to(DT[dtype])  # code * scale: one float rounding, then dtype's
                assert torch.equal(got[b, :len(want), h].cpu(), want)
                assert (got[b, len(want):, h] == 7).all()  # rows behind the last token
    assert tq.check_device_error() == 0


# ---------------------------------------------------------------------------------------------- decode

DECODE = [
    (128, None, 2, 4, 32, "bf16", [200, 37]), (128, None, 1, 1, 1, "f32", [1, 17, 0]), (256, None, 2, 8, 16, "f16", [130, 16, 95]),
    (128, 80, 2, 3, 24, "bf16", [77]), (256, 168, 1, 5, 100, "f32", [150, 20]), (128, None, 4, 8, 128, "bf16", [1000, 3]),
    (128, None, 3, 2, 7, "f16", [333, 8, 7, 6]),
]


@pytest.mark.parametrize("d,head_dim,hkv,g,window,dtype,lens", DECODE)
@pytest.mark.parametrize("n_splits", [0, 1, 3])
def test_decode(tq, d, head_dim, hkv, g, window, dtype, lens, n_splits):
    L = layer(tq, d, hkv, g, window, head_dim)
    T = max(lens)
    k, v = data((len(lens), T, hkv, L.head_dim), dtype, 11), data((len(lens), T, hkv, L.head_dim), dtype, 12)
    pc = tq.PagedCache(L, len(lens), T, pool_pages=len(lens) * -(-T // 16))
    pc.block_table.copy_(torch.randperm(pc.n_pages, generator=torch.Generator().manual_seed(1)).reshape(len(lens), -1).int())
    pc.pool.fill_(0x7f)  # unwritten pages: scales of 3e38 and NaN-like garbage
    pc.prefill(k, v)
    # ragged: a shorter sequence holds the window its own length leaves
    m = Mirror(L, k, v)
    for b, n in enumerate(lens):
        one = tq.PagedCache(L, 1, T)
        one.share_pages(pc)
        one.block_table.copy_(pc.block_table[b:b + 1])
        if n:
            one.prefill(k[b:b + 1, :n], v[b:b + 1, :n])
        pc.seq_len[b], pc.n_compressed[b] = n, O8.n_compressed(n, window)
        if n:
            pc.win_k[b], pc.win_v[b] = one.win_k[0], one.win_v[0]
        ring = window + 16
        for slot in range(ring):  # rows of no token: NaN
            if not any(p % ring == slot for p in range(O8.n_compressed(n, window), n)):
                pc.win_k[b, :, slot] = math.nan
                pc.win_v[b, :, slot] = math.nan
    q = data((len(lens), hkv * g, L.head_dim), dtype, 13)
    out, lse, sc = decode(tq, pc, q, T, n_splits, scores=True)
    assert tq.check_device_error() == 0
    scale = L.head_dim**-0.5
    for b, n in enumerate(lens):
        for h in range(hkv * g):
            kk, vv = m.values(b, h // g, n, n)
            qq = f64(q)[b, h]
            check_attention(qq, f64(out)[b, h], float(lse[b, h]), kk, vv, scale, (b, h))
            got = f64(sc)[b, h]
            assert np.isnan(got[n:]).all()  # rows of no token are left as they were
            l = O8.attend(qq, kk, vv, scale)[2]
            if n:
                assert np.abs(got[:n] - l).max() <= scale * (np.abs(kk).sum(1) * np.abs(qq).max()).max() * 2.0**-18


def test_decode_with_queries_and_scales_far_apart(tq):
    """Value scales from 1e-18 to 1e18 in one sequence, query rows from 1e-30 to 1e30, a zero row."""
    L = layer(tq, 128, 1, 8, 4)
    T = 16 * 12 + 4
    k, v = data((1, T, 1, 128), "f32", 14), data((1, T, 1, 128), "f32", 15)
    for i in range(12):
        v[0, 16 * i:16 * i + 16] *= 10.0 ** (3 * ((5 * i) % 12) - 18)
    q = data((1, 8, 128), "f32", 16)
    q[0, 0] = 0
    q[0, 1] *= 1e-30
    q[0, 2] *= 1e-4
    q[0, 3, 64:] = 0
    k16 = k.clone()
    pc = tq.PagedCache(L, 1, T)
    pc.prefill(k, v)
    out, lse, _ = decode(tq, pc, q, T, 2)
    m = Mirror(L, k16, v)
    kk, vv = m.values(0, 0, T, T)
    for h in range(8):
        check_attention(f64(q)[0, h], f64(out)[0, h], float(lse[0, h]), kk, vv, 128**-0.5, h)
    # 1e30: one token takes all the weight in either arithmetic unless two logits tie
    q[0, 4] *= 1e30
    out, lse, _ = decode(tq, pc, q, T, 2)
    l = O8.attend(f64(q)[0, 4], kk, vv, 128**-0.5)[2]
    top = int(np.argmax(l))
    assert np.sort(l)[-1] - np.sort(l)[-2] > 1e20
    # a single weight of 1: the two limbs' 2^-22 and the value scale's product
    assert np.abs(f64(out)[0, 4] - vv[top]).max() <= np.abs(vv[top]).max() * 2.0**-20
    # a NaN in one query row stays in that row
    q[0, 5, 3] = math.nan
    out2, lse2, _ = decode(tq, pc, q, T, 2)
    assert torch.isnan(out2[0, 5]).all() and torch.isnan(lse2[0, 5])
    keep = [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(out2[0, keep], out[0, keep])


def outlier_pages(kind):
    """(k, v, q) of 12 pages + 4 window tokens, one head, d = 128, whose value scales are far apart: page 3 holds values
    of 1e18 that weigh nothing (its keys are far from the query), or zeros that take all of the weight, or all of the
    values are tiny."""
    g = torch.Generator().manual_seed(70)
    k, v = torch.randn((1, 196, 1, 128), generator=g) * 0.1, torch.randn((1, 196, 1, 128), generator=g)
    q = torch.randn((1, 8, 128), generator=g)
    far = q[0].mean(0) * 40
    if kind == "huge_but_light":
        k[0, 48:64, 0] = -far * 10
        v[0, 48:64] *= 1e18
    elif kind == "zero_but_heavy":
        k[0, 48:64, 0] = far * 40
        v[0, 48:64] = 0
        v[0, 192:] = 0
    elif kind == "all_tiny":
        v *= 1e-36
        v[0, 192:] = 0
    return k.cuda(), v.cuda(), q.cuda()


@pytest.mark.parametrize("kind", ["huge_but_light", "zero_but_heavy", "all_tiny"])
@pytest.mark.parametrize("chunk", [1, 5, 20])
def test_value_scales_far_apart_keep_the_output_precise(tq, kind, chunk):
    """Against the output itself, not the largest value of the cache: dl <= 2^-12 here (|l| under 2^9 with 2^-21 each
    way), so 2 dl + 2^-12 of the terms that make up the output."""
    L = layer(tq, 128, 1, 8, 4)
    k, v, q = outlier_pages(kind)
    pc = tq.PagedCache(L, 1, 196)
    pc.prefill(k, v)
    qs = q[:, None].repeat(1, chunk, 1, 1).contiguous()
    out, lse = torch.full(qs.shape, float("nan"), device="cuda"), torch.full(qs.shape[:-1], float("nan"), device="cuda")
    ws = torch.empty(tq.prefill_workspace_size(L.params, 1, chunk, 196), dtype=torch.uint8, device="cuda")
    tq.prefill_attention(L.params, pc.cache, chunk, qs, 128**-0.5, out, lse, ws, 196)
    assert tq.check_device_error() == 0
    kk, vv = Mirror(L, k, v).values(0, 0, 196, 196)
    for i in range(chunk):
        n = 196 - chunk + i + 1
        for h in range(8):
            l = 128**-0.5 * kk[:n] @ f64(q)[0, h]
            p = np.exp(l - l.max())
            want = p @ vv[:n] / p.sum()
            terms = (p[:, None] * np.abs(vv[:n])).sum(0).max() / p.sum()
            got = f64(out)[0, i, h]
            assert np.isfinite(got).all()
            # results under 2^-120 may come out as 0
            assert (np.abs(got - want) <= 2.0**-10 * terms + 2.0**-120).all(), (i, h, np.abs(got - want).max(), terms)


def test_decode_flags_bad_state_and_skips_it(tq):
    L = layer(tq, 128, 2, 2, 16)
    T = 100
    k = data((3, T, 2, 128), "bf16", 17)
    pc = tq.PagedCache(L, 3, T)
    pc.prefill(k, k)
    q = data((3, 4, 128), "bf16", 18)
    ref, _, _ = decode(tq, pc, q, T)
    table = pc.block_table.clone()
    pc.block_table[0, 1] = -5
    pc.block_table[1, 2] = 10**6
    out, _, _ = decode(tq, pc, q, T)
    assert tq.check_device_error() == 0x1
    assert torch.equal(out[2], ref[2]) and torch.isfinite(out).all()
    pc.block_table.copy_(table)
    for n, nc in ((T + 1, 80), (T, T + 16), (-3, 0), (T, -16), (T, 16)):
        pc.seq_len[1], pc.n_compressed[1] = n, nc
        out, _, _ = decode(tq, pc, q, T)
        assert tq.check_device_error() == 0x2, (n, nc)
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])


def test_decode_static_and_captured_and_on_another_stream(tq):
    L = layer(tq, 128, 2, 4, 16)
    T = 300
    k, v = data((2, T + 4, 2, 128), "bf16", 19), data((2, T + 4, 2, 128), "bf16", 20)
    q = data((2, 8, 128), "bf16", 21)
    pc = tq.PagedCache(L, 2, T + 4)
    pc.prefill(k[:, :T], v[:, :T])
    ref, rl, _ = decode(tq, pc, q, T + 4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(tq.decode_workspace_size(L.params, 2, T + 4), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(ref), torch.zeros_like(rl)
    with torch.cuda.stream(st):
        tq.decode_attention(L.params, pc.cache, q, 128**-0.5, out, lse, None, ws, T + 4)
    st.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    s_out, s_lse = torch.zeros_like(ref), torch.zeros_like(rl)
    tq._lib.decode_attention_static(L.params, pc.cache, q, 128**-0.5, s_out, s_lse, None, T + 4)
    torch.cuda.synchronize()
    assert torch.equal(s_out, ref) and torch.equal(s_lse, rl)
    # a captured step (append, then decode) replayed over the same buffers
    kt, vt = k[:, T].contiguous(), v[:, T].contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pc.append(kt, vt)
        tq.decode_attention(L.params, pc.cache, q, 128**-0.5, out, lse, None, ws, T + 4)
    for t in range(T, T + 3):
        kt.copy_(k[:, t])
        vt.copy_(v[:, t])
        graph.replay()
        eager = tq.PagedCache(L, 2, T + 4)
        eager.prefill(k[:, :T], v[:, :T])
        for u in range(T, t + 1):
            eager.append(k[:, u].contiguous(), v[:, u].contiguous())
        ref, rl, _ = decode(tq, eager, q, T + 4)
        assert torch.equal(out, ref) and torch.equal(lse, rl), t
    assert pc.seq_len.tolist() == [T + 3] * 2 and tq.check_device_error() == 0


# ---------------------------------------------------------------------------------------------- prefill attention

@pytest.mark.parametrize("d,head_dim,hkv,g,window,dtype,T,nq", [
    (128, None, 2, 4, 32, "bf16", 200, 64), (128, None, 1, 1, 5, "f32", 1, 1), (128, None, 2, 3, 16, "f16", 150, 150),
    (256, None, 1, 8, 40, "bf16", 130, 33), (128, 80, 2, 5, 8, "f32", 90, 41), (256, 144, 1, 2, 16, "f16", 80, 80),
    (128, None, 1, 7, 3, "bf16", 530, 129), (128, None, 2, 8, 64, "bf16", 20, 13), (128, None, 2, 3, 16, "bf16", 300, 5),
    (128, None, 1, 1, 20, "f16", 90, 19), (128, None, 2, 2, 40, "f32", 200, 23), (256, None, 2, 1, 16, "bf16", 100, 21),
    (256, 160, 1, 3, 5, "f32", 77, 11),
])
def test_prefill_attention(tq, d, head_dim, hkv, g, window, dtype, T, nq):
    L = layer(tq, d, hkv, g, window, head_dim)
    B = 2
    k, v = data((B, T, hkv, L.head_dim), dtype, 22), data((B, T, hkv, L.head_dim), dtype, 23)
    pc = tq.PagedCache(L, B, T)
    pc.pool.fill_(0x7f)
    pc.prefill(k, v)
    ring = window + 16
    for slot in range(ring):
        if not any(p % ring == slot for p in range(O8.n_compressed(T, window), T)):
            pc.win_k[:, :, slot] = math.nan
            pc.win_v[:, :, slot] = math.nan
    q = data((B, nq, hkv * g, L.head_dim), dtype, 24)
    ws = torch.empty(tq.prefill_workspace_size(L.params, B, nq, T), dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:-1], float("nan"), device="cuda")
    tq.prefill_attention(L.params, pc.cache, nq, q, L.head_dim**-0.5, out, lse, ws, T)
    assert tq.check_device_error() == 0
    m = Mirror(L, k, v)
    qq, oo, zz = f64(q), f64(out), f64(lse)
    for b in range(B):
        for h in range(hkv * g):
            kk, vv = m.values(b, h // g, T, T)
            for i in sorted({0, 1, nq // 2, nq - 2, nq - 1} & set(range(nq))):
                n = T - nq + i + 1
                check_attention(qq[b, i, h], oo[b, i, h], zz[b, i, h], kk[:n], vv[:n], L.head_dim**-0.5, (b, h, i))
    assert np.isfinite(oo).all()


@pytest.mark.parametrize("nq", [20, 11])
def test_prefill_attention_of_ragged_sequences(tq, nq):
    """Sequences of different lengths, one shorter than the chunk (flagged; its first queries see nothing)."""
    L = layer(tq, 128, 2, 4, 16)
    lens, T = [140, 33, 9], 140
    k = data((3, T, 2, 128), "bf16", 25)
    pc = tq.PagedCache(L, 3, T)
    for b, n in enumerate(lens):
        one = tq.PagedCache(L, 1, T)
        one.share_pages(pc)
        one.block_table.copy_(pc.block_table[b:b + 1])
        one.prefill(k[b:b + 1, :n], k[b:b + 1, :n])
        pc.seq_len[b], pc.n_compressed[b] = n, O8.n_compressed(n, 16)
        pc.win_k[b], pc.win_v[b] = one.win_k[0], one.win_v[0]
    q = data((3, nq, 8, 128), "bf16", 26)
    ws = torch.empty(tq.prefill_workspace_size(L.params, 3, nq, T), dtype=torch.uint8, device="cuda")
    out, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:-1], float("nan"), device="cuda")
    tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, out, lse, ws, T)
    assert tq.check_device_error() == 0x2
    m = Mirror(L, k, k)
    for b, n in enumerate(lens):
        for h in range(8):
            kk, vv = m.values(b, h // 4, n, n)
            for i in range(nq):
                see = max(0, n - nq + i + 1)
                check_attention(f64(q)[b, i, h], f64(out)[b, i, h], float(lse[b, i, h]), kk[:see], vv[:see], 128**-0.5, (b, h, i))


@pytest.mark.parametrize("B,hkv,g,nq,T,window,dtype,seqs,heads,queries", [
    (39, 4, 2, 65, 1100, 16, "bf16", (0, 36, 37, 38), (0, 5, 7), (0, 63, 64)),
    (1, 8, 8, 640, 1070, 5, "f16", (0,), (0, 55, 56, 63), (0, 1, 383, 384, 385, 639)),
    (39, 4, 2, 65, 1100, 16, "f32", (0, 38), (0, 7), (0, 64)),
])
def test_prefill_attention_of_more_row_tiles_than_places(tq, B, hkv, g, nq, T, window, dtype, seqs, heads, queries):
    """156 and 160 units of work: those behind the last full wave are split over the keys."""
    L = layer(tq, 128, hkv, g, window)
    lens = [T - 3 * (b % 11) for b in range(B)]
    k = data((B, T, hkv, 128), dtype, 27)
    pc = tq.PagedCache(L, B, T)
    for b, n in enumerate(lens):
        one = tq.PagedCache(L, 1, T, pool_pages=1)
        one.share_pages(pc)
        one.block_table.copy_(pc.block_table[b:b + 1])
        one.prefill(k[b:b + 1, :n].contiguous(), k[b:b + 1, :n].contiguous())
        pc.seq_len[b], pc.n_compressed[b] = n, O8.n_compressed(n, window)
        pc.win_k[b], pc.win_v[b] = one.win_k[0], one.win_v[0]
    q = data((B, nq, hkv * g, 128), dtype, 28)
    ws = torch.empty(tq.prefill_workspace_size(L.params, B, nq, T), dtype=torch.uint8, device="cuda")
    out, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:-1], float("nan"), device="cuda")
    tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, out, lse, ws, T)
    assert tq.check_device_error() == 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    again = torch.empty_like(out)
    tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, again, None, ws, T)
    assert torch.equal(out, again)
    for b in seqs:
        n = lens[b]
        m = Mirror(L, k[b:b + 1], k[b:b + 1])
        for h in heads:
            kk, vv = m.values(0, h // g, n, n)
            for i in queries:
                see = n - nq + i + 1
                check_attention(f64(q[b, i, h]), f64(out[b, i, h]), float(lse[b, i, h]), kk[:see], vv[:see], 128**-0.5, (b, h, i))


def test_chunked_prefill_equals_decode_of_its_last_query(tq):
    """The chunk's last query is a decode query: both calls within the tolerance of the same definition."""
    L = layer(tq, 128, 4, 4, 32)
    T = 700
    k, v = data((1, T, 4, 128), "bf16", 27), data((1, T, 4, 128), "bf16", 28)
    pc = tq.PagedCache(L, 1, T)
    pc.prefill(k, v)
    q = data((1, 100, 16, 128), "bf16", 29)
    ws = torch.empty(tq.prefill_workspace_size(L.params, 1, 100, T), dtype=torch.uint8, device="cuda")
    out = torch.empty(q.shape, device="cuda")
    tq.prefill_attention(L.params, pc.cache, 100, q, 128**-0.5, out, None, ws, T)
    ref, _, _ = decode(tq, pc, q[:, -1].contiguous(), T)
    qn, kn = f64(q)[0, -1], np.abs(f64(k)).sum(-1).max()
    tol = 2 * (2 * 128**-0.5 * kn * np.abs(qn).max() * 2.0**-18 + 2.0**-16) * float(v.abs().max())
    assert (out[:, -1] - ref).abs().max() <= tol


@pytest.mark.parametrize("dtype,nq,g", [("bf16", 60, 4), ("f32", 60, 2), ("bf16", 200, 2), ("bf16", 5, 4)])
def test_non_finite_window_values_reach_only_the_queries_that_see_them(tq, dtype, nq, g):
    """A query attends to nothing behind itself, whatever lies there: infinities and NaN among the window's values (and
    keys) change no query before them, and do reach those after."""
    L = layer(tq, 128, 2, g, 100)
    T = 300
    k, v = data((1, T, 2, 128), dtype, 30), data((1, T, 2, 128), dtype, 31)
    pc = tq.PagedCache(L, 1, T)
    pc.prefill(k, v)
    q = data((1, nq, 2 * g, 128), dtype, 32)
    ws = torch.empty(tq.prefill_workspace_size(L.params, 1, nq, T), dtype=torch.uint8, device="cuda")

    def run():
        out = torch.empty(q.shape, device="cuda")
        tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, out, None, ws, T)
        return out

    ref = run()
    at = T - 3  # seen by the last three queries only
    pc.win_v[0, :, at % 116, 5] = math.inf
    pc.win_v[0, :, at % 116, 9] = math.nan
    out = run()
    assert torch.equal(out[:, :-3], ref[:, :-3])
    assert not torch.isfinite(out[:, -3:, :, 5]).any() and not torch.isfinite(out[:, -3:, :, 9]).any()
    keep = [c for c in range(128) if c not in (5, 9)]
    assert torch.equal(out[:, -3:][..., keep], ref[:, -3:][..., keep])
    pc.win_k[0, :, at % 116, 7] = math.nan
    out = run()
    assert torch.equal(out[:, :-3], ref[:, :-3]) and torch.isnan(out[:, -3:]).all()


def test_prefill_attention_skips_pages_that_are_not_there(tq):
    L = layer(tq, 128, 2, 4, 16)
    k = data((2, 200, 2, 128), "bf16", 33)
    pc = tq.PagedCache(L, 2, 200)
    pc.prefill(k, k)
    for nq in (40, 3):
        q = data((2, nq, 8, 128), "bf16", 34)
        ws = torch.empty(tq.prefill_workspace_size(L.params, 2, nq, 200), dtype=torch.uint8, device="cuda")
        out = [torch.full(q.shape, float("nan"), device="cuda") for _ in range(2)]
        tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, out[0], None, ws, 200)
        table = pc.block_table.clone()
        pc.block_table[0, 2], pc.block_table[0, 9] = -1, 10**6
        tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, out[1], None, ws, 200)
        assert tq.check_device_error() == 0x1
        assert torch.equal(out[0][1], out[1][1]) and torch.isfinite(out[1]).all()
        rows = [i for i in range(200) if i // 16 not in (2, 9)]
        kk, vv = Mirror(L, k, k).values(0, 0, 200, 200)
        check_attention(f64(q)[0, -1, 0], f64(out[1])[0, -1, 0], O8.attend(f64(q)[0, -1, 0], kk[rows], vv[rows], 128**-0.5)[1],
                        kk[rows], vv[rows], 128**-0.5, nq)
        pc.block_table.copy_(table)


def test_prefill_attention_captured_and_replayed(tq):
    L = layer(tq, 128, 2, 8, 16)
    T, nq = 600, 70
    k, v = data((1, T, 2, 128), "bf16", 35), data((1, T, 2, 128), "bf16", 36)
    pc = tq.PagedCache(L, 1, T)
    pc.prefill(k, v)
    q = data((1, nq, 16, 128), "bf16", 37)
    ws = torch.empty(tq.prefill_workspace_size(L.params, 1, nq, T), dtype=torch.uint8, device="cuda")
    ref, out = torch.empty(q.shape, device="cuda"), torch.empty(q.shape, device="cuda")
    tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, ref, None, ws, T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, out, None, ws, T)
    ws.fill_(0xFF)  # the workspace holds nothing from call to call
    graph.replay()
    assert torch.equal(out, ref)
    q.mul_(0.5)
    graph.replay()
    tq.prefill_attention(L.params, pc.cache, nq, q, 128**-0.5, ref, None, ws, T)
    assert torch.equal(out, ref) and tq.check_device_error() == 0


@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_scales_below_and_at_zero(tq, scale):
    L = layer(tq, 128, 1, 4, 16)
    T = 300
    k, v = data((1, T, 1, 128), "bf16", 38), data((1, T, 1, 128), "bf16", 39)
    pc = tq.PagedCache(L, 1, T)
    pc.prefill(k, v)
    kk, vv = Mirror(L, k, v).values(0, 0, T, T)
    for nq in (30, 2):
        q = data((1, nq, 4, 128), "bf16", 40)
        ws = torch.empty(tq.prefill_workspace_size(L.params, 1, nq, T), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
        tq.prefill_attention(L.params, pc.cache, nq, q, scale, out, lse, ws, T)
        for i in (0, nq - 1):
            n = T - nq + i + 1
            for h in range(4):
                o, z, _ = O8.attend(f64(q)[0, i, h], kk[:n], vv[:n], scale)
                dl = abs(scale) * (np.abs(kk).sum(1) * np.abs(f64(q)[0, i, h]).max()).max() * 2.0**-18
                assert np.abs(f64(out)[0, i, h] - o).max() <= (2 * dl + 2.0**-16) * np.abs(vv).max()
                assert abs(float(lse[0, i, h]) - z) <= dl + 2.0**-18 * max(1, abs(z))

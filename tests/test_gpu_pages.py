"""Page selection, attention over chosen pages, attention totals and eviction, against float64 definitions.

Choices are whole numbers and compared exactly.  Totals are float sums of at most 2^10 non-negative weights:
exp of a float difference is 2^-22 relative plus the difference's rounding (|l - lse| 2^-24, under 2^-18 here), the
sum 2^-20: 2^-17 relative.
"""

import math

import numpy as np
import pytest

from oracle import int8 as O8
from test_gpu_int8 import Mirror, check_attention, data, decode, f64, layer, tq  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def filled(tq, L, lens, seed, dtype="bf16", T=None):
    """A cache of sequences of these lengths over a shuffled pool, and its inputs."""
    T = T or max(lens)
    k, v = data((len(lens), T, L.n_kv_heads, L.head_dim), dtype, seed), data((len(lens), T, L.n_kv_heads, L.head_dim), dtype, seed + 1)
    pc = tq.PagedCache(L, len(lens), T)
    pc.block_table.copy_(torch.randperm(pc.n_pages, generator=torch.Generator().manual_seed(seed)).reshape(len(lens), -1).int())
    pc.prefill(k, v)
    for b, n in enumerate(lens):
        one = tq.PagedCache(L, 1, T)
        one.share_pages(pc)
        one.block_table.copy_(pc.block_table[b:b + 1])
        one.prefill(k[b:b + 1, :n], v[b:b + 1, :n])
        pc.seq_len[b], pc.n_compressed[b] = n, O8.n_compressed(n, L.window) if L.window else n
        if L.window:
            pc.win_k[b], pc.win_v[b] = one.win_k[0], one.win_v[0]
    return pc, k, v


def select(tq, pc, q, n_sel, sink, recent, T):
    L = pc.layer
    ws = torch.empty(tq.select_workspace_size(L.params, pc.batch, T), dtype=torch.uint8, device="cuda")
    pages = torch.full((pc.batch, L.n_kv_heads, n_sel), 12345, dtype=torch.int32, device="cuda")
    counts = torch.full((pc.batch, L.n_kv_heads), 12345, dtype=torch.int32, device="cuda")
    tq.select_pages(L.params, pc.cache, q, n_sel, sink, recent, pages, counts, ws, T)
    return pages, counts


@pytest.mark.parametrize("d,head_dim,hkv,g,window,lens,n_sel,sink,recent,dtype", [
    (128, None, 2, 4, 16, [500, 90, 16, 333], 7, 1, 2, "bf16"), (256, None, 1, 8, 5, [700, 0, 1], 9, 0, 0, "f16"),
    (128, 96, 3, 1, 20, [260], 16, 15, 1, "f32"), (128, None, 1, 3, 16, [400], 400, 2, 2, "bf16"),
    (256, 200, 2, 5, 16, [1300, 40], 1, 0, 0, "f32"), (128, None, 1, 2, 16, [3000], 70, 0, 3, "bf16"),
])
def test_selected_pages_are_the_best(tq, d, head_dim, hkv, g, window, lens, n_sel, sink, recent, dtype):
    L = layer(tq, d, hkv, g, window, head_dim)
    T = max(lens)
    pc, k, v = filled(tq, L, lens, 31, dtype)
    q = data((len(lens), hkv * g, L.head_dim), dtype, 33)
    q[0, :g] *= 3.0
    pages, counts = select(tq, pc, q, n_sel, sink, recent, T)
    assert tq.check_device_error() == 0
    for b, n in enumerate(lens):
        nc = O8.n_compressed(n, window)
        for h in range(hkv):
            key = O8.page_scores(f64(q)[b, h * g:(h + 1) * g], f64(k)[b, :n, h], nc)
            want = O8.choose(key, n_sel, sink, recent)
            assert int(counts[b, h]) == len(want)
            assert pages[b, h].tolist() == want + [-1] * (n_sel - len(want)), (b, h)


def test_selection_among_equals_takes_the_lower_page(tq):
    L = layer(tq, 128, 2, 2, 16)
    T = 16 * 40 + 16
    k = data((1, 16, 2, 128), "bf16", 34).repeat(1, T // 16, 1, 1)
    k[:, 16 * 20:16 * 21] *= 2
    pc = tq.PagedCache(L, 1, T)
    pc.prefill(k, k)
    q = data((1, 4, 128), "bf16", 35)
    assert select(tq, pc, q, 5, 0, 1, T)[0][0].tolist() == [[0, 1, 2, 20, 39]] * 2
    assert select(tq, pc, torch.zeros_like(q), 3, 0, 0, T)[0][0].tolist() == [[0, 1, 2]] * 2  # all scores 0
    q[0, 0, 5] = math.nan  # non-finite entries count as in a page: NaN 0, infinities the largest code
    q[0, 1, 7] = math.inf
    key = O8.page_scores(f64(q)[0, :2], f64(k)[0, :, 0], T - 16)
    assert select(tq, pc, q, 5, 0, 1, T)[0][0, 0].tolist() == O8.choose(key, 5, 0, 1)


def test_selection_of_a_bad_state_takes_nothing(tq):
    L = layer(tq, 128, 1, 2, 16)
    pc, k, v = filled(tq, L, [200, 200], 36)
    q = data((2, 2, 128), "bf16", 37)
    pc.seq_len[1] = 300
    pages, counts = select(tq, pc, q, 3, 0, 0, 200)
    assert tq.check_device_error() == 0x2
    assert counts[:, 0].tolist() == [3, 0] and pages[1, 0].tolist() == [-1] * 3


@pytest.mark.parametrize("d,hkv,g,window,lens", [(128, 2, 4, 16, [500, 40, 16]), (256, 1, 8, 30, [400, 100])])
def test_attention_over_listed_pages(tq, d, hkv, g, window, lens):
    L = layer(tq, d, hkv, g, window)
    T, n_sel = max(lens), 6
    pc, k, v = filled(tq, L, lens, 38)
    q = data((len(lens), hkv * g, d), "bf16", 40)
    rng = np.random.default_rng(3)
    pages = torch.full((len(lens), hkv, n_sel), -7, dtype=torch.int32)
    lists = {}
    for b, n in enumerate(lens):
        for h in range(hkv):
            np_ = O8.n_compressed(n, window) // 16
            take = list(rng.permutation(np_)[:rng.integers(0, min(np_, n_sel) + 1)])
            if len(take) in (2, 3, 4):
                take.append(take[0])  # one page twice: it counts twice
            lists[b, h] = [int(x) for x in take]
            pages[b, h, :len(take)] = torch.tensor(lists[b, h], dtype=torch.int32)
    counts = torch.tensor([[len(lists[b, h]) for h in range(hkv)] for b in range(len(lens))], dtype=torch.int32, device="cuda")
    pages = pages.cuda()
    m = Mirror(L, k, v)
    for splits in (0, 1, 4):
        ws = torch.empty(tq.decode_pages_workspace_size(L.params, len(lens), n_sel, splits), dtype=torch.uint8, device="cuda")
        out = torch.full((len(lens), hkv * g, d), float("nan"), device="cuda")
        lse = torch.full((len(lens), hkv * g), float("nan"), device="cuda")
        tq.decode_attention_pages(L.params, pc.cache, q, d**-0.5, pages, counts, n_sel, out, lse, ws, T, splits)
        assert tq.check_device_error() == 0
        for b, n in enumerate(lens):
            for h in range(hkv * g):
                kk, vv = m.values(b, h // g, n, n)
                rows = [16 * p + i for p in lists[b, h // g] for i in range(16)] + list(range(O8.n_compressed(n, window), n))
                check_attention(f64(q)[b, h], f64(out)[b, h], float(lse[b, h]), kk[rows], vv[rows], d**-0.5, (b, h, splits))
    # ordinals outside the sequence and counts outside the list are flagged and skipped
    bad = pages.clone()
    bad[0, 0, 0] = 10**6
    counts2 = counts.clone()
    counts2[0, 0] = max(1, int(counts[0, 0]))
    tq.decode_attention_pages(L.params, pc.cache, q, d**-0.5, bad, counts2, n_sel, out, lse, ws, T, 4)
    assert tq.check_device_error() == 0x1 and torch.isfinite(out).all()
    counts2[0, 0] = n_sel + 1
    tq.decode_attention_pages(L.params, pc.cache, q, d**-0.5, pages, counts2, n_sel, out, lse, ws, T, 4)
    assert tq.check_device_error() & 0x2


# ---------------------------------------------------------------------------------------------- totals and eviction

@pytest.mark.parametrize("hq,lens,max_ctx", [(8, [200, 17, 130], 200), (3, [61], 67), (32, [1000, 0], 1000)])
def test_totals(tq, hq, lens, max_ctx):
    L = tq.TQLayer(128, 1 if hq < 8 else hq // 4, hq, 8, 8, tq.TQ_FWHT, window=16, key_qjl=tq.KEY_MSE, int8=True)
    pc = tq.PagedCache(L, len(lens), max_ctx, pool_pages=1)
    g = torch.Generator().manual_seed(5)
    scores = torch.randn((len(lens), hq, max_ctx), generator=g) * 2
    lse = torch.full((len(lens), hq), -math.inf)
    for b, n in enumerate(lens):
        pc.seq_len[b], pc.n_compressed[b] = n, O8.n_compressed(n, 16)
        if n:
            lse[b] = scores[b, :, :n].double().logsumexp(-1).float()
        scores[b, :, n:] = math.nan
    mass = torch.rand((len(lens), pc.max_pages), generator=g)
    got = mass.cuda()
    for _ in range(2):
        tq.track_pages(L.params, pc.cache, scores.cuda(), lse.cuda(), got, max_ctx)
    assert tq.check_device_error() == 0
    for b, n in enumerate(lens):
        np_ = O8.n_compressed(n, 16) // 16
        p = np.exp(f64(scores)[b, :, :16 * np_] - f64(lse)[b][:, None]) if n else np.zeros((hq, 0))
        want = f64(mass)[b].copy()
        want[:np_] += 2 * p.reshape(hq, np_, 16).sum((0, 2))
        assert (np.abs(f64(got)[b] - want) <= 2.0**-17 * want).all()
        assert np.array_equal(f64(got)[b, np_:], f64(mass)[b, np_:])
    again = mass.cuda()
    for _ in range(2):
        tq.track_pages(L.params, pc.cache, scores.cuda(), lse.cuda(), again, max_ctx)
    assert torch.equal(again, got)


def evict(tq, pc, mass, budget, sink, recent, after=None, mass_after=None):
    L = pc.layer
    after, mass_after = after or pc, mass if mass_after is None else mass_after
    kept = torch.full((pc.batch, budget), 777, dtype=torch.int32, device="cuda")
    ws = torch.empty(tq.evict_workspace_size(L.params, pc.batch, pc.max_pages), dtype=torch.uint8, device="cuda")
    tq.evict_pages(L.params, pc.cache, after.cache, mass, mass_after, budget, sink, recent, kept, ws)
    return kept


def expected_eviction(table, mass, n, nc, budget, sink, recent):
    np_, part = nc // 16, 1 if nc % 16 else 0
    keep = O8.choose(mass[:np_], budget, sink, recent)
    gone = [i for i in range(np_) if i not in set(keep)]
    order = keep + [np_] * part + gone + list(range(np_ + part, len(table)))
    m = np.zeros(len(table), np.float32)
    m[:len(keep) + part] = mass[keep + [np_] * part]
    return [table[i] for i in order], m, n - 16 * len(gone), nc - 16 * len(gone), keep


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("window,lens,budget,sink,recent", [
    (16, [500, 90, 16, 0, 333], 7, 1, 2), (5, [1000, 700], 20, 0, 0), (40, [400, 300], 3, 1, 2), (130, [2000], 1, 0, 0),
    (1, [333], 300, 4, 4), (16, [50000], 1000, 4, 16),
])
def test_eviction(tq, in_place, window, lens, budget, sink, recent):
    L = layer(tq, 128, 2, 2, window)
    T = max(lens)
    pc = tq.PagedCache(L, len(lens), T, pool_pages=1)
    g = torch.Generator().manual_seed(6)
    pc.block_table.copy_(torch.randint(0, 10**6, pc.block_table.shape, generator=g, dtype=torch.int32))
    mass = torch.rand(pc.block_table.shape, generator=g)
    mass[:, ::3] = 0.25  # equals
    mass[0, 1] = math.nan
    for b, n in enumerate(lens):
        pc.seq_len[b], pc.n_compressed[b] = n, O8.n_compressed(n, window)
    pc.win_k.copy_(torch.randn(pc.win_k.shape, generator=g))
    pc.win_v.copy_(torch.randn(pc.win_v.shape, generator=g))
    old = dict(t=pc.block_table.tolist(), m=mass.numpy().copy(), k=pc.win_k.clone(), v=pc.win_v.clone())
    mg = mass.cuda()
    after, ma = pc, mg
    if not in_place:
        after, ma = tq.PagedCache(L, len(lens), T, pool_pages=1), torch.full_like(mg, 9.0)
        after.share_pages(pc)
    kept = evict(tq, pc, mg, budget, sink, recent, after, ma)
    assert tq.check_device_error() == 0
    ring = window + 16
    for b, n in enumerate(lens):
        nc = O8.n_compressed(n, window)
        t, m, n2, nc2, keep = expected_eviction(old["t"][b], old["m"][b], n, nc, budget, sink, recent)
        assert after.block_table[b].tolist() == t
        assert np.array_equal(ma[b].cpu().numpy(), m, equal_nan=True)
        assert (int(after.seq_len[b]), int(after.n_compressed[b])) == (n2, nc2)
        assert kept[b].tolist() == keep + [-1] * (budget - len(keep))
        for p in range(nc2, n2):
            for now, was in ((after.win_k, old["k"]), (after.win_v, old["v"])):
                assert torch.equal(now[b, :, p % ring], was[b, :, (p + n - n2) % ring])
    if not in_place:  # the source is as it was
        assert pc.block_table.tolist() == old["t"] and torch.equal(pc.win_k, old["k"])
        assert pc.seq_len.tolist() == lens and np.array_equal(mg.cpu().numpy(), old["m"], equal_nan=True)


def test_eviction_of_a_bad_state_changes_nothing(tq):
    L = layer(tq, 128, 1, 1, 16)
    pc = tq.PagedCache(L, 3, 160, pool_pages=1)
    pc.seq_len.copy_(torch.tensor([160, 10, 300]))
    pc.n_compressed.copy_(torch.tensor([144, 16, 288]))
    mass = torch.rand((3, 10), device="cuda")
    old = (pc.block_table.clone(), mass.clone())
    evict(tq, pc, mass, 4, 0, 0)
    assert tq.check_device_error() == 0x2
    assert pc.seq_len.tolist() == [80, 10, 300] and pc.n_compressed.tolist() == [64, 16, 288]
    assert torch.equal(pc.block_table[1:], old[0][1:]) and torch.equal(mass[1:], old[1][1:])


def test_counters_that_hold_anything_are_flagged(tq):
    big = 2**31 - 1
    L = layer(tq, 128, 1, 2, 16)
    states = [(160, 144), (big, big), (big, big - 15), (big, 144), (-1, -1), (160, -16), (-2**31, 0)]
    pc = tq.PagedCache(L, len(states), 160, pool_pages=10)
    pc.seq_len.copy_(torch.tensor([s[0] for s in states]))
    pc.n_compressed.copy_(torch.tensor([s[1] for s in states]))
    mass = torch.rand((len(states), 10), device="cuda")
    old = (pc.block_table.clone(), mass.clone())
    scores, lse = torch.zeros((len(states), 2, 160), device="cuda"), torch.zeros((len(states), 2), device="cuda")
    tq.track_pages(L.params, pc.cache, scores, lse, mass, 160)
    assert tq.check_device_error() == 0x2
    assert torch.equal(mass[1:], old[1][1:]) and not torch.equal(mass[0], old[1][0])
    q = data((len(states), 2, 128), "f32", 50)
    pages, counts = torch.empty((len(states), 1, 4), dtype=torch.int32, device="cuda"), torch.empty((len(states), 1), dtype=torch.int32, device="cuda")
    ws = torch.empty(tq.select_workspace_size(L.params, len(states), 160), dtype=torch.uint8, device="cuda")
    tq.select_pages(L.params, pc.cache, q, 4, 1, 1, pages, counts, ws, 160)
    assert tq.check_device_error() == 0x2 and counts.flatten().tolist() == [4] + [0] * (len(states) - 1)
    kept = evict(tq, pc, mass, 4, 0, 0)
    assert tq.check_device_error() == 0x2
    assert [tuple(s) for s in zip(pc.seq_len.tolist(), pc.n_compressed.tolist())] == [(80, 64)] + states[1:]
    assert torch.equal(pc.block_table[1:], old[0][1:]) and torch.equal(mass[1:], old[1][1:]) and (kept[1:] == -1).all()


def test_a_thinned_turboquant_cache_attends_to_what_is_left(tq):
    """Eviction moves pages of any arm: 3-bit keys without a window, the last page partly filled.  The thinned cache's
    decode equals that of a cache that was given the kept tokens only (equal records: the same bits)."""
    L = tq.TQLayer(128, 2, 8, 3, 4, tq.TQ_FWHT, window=0, key_qjl=tq.KEY_QJL)
    T = 16 * 11 + 5
    pc, k, v = filled(tq, L, [T, T], 41)
    q = data((2, 8, 128), "bf16", 43)
    out, lse, sc = decode(tq, pc, q, T, scores=True)
    mass = torch.zeros((2, pc.max_pages), device="cuda")
    tq.track_pages(L.params, pc.cache, sc, lse, mass, T)
    w = torch.exp(sc.double() - lse.double()[..., None]).sum(1)
    w = torch.nn.functional.pad(w, (0, 16 * 12 - T)).reshape(2, 12, 16).sum(-1)
    assert ((mass - w).abs() <= 2.0**-17 * w).all()
    kept = evict(tq, pc, mass, 5, 1, 1).tolist()
    assert pc.seq_len.tolist() == [16 * 5 + 5] * 2 and pc.n_compressed.tolist() == [16 * 5 + 5] * 2
    rows = torch.tensor([[16 * p + i for p in kp for i in range(16)] + list(range(T - 5, T)) for kp in kept], device="cuda")
    take = lambda x: torch.stack([x[b, rows[b]] for b in range(2)])  # noqa: E731
    ref = tq.PagedCache(L, 2, T)
    ref.prefill(take(k), take(v))
    a, b = decode(tq, pc, q, T), decode(tq, ref, q, T)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # and goes on: appended tokens fill the partly filled page, then the pages that were dropped
    more, mv = data((2, 30, 2, 128), "bf16", 44), data((2, 30, 2, 128), "bf16", 45)
    for t in range(30):
        for c in (pc, ref):
            c.append(more[:, t].contiguous(), mv[:, t].contiguous())
    a, b = decode(tq, pc, q, T), decode(tq, ref, q, T)
    assert torch.equal(a[0], b[0]) and tq.check_device_error() == 0


def test_a_run_of_them_together(tq):
    """A prompt, steps that select, attend and track, an eviction in place, and more steps: every output against the
    definition over what the cache holds."""
    W, T0, hkv, g = 20, 300, 2, 4
    L = layer(tq, 128, hkv, g, W)
    steps = 40
    k, v = data((2, T0 + steps, hkv, 128), "bf16", 46), data((2, T0 + steps, hkv, 128), "bf16", 47)
    pc = tq.PagedCache(L, 2, T0 + steps)
    pc.prefill(k[:, :T0], v[:, :T0])
    mx, n_sel, scale = T0 + steps, 6, 128**-0.5
    ws = torch.empty(max(tq.select_workspace_size(L.params, 2, mx), tq.decode_pages_workspace_size(L.params, 2, n_sel)),
                     dtype=torch.uint8, device="cuda")
    mass = torch.zeros((2, pc.max_pages), device="cuda")
    # what each (sequence, head) holds: raw inputs as quantized (float16 where they went through the window)
    nc0 = O8.n_compressed(T0, W)
    hold = []
    for x in (f64(k), f64(v)):
        x = x.copy()
        x[:, nc0:] = x[:, nc0:].astype(np.float16).astype(np.float64)
        hold.append([[list(x[b, :T0, h]) for h in range(hkv)] for b in range(2)])
        full = x
        hold[-1].append(full)
    n, nc = T0, nc0
    for t in range(T0, T0 + steps):
        pc.append(k[:, t].contiguous(), v[:, t].contiguous())
        n += 1
        if n - nc == W + 16:
            nc += 16
        for i in range(2):
            for b in range(2):
                for h in range(hkv):
                    hold[i][b][h].append(hold[i][2][b, t, h])
        q = data((2, hkv * g, 128), "bf16", 100 + t)
        pages = torch.empty((2, hkv, n_sel), dtype=torch.int32, device="cuda")
        counts = torch.empty((2, hkv), dtype=torch.int32, device="cuda")
        out, lse = torch.empty((2, hkv * g, 128), device="cuda"), torch.empty((2, hkv * g), device="cuda")
        tq.select_pages(L.params, pc.cache, q, n_sel, 1, 1, pages, counts, ws, mx)
        tq.decode_attention_pages(L.params, pc.cache, q, scale, pages, counts, n_sel, out, lse, ws, mx)
        if t % 8 == 0 or t == T0 + 21:
            for b in range(2):
                for h in range(hkv):
                    kk, vv = np.array(hold[0][b][h]), np.array(hold[1][b][h])
                    want = O8.choose(O8.page_scores(f64(q)[b, h * g:h * g + g], kk, nc), n_sel, 1, 1)
                    assert pages[b, h, :len(want)].tolist() == want, (t, b, h)
                    rows = [16 * p + i for p in want for i in range(16)] + list(range(nc, n))
                    hk, hv = O8.held(kk, nc)[rows], O8.held(vv, nc)[rows]
                    for j in range(g):
                        check_attention(f64(q)[b, h * g + j], f64(out)[b, h * g + j], float(lse[b, h * g + j]), hk, hv, scale, (t, b, h, j))
        _, full_lse, sc = decode(tq, pc, q, mx, scores=True)
        tq.track_pages(L.params, pc.cache, sc, full_lse, mass, mx)
        if t == T0 + 20:
            before = mass.cpu().numpy()
            kept = evict(tq, pc, mass, 8, 1, 2).tolist()
            for b in range(2):
                keep = O8.choose(before[b, :nc // 16], 8, 1, 2)
                assert kept[b] == keep
                for i in range(2):
                    for h in range(hkv):
                        x = hold[i][b][h]
                        hold[i][b][h] = [x[16 * p + j] for p in keep for j in range(16)] + x[nc:]
            e = 16 * (nc // 16 - 8)
            n, nc = n - e, nc - e
            assert pc.seq_len.tolist() == [n] * 2 and pc.n_compressed.tolist() == [nc] * 2
    assert tq.check_device_error() == 0


def test_pages_behind_4_gb_of_the_pool(tq):
    """The same sequence in the pool's first and in its last pages (byte offsets past 32 bits): equal bits everywhere."""
    L = layer(tq, 128, 1, 4, 16)
    T, far = 400, 1000100
    assert (far - 64) * L.sub_bytes > 2**32
    low = tq.PagedCache(L, 1, T + 16, pool_pages=far)
    high = tq.PagedCache(L, 1, T + 16, pool_pages=1)
    high.share_pages(low)
    high.block_table.copy_(far - 1 - torch.arange(high.max_pages, dtype=torch.int32)[None])
    k, v = data((1, T + 16, 1, 128), "bf16", 60), data((1, T + 16, 1, 128), "bf16", 61)
    got = []
    for pc in (low, high):
        pc.prefill(k[:, :T], v[:, :T])
        for t in range(T, T + 16):
            pc.append(k[:, t].contiguous(), v[:, t].contiguous())
        n = T + 16
        rk, rv = torch.zeros((1, n, 1, 128), device="cuda"), torch.zeros((1, n, 1, 128), device="cuda")
        tq.read_cache(L.params, pc.cache, rk, rv, 0, n)
        q = data((1, 4, 128), "bf16", 62)
        out, lse, _ = decode(tq, pc, q, n)
        chunk = data((1, 40, 4, 128), "bf16", 63)  # 160 rows
        o2 = torch.empty((1, 40, 4, 128), device="cuda")
        ws = torch.empty(tq.prefill_workspace_size(L.params, 1, 40, n), dtype=torch.uint8, device="cuda")
        tq.prefill_attention(L.params, pc.cache, 40, chunk, 128**-0.5, o2, None, ws, n)
        pages, counts = select(tq, pc, q, 5, 1, 1, n)
        o3 = torch.empty((1, 4, 128), device="cuda")
        ws = torch.empty(tq.decode_pages_workspace_size(L.params, 1, 5), dtype=torch.uint8, device="cuda")
        tq.decode_attention_pages(L.params, pc.cache, q, 128**-0.5, pages, counts, 5, o3, None, ws, n)
        got.append((rk, rv, out, lse, o2, pages, counts, o3))
    assert tq.check_device_error() == 0
    assert got[0][0].abs().sum() > 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_captured_step_selects_tracks_and_evicts(tq):
    """One graph of a whole serving step, replayed, against the same calls made one by one."""
    L = layer(tq, 128, 2, 4, 5)
    T, steps, budget, n_sel, scale = 150, 40, 6, 3, 128**-0.5
    k, v = data((2, T + steps, 2, 128), "bf16", 70), data((2, T + steps, 2, 128), "bf16", 71)
    qs = data((steps, 2, 8, 128), "bf16", 72)
    mx = T + 16

    def make():
        pc = tq.PagedCache(L, 2, mx)
        pc.prefill(k[:, :T], v[:, :T])
        b = dict(pc=pc, k=k[:, 0].clone(), v=v[:, 0].clone(), q=qs[0].clone(), mass=torch.zeros((2, pc.max_pages), device="cuda"),
                 pages=torch.zeros((2, 2, n_sel), dtype=torch.int32, device="cuda"),
                 counts=torch.zeros((2, 2), dtype=torch.int32, device="cuda"),
                 kept=torch.zeros((2, budget), dtype=torch.int32, device="cuda"), out=torch.zeros((2, 8, 128), device="cuda"),
                 few=torch.zeros((2, 8, 128), device="cuda"), lse=torch.zeros((2, 8), device="cuda"),
                 scores=torch.zeros((2, 8, mx), device="cuda"))
        size = max(tq.select_workspace_size(L.params, 2, mx), tq.decode_pages_workspace_size(L.params, 2, n_sel),
                   tq.decode_workspace_size(L.params, 2, mx), tq.evict_workspace_size(L.params, 2, pc.max_pages))
        b["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")  # one for all: the calls follow one another
        return b

    def step(b):
        c = b["pc"].cache
        b["pc"].append(b["k"], b["v"])
        tq.select_pages(L.params, c, b["q"], n_sel, 1, 1, b["pages"], b["counts"], b["ws"], mx)
        tq.decode_attention_pages(L.params, c, b["q"], scale, b["pages"], b["counts"], n_sel, b["few"], None, b["ws"], mx)
        tq.decode_attention(L.params, c, b["q"], scale, b["out"], b["lse"], b["scores"], b["ws"], mx)
        tq.track_pages(L.params, c, b["scores"], b["lse"], b["mass"], mx)
        tq.evict_pages(L.params, c, c, b["mass"], b["mass"], budget, 1, 1, b["kept"], b["ws"])

    eager, played = make(), make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(played)
    for t in range(steps):
        for b in (eager, played):
            b["k"].copy_(k[:, T + t])
            b["v"].copy_(v[:, T + t])
            b["q"].copy_(qs[t])
        step(eager)
        graph.replay()
        for name in ("out", "few", "lse", "mass", "pages", "counts", "kept"):
            assert torch.equal(eager[name], played[name]), (t, name)
        for name in ("block_table", "seq_len", "n_compressed"):
            assert torch.equal(getattr(eager["pc"], name), getattr(played["pc"], name)), (t, name)
    assert tq.check_device_error() == 0
    assert played["pc"].n_compressed.tolist() == [budget * 16] * 2

"""Eviction on the GPU against the plain definition (exact), and the whole run of a cache
that is filled, read, evicted and read on."""

import numpy as np
import pytest
import torch

import kv4_ref
import oracle
from parity import dev_i32
from test_gpu_kv4 import DIM, bf16, f64, new_rows

pytestmark = pytest.mark.gpu


def H():
    import sparse_attention_top_hisa_b200 as mod
    return mod


def regions(lens, spare=1):
    return np.concatenate([[0], np.cumsum([(x // 128 + 1 + spare) * 128 for x in lens])]) \
        .astype(np.int32)


def weights_of(kind, n, rng):
    if kind == "ties":
        return rng.integers(0, 4, n)
    if kind == "equal":
        return np.full(n, 77)
    if kind == "zero":
        return np.zeros(n, np.int64)
    if kind == "wide":  # every magnitude, both signs, the extremes
        w = rng.integers(-2 ** 62, 2 ** 62, n) >> rng.integers(0, 63, n)
        w[rng.integers(0, n, max(1, n // 50))] = np.iinfo(np.int64).max
        w[rng.integers(0, n, max(1, n // 50))] = np.iinfo(np.int64).min
        return w
    if kind == "close":  # differ in the low bits only
        return (1 << 52) + rng.integers(0, 3000, n)
    w = np.exp(rng.standard_normal(n) * 2.5) * (rng.random(n) < 0.6)
    return (w * 2.0 ** 26).astype(np.int64)


def run_select(w, cu_k, lens, keep, sink, recent, max_len=None):
    h = H()
    kept = torch.full((len(w),), -9, dtype=torch.int32, device="cuda")
    n = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    h.hisa_evict_select(torch.from_numpy(w.astype(np.int64)).cuda(), dev_i32(cu_k), dev_i32(lens),
                        dev_i32(keep), max(lens) if max_len is None else max_len, sink, recent,
                        kept=kept, kept_len=n)
    return kept.cpu().numpy(), n.cpu().numpy()


@pytest.mark.parametrize("kind", ["real", "ties", "equal", "zero", "wide", "close"])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1], [0], 0, 0), ([1, 0, 2], [1, 1, 1], 0, 0), ([100, 1000], [99, 1], 4, 32),
    ([4096, 4097, 5000], [2048, 4096, 5000], 4, 128), ([3000, 3001], [100, 60], 50, 30),
    ([2500], [2499], 0, 0), ([2049], [700], 0, 700), ([20000, 300], [9000, 17], 64, 512)])
def test_select(kind, lens, keep, sink, recent):
    h = H()
    rng = np.random.Generator(np.random.PCG64(sum(lens) + sink))
    cu_k = regions(lens)
    w = weights_of(kind, int(cu_k[-1]), rng)
    h.hisa_device_status(clear=True)
    kept, n = run_select(w, cu_k, lens, keep, sink, recent)
    assert h.hisa_device_status() == 0
    for s, length in enumerate(lens):
        c = int(cu_k[s])
        want = kv4_ref.evict_select(w[c:c + length], length, keep[s], sink, recent)
        assert n[s] == len(want)
        assert np.array_equal(kept[c:c + len(want)], want)
        assert (kept[c + len(want):cu_k[s + 1]] == -9).all()  # left as they were


def test_select_long_sequences():
    """Sequences of 300000 tokens, one with its weights in ascending order."""
    rng = np.random.Generator(np.random.PCG64(2))
    lens, keep = [300000, 131072, 7], [100001, 32768, 3]
    cu_k = regions(lens)
    w = weights_of("real", int(cu_k[-1]), rng)
    w[:300000] = np.sort(w[:300000])
    kept, n = run_select(w, cu_k, lens, keep, 128, 4096)
    for s, length in enumerate(lens):
        c = int(cu_k[s])
        x = w[c:c + length]
        if length > 4096:
            order = np.argsort(-x[128:length - 4096], kind="stable")[:keep[s] - 128 - 4096] + 128
            want = np.sort(np.concatenate([np.arange(128), order,
                                           np.arange(length - 4096, length)]))
        else:
            want = kv4_ref.evict_select(x, length, keep[s], 128, 4096)
        assert n[s] == keep[s] and np.array_equal(kept[c:c + n[s]], want)


def test_select_bad_sequences_are_reported():
    h = H()
    cu_k, w = regions([100, 100, 100, 100]), np.arange(1024)
    h.hisa_device_status(clear=True)
    kept, n = run_select(w, cu_k, [100, 300, 100, 90], [5, 5, -1, 5], 0, 0, max_len=100)
    assert h.hisa_device_status(clear=True) == 1 << 1
    assert n.tolist() == [5, -1, -1, 5] and kept[:5].tolist() == [95, 96, 97, 98, 99]
    assert (kept[256:768] == -9).all()
    kept, n = run_select(w, cu_k, [100, 100, 100, 90], [5, 5, 1, 5], 0, 0, max_len=99)
    assert h.hisa_device_status(clear=True) == 1 << 1
    assert n.tolist() == [-1, -1, -1, 5]


def arrays_of(rows, rng, widest=True):
    """Row arrays of every piece width: 4, 8, 12, 16, 24, 48, 128 and 4096 bytes."""
    out = [torch.from_numpy(rng.integers(0, 2 ** 31, (rows, n)).astype(np.int32)).cuda()
           for n in (1, 2, 3, 4, 6, 12)]
    out[0] = out[0].view(rows)
    out.append(torch.from_numpy(rng.integers(0, 256, (rows, 128)).astype(np.uint8)).cuda())
    if widest:
        out.append(torch.from_numpy(rng.integers(0, 2 ** 15, (rows, 16, 128), dtype=np.int16))
                   .cuda())
    return out


def kept_of(lens, keep, cu, rng):
    kept = np.full(int(cu[-1]), -5, np.int32)
    for s, (n, k) in enumerate(zip(lens, keep)):
        kept[cu[s]:cu[s] + k] = np.sort(rng.choice(n, k, replace=False))
    return kept


MOVES = [([1], [1]), ([200, 0, 300], [130, 0, 1]), ([5000], [4999]), ([9000, 700], [4321, 700]),
         ([300] * 40, [77] * 40)]


@pytest.mark.parametrize("lens,keep", MOVES)
def test_rows_to_another_cache(lens, keep):
    h = H()
    rng = np.random.Generator(np.random.PCG64(sum(keep)))
    cu, cd = regions(lens), regions(keep, 0)
    kept = kept_of(lens, keep, cu, rng)
    src = arrays_of(int(cu[-1]), rng)
    dst = [torch.full((int(cd[-1]),) + t.shape[1:], 3, dtype=t.dtype, device="cuda") for t in src]
    want = [t.clone() for t in dst]
    for s, k in enumerate(keep):
        at = torch.from_numpy(cu[s] + kept[cu[s]:cu[s] + k].astype(np.int64)).cuda()
        for a, b in zip(src, want):
            b[cd[s]:cd[s] + k] = a[at]
    h.hisa_device_status(clear=True)
    h.hisa_evict_rows(src, dst, dev_i32(cu), dev_i32(cd), dev_i32(kept), dev_i32(keep), max(keep))
    assert h.hisa_device_status() == 0
    for a, b in zip(dst, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens,keep", MOVES + [([70000], [50001]), ([40000, 30000], [39999, 9])])
@pytest.mark.parametrize("which", ["all", "one"])
def test_rows_in_place(lens, keep, which):
    """All widths at once, and one narrow array (whose columns are split over clusters)."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(sum(keep) + 1))
    cu = regions(lens)
    kept = kept_of(lens, keep, cu, rng)
    src = arrays_of(int(cu[-1]), rng, max(lens) < 10000)[:8 if which == "all" else 1]
    want = [t.clone() for t in src]
    for s, k in enumerate(keep):
        at = torch.from_numpy(cu[s] + kept[cu[s]:cu[s] + k].astype(np.int64)).cuda()
        for a, b in zip(src, want):
            b[cu[s]:cu[s] + k] = a[at]
    c = dev_i32(cu)
    h.hisa_device_status(clear=True)
    h.hisa_evict_rows(src, src, c, c, dev_i32(kept), dev_i32(keep), max(keep))
    assert h.hisa_device_status() == 0
    for a, b in zip(src, want):
        assert torch.equal(a, b)


def test_rows_some_in_place_some_not():
    h = H()
    rng = np.random.Generator(np.random.PCG64(8))
    cu = regions([1000])
    kept = kept_of([1000], [600], cu, rng)
    a, b = arrays_of(int(cu[-1]), rng, False)[:2]
    a0, b2 = a.clone(), torch.zeros_like(b)
    c, at = dev_i32(cu), torch.from_numpy(kept[:600].astype(np.int64)).cuda()
    h.hisa_evict_rows([a, b], [a, b2], c, c, dev_i32(kept), dev_i32([600]), 1000)
    assert torch.equal(a[:600], a0[at]) and torch.equal(a[600:], a0[600:])
    assert torch.equal(b2[:600], b[at]) and int(b2[600:].abs().max()) == 0


def test_rows_bad_sequences_are_skipped():
    h = H()
    cu, cd = dev_i32([0, 256, 512, 768]), dev_i32([0, 128, 256, 384])
    kept = torch.arange(256, dtype=torch.int32, device="cuda").repeat(3)
    a = torch.arange(1, 769, dtype=torch.int32, device="cuda")

    def go(n, most, k=kept, d=cd):
        b = torch.zeros(int(d[-1]), dtype=torch.int32, device="cuda")
        h.hisa_evict_rows([a], [b], cu, d, k, dev_i32(n), most)
        return [int((b[d[s]:d[s + 1]] != 0).sum()) for s in range(3)], \
            h.hisa_device_status(clear=True)
    h.hisa_device_status(clear=True)
    assert go([3, 128, 128], 128) == ([3, 128, 128], 0)
    assert go([3, 129, 128], 200) == ([3, 0, 128], 1 << 7)
    assert go([3, -1, 128], 200) == ([3, 0, 128], 1 << 1)
    assert go([3, 100, 101], 100) == ([3, 100, 0], 1 << 1)
    assert go([3, 257, 5], 300, d=dev_i32([0, 300, 600, 900])) == ([3, 0, 5], 1 << 1)
    bad = kept.clone()
    bad[1], bad[257] = -3, 256
    assert go([3, 2, 1], 128, k=bad) == ([2, 1, 1], 1 << 1)
    # in place: regions that differ, rows that would move backwards
    b = a.clone()
    h.hisa_evict_rows([b], [b], cu, dev_i32([0, 256, 513, 768]), kept, dev_i32([3, 3, 3]), 3)
    assert h.hisa_device_status(clear=True) == 1 << 1 and torch.equal(a, b)
    back = kept.clone()
    back[:5] = torch.tensor([1, 2, 3, 2, 9], device="cuda")
    h.hisa_evict_rows([b], [b], cu, cu, back, dev_i32([5, 0, 0]), 5)
    assert h.hisa_device_status(clear=True) == 1 << 1
    assert b[:5].tolist() == [2, 3, 4, 4, 10] and torch.equal(b[5:], a[5:])


def test_binding_refusals():
    h = H()
    cu = dev_i32([0, 128])
    kept, n = torch.zeros(128, dtype=torch.int32, device="cuda"), dev_i32([1])
    a = torch.zeros(128, 4, dtype=torch.int32, device="cuda")
    big = torch.zeros(300, 4, dtype=torch.int32, device="cuda")
    for src, dst, what in (([a], [], "as many"), ([a], [a.long()], "type"),
                           ([a], [big[:, :2].contiguous()], "type"),
                           ([a[:, ::2]], [a[:, ::2]], "contiguous"),
                           ([big[:100]], [a], "source row"),
                           ([big[:128]], [big[64:192]], "overlaps a source"),
                           ([big[:128], a], [big[128:256], big[200:]], "destinations overlap"),
                           ([big[:128]], [big], "overlaps a source")):
        with pytest.raises(ValueError, match=what):
            h.hisa_evict_rows(src, dst, cu, cu, kept, n, 1)
    w = torch.zeros(128, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="budget"):
        h.hisa_evict_select(w, cu, None, dev_i32([1, 2]), 128, 0, 0)
    with pytest.raises(ValueError, match="kept"):
        h.hisa_evict_select(w, cu, None, n, 128, 0, 0, kept=kept[:5])
    with pytest.raises(ValueError, match="weights"):
        h.hisa_evict_select(w.int(), cu, None, n, 128, 0, 0)


def test_prefill_evict_decode():
    """The operators together, as a server runs them: two prompts are selected and attended
    over a 4-bit cache with the token weights, the cache is cut in place to a budget, the
    representatives are renewed, and decode steps go on in the smaller cache.  Every stage is
    compared with the plain definitions on the host's copy of the state."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(77))
    lens, m, topk, heads, scale = [900, 1400], 4, 256, 16, DIM ** -0.5
    S, budget, steps = 2, [512, 600], 3
    cu_k = regions(lens)
    rows = int(cu_k[-1])
    cu_q = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ck, n_live, cq = dev_i32(cu_k), dev_i32(lens), dev_i32(cu_q)
    ikeys = np.zeros((rows, 64))
    live = new_rows(lens, lens, cu_k)
    ikeys[live] = rng.integers(-4, 5, (len(live), 64))
    keys = bf16(ikeys)
    kv4 = torch.zeros(rows, 128, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(rows, 16, dtype=torch.uint8, device="cuda")
    w = torch.zeros(rows, dtype=torch.int64, device="cuda")
    pos = torch.from_numpy((np.arange(rows) - np.repeat(cu_k[:-1], np.diff(cu_k)))
                           .astype(np.int32)).cuda()
    h.hisa_device_status(clear=True)
    # prompt
    total = int(cu_q[-1])
    iq = bf16(rng.integers(-4, 5, (total, 64)))
    q = bf16(rng.standard_normal((total, heads, DIM)))
    k, v = bf16(rng.standard_normal((total, DIM))), bf16(rng.standard_normal((total, DIM)))
    reps = h.hisa_pool_blocks(keys, ck, n_live, max(lens))
    h.hisa_kv4_store(k, v, cq, ck, n_live, kv4, sc)
    idx = h.hisa_select(iq, keys, reps, cq, ck, n_live, max(lens), m, topk)
    lse = torch.empty(total, heads, device="cuda")
    out = h.hisa_sparse_attention_kv4(q, kv4, sc, idx, cq, ck, scale, lse=lse, weights=w)
    kr, vr = kv4_ref.values(kv4.cpu().numpy(), sc.cpu().numpy())
    ref = kv4_ref.Attention(f64(q), kr, vr, idx.cpu().numpy(), cu_q, cu_k,
                            np.float64(np.float32(scale)))
    ref.check_out(f64(out), np.abs(vr).max())
    ref.check_lse(f64(lse))
    ref.check_weights(w.cpu().numpy(), rows)
    # eviction in place
    before = [t.cpu().numpy().copy() for t in (keys.view(torch.int16), kv4, sc, w, pos)]
    kept, n_live = h.hisa_evict_select(w, ck, n_live, dev_i32(budget), max(lens), 4, 128)
    state = [keys, kv4, sc, w, pos]
    h.hisa_evict_rows(state, state, ck, ck, kept, n_live, max(budget))
    for s in range(S):
        c, n = int(cu_k[s]), budget[s]
        stay = kv4_ref.evict_select(before[3][c:c + lens[s]], lens[s], n, 4, 128)
        for x, t in zip(before, (keys.view(torch.int16), kv4, sc, w, pos)):
            assert np.array_equal(t.cpu().numpy()[c:c + n], x[c + stay])
    reps = h.hisa_pool_blocks(keys, ck, n_live, max(lens))
    # decode
    one = np.arange(S + 1, dtype=np.int32)
    d1 = dev_i32(one)
    for t in range(steps):
        iq1, ik1 = (bf16(rng.integers(-4, 5, (S, 64))) for _ in range(2))
        q1 = bf16(rng.standard_normal((S, heads, DIM)))
        k1, v1 = bf16(rng.standard_normal((S, DIM))), bf16(rng.standard_normal((S, DIM)))
        idx = h.hisa_decode_step(keys, reps, ck, n_live, ik1, iq1, max(lens), m, topk)
        h.hisa_kv4_store(k1, v1, d1, ck, n_live, kv4, sc)
        lse = torch.empty(S, heads, device="cuda")
        out = h.hisa_sparse_attention_kv4(q1, kv4, sc, idx, d1, ck, scale, lse=lse, weights=w)
        now = [b + t + 1 for b in budget]
        assert n_live.cpu().tolist() == now
        r_idx, _, _, _ = oracle.hisa(iq1.view(torch.int16).cpu().numpy().view(np.uint16),
                                  keys.view(torch.int16).cpu().numpy().view(np.uint16), one, cu_k,
                                  np.array(now, np.int32), 128, m, topk)
        assert np.array_equal(idx.cpu().numpy(), r_idx)
        kr, vr = kv4_ref.values(kv4.cpu().numpy(), sc.cpu().numpy())
        ref = kv4_ref.Attention(f64(q1), kr, vr, r_idx, one, cu_k, np.float64(np.float32(scale)))
        ref.check_out(f64(out), np.abs(vr).max())
        ref.check_lse(f64(lse))
    assert h.hisa_device_status() == 0


def test_kept_may_not_be_overwritten():
    h = H()
    cu = dev_i32([0, 128])
    kept, n = torch.arange(128, dtype=torch.int32, device="cuda"), dev_i32([1])
    for arrays in ([kept], [n]):
        with pytest.raises(ValueError, match="kept"):
            h.hisa_evict_rows([torch.zeros(128, dtype=torch.int32, device="cuda")], arrays, cu, cu,
                              kept, n, 1)


def test_lengths_past_the_limit_are_refused():
    h = H()
    w = torch.zeros(128, dtype=torch.int64, device="cuda")
    with pytest.raises(h.HisaError):
        h.hisa_evict_select(w, dev_i32([0, 128]), None, dev_i32([5]), (1 << 30) + 1, 0, 0)


@pytest.mark.parametrize("seqs,top", [(1, 40000), (3, 33000), (20, 17000), (100, 9000), (160, 700)])
def test_select_every_split_of_a_sequence(seqs, top):
    """One to eight CTAs per sequence, keys in registers or read again, odd lengths."""
    rng = np.random.Generator(np.random.PCG64(seqs))
    lens = (top - rng.integers(0, top // 2, seqs)).tolist()
    lens[0] = top
    keep = [int(rng.integers(0, n + 1)) for n in lens]
    cu_k = regions(lens)
    w = weights_of("real", int(cu_k[-1]), rng)
    w[: top // 3] //= 1 << 30  # ties in the first sequence
    kept, n = run_select(w, cu_k, lens, keep, 7, 100)
    for s, length in enumerate(lens):
        c, b = int(cu_k[s]), keep[s]
        sink = min(7, b)
        recent = min(100, b - sink)
        if length <= b:
            want = np.arange(length)
        else:
            x = w[c + sink:c + length - recent]
            free = np.argsort(-x, kind="stable")[:b - sink - recent] + sink
            want = np.sort(np.concatenate([np.arange(sink), free,
                                           np.arange(length - recent, length)]))
        assert n[s] == len(want) and np.array_equal(kept[c:c + len(want)], want)


def test_select_and_move_in_a_graph():
    """Captured once, replayed on changed weights and lengths."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(6))
    cu = regions([3000, 3000])
    rows = int(cu[-1])
    c, keep = dev_i32(cu), dev_i32([500, 700])
    w = torch.zeros(rows, dtype=torch.int64, device="cuda")
    lens, x = dev_i32([3000, 3000]), torch.zeros(rows, 8, dtype=torch.int32, device="cuda")
    kept = torch.zeros(rows, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")

    def step():
        h.hisa_evict_select(w, c, lens, keep, 3000, 4, 64, kept=kept, kept_len=n)
        h.hisa_evict_rows([x], [x], c, c, kept, n, 700)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        hw = weights_of("real", rows, rng)
        hl = rng.integers(300, 3001, 2)
        hx = rng.integers(0, 1 << 30, (rows, 8)).astype(np.int32)
        w.copy_(torch.from_numpy(hw))
        lens.copy_(torch.from_numpy(hl.astype(np.int32)))
        x.copy_(torch.from_numpy(hx))
        g.replay()
        torch.cuda.synchronize()
        for s in range(2):
            at = int(cu[s])
            want = kv4_ref.evict_select(hw[at:at + hl[s]], int(hl[s]), [500, 700][s], 4, 64)
            assert int(n[s]) == len(want)
            assert np.array_equal(x[at:at + len(want)].cpu().numpy(), hx[at + want])


def test_rows_with_the_largest_max_keep():
    """max_keep only has to be at least every count."""
    h = H()
    cu, kept = dev_i32([0, 256]), torch.arange(3, 259, dtype=torch.int32, device="cuda")
    a = torch.arange(256, dtype=torch.int32, device="cuda")
    for most in (2 ** 31 - 1, 2 ** 31 - 128):
        b = torch.zeros_like(a)
        h.hisa_device_status(clear=True)
        h.hisa_evict_rows([a], [b], cu, cu, kept, dev_i32([200]), most)
        assert h.hisa_device_status() == 0
        assert torch.equal(b[:200], a[3:203]) and not b[200:].any()
        b = a.clone()
        h.hisa_evict_rows([b], [b], cu, cu, kept, dev_i32([200]), most)
        assert h.hisa_device_status() == 0
        assert torch.equal(b[:200], a[3:203]) and torch.equal(b[200:], a[200:])


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("lens,keep", [([1500, 4097], [700, 4096]), ([70001], [30000]),
                                       ([150003], [50001])])
def test_select_weights_at_any_address(lens, keep, shift):
    """Regions that start at any row, weights aligned to 8 bytes only."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(shift + len(lens)))
    cu = (np.cumsum([0] + [n + 5 for n in lens]) + shift).astype(np.int32)
    for kind in ("real", "ties", "wide"):
        w = weights_of(kind, int(cu[-1]), rng)
        dev = torch.from_numpy(np.concatenate([[0], w]).astype(np.int64)).cuda()[1:]
        kept, n = h.hisa_evict_select(dev, dev_i32(cu), dev_i32(lens), dev_i32(keep), max(lens), 3,
                                      50)
        assert n.tolist() == keep
        for s, length in enumerate(lens):
            got = kept[cu[s]:cu[s] + keep[s]].cpu().numpy()
            want = kv4_ref.evict_select(w[cu[s]:cu[s] + length], length, keep[s], 3, 50)
            assert np.array_equal(got, want), (kind, s)

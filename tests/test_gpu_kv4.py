"""The 4-bit cache and the attention over it on the GPU, against the 64-bit reference of
kv4_ref.py (which derives the tolerances).  Storing and loading are exact."""

import math

import numpy as np
import pytest
import torch

import kv4_ref
from parity import dev_i32

pytestmark = pytest.mark.gpu

DIM = 128


def H():
    import sparse_attention_top_hisa_b200 as mod
    return mod


def bf16(x, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).to(device)


def f64(t):
    return t.double().cpu().numpy()


def layout(lens, news, spare=1):
    """Offsets of the query rows and of the regions, whole blocks and `spare` blocks more."""
    cu_q = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    cap = [(x // 128 + 1 + spare) * 128 for x in lens]
    return cu_q, np.concatenate([[0], np.cumsum(cap)]).astype(np.int32)


def new_rows(lens, news, cu_k):
    return np.concatenate([np.arange(c + x - n, c + x) for x, n, c in zip(lens, news, cu_k)]
                          + [np.zeros(0, int)]).astype(int)


def hard_rows(n, rng):
    """Rows whose groups go over the whole range: plain, tiny, huge, ties, zeros, one spike."""
    x = rng.standard_normal((n, 8, 16))
    kind = rng.integers(0, 8, (n, 8))
    x *= np.where(kind == 0, 1e-6, np.where(kind == 1, 3e-4, np.where(kind == 2, 1e5, 1.0)))[..., None]
    ties = rng.integers(-14, 15, (n, 8, 16)) / 2.0  # halves under scales that are powers of two
    ties[..., 0] = 7.0
    ties *= 2.0 ** rng.integers(-16, 9, (n, 8, 1))
    x = np.where((kind == 3)[..., None], ties, x)
    x = np.where((kind == 4)[..., None], 0.0, x)
    grid = kv4_ref.scale_grid()
    mid = 7 * (grid[:-1] + grid[1:]) / 2  # borders between scales
    spike = np.zeros((n, 8, 16))
    spike[..., 3] = mid[rng.integers(0, len(mid), (n, 8))]
    spike[..., 5] = -spike[..., 3] / 4
    x = np.where((kind == 5)[..., None], spike, x)
    x = np.where((kind == 6)[..., None], x * 2.0 ** rng.integers(-140, 100, (n, 8, 1)), x)
    return x.reshape(n, DIM)


@pytest.mark.parametrize("lens,news", [
    ([1], [1]), ([300], [300]), ([5, 0, 129, 4096], [1, 0, 129, 17]), ([700, 701], [0, 333]),
    ([130] * 33, [1] * 33)])
def test_store_and_load_exactly(lens, news):
    h = H()
    rng = np.random.Generator(np.random.PCG64(len(lens) * 100 + sum(news)))
    cu_q, cu_k = layout(lens, news)
    n, rows = int(cu_q[-1]), int(cu_k[-1])
    k, v = bf16(hard_rows(n, rng)), bf16(hard_rows(n, rng))
    kv4 = torch.full((rows, 128), 0xA5, dtype=torch.uint8, device="cuda")
    sc = torch.full((rows, 16), 0x5A, dtype=torch.uint8, device="cuda")
    args = dev_i32(cu_q), dev_i32(cu_k), dev_i32(lens)
    h.hisa_device_status(clear=True)
    h.hisa_kv4_store(k, v, *args, kv4, sc)
    kb, vb = h.hisa_kv4_load(kv4, sc, *args, n)
    assert h.hisa_device_status() == 0
    codes, scales = kv4_ref.pack(*kv4_ref.quantise(f64(k)), *kv4_ref.quantise(f64(v)))
    want = np.full((rows, 128), 0xA5, np.uint8), np.full((rows, 16), 0x5A, np.uint8)
    at = new_rows(lens, news, cu_k)
    want[0][at], want[1][at] = codes, scales
    assert np.array_equal(sc.cpu().numpy(), want[1])
    assert np.array_equal(kv4.cpu().numpy(), want[0])  # rows of no new token as they were
    kr, vr = kv4_ref.values(codes, scales)
    assert np.array_equal(f64(kb), kr) and np.array_equal(f64(vb), vr)


def test_not_finite_groups_are_marked():
    h = H()
    rng = np.random.Generator(np.random.PCG64(3))
    x = rng.standard_normal((4, DIM))
    x[0, 17], x[1, 100], x[2, 0] = np.inf, np.nan, -np.inf
    k, v = bf16(x), bf16(rng.standard_normal((4, DIM)))
    kv4 = torch.zeros(256, 128, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(256, 16, dtype=torch.uint8, device="cuda")
    args = dev_i32([0, 4]), dev_i32([0, 256]), dev_i32([4])
    h.hisa_device_status(clear=True)
    h.hisa_kv4_store(k, v, *args, kv4, sc)
    assert h.hisa_device_status(clear=True) == 1 << 1
    kb, vb = h.hisa_kv4_load(kv4, sc, *args, 4)
    codes, scales = kv4_ref.pack(*kv4_ref.quantise(f64(k)), *kv4_ref.quantise(f64(v)))
    kr, vr = kv4_ref.values(codes, scales)
    assert np.isnan(kr).sum() == 48
    assert np.array_equal(f64(kb), kr, equal_nan=True) and np.array_equal(f64(vb), vr)


def test_bad_sequences_are_skipped():
    """A length beyond its region, more query rows than tokens, an unaligned region."""
    h = H()
    x = bf16(np.ones((6, DIM)))
    for cu_k, lens, cu_q, bit in (([0, 128, 256], [200, 5], [0, 2, 6], 1),
                                  ([0, 128, 256], [1, 5], [0, 2, 6], 1),
                                  ([0, 100, 256], [5, 5], [0, 2, 6], 2)):
        kv4 = torch.zeros(256, 128, dtype=torch.uint8, device="cuda")
        sc = torch.zeros(256, 16, dtype=torch.uint8, device="cuda")
        args = dev_i32(cu_q), dev_i32(cu_k), dev_i32(lens)
        h.hisa_device_status(clear=True)
        h.hisa_kv4_store(x, x, *args, kv4, sc)
        kb, _ = h.hisa_kv4_load(kv4, sc, *args, 6)
        assert h.hisa_device_status(clear=True) == 1 << bit
        good = [1 if bit == 1 else 0]
        want = np.zeros(6)
        s = good[0]
        want[cu_q[s]:cu_q[s + 1]] = 1
        assert np.array_equal((f64(kb) != 0).any(1), want.astype(bool))
        assert (sc.cpu().numpy() != 0).any(1).sum() == want.sum()


class Case:
    """A cache of random rows, queries and indices, on the host and on the GPU."""

    def __init__(self, seed, heads, topk, lens, news, scale=0.09, q_gain=1.0, idx=None,
                 empty=4):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.heads, self.scale = heads, scale
        self.cu_q, self.cu_k = layout(lens, news)
        n, rows = int(self.cu_q[-1]), int(self.cu_k[-1])
        gain = np.exp(rng.standard_normal((2, DIM)) * 0.5)
        k = kv4_ref.quantise(f64(bf16(rng.standard_normal((rows, DIM)) * gain[0], "cpu")))
        v = kv4_ref.quantise(f64(bf16(rng.standard_normal((rows, DIM)) * gain[1], "cpu")))
        self.codes, self.scales = kv4_ref.pack(*k, *v)
        self.q = bf16(rng.standard_normal((n, heads, DIM)) * q_gain)
        if idx is None:
            idx = np.full((n, topk), -1, np.int32)
            for s, length in enumerate(lens):
                for r in range(int(self.cu_q[s]), int(self.cu_q[s + 1])):
                    if empty and r % empty == empty - 1:
                        continue  # a row with no index
                    m = int(rng.integers(1, min(topk, length) + 1)) if r % 3 else min(topk, length)
                    idx[r, rng.choice(topk, m, replace=False)] = rng.choice(length, m,
                                                                            replace=False)
        self.idx = idx
        self.rows = rows

    def ref(self):
        self.k, self.v = kv4_ref.values(self.codes, self.scales)
        return kv4_ref.Attention(f64(self.q), self.k, self.v, self.idx, self.cu_q, self.cu_k,
                                 np.float32(self.scale).astype(np.float64))

    def run(self, weights=False, out=None):
        h = H()
        n = len(self.idx)
        out = torch.full((n, self.heads, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, self.heads), 7.0, dtype=torch.float32, device="cuda")
        w = torch.zeros(self.rows, dtype=torch.int64, device="cuda") if weights else None
        h.hisa_sparse_attention_kv4(self.q, torch.from_numpy(self.codes).cuda(),
                                    torch.from_numpy(self.scales).cuda(), dev_i32(self.idx),
                                    dev_i32(self.cu_q), dev_i32(self.cu_k), self.scale, out=out,
                                    lse=lse, weights=w)
        torch.cuda.synchronize()
        return f64(out), f64(lse), None if w is None else w.cpu().numpy()

    def check(self, weights=True):
        h = H()
        h.hisa_device_status(clear=True)
        out, lse, w = self.run(weights)
        assert h.hisa_device_status() == 0
        ref = self.ref()
        ref.check_lse(lse)
        ref.check_out(out, np.abs(self.v).max())
        assert np.all(out[np.isinf(ref.lse)] == 0)
        if weights:
            ref.check_weights(w, self.rows)
        return out, lse, w


@pytest.mark.parametrize("heads", [1, 3, 8, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("topk", [1, 33, 500])
def test_attention_heads(heads, topk):
    Case(heads * 1000 + topk, heads, topk, [600, 1500], [5, 6]).check()


@pytest.mark.parametrize("topk", [7, 31, 32, 64, 127, 128, 129, 256, 257, 1000, 1024, 2048, 4500])
def test_attention_lengths_of_the_index_row(topk):
    """Every split of a row over warps and CTAs, for few queries."""
    Case(topk, 16, topk, [4600], [3], empty=3).check()


@pytest.mark.parametrize("heads,topk,news", [(16, 300, [200, 1, 219]), (32, 130, [400, 0, 7]),
                                             (5, 64, [80, 80, 80]), (20, 40, [90, 91, 92])])
def test_attention_many_rows(heads, topk, news):
    Case(heads + topk, heads, topk, [700, 130, 900], news).check()


@pytest.mark.parametrize("lens", [[1], [1, 2, 3], [128], [129]])
def test_attention_shortest_sequences(lens):
    Case(len(lens), 4, 16, lens, [1] * len(lens), empty=0).check()


def test_attention_repeated_indices():
    """The same index several times in a row counts that often, as in the bf16 attention."""
    rng = np.random.Generator(np.random.PCG64(5))
    idx = rng.integers(0, 20, (7, 200)).astype(np.int32)
    Case(6, 12, 200, [300], [7], idx=idx).check()


@pytest.mark.parametrize("q_gain", [0.0, 1e-30, 2.0 ** -120, 1e-3, 30.0])
def test_attention_query_magnitudes(q_gain):
    Case(9, 10, 100, [400], [6], q_gain=q_gain).check()


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-20])
def test_attention_scales(scale):
    Case(11, 10, 100, [400], [6], scale=scale).check()


@pytest.mark.parametrize("order", ["rising", "falling", "shuffled"])
@pytest.mark.parametrize("heads,nq", [(8, 1), (20, 1), (8, 150), (20, 150)])
def test_attention_score_ramp(order, heads, nq):
    """Scores that climb by about 200 nats over the row: the reference maximum is raised
    again and again, or the later weights vanish."""
    c = Case(heads + nq, heads, 2048, [2048], [nq], scale=1.0, empty=0,
             idx=np.tile(np.arange(2048, dtype=np.int32), (nq, 1)))
    rng = np.random.Generator(np.random.PCG64(nq))
    u = rng.standard_normal(DIM)
    u /= np.linalg.norm(u)
    k = np.zeros((c.rows, DIM))
    k[:2048] = np.outer(np.arange(2048) * (200.0 / 2048 / 15.0), u)
    c.codes, c.scales = kv4_ref.pack(*kv4_ref.quantise(f64(bf16(k, "cpu"))),
                                     *kv4_ref.quantise(f64(bf16(rng.standard_normal(k.shape),
                                                                "cpu"))))
    c.q = bf16(np.broadcast_to(15.0 * u, (nq, heads, DIM))
               * rng.uniform(0.5, 1.0, (nq, heads, 1)))
    if order == "falling":
        c.idx = c.idx[:, ::-1].copy()
    elif order == "shuffled":
        c.idx = np.stack([rng.permutation(2048) for _ in range(nq)]).astype(np.int32)
    c.check()


def test_attention_index_outside_the_region_is_reported():
    h = H()
    c = Case(21, 3, 4, [100], [2], idx=np.array([[0, 5, 300, -1], [7, -2, -1, 1]], np.int32))
    assert c.rows == 256
    h.hisa_device_status(clear=True)
    out, lse, w = c.run(True)
    assert h.hisa_device_status(clear=True) == 1 << 1
    c.idx = np.array([[0, 5, -1, -1], [7, -1, -1, 1]], np.int32)  # the entry is ignored
    ref = c.ref()
    ref.check_lse(lse)
    ref.check_out(out, np.abs(c.v).max())
    ref.check_weights(w, c.rows)


def test_attention_infinities_stay_in_their_rows():
    """An infinity or a NaN in a query's head, or in a selected row's group, makes exactly
    those outputs NaN; rows that nobody selects may hold anything."""
    c = Case(22, 18, 64, [400], [9], empty=0)
    q = c.q.float()
    q[3, 2, 7], q[5, 17, 100] = float("inf"), float("nan")
    c.q = q.to(torch.bfloat16)
    picked = np.unique(c.idx[c.idx >= 0])
    other = np.setdiff1d(np.arange(c.rows), picked)
    c.scales[other] = 255  # NaN
    h = H()
    h.hisa_device_status(clear=True)
    out, lse, w = c.run(False)
    bad = np.zeros(out.shape[:2], bool)
    bad[3, 2] = bad[5, 17] = True
    assert np.isnan(out[bad]).all() and not np.isnan(out[~bad]).any()
    assert np.isnan(lse[bad]).all() and not np.isnan(lse[~bad]).any()
    # with weights: the poisoned rows add nothing for the poisoned queries, and say so
    _, _, w = c.run(True)
    assert h.hisa_device_status(clear=True) == 1 << 1
    assert (w[other] == 0).all() and w.min() >= 0
    # a poisoned value group: its 16 dimensions of every row that selects it
    c = Case(23, 4, 40, [300], [6], empty=0)
    j = int(c.idx[0][c.idx[0] >= 0][0])
    c.scales[j, 8 + 2] = 255
    out, lse, _ = c.run(False)
    hit = (c.idx == j).any(1)
    assert np.isnan(out[hit][:, :, 32:48]).all() and not np.isnan(lse).any()
    assert not np.isnan(out[hit][:, :, :32]).any() and not np.isnan(out[~hit]).any()


def test_weights_add_up_and_repeat_bit_for_bit():
    """Accumulation into what is there; the same bits on every run; the total is the number
    of heads for every row with an index."""
    h = H()
    c = Case(31, 16, 300, [900, 300], [150, 90])
    _, _, w1 = c.run(True)
    _, _, w2 = c.run(True)
    assert np.array_equal(w1, w2)
    rows = (c.idx >= 0).any(1).sum()
    entries = (c.idx >= 0).sum()
    assert abs(w1.sum() * 2.0 ** -32 - rows * 16) <= rows * 16 * 2.0 ** -11 + entries * 2.0 ** -33
    dev = [torch.from_numpy(x).cuda() for x in (c.codes, c.scales)]
    w = torch.from_numpy(w1).cuda()
    lse = torch.empty(len(c.idx), 16, device="cuda")
    h.hisa_sparse_attention_kv4(c.q, *dev, dev_i32(c.idx), dev_i32(c.cu_q), dev_i32(c.cu_k),
                                c.scale, lse=lse, weights=w)
    assert np.array_equal(w.cpu().numpy(), 2 * w1)


@pytest.mark.parametrize("heads,topk,news", [(1, 5, [3, 2]), (16, 700, [60, 3]),
                                             (17, 100, [1, 1]), (32, 65, [300, 200])])
def test_token_weights_of_the_bf16_cache(heads, topk, news):
    h = H()
    c = Case(heads * 7 + topk, heads, topk, [800, 500], news)
    rng = np.random.Generator(np.random.PCG64(heads))
    k, v = bf16(rng.standard_normal((c.rows, DIM))), bf16(rng.standard_normal((c.rows, DIM)))
    idx, cu_q, cu_k = dev_i32(c.idx), dev_i32(c.cu_q), dev_i32(c.cu_k)
    lse = torch.empty(len(c.idx), heads, device="cuda")
    h.hisa_device_status(clear=True)
    h.hisa_sparse_attention(c.q, k, v, idx, cu_q, cu_k, c.scale, lse=lse)
    w = torch.zeros(c.rows, dtype=torch.int64, device="cuda")
    h.hisa_token_weights(c.q, k, idx, lse, cu_q, cu_k, c.scale, w)
    assert h.hisa_device_status() == 0
    ref = kv4_ref.Attention(f64(c.q), f64(k), None, c.idx, c.cu_q, c.cu_k,
                            np.float32(c.scale).astype(np.float64))
    ref.check_weights(w.cpu().numpy(), c.rows)
    # an index outside the region is ignored and reported
    bad = c.idx.copy()
    at = np.argwhere(bad[0] >= 0)[0]
    bad[0, at] = 1 << 20
    w2 = torch.zeros_like(w)
    h.hisa_token_weights(c.q, k, dev_i32(bad), lse, cu_q, cu_k, c.scale, w2)
    assert h.hisa_device_status(clear=True) == 1 << 1
    assert int((w - w2).sum()) > 0


def test_rows_past_32_bits():
    """A cache of more than 2^32 bytes: rows on both sides of the border."""
    h = H()
    rows = (1 << 25) + 4096
    kv4 = torch.zeros(rows, 128, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(rows, 16, dtype=torch.uint8, device="cuda")
    w = torch.zeros(rows, dtype=torch.int64, device="cuda")
    cu_q, cu_k, lens = dev_i32([0, 64]), dev_i32([0, rows]), dev_i32([rows - 7])
    rng = np.random.Generator(np.random.PCG64(41))
    k, v = bf16(rng.standard_normal((64, DIM))), bf16(rng.standard_normal((64, DIM)))
    h.hisa_device_status(clear=True)
    h.hisa_kv4_store(k, v, cu_q, cu_k, lens, kv4, sc)
    kb, vb = h.hisa_kv4_load(kv4, sc, cu_q, cu_k, lens, 64)
    assert torch.equal(kb, h.hisa_kv4_load(kv4[-4096:].contiguous(), sc[-4096:].contiguous(),
                                           cu_q, dev_i32([0, 4096]), dev_i32([4096 - 7]), 64)[0])
    heads = 16
    q = bf16(rng.standard_normal((64, heads, DIM)))
    local = np.stack([rng.permutation(64)[:50] for _ in range(64)]) + 4096 - 7 - 64
    args = q, kv4, sc
    lse = torch.empty(64, heads, device="cuda")
    out = h.hisa_sparse_attention_kv4(*args, dev_i32(local + rows - 4096), cu_q, cu_k, 0.1,
                                      lse=lse, weights=w)
    lse2, w2 = torch.empty_like(lse), torch.zeros(4096, dtype=torch.int64, device="cuda")
    out2 = h.hisa_sparse_attention_kv4(q, kv4[-4096:].contiguous(), sc[-4096:].contiguous(),
                                       dev_i32(local), cu_q, dev_i32([0, 4096]), 0.1, lse=lse2,
                                       weights=w2)
    assert h.hisa_device_status() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert torch.equal(w[-4096:], w2) and int(w[:-4096].abs().max()) == 0


def test_other_stream_and_graphs():
    """Eager calls on a side stream, and two captured graphs replayed in turn, give the bits
    of the plain call."""
    h = H()
    c = Case(51, 16, 600, [1000, 1000], [1, 1], empty=0)
    out0, lse0, w0 = c.run(True)
    dev = [torch.from_numpy(x).cuda() for x in (c.codes, c.scales)]
    idx, cu_q, cu_k = dev_i32(c.idx), dev_i32(c.cu_q), dev_i32(c.cu_k)
    lens = dev_i32([1000, 1000])
    k, v = bf16(np.ones((2, DIM))), bf16(np.ones((2, DIM)))
    side = torch.cuda.Stream()
    bufs = [(torch.empty(2, 16, DIM, dtype=torch.bfloat16, device="cuda"),
             torch.empty(2, 16, device="cuda"),
             torch.zeros(c.rows, dtype=torch.int64, device="cuda")) for _ in range(3)]

    def step(b, cache):
        h.hisa_kv4_store(k, v, cu_q, cu_k, lens, *cache)
        h.hisa_sparse_attention_kv4(c.q, *dev, idx, cu_q, cu_k, c.scale, out=b[0], lse=b[1],
                                    weights=b[2])
    spare = [torch.zeros_like(x) for x in dev]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(bufs[0], spare)
    side.synchronize()
    graphs = []
    for b in bufs[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b, spare)
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for i, b in enumerate(bufs):
        assert np.array_equal(f64(b[0]), out0) and np.array_equal(f64(b[1]), lse0)
        assert np.array_equal(b[2].cpu().numpy(), w0 * (2 if i else 1))


def test_binding_refusals():
    h = H()
    c = Case(61, 4, 8, [100], [2])
    dev = [torch.from_numpy(x).cuda() for x in (c.codes, c.scales)]
    idx, cu_q, cu_k = dev_i32(c.idx), dev_i32(c.cu_q), dev_i32(c.cu_k)
    ok = dict(q_att=c.q, kv4=dev[0], kv4_scale=dev[1], topk_idx=idx, cu_seqlens_q=cu_q,
              cu_seqlens_k=cu_k, scale=0.1)
    w = torch.zeros(c.rows, dtype=torch.int64, device="cuda")
    lse = torch.empty(2, 4, device="cuda")
    for change, what in ((dict(q_att=c.q.half()), "q_att"), (dict(q_att=c.q[:1]), "topk_idx"),
                         (dict(kv4=dev[0][:, :64].contiguous()), "kv4"),
                         (dict(kv4_scale=dev[1][:-1]), "rows"), (dict(topk_idx=idx.long()), "topk"),
                         (dict(topk_idx=idx.t()), "topk_idx"), (dict(weights=w), "lse"),
                         (dict(weights=w[:-1], lse=lse), "weights"),
                         (dict(weights=w.int(), lse=lse), "weights"),
                         (dict(lse=lse[:, :3].contiguous()), "lse"),
                         (dict(out=c.q.float()), "out"), (dict(out=c.q[:, :2].contiguous()), "out"),
                         (dict(cu_seqlens_k=dev_i32([0, 128, 256])), "sequences"),
                         (dict(cu_seqlens_k=cu_k.cpu()), "CUDA")):
        with pytest.raises(ValueError, match=what):
            h.hisa_sparse_attention_kv4(**{**ok, **change})
    with pytest.raises(h.HisaError):
        h.hisa_sparse_attention_kv4(**{**ok, "scale": math.nan})
    with pytest.raises(ValueError, match="same shape"):
        h.hisa_kv4_store(bf16(np.ones((2, DIM))), bf16(np.ones((3, DIM))), cu_q, cu_k, None, *dev)
    with pytest.raises(ValueError, match="sequences"):
        h.hisa_kv4_load(*dev, cu_q, cu_k, dev_i32([1, 2]), 2)


@pytest.mark.parametrize("seqs", [31, 33, 129, 700])
def test_many_sequences(seqs):
    """Rows find their sequence among many, empty ones and ones without queries among them."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(seqs))
    lens = rng.integers(0, 60, seqs)
    news = [int(rng.integers(0, min(4, n) + 1)) if n else 0 for n in lens]
    lens[-1], news[-1] = 40, 0
    c = Case(seqs, 6, 24, lens.tolist(), news, empty=5)
    c.check()
    cu_q, cu_k, n = c.cu_q, c.cu_k, int(c.cu_q[-1])
    k, v = bf16(hard_rows(n, rng)), bf16(hard_rows(n, rng))
    kv4 = torch.zeros(c.rows, 128, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(c.rows, 16, dtype=torch.uint8, device="cuda")
    args = dev_i32(cu_q), dev_i32(cu_k), dev_i32(lens)
    h.hisa_device_status(clear=True)
    h.hisa_kv4_store(k, v, *args, kv4, sc)
    kb, vb = h.hisa_kv4_load(kv4, sc, *args, n)
    assert h.hisa_device_status() == 0
    codes, scales = kv4_ref.pack(*kv4_ref.quantise(f64(k)), *kv4_ref.quantise(f64(v)))
    at = new_rows(lens.tolist(), news, cu_k)
    assert np.array_equal(kv4.cpu().numpy()[at], codes)
    assert np.array_equal(sc.cpu().numpy()[at], scales)
    assert int((sc.cpu().numpy() != 0).any(1).sum()) <= n
    kr, vr = kv4_ref.values(codes, scales)
    assert np.array_equal(f64(kb), kr) and np.array_equal(f64(vb), vr)
    # the bf16 token weights look their rows up the same way
    keys = bf16(rng.standard_normal((c.rows, DIM)))
    lse = torch.empty(n, 6, device="cuda")
    h.hisa_sparse_attention(c.q, keys, keys, dev_i32(c.idx), args[0], args[1], c.scale, lse=lse)
    w = torch.zeros(c.rows, dtype=torch.int64, device="cuda")
    h.hisa_token_weights(c.q, keys, dev_i32(c.idx), lse, args[0], args[1], c.scale, w)
    ref = kv4_ref.Attention(f64(c.q), f64(keys), None, c.idx, cu_q, cu_k,
                            np.float64(np.float32(c.scale)))
    ref.check_weights(w.cpu().numpy(), c.rows)


@pytest.mark.parametrize("rows", [1183, 4800, 9473])
def test_store_many_rows(rows):
    """Enough rows for several per thread, in a chunk that ends anywhere: the last warp is
    part empty, two sequences meet inside one."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(rows))
    lens, news = [rows, 700], [rows - 333, 333]
    cu_q, cu_k = layout(lens, news)
    k, v = bf16(hard_rows(rows, rng)), bf16(hard_rows(rows, rng))
    kv4 = torch.full((int(cu_k[-1]), 128), 7, dtype=torch.uint8, device="cuda")
    sc = torch.full((int(cu_k[-1]), 16), 7, dtype=torch.uint8, device="cuda")
    args = dev_i32(cu_q), dev_i32(cu_k), dev_i32(lens)
    h.hisa_kv4_store(k, v, *args, kv4, sc)
    kb, vb = h.hisa_kv4_load(kv4, sc, *args, rows)
    codes, scales = kv4_ref.pack(*kv4_ref.quantise(f64(k)), *kv4_ref.quantise(f64(v)))
    want = np.full((int(cu_k[-1]), 128), 7, np.uint8), np.full((int(cu_k[-1]), 16), 7, np.uint8)
    at = new_rows(lens, news, cu_k)
    want[0][at], want[1][at] = codes, scales
    assert np.array_equal(kv4.cpu().numpy(), want[0]) and np.array_equal(sc.cpu().numpy(), want[1])
    kr, vr = kv4_ref.values(codes, scales)
    assert np.array_equal(f64(kb), kr) and np.array_equal(f64(vb), vr)


@pytest.mark.parametrize("heads,rows,topk", [(16, 7000, 40), (9, 1500, 150), (32, 5000, 33),
                                             (20, 900, 260)])
def test_attention_one_warp_per_row(heads, rows, topk):
    """Row counts at which a warp has a row to itself, not a multiple of a CTA's warps; a
    sample of the rows against the reference, the weights' total over all."""
    rng = np.random.Generator(np.random.PCG64(rows))
    length = 900
    idx = np.argsort(rng.random((rows, length)), 1)[:, :topk].astype(np.int32)
    idx[rng.random(idx.shape) < 0.1] = -1
    idx[5] = -1
    c = Case(rows, heads, topk, [length + rows], [rows], idx=idx)
    h = H()
    h.hisa_device_status(clear=True)
    out, lse, w = c.run(True)
    assert h.hisa_device_status() == 0
    k, v = kv4_ref.values(c.codes, c.scales)
    pick = np.unique(np.concatenate([np.arange(9), np.arange(rows - 9, rows),
                                     rng.integers(0, rows, 60)]))
    ref = kv4_ref.Attention(f64(c.q)[pick], k, v, idx[pick], np.array([0, len(pick)]), c.cu_k,
                            np.float64(np.float32(c.scale)))
    ref.check_out(out[pick], np.abs(v).max())
    ref.check_lse(lse[pick])
    n = (idx >= 0).any(1).sum()
    assert abs(w.sum() * 2.0 ** -32 - n * heads) <= \
        n * heads * 2.0 ** -11 + (idx >= 0).sum() * 2.0 ** -33
    out2, lse2, w2 = c.run(True)
    assert np.array_equal(w, w2) and np.array_equal(out, out2)
    out3, _, _ = c.run(False)  # without weights: another kernel, the same values
    assert np.array_equal(out, out3)


def test_calls_on_two_streams_add_to_one_accumulator():
    h = H()
    c = Case(71, 16, 300, [900], [64], empty=0)
    _, _, w1 = c.run(True)
    dev = [torch.from_numpy(x).cuda() for x in (c.codes, c.scales)]
    idx, cu_q, cu_k = dev_i32(c.idx), dev_i32(c.cu_q), dev_i32(c.cu_k)
    w = torch.zeros(c.rows, dtype=torch.int64, device="cuda")
    lse = [torch.empty(64, 16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x in zip(streams, lse):
            with torch.cuda.stream(s):
                h.hisa_sparse_attention_kv4(c.q, *dev, idx, cu_q, cu_k, c.scale, lse=x, weights=w)
    torch.cuda.synchronize()
    assert np.array_equal(w.cpu().numpy(), 10 * w1)


def test_empty_calls():
    h = H()
    c = Case(81, 4, 8, [100], [2])
    dev = [torch.from_numpy(x).cuda() for x in (c.codes, c.scales)]
    cu_k, none = dev_i32(c.cu_k), dev_i32([0, 0])
    q = torch.empty(0, 4, DIM, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(0, 8, dtype=torch.int32, device="cuda")
    x = torch.empty(0, DIM, dtype=torch.bfloat16, device="cuda")
    assert h.hisa_sparse_attention_kv4(q, *dev, idx, none, cu_k, 0.1).shape == (0, 4, DIM)
    h.hisa_kv4_store(x, x, none, cu_k, dev_i32([100]), *dev)
    assert h.hisa_kv4_load(*dev, none, cu_k, dev_i32([100]), 0)[0].shape == (0, DIM)
    with pytest.raises(h.HisaError):  # no entry per row at all
        h.hisa_sparse_attention_kv4(c.q, *dev, dev_i32(np.zeros((2, 0))), dev_i32(c.cu_q), cu_k,
                                    0.1)


@pytest.mark.parametrize("heads,topk,news", [(16, 300, [3, 2]), (16, 40, [3000, 2]),
                                             (20, 300, [3, 2]), (20, 40, [3000, 2])])
def test_rows_behind_the_last_sequence_add_nothing(heads, topk, news):
    """A padded batch: rows past cu_seqlens_q[S] have no tokens, whatever their indices say."""
    h = H()
    pad = 7
    c = Case(heads + topk, heads, topk, [4000, 500], news)
    n = len(c.idx)
    rng = np.random.Generator(np.random.PCG64(5))
    k, v = bf16(rng.standard_normal((c.rows, DIM))), bf16(rng.standard_normal((c.rows, DIM)))
    q = torch.cat([c.q, c.q[:pad - 2], c.q[:2]])
    dev = [torch.from_numpy(x).cuda() for x in (c.codes, c.scales)]
    cu_q, cu_k = dev_i32(c.cu_q), dev_i32(c.cu_k)
    want, _, want_w = c.check()
    lse_bf = torch.empty(n, heads, device="cuda")
    h.hisa_sparse_attention(c.q, k, v, dev_i32(c.idx), cu_q, cu_k, c.scale, lse=lse_bf)
    want_tw = torch.zeros(c.rows, dtype=torch.int64, device="cuda")
    h.hisa_token_weights(c.q, k, dev_i32(c.idx), lse_bf, cu_q, cu_k, c.scale, want_tw)
    for fill, status in ((-1, 0), (3, 1 << 1)):
        idx = dev_i32(np.concatenate([c.idx, np.full((pad, topk), fill, np.int32)]))
        h.hisa_device_status(clear=True)
        lse = torch.empty(n + pad, heads, device="cuda")
        w = torch.zeros(c.rows, dtype=torch.int64, device="cuda")
        out = h.hisa_sparse_attention_kv4(q, *dev, idx, cu_q, cu_k, c.scale, lse=lse, weights=w)
        assert h.hisa_device_status(clear=True) == status
        assert np.array_equal(f64(out[:n]), want) and not out[n:].any()
        assert np.array_equal(w.cpu().numpy(), want_w) and torch.isneginf(lse[n:]).all()
        tw = torch.zeros_like(w)
        lse_pad = torch.cat([lse_bf, torch.ones(pad, heads, device="cuda")])
        h.hisa_token_weights(q, k, idx, lse_pad, cu_q, cu_k, c.scale, tw)
        assert h.hisa_device_status(clear=True) == status
        assert torch.equal(tw, want_tw)


@pytest.mark.parametrize("heads", [1, 2, 5, 7, 16, 17, 31, 32])
@pytest.mark.parametrize("rows,topk", [(1, 2048), (3, 1000), (20, 2048), (70, 512)])
def test_attention_rows_over_clusters(heads, rows, topk):
    """Every number of CTAs of a row, with fewer heads than CTAs and heads that do not divide
    among them; some rows without an index, and some whose first CTAs have none."""
    c = Case(3 * heads + rows, heads, topk, [3000, 2500], [(rows + 1) // 2, rows // 2],
             empty=5)
    c.idx[0, :topk * 3 // 4] = -1
    c.check()
    c.check(weights=False)

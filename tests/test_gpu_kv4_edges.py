"""Edges of the 4-bit cache on the GPU: small softmax weights beside a large one of no value,
rows behind the last sequence, scale bytes that the store does not write."""

import numpy as np
import pytest
import torch

import kv4_ref
from parity import dev_i32
from test_gpu_kv4 import DIM, H, bf16, f64, hard_rows, layout, new_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nats", [12.0, 17.4, 19.0])
@pytest.mark.parametrize("heads", [8, 20])
@pytest.mark.parametrize("rows", [1, 40, 1500])
def test_small_weights_beside_a_sink_of_no_value(nats, heads, rows):
    """A first token whose score lies far above all others' and whose value is zero: the output
    is the others', however small their weights are beside its own.

    A weight enters the value product as fp16, taken against a reference under which the largest
    weight of its share is at least 2^7: it is off by 2^-11 of itself or by 2^-25, half the
    smallest fp16 number, so n of them by n 2^-32 of the largest value after the division by the
    sum.  The rest of the tolerance is that of Attention.check_out."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(int(nats * 10) + heads + rows))
    length, topk, cap = 2100, 2048, 2176
    k = np.zeros((cap, DIM))
    k[0, 0] = 7.0  # held exactly: scale 1, q = 7
    v = rng.uniform(1.0, 2.0, (cap, DIM))
    v[0] = 0.0
    codes, scales = kv4_ref.pack(*kv4_ref.quantise(k), *kv4_ref.quantise(f64(bf16(v, "cpu"))))
    q = np.zeros((rows, heads, DIM))
    q[:, :, 0] = 1.0
    scale = nats / 7.0
    picked = [rng.permutation(np.arange(1, length))[:topk - 1] for _ in range(min(rows, 40))]
    idx = np.stack([np.insert(picked[r % len(picked)], r * 37 % topk, 0) for r in range(rows)]) \
        .astype(np.int32)
    lse = torch.empty(rows, heads, device="cuda")
    w = torch.zeros(cap, dtype=torch.int64, device="cuda")
    args = (bf16(q), torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
            dev_i32(idx), dev_i32([0, rows]), dev_i32([0, cap]), scale)
    outs = [h.hisa_sparse_attention_kv4(*args),
            h.hisa_sparse_attention_kv4(*args, lse=lse, weights=w)]
    kr, vr = kv4_ref.values(codes, scales)
    n = min(rows, 40)
    ref = kv4_ref.Attention(q[:n], kr, vr, idx[:n], [0, n], [0, cap],
                            np.float64(np.float32(scale)))
    rel = 2.0 ** -11 + 2 * ref.score_error() + topk * 2.0 ** -22
    tol = 2.0 ** -8 * np.abs(ref.out) + rel[..., None] * ref.spread * (1 + 2.0 ** -8) \
        + topk * 2.0 ** -32 * np.abs(vr).max() * (1 + 2.0 ** -7)
    assert tol.max() < ref.out.min() / 6  # the weights of this test are within its reach
    for out in outs:
        err = np.abs(f64(out[:n]) - ref.out)
        assert np.all(err <= tol), float((err / ref.out).max())
    ref.check_lse(f64(lse[:n]))


@pytest.mark.parametrize("news,pad", [([1, 1, 1], 5), ([3, 0, 2], 3), ([40, 0, 1], 1),
                                      ([0, 0, 0], 4), ([5000, 300, 7], 777)])
def test_store_and_load_pass_over_rows_behind_the_last_sequence(news, pad):
    """A padded batch, as the attention and the token weights take it: no error, nothing of the
    cache touched by the padding, zeros read back for it."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(sum(news) + pad))
    lens = [n + 100 for n in news]
    cu_q, cu_k = layout(lens, news)
    n, rows = int(cu_q[-1]), int(cu_k[-1])
    k, v = bf16(hard_rows(n + pad, rng)), bf16(hard_rows(n + pad, rng))
    k[n:], v[n:] = float("nan"), float("inf")  # what stands in the padding is not looked at
    kv4 = torch.full((rows, 128), 0xA5, dtype=torch.uint8, device="cuda")
    sc = torch.full((rows, 16), 0x5A, dtype=torch.uint8, device="cuda")
    args = dev_i32(cu_q), dev_i32(cu_k), dev_i32(lens)
    h.hisa_device_status(clear=True)
    h.hisa_kv4_store(k, v, *args, kv4, sc)
    out = [torch.full((n + pad, DIM), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    h.hisa_kv4_load(kv4, sc, *args, n + pad, *out)
    assert h.hisa_device_status(clear=True) == 0
    codes, scales = np.zeros((0, 128), np.uint8), np.zeros((0, 16), np.uint8)
    if n:
        codes, scales = kv4_ref.pack(*kv4_ref.quantise(f64(k[:n])),
                                     *kv4_ref.quantise(f64(v[:n])))
    want = np.full((rows, 128), 0xA5, np.uint8), np.full((rows, 16), 0x5A, np.uint8)
    at = new_rows(lens, news, cu_k)
    want[0][at], want[1][at] = codes, scales
    assert np.array_equal(kv4.cpu().numpy(), want[0]) and np.array_equal(sc.cpu().numpy(), want[1])
    for got, ref in zip(out, kv4_ref.values(codes, scales)):
        assert np.array_equal(f64(got[:n]), ref) and not got[n:].any()
    # a sequence that does not fit is still reported, padding or not
    h.hisa_kv4_store(k, v, args[0], args[1], dev_i32([lens[0], lens[1], rows]), kv4, sc)
    assert h.hisa_device_status(clear=True) == (1 << 1 if news[2] else 0)


def test_eviction_counts_over_an_input_are_refused():
    h = H()
    w = torch.zeros(256, dtype=torch.int64, device="cuda")
    cu, lens, keep = dev_i32([0, 128, 256]), dev_i32([100, 128]), dev_i32([50, 60])
    kept, n = torch.zeros(256, dtype=torch.int32, device="cuda"), dev_i32([0, 0])
    both = torch.zeros(258, dtype=torch.int32, device="cuda")
    for out in (dict(kept_len=lens), dict(kept_len=keep), dict(kept_len=cu[:2]),
                dict(kept_len=cu[1:]), dict(kept=w.view(torch.int32)[:256]),
                dict(kept=w.view(torch.int32)[256:]), dict(kept=both[:256], kept_len=both[255:257])):
        with pytest.raises(ValueError, match="overlaps"):
            h.hisa_evict_select(w, cu, lens, keep, 128, 4, 4, **{**dict(kept=kept, kept_len=n), **out})
    h.hisa_device_status(clear=True)
    h.hisa_evict_select(w, cu, lens, keep, 128, 4, 4, kept=both[:256], kept_len=both[256:])
    assert both[256:].tolist() == [50, 60] and h.hisa_device_status() == 0


@pytest.mark.parametrize("seqs", [1, 3, 2000, 65535])
def test_rows_move_whatever_the_bound_of_their_count(seqs):
    """max_keep only has to be at least every count: the launch does not grow with it (a grid of
    65535 sequences times 2^31 rows would keep the GPU for hours).  The first sequence has more
    rows than its CTAs have in one turn."""
    h = H()
    long = {1: 6200000, 3: 2100000}.get(seqs, 10000)
    lens = np.full(seqs, 3)
    lens[0] = long
    keep = np.full(seqs, 2)
    keep[0] = long - 5
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(cu[-1])
    kept = np.full(rows, -1, np.int32)
    kept[cu[1:-1]], kept[cu[1:-1] + 1] = 0, 2
    kept[:long - 5] = np.arange(5, long)
    src = torch.arange(rows * 3, dtype=torch.int32, device="cuda").view(rows, 3)
    dst, want = torch.zeros_like(src), np.zeros((rows, 3), np.int32)
    host = src.cpu().numpy()
    want[:long - 5] = host[5:long]
    want[cu[1:-1]], want[cu[1:-1] + 1] = host[cu[1:-1]], host[cu[1:-1] + 2]
    c, kept, n = dev_i32(cu), dev_i32(kept), dev_i32(keep)
    h.hisa_device_status(clear=True)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    h.hisa_evict_rows([src], [dst], c, c, kept, n, long)
    assert np.array_equal(dst.cpu().numpy(), want)
    dst.zero_()
    torch.cuda.synchronize()
    start.record()
    h.hisa_evict_rows([src], [dst], c, c, kept, n, 2 ** 31 - 1)
    end.record()
    torch.cuda.synchronize()
    assert h.hisa_device_status() == 0
    assert np.array_equal(dst.cpu().numpy(), want)
    # 47360 CTAs, or one per sequence: well under a millisecond; 2^24 and more of them without
    # work take several
    assert start.elapsed_time(end) < 3


def test_rows_over_the_offsets_are_refused():
    h = H()
    cu, other = dev_i32([0, 2]), dev_i32([0, 2])
    kept, n, src = dev_i32([0, 1]), dev_i32([1]), dev_i32([5, 6])
    for c, d in ((cu, other), (other, cu)):
        with pytest.raises(ValueError, match="overlaps"):
            h.hisa_evict_rows([src], [cu], c, d, kept, n, 1)
    with pytest.raises(ValueError, match="overlaps"):
        h.hisa_evict_rows([cu], [cu], cu, cu, kept, n, 1)
    h.hisa_evict_rows([cu], [src], cu, cu, kept, n, 1)  # offsets may be read as any row
    assert src.tolist() == [0, 6]


@pytest.mark.parametrize("byte", [0, 1, 8, 197, 198, 199, 200, 207, 223, 247, 248, 249, 254, 255])
def test_scale_bytes_of_the_format_and_others(byte):
    """A cache that something else than the store filled: up to byte 198 (896) both readers give
    (nibble - 8) * scale, above it neither gives a finite number: NaN in the load and, where the
    byte is 255, in the attention."""
    h = H()
    nib = np.tile(np.arange(16, dtype=np.uint8), 8)[None]
    half = nib[:, 0::2] | (nib[:, 1::2] << 4)
    for which in (0, 1):  # the scales of the key, of the value
        codes = np.tile(np.concatenate([half, half], 1), (128, 1))
        scales = np.full((128, 16), 0x70, np.uint8)
        scales[5, 8 * which:8 * which + 8] = byte
        dev = [torch.from_numpy(x).cuda() for x in (codes, scales)]
        kb, vb = h.hisa_kv4_load(*dev, dev_i32([0, 6]), dev_i32([0, 128]), dev_i32([6]), 6)
        ref = kv4_ref.values(codes[:6], scales[:6])
        if byte > 198:
            ref[which][5] = np.nan
        assert np.array_equal(f64(kb), ref[0], equal_nan=True)
        assert np.array_equal(f64(vb), ref[1], equal_nan=True)
        for heads in (3, 20):
            for rows in (1, 1000):  # over a cluster, one warp a row
                q = np.zeros((rows, heads, DIM))
                q[:, :, 3] = 1.0
                lse = torch.empty(rows, heads, device="cuda")
                out = h.hisa_sparse_attention_kv4(
                    bf16(q), *dev, dev_i32(np.full((rows, 1), 5)), dev_i32([0, rows]),
                    dev_i32([0, 128]), 1.0, lse=lse)
                # one token: its value, and its score as the log-sum-exp (fp32, and 2^-16 of it)
                got, x = f64(lse), float(ref[0][5, 3])
                if byte > 198:
                    none = np.isnan if byte == 255 else lambda y: ~np.isfinite(y)
                    assert none(f64(out)).all() and (which or none(got).all())
                else:
                    assert np.array_equal(f64(out), np.broadcast_to(ref[1][5], out.shape))
                if byte <= 198 or which:
                    assert np.abs(got - x).max() <= 2.0 ** -16 * (1 + abs(x))


def given_lse_run(q, k, idx, lse, scale):
    """hisa_token_weights of one sequence: the weights of every cache row, as numbers."""
    h = H()
    rows = len(k)
    w = torch.zeros(rows, dtype=torch.int64, device="cuda")
    h.hisa_device_status(clear=True)
    h.hisa_token_weights(bf16(q), bf16(k), dev_i32(idx), torch.from_numpy(lse).cuda(),
                         dev_i32([0, len(q)]), dev_i32([0, rows]), scale, w)
    assert h.hisa_device_status() == 0
    return w.cpu().numpy() * 2.0 ** -32


@pytest.mark.parametrize("heads", [1, 20])
def test_token_weights_of_exact_sums_against_a_given_lse(heads):
    """Whole numbers, whose products the matrix unit sums exactly, at scores of about 215: here
    the rounding of one fp32 scale or log-sum-exp would move a weight by up to 1e-5, and the
    2^-24 of the score that is added for what the unit cuts off elsewhere does so, which the
    reference adds too.

    Left: the exponent e is rounded twice (2^-24 of it each), 2^e is off by 2^-22, a lane adds up
    to 4 heads and 8 lanes their sums (7 additions), half a unit of 2^-32."""
    rng = np.random.Generator(np.random.PCG64(heads))
    n, topk = 24, 40
    k = rng.integers(-2, 3, (n * topk, DIM)).astype(float)
    q = rng.integers(-2, 3, (n, heads, DIM)).astype(float)
    k[:, :64], q[:, :, :64] = 7.0, 7.0
    q[:, :, 0] = rng.integers(0, 8, (n, 1))
    idx = np.stack([rng.permutation(topk) + r * topk for r in range(n)]).astype(np.int32)
    scale = np.float32(0.0687)
    s = np.einsum("nhd,ntd->nht", q, k[idx]) * np.float64(scale)
    lse = (np.log(np.exp(s - 200).sum(-1)) + 200).astype(np.float32)
    p = np.exp(s - lse.astype(np.float64)[..., None])
    biased = p * np.exp(s * 2.0 ** -24)
    ref = np.zeros(len(k))
    ref[idx.ravel()] = biased.sum(1).ravel()
    got = given_lse_run(q, k, idx, lse, float(scale))
    e = np.abs(np.log2(p)).max()
    assert e < 16
    tol = ref * (2 * np.log(2) * 16 * 2.0 ** -24 + 2.0 ** -22 + 7 * 2.0 ** -24) + 2.0 ** -33
    err = np.abs(got - ref)
    assert np.all(err <= tol), float((err / ref).max())


@pytest.mark.parametrize("heads", [16, 32])
def test_token_weights_of_rounded_sums_have_no_bias(heads):
    """Random rows: what the matrix unit cuts off lowers every score.  2^-24 of the score is added
    for it; unless that takes more than half of the bias away it is the wrong number."""
    rng = np.random.Generator(np.random.PCG64(heads))
    n, topk = 64, 256
    k = bf16(rng.standard_normal((n * topk, DIM)), "cpu").double().numpy()
    q = bf16(2 * rng.standard_normal((n, heads, DIM)), "cpu").double().numpy()
    idx = np.arange(n * topk, dtype=np.int32).reshape(n, topk)
    scale = np.float32(DIM ** -0.5)
    s = np.einsum("nhd,ntd->nht", q, k.reshape(n, topk, DIM)) * np.float64(scale)
    lse = np.log(np.exp(s).sum(-1)).astype(np.float32)
    p = np.exp(s - lse.astype(np.float64)[..., None])
    got = given_lse_run(q, k, idx, lse, float(scale))
    added = (p * s).sum() * 2.0 ** -24  # by the correction, over all weights
    assert added > 4 * len(k) * 2.0 ** -33  # far above the accumulators' half units
    bias = got.sum() - p.sum()
    assert abs(bias) <= added / 2 + len(k) * 2.0 ** -33, bias / p.sum()


def test_a_padded_decode_step_in_a_graph():
    """A step of fixed size, captured once: the sequences that take part, and their number of
    rows, change from replay to replay, the rest of the rows is padding."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(4))
    lens, heads, topk, size = [700, 300, 500, 150], 12, 96, 6
    cap = np.array([(n // 128 + 2) * 128 for n in lens])
    cu_k = np.concatenate([[0], np.cumsum(cap)]).astype(np.int32)
    rows = int(cu_k[-1])
    ck, ln, cq = dev_i32(cu_k), dev_i32(lens), dev_i32([0] * 5)
    codes, scales = kv4_ref.pack(*kv4_ref.quantise(rng.standard_normal((rows, DIM))),
                                 *kv4_ref.quantise(rng.standard_normal((rows, DIM))))
    kv4, sc = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    k, v = (torch.zeros(size, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(size, heads, DIM, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((size, topk), -1, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(size, heads, device="cuda")
    w = torch.zeros(rows, dtype=torch.int64, device="cuda")

    def step():
        h.hisa_kv4_store(k, v, cq, ck, ln, kv4, sc)
        h.hisa_sparse_attention_kv4(q, kv4, sc, idx, cq, ck, 0.09, out=out, lse=lse, weights=w)
    h.hisa_device_status(clear=True)
    step()
    assert h.hisa_device_status() == 0  # no sequence has a row: all of it is padding
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for news in ([1, 1, 1, 1], [0, 1, 0, 1], [2, 0, 0, 0], [0, 0, 0, 0], [1, 2, 3, 0]):
        cu_q = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        n = int(cu_q[-1])
        hk, hv = (rng.standard_normal((size, DIM)) for _ in range(2))
        hi = np.full((size, topk), -1, np.int32)
        for s in range(4):
            for r in range(int(cu_q[s]), int(cu_q[s + 1])):
                hi[r] = rng.permutation(lens[s])[:topk]
        q.copy_(bf16(rng.standard_normal((size, heads, DIM))))
        k.copy_(bf16(hk))
        v.copy_(bf16(hv))
        idx.copy_(torch.from_numpy(hi))
        cq.copy_(torch.from_numpy(cu_q))
        w.zero_()
        out.fill_(7.0)
        g.replay()
        assert h.hisa_device_status() == 0
        if n:
            at = new_rows(lens, news, cu_k)
            codes[at], scales[at] = kv4_ref.pack(*kv4_ref.quantise(f64(k[:n])),
                                                 *kv4_ref.quantise(f64(v[:n])))
        assert np.array_equal(kv4.cpu().numpy(), codes)
        assert np.array_equal(sc.cpu().numpy(), scales)
        if n:
            kr, vr = kv4_ref.values(codes, scales)
            ref = kv4_ref.Attention(f64(q[:n]), kr, vr, hi[:n], cu_q, cu_k,
                                    np.float64(np.float32(0.09)))
            ref.check_out(f64(out[:n]), np.abs(vr).max())
            ref.check_lse(f64(lse[:n]))
            ref.check_weights(w.cpu().numpy(), rows)
        else:
            assert not w.any()
        assert not out[n:].any() and torch.isneginf(lse[n:]).all()


def test_a_named_stream_and_no_lengths():
    """Every call on a stream that is named, with the outputs made by the call; without
    seqlens_k the regions are full."""
    h = H()
    rng = np.random.Generator(np.random.PCG64(12))
    cu_q, cu_k, heads = [0, 256, 260], [0, 256, 640], 5
    n, rows = 260, 640
    k, v = bf16(rng.standard_normal((n, DIM))), bf16(rng.standard_normal((n, DIM)))
    q = bf16(rng.standard_normal((n, heads, DIM)))
    hi = np.stack([rng.permutation(256)[:40] for _ in range(n)]).astype(np.int32)
    hw = rng.integers(0, 1 << 40, rows)
    cq, ck, idx, keep = dev_i32(cu_q), dev_i32(cu_k), dev_i32(hi), dev_i32([100, 384])
    for s in (torch.cuda.Stream(), torch.cuda.default_stream()):
        kv4 = torch.zeros(rows, 128, dtype=torch.uint8, device="cuda")
        sc = torch.zeros(rows, 16, dtype=torch.uint8, device="cuda")
        w, w2 = torch.from_numpy(hw).cuda(), torch.zeros(rows, dtype=torch.int64, device="cuda")
        lse = torch.empty(n, heads, device="cuda")
        torch.cuda.synchronize()
        h.hisa_kv4_store(k, v, cq, ck, None, kv4, sc, stream=s)
        kb, vb = h.hisa_kv4_load(kv4, sc, cq, ck, None, n, stream=s)
        out = h.hisa_sparse_attention_kv4(q, kv4, sc, idx, cq, ck, 0.1, lse=lse, stream=s)
        keys = torch.zeros(rows, DIM, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        h.hisa_token_weights(q, keys, idx, lse, cq, ck, 0.0, w2, stream=s)
        kept, kept_len = h.hisa_evict_select(w, ck, None, keep, 384, 3, 9, stream=s)
        h.hisa_evict_rows([kv4, w], [kv4, w], ck, ck, kept, kept_len, 384, stream=s)
        s.synchronize()
        at = np.concatenate([np.arange(256), np.arange(636, 640)])
        codes, scales = np.zeros((rows, 128), np.uint8), np.zeros((rows, 16), np.uint8)
        codes[at], scales[at] = kv4_ref.pack(*kv4_ref.quantise(f64(k)), *kv4_ref.quantise(f64(v)))
        kr, vr = kv4_ref.values(codes, scales)
        assert np.array_equal(f64(kb), kr[at]) and np.array_equal(f64(vb), vr[at])
        ref = kv4_ref.Attention(f64(q), kr, vr, hi, cu_q, cu_k, np.float64(np.float32(0.1)))
        ref.check_out(f64(out), np.abs(vr).max())
        ref.check_lse(f64(lse))
        total = np.exp(-f64(lse)).sum() * hi.shape[1]  # scores of nothing: exp(0 - lse)
        assert abs(float(w2.sum()) * 2.0 ** -32 - total) <= 1e-5 * total
        stay = kv4_ref.evict_select(hw[:256], 256, 100, 3, 9)
        assert kept_len.tolist() == [100, 384]
        assert np.array_equal(kept[:100].cpu().numpy(), stay)
        assert np.array_equal(kept[256:640].cpu().numpy(), np.arange(384))
        assert np.array_equal(kv4[:100].cpu().numpy(), codes[stay])
        assert np.array_equal(w[:100].cpu().numpy(), hw[stay])
        assert np.array_equal(kv4[100:].cpu().numpy(), codes[100:])

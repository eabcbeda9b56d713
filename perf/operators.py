"""Workloads of the 4-bit attention cache and of cache eviction, with the operators in plain torch.

Four operators, each as a user's program runs it:

  cache    rows of a prefill chunk or a decode step are stored in the 4-bit cache and read back;
  attend   sparse attention over the 4-bit cache along the selected token indices, with the
           accumulated attention weight of every token where a case asks for it;
  weights  the accumulated attention weight for a bf16 cache, from the attention's log-sum-exp;
  evict    the tokens of every sequence that stay are chosen by their accumulated weight and
           their rows move into the regions of a smaller cache.

The 4-bit format: groups of 16 dimensions share a scale s, an unsigned 8-bit float with 5 exponent
and 3 mantissa bits (bits 14..7 of the fp16 pattern of s); s is amax / 7 rounded to nearest even,
at most 896.  A value is q * s with q = x / s rounded to nearest even and clamped to -7..7, stored
as the nibble q + 8, low nibble first.  A cache row is 64 bytes of key nibbles then 64 bytes of
value nibbles; its 16 scale bytes are the 8 groups of the key, then the 8 of the value.
"""

import torch

own = False

DIM = 128            # width of a key or value row
INDEX_DIM = 64       # width of an index key row
GROUP = 16           # dimensions that share a scale
BLOCK = 128          # region starts are multiples of this
UNIT = 2.0 ** -32    # accumulated weights are whole multiples of this


def listed():
    return [
        # one decode step of a batch of 16: one new row per sequence
        dict(name="cache decode 16", op="cache", seqs=16, len=32768, new=1, ragged=False),
        # a 131072-token prompt stored in one go
        dict(name="cache prefill 131072", op="cache", seqs=1, len=131072, new=131072, ragged=False),
        # one short sequence, one query: latency alone
        dict(name="attend decode 1 short", op="attend", seqs=1, len=600, new=1, heads=8, k=256,
             ragged=False, weights=False),
        # the decode batch of the benchmark: 16 sequences of 32768 keys, 2048 selected
        dict(name="attend decode 16x32K", op="attend", seqs=16, len=32768, new=1, heads=16, k=2048,
             ragged=False, weights=False),
        # a larger ragged decode batch that also keeps the accumulated weights
        dict(name="attend decode 64 weights", op="attend", seqs=64, len=8192, new=1, heads=32,
             k=1000, ragged=True, weights=True),
        # the last 8192 queries of a 32768-token prompt
        dict(name="attend prefill 8192", op="attend", seqs=1, len=32768, new=8192, heads=16, k=2048,
             ragged=False, weights=False),
        # packed prompts of odd lengths, every query, with the accumulated weights
        dict(name="attend packed weights", op="attend", seqs=5, len=1777, new=1777, heads=12, k=512,
             ragged=True, weights=True),
        # the observation window before an eviction: the last 64 queries of 8 prompts
        dict(name="weights window 8x64", op="weights", seqs=8, len=16384, new=64, heads=16, k=2048,
             ragged=True),
        # every query of a chunk, 32 heads
        dict(name="weights chunk 4096", op="weights", seqs=1, len=20000, new=4096, heads=32, k=1024,
             ragged=False),
        # one sequence gone a little over its budget
        dict(name="evict 1 small", op="evict", seqs=1, len=1100, keep=1024, sink=4, recent=128,
             ragged=False),
        # a decode batch halved
        dict(name="evict 16x32K", op="evict", seqs=16, len=32768, keep=16384, sink=64, recent=1024,
             ragged=True),
        # one long prompt cut to a quarter before decoding
        dict(name="evict 1x131072", op="evict", seqs=1, len=131072, keep=32768, sink=128,
             recent=4096, ragged=False),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "attend", "weights", "evict"])
    ragged = rng.random() < 0.6
    if op == "cache":
        seqs = _log(rng, 1, 48)
        length = _log(rng, 64, 131072 // seqs)
        new = 1 if rng.random() < 0.3 else _log(rng, 1, length)
        return dict(op=op, seqs=seqs, len=length, new=new, ragged=ragged)
    if op == "evict":
        seqs = _log(rng, 1, 32)
        length = _log(rng, 200, min(131072, 524288 // seqs))
        keep = rng.randint(length // 8, length - 1)
        return dict(op=op, seqs=seqs, len=length, keep=keep, sink=rng.randint(0, keep // 16),
                    recent=rng.randint(0, keep // 4), ragged=ragged)
    heads, k = rng.randint(1, 32), _log(rng, 16, 2048)
    if op == "attend" and rng.random() < 0.5:  # decode
        seqs, new = _log(rng, 1, 64), 1
        length = _log(rng, 100, 32768 if seqs <= 16 else 8192)
    else:
        seqs = rng.randint(1, 8)
        length = _log(rng, 100, 32768 if seqs <= 2 else 8192)
        entries = (4096 * 2048) // (2 if heads > 16 else 1)
        new = _log(rng, 1, max(1, min(length, 8192, entries // (seqs * k))))
    case = dict(op=op, seqs=seqs, len=length, new=new, heads=heads, k=k, ragged=ragged)
    if op == "attend":
        case["weights"] = rng.random() < 0.5
    return case


def _lengths(case):
    """Live length and new (query) rows of every sequence: equal, or falling to a quarter."""
    n, top = case["seqs"], case["len"]
    lens = [top - (3 * top * s) // (4 * n) if case["ragged"] else top for s in range(n)]
    return lens, [min(case.get("new", 1), x) for x in lens]


def _offsets(sizes):
    at = [0]
    for x in sizes:
        at.append(at[-1] + x)
    return at


def _regions(lens):
    """Region starts: live rows rounded up to whole blocks, and one block more."""
    return _offsets([(x // BLOCK + 2) * BLOCK for x in lens])


def _owner(cu, rows):
    """The sequence of each of `rows` rows under the offsets cu, and the row's place in it."""
    at = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), at, right=True).clamp(max=cu.numel() - 2)
    return seq, at - cu.long()[seq]


def _new_rows(st):
    """The cache row of every query row: the last positions of its sequence."""
    seq, at = _owner(st["cu_q"], st["total_q"])
    new = (st["cu_q"][1:] - st["cu_q"][:-1]).long()[seq]
    return st["cu_k"].long()[seq] + st["lens"].long()[seq] - new + at


def _entry_rows(st):
    """The cache row of every selected entry (of none: the region's first)."""
    seq, _ = _owner(st["cu_q"], st["total_q"])
    return st["cu_k"].long()[seq][:, None] + st["idx"].clamp(min=0)


def _keys(n, width, gen):
    """Rows as a model leaves them: Gaussian, with a few channels several times larger."""
    x = torch.randn(n, width, generator=gen, device=gen.device)
    channel = torch.randn(width, generator=gen, device=gen.device).mul_(0.7).exp_()
    return (x * channel).to(torch.bfloat16)


def _selected(lens, cu_q, k, gen):
    """Indices as the selection leaves them: distinct causal tokens that cluster in blocks, in no
    order of position, padded with -1; one query in about 500 has none."""
    out = []
    for s, length in enumerate(lens):
        n = cu_q[s + 1] - cu_q[s]
        score = torch.rand(n, length, generator=gen, device=gen.device)
        score += torch.rand(n, length // BLOCK + 1, generator=gen, device=gen.device) \
            .repeat_interleave(BLOCK, dim=1)[:, :length]
        pos = torch.arange(length - n, length, device=gen.device)
        score[torch.arange(length, device=gen.device)[None, :] > pos[:, None]] = -1.0
        best, at = score.topk(min(k, length), dim=1)
        at = torch.where(best < 0, -1, at).to(torch.int32)
        out.append(torch.nn.functional.pad(at, (0, k - at.shape[1]), value=-1))
        del score, best
    idx = torch.cat(out)
    if idx.shape[0] > 1:
        none = torch.rand(idx.shape[0], generator=gen, device=gen.device) < 0.002
        none[0] = False
        idx[none] = -1
    return idx.contiguous()


def _scale_of(amax):
    """amax / 7 rounded to the nearest unsigned e5m3 number (ties to even), at most 896."""
    t = amax.double() / 7
    exponent = torch.frexp(t)[1].double() - 1
    step = torch.exp2(exponent.clamp(min=-14) - 3)
    return (torch.round(t / step) * step).clamp(max=896.0)


def _quantise(x):
    """Rows bf16 [n, 128] -> whole numbers -7..7 [n, 8, 16] and scales [n, 8], in 64 bits since
    ties are common."""
    g = x.double().view(x.shape[0], -1, GROUP)
    s = _scale_of(g.abs().amax(dim=-1))
    q = torch.where(s[..., None] > 0, g / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    return torch.round(q).clamp(-7, 7), s


def _pack(q, s):
    """Nibbles and scale bytes of _quantise's answer: uint8 [n, 64] and [n, 8]."""
    u = (q.reshape(q.shape[0], DIM) + 8).to(torch.uint8)
    bits = s.to(torch.float16).view(torch.int16).to(torch.int32) >> 7
    return u[:, 0::2] | (u[:, 1::2] << 4), bits.to(torch.uint8)


def _unpack(codes, scales):
    """Nibbles uint8 [n, 64] and scale bytes uint8 [n, 8] -> values fp32 [n, 128]."""
    u = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(codes.shape[0], -1, GROUP)
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return ((u.float() - 8) * s[..., None]).view(codes.shape[0], DIM)


def prepare(case, seed):
    device = "cuda"
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    lens, news = _lengths(case)
    cu_q, cu_k = _offsets(news), _regions(lens)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    st = dict(op=case["op"], case=case, cu_q=i32(cu_q), cu_k=i32(cu_k), lens=i32(lens),
              total_q=cu_q[-1], max_len=max(lens))
    rows = cu_k[-1]
    if case["op"] == "cache":
        st["k"], st["v"] = _keys(cu_q[-1], DIM, gen), _keys(cu_q[-1], DIM, gen)
        st["kv4"] = torch.zeros(rows, DIM, dtype=torch.uint8, device=device)
        st["kv4_scale"] = torch.zeros(rows, DIM // GROUP * 2, dtype=torch.uint8, device=device)
        return st
    if case["op"] == "evict":
        keep = [min(case["keep"], x) for x in lens]
        cu_d = _regions(keep)
        st.update(keep=i32(keep), cu_d=i32(cu_d), max_keep=max(keep), sink=case["sink"],
                  recent=case["recent"])
        # most tokens were never selected, a few carry most of the weight
        w = torch.randn(rows, generator=gen, device=device).mul_(2.5).exp_().double()
        w *= torch.rand(rows, generator=gen, device=device) < 0.6
        st["weights"] = torch.round(w * 2.0 ** 32 / 64).to(torch.int64)
        st["keys"] = _keys(rows, INDEX_DIM, gen)
        st["kv4"] = torch.randint(0, 256, (rows, DIM), generator=gen, device=device,
                                  dtype=torch.uint8)
        st["kv4_scale"] = torch.randint(0, 200, (rows, 16), generator=gen, device=device,
                                        dtype=torch.uint8)
        st["pos"] = _owner(st["cu_k"], rows)[1].to(torch.int32)
        st["kept"] = torch.full((rows,), -1, dtype=torch.int32, device=device)
        st["kept_len"] = torch.zeros(len(lens), dtype=torch.int32, device=device)
        names = ("keys", "kv4", "kv4_scale", "weights", "pos")
        st["src"] = [st[n] for n in names]
        st["dst"] = [torch.zeros((cu_d[-1],) + tuple(t.shape[1:]), dtype=t.dtype, device=device)
                     for t in st["src"]]
        return st
    st["q"] = _keys(cu_q[-1] * case["heads"], DIM, gen).view(cu_q[-1], case["heads"], DIM)
    st["idx"] = _selected(lens, cu_q, case["k"], gen)
    st["scale"] = DIM ** -0.5
    st["weights"] = torch.zeros(rows, dtype=torch.int64, device=device)
    k = _keys(rows, DIM, gen)
    if case["op"] == "attend":
        v = _keys(rows, DIM, gen)
        parts = [_pack(*_quantise(x)) for x in (k, v)]
        st["kv4"] = torch.cat([p[0] for p in parts], dim=1).contiguous()
        st["kv4_scale"] = torch.cat([p[1] for p in parts], dim=1).contiguous()
    else:
        st["k"] = k
        logits = _logits(st, k.float())
        st["lse"] = torch.logsumexp(logits, dim=-1)
        del logits
    return st


def _logits(st, k):
    """Scaled scores of every selected entry, -inf where there is none: fp32 [total_q, H, k]."""
    s = torch.einsum("qhd,qkd->qhk", st["q"].float(), k[_entry_rows(st)]) * st["scale"]
    return s.masked_fill_((st["idx"] < 0)[:, None, :], float("-inf"))


def _accumulate(st, p):
    """Weights p [total_q, H, k] summed over heads and queries, per cache row, in 64 bits."""
    w = torch.where(st["idx"] >= 0, p.sum(1).double(), 0.0)
    total = torch.zeros(st["weights"].shape[0], dtype=torch.float64, device=p.device)
    return total.index_add_(0, _entry_rows(st).view(-1), w.view(-1)).float()


def _cache_plain(st):
    out = []
    for name in ("k", "v"):
        q, s = _quantise(st[name])
        out.append(_pack(q, s))
    row = _new_rows(st)
    st["kv4"][row] = torch.cat([o[0] for o in out], dim=1)
    st["kv4_scale"][row] = torch.cat([o[1] for o in out], dim=1)
    codes, scales = st["kv4"][row], st["kv4_scale"][row]
    return dict(k=_unpack(codes[:, :64], scales[:, :8]).to(torch.bfloat16),
                v=_unpack(codes[:, 64:], scales[:, 8:]).to(torch.bfloat16))


def _attend_plain(st):
    k = _unpack(st["kv4"][:, :64], st["kv4_scale"][:, :8])
    v = _unpack(st["kv4"][:, 64:], st["kv4_scale"][:, 8:])
    s = _logits(st, k)
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(dim=-1, keepdim=True)
    lse = (torch.log(total) + top).squeeze(-1)
    p = p / torch.where(total > 0, total, 1.0)
    out = torch.einsum("qhk,qkd->qhd", p, v[_entry_rows(st)]).to(torch.bfloat16)
    got = dict(out=out, lse=lse)
    if st["case"]["weights"]:
        got["weights"] = _accumulate(st, p)
    return got


def _weights_plain(st):
    lse = st["lse"][..., None]
    p = torch.exp(_logits(st, st["k"].float()) - torch.where(torch.isinf(lse), 0.0, lse))
    return dict(weights=_accumulate(st, p))


def _evict_plain(st):
    rows = st["kept"].shape[0]
    col = torch.arange(st["max_len"], device=st["kept"].device)[None, :]
    cell = (st["cu_k"].long()[:-1, None] + col).clamp(max=rows - 1)
    n, budget = st["lens"].long()[:, None], st["keep"].long()[:, None]
    first = budget.clamp(max=st["sink"])
    last = (budget - first).clamp(max=st["recent"])
    fixed = ((col < first) | (col >= n - last) | (n <= budget)) & (col < n)
    free = (col < n) & ~fixed
    quota = budget - fixed.sum(1, keepdim=True)
    w = torch.where(free, st["weights"][cell], -1)
    order = torch.argsort(w, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, col.expand_as(order).contiguous())
    stay = fixed | (free & (rank < quota))
    count = stay.sum(1)
    # positions that stay, ascending, at the front of every row
    pos = torch.argsort((~stay).to(torch.int8), dim=1, stable=True)
    # a table cell beyond its sequence's count goes to a spare cell behind the last row
    spare = torch.cat((st["kept"], st["kept"].new_zeros(1)))
    at = torch.where(col < count[:, None], st["cu_k"].long()[:-1, None] + col, rows)
    spare[at] = pos.to(torch.int32)
    st["kept"].copy_(spare[:rows])
    st["kept_len"].copy_(count)
    seq, dpos = _owner(st["cu_d"], st["dst"][0].shape[0])
    live = dpos < count[seq]
    base = st["cu_k"].long()[seq]
    src = base + torch.where(live, st["kept"][(base + dpos).clamp(max=rows - 1)].long(), 0)
    for a, b in zip(st["src"], st["dst"]):
        m = live.view(-1, *([1] * (a.dim() - 1)))
        b.copy_(torch.where(m, a[src], b))
    return _evicted(st)


def _evicted(st):
    keys, kv4, kv4_scale, weights, pos = st["dst"]
    # moved bytes come back as the whole numbers that they spell, four to a number
    return dict(kept=st["kept"], kept_len=st["kept_len"], keys=keys, kv4=kv4.view(torch.int32),
                kv4_scale=kv4_scale.view(torch.int32), weights=weights, pos=pos)


def _run_own(st):
    import sparse_attention_top_hisa_b200 as hisa
    if st["op"] == "cache":
        hisa.hisa_kv4_store(st["k"], st["v"], st["cu_q"], st["cu_k"], st["lens"], st["kv4"],
                            st["kv4_scale"])
        k, v = hisa.hisa_kv4_load(st["kv4"], st["kv4_scale"], st["cu_q"], st["cu_k"], st["lens"],
                                  st["total_q"])
        return dict(k=k, v=v)
    if st["op"] == "attend":
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=st["q"].device)
        w = st["weights"].zero_() if st["case"]["weights"] else None
        out = hisa.hisa_sparse_attention_kv4(st["q"], st["kv4"], st["kv4_scale"], st["idx"],
                                             st["cu_q"], st["cu_k"], st["scale"], lse=lse,
                                             weights=w)
        got = dict(out=out, lse=lse)
        if w is not None:
            got["weights"] = w * UNIT
        return got
    if st["op"] == "weights":
        w = st["weights"].zero_()
        hisa.hisa_token_weights(st["q"], st["k"], st["idx"], st["lse"], st["cu_q"], st["cu_k"],
                                st["scale"], w)
        return dict(weights=w * UNIT)
    hisa.hisa_evict_select(st["weights"], st["cu_k"], st["lens"], st["keep"], st["max_len"],
                           st["sink"], st["recent"], kept=st["kept"], kept_len=st["kept_len"])
    hisa.hisa_evict_rows(st["src"], st["dst"], st["cu_k"], st["cu_d"], st["kept"],
                         st["kept_len"], st["max_keep"])
    return _evicted(st)


def run(state):
    if own:
        return _run_own(state)
    return dict(cache=_cache_plain, attend=_attend_plain, weights=_weights_plain,
                evict=_evict_plain)[state["op"]](state)


def _counts(case):
    """Query rows, selected entries and live rows of a case."""
    lens, news = _lengths(case)
    entries = 0
    for length, n in zip(lens, news):
        full = max(0, length - max(length - n, case["k"] - 1))  # queries that see k tokens or more
        first = length - n + 1
        entries += full * case["k"] + sum(range(first, first + n - full))
    return sum(news), entries, sum(lens)


def work(case):
    if case["op"] == "cache":
        rows = sum(_lengths(case)[1])
        # 256 values of a row: about eight operations each, quantised and read back
        return {"bytes": rows * (512 + 144 + 512), "flops": rows * 256 * 8}
    if case["op"] == "evict":
        lens, _ = _lengths(case)
        kept = sum(min(case["keep"], x) for x in lens)
        row = 2 * INDEX_DIM + 128 + 16 + 8 + 4
        return {"bytes": 8 * sum(lens) + 4 * kept + 2 * row * kept, "flops": sum(lens)}
    queries, entries, live = _counts(case)
    heads, k = case["heads"], case["k"]
    read = queries * (heads * DIM * 2 + 4 * k)
    touched = min(live, entries)
    if case["op"] == "weights":
        return {"bytes": read + queries * heads * 4 + touched * (DIM * 2 + 8),
                "flops": entries * heads * (2 * DIM + 4)}
    moved = read + queries * heads * (DIM * 2 + 4) + touched * (144 + (8 if case["weights"] else 0))
    return {"bytes": moved, "flops": entries * heads * (4 * DIM + 4)}


def _value_table(device):
    """Every nibble's value under every scale byte: float64 [256, 16], from the definition."""
    byte = torch.arange(256, device=device)
    e, m = (byte >> 3).double(), (byte & 7).double()
    s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 15), (m / 8) * 2.0 ** -14)
    return s[:, None] * (torch.arange(16, device=device).double() - 8)[None, :]


def _exact_rows(rows, half, st, table):
    """Values float64 [..., 128] of the key (half 0) or value (half 1) of cache rows."""
    code = st["kv4"][rows][..., 64 * half:64 * half + 64].long()
    byte = st["kv4_scale"][rows][..., 8 * half:8 * half + 8].long()
    dim = torch.arange(DIM, device=code.device)
    nibble = (code[..., dim // 2] >> (4 * (dim % 2))) & 15
    return table[byte[..., dim // GROUP], nibble]


def _exact_cache(x):
    """What a row stands for once stored: the nearest of the scale's multiples, by comparing with
    every candidate."""
    grid = _value_table(x.device)[:, 9].contiguous()  # the scales themselves, ascending
    grid = grid[grid <= 896.0]
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[0], 8192):
        g = x[at:at + 8192].double().view(-1, 8, GROUP)
        want = g.abs().amax(-1) / 7
        hi = torch.searchsorted(grid, want).clamp(max=grid.numel() - 1)
        lo = (hi - 1).clamp(min=0)
        a, b = (want - grid[lo]).abs(), (grid[hi] - want).abs()
        even = torch.where(lo % 2 == 0, lo, hi)
        s = grid[torch.where(a < b, lo, torch.where(b < a, hi, even))][..., None]
        q = torch.arange(-7, 8, device=x.device).double()
        far = (g[..., None] - q * s[..., None]).abs()
        best = far.amin(-1, keepdim=True)
        # of two equally near multiples the even one
        tie = (far == best).double() * torch.where(q % 2 == 0, 2.0, 1.0)
        out[at:at + 8192] = (q[tie.argmax(-1)] * s).reshape(-1, DIM)
    return out


def exact(case, seed):
    if case["op"] == "evict":
        return None  # positions and moved bytes: nothing computed
    st = prepare(case, seed)
    if case["op"] == "cache":
        return dict(k=_exact_cache(st["k"]), v=_exact_cache(st["v"]))
    queries, heads = st["q"].shape[:2]
    device, table = st["q"].device, _value_table(st["q"].device)
    base = torch.cat([torch.full((n,), c, device=device) for n, c in
                      zip(st["cu_q"].diff().tolist(), st["cu_k"].tolist())])
    out = torch.zeros(queries, heads, DIM, dtype=torch.float64, device=device)
    lse = torch.zeros(queries, heads, dtype=torch.float64, device=device)
    weights = torch.zeros(st["weights"].shape[0], dtype=torch.float64, device=device)
    step = max(1, (1 << 18) // case["k"])
    for a in range(0, queries, step):
        b = min(queries, a + step)
        idx = st["idx"][a:b].long()
        rows = (base[a:b, None] + idx.clamp(min=0))
        none = idx < 0
        keys = _exact_rows(rows, 0, st, table) if case["op"] == "attend" else st["k"][rows].double()
        s = torch.matmul(st["q"][a:b].double(), keys.transpose(1, 2)) * st["scale"]
        s = torch.where(none[:, None, :], -torch.inf, s)
        if case["op"] == "attend":
            lse[a:b] = torch.logsumexp(s, dim=-1)
            of = lse[a:b]
        else:
            of = st["lse"][a:b].double()
        p = torch.exp(s - torch.where(torch.isinf(of), 0.0, of)[..., None])
        weights.index_add_(0, rows.reshape(-1),
                           torch.where(none, 0.0, p.sum(1)).reshape(-1))
        if case["op"] == "attend":
            out[a:b] = torch.matmul(p, _exact_rows(rows, 1, st, table))
    if case["op"] == "weights":
        return dict(weights=weights)
    got = dict(out=out, lse=lse)
    if case["weights"]:
        got["weights"] = weights
    return got

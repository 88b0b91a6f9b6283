"""The 4-bit cache on the GPU at the edges of what its calls accept, against the plain restatement
in 64 bits."""
import numpy as np
import pytest
import torch

import nibble_ref as ref
import test_gpu_nibble as base

pytestmark = pytest.mark.gpu

dw = pytest.importorskip("decode_attention_depthweave_b200")

BF, FP = torch.bfloat16, torch.float16
i32, ops = base.i32, base.ops


# ------------------------------------------------------------------------------ tables
@pytest.mark.parametrize("new", [
    [1 << 30, 1 << 30, 1, 1], [1 << 30, 1 << 30, 1 << 30, 1 << 30, 5, 2], [2**31 - 1] * 6 + [3, 0, 2], [4, 1 << 30, 1, (1 << 30) - 1, 2],
    [1] * 40 + [1 << 30] * 4 + [2] * 90, [1 << 30, 0] * 150 + [3]])
def test_totals_of_refused_counts_stay_at_their_cap(new):
    """Counts that no table holds are refused, and so is every row behind them: lengths, pages and slots
    stay as they were, whatever the counts add up to."""
    n, page, pages, width = len(new), 16, 400, 4
    nb = ops(page=page, pages=pages, seqs=n, blocks=width)
    st = dict(seq_lens=[0] * n, block_tables=[[0] * width for _ in range(n)], free_list=list(range(pages)), free_count=[pages])
    base.step(nb, st, new, [0] * n, page, 64)
    with pytest.raises(dw.DwkvError, match="length or count|do not fit"):
        nb.sync()
    # and in a step that releases too
    st = dict(st, seq_lens=[1] * n, block_tables=[[b, 0, 0, 0] for b in range(n)], free_list=list(range(n, pages)) + [0] * n,
              free_count=[pages - n])
    base.step(nb, st, new, [b % 3 == 0 for b in range(n)], page, 64, in_place=False)
    with pytest.raises(dw.DwkvError, match="length or count|do not fit"):
        nb.sync()


# ------------------------------------------------------------------------------ windows
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 16, 2**30, 4096, 1088, 1087, 1086])
@pytest.mark.parametrize("lens,qs", [([2, 1000], [6, 1]), ([2, 0, 700], [3, 2, 1]), ([3, 1000], [200, 60]), ([0, 1, 1087], [40, 90, 1])])
def test_windows_as_long_as_a_request_or_longer(window, lens, qs):
    """Up to the largest that a configuration takes, with rows that stand before the first token."""
    width = 17 - -(-max(lens) // 64)                              # rows of 17 pages: 1088 tokens
    r = base.Requests(61, 8, 2, 128, 64, BF, lens, qs, window, extra_blocks=width)
    assert r.nb.max_blocks == 17
    out, lse = r.run()
    r.nb.sync()
    r.check(out, lse)


# ------------------------------------------------------------------------------ streams
@pytest.mark.parametrize("raw", [False, True])
def test_a_stream_of_its_own_while_another_is_current(raw):
    """step, append, attention and read on a stream that is given and not current, with work pending on
    both: nothing of a call is done on the current stream, and no memory that the current one still uses is
    taken for it."""
    hq, hkv, d, rows = 8, 2, 128, 500
    g = torch.Generator().manual_seed(71)
    qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g).to(BF).cuda()
    new = i32([300, 200])

    def run(c, stream):
        c.step(new, stream=stream)
        c.append(0, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], stream=stream)
        out, lse = c.attention(0, qkv[:, :hq], 300, want_lse=True, stream=stream)
        return (out, lse, *c.read(0, 0, 300, stream=stream), *c.read(0, 1, 200, stream=stream))

    def cache(stream):
        return dw.NibbleCache(1, hq, hkv, d, num_pages=40, max_seqs=2, max_context=512, page_tokens=32, max_rows=rows, stream=stream)
    want = run(cache(None), None)                                 # also loads what torch loads at first use
    torch.cuda.synchronize()
    for late in ("given", "current"):
        s = torch.cuda.Stream()
        stream = s.cuda_stream if raw else s
        # of the current stream: blocks of the outputs' sizes, freed with their last use pending
        filled = [torch.empty_like(x) for x in want]
        with torch.cuda.stream(s) if late == "given" else torch.cuda.stream(torch.cuda.current_stream()):
            torch.cuda._sleep(40_000_000)
        for x in filled:
            x.fill_(7)
        del x, filled
        c = cache(stream)
        if late == "given":
            with torch.cuda.stream(s):
                torch.cuda._sleep(40_000_000)                     # the step is late: what reads its tables waits for it
        got = run(c, stream)
        s.synchronize()
        copies = [x.cpu() for x in got]                           # (waits for the current stream's work too)
        torch.cuda.synchronize()
        for a, b, e in zip(want, got, copies):
            assert torch.equal(a, b) and torch.equal(a.cpu(), e)
        c.sync(stream)


def test_a_stream_for_the_wrappers_outputs():
    """Outputs that attention and read allocate are memory of the given stream: not a block that pending work
    of the current one still writes."""
    r = base.Requests(72, 8, 2, 128, 64, BF, [900, 333], [1, 1])
    want, want_lse = r.run()
    dev = [i32(x) for x in (r.cu, r.lens, r.table.tolist())]
    q, slots = r.q.cuda(), torch.arange(128, dtype=torch.int32, device="cuda")
    k, v = r.nb.read(slots, r.dev_pool)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.empty_like(x) for x in (want, want_lse, k, v)]
        torch.cuda._sleep(40_000_000)
        for x in old:
            x.zero_()
        del x, old
        out, lse = r.nb.attention(q, *dev, r.dev_pool, 1, want_lse=True, stream=s)
        rk, rv = r.nb.read(slots, r.dev_pool, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(rk, k) and torch.equal(rv, v)


# ------------------------------------------------------------------------------ queries
def one_request(hq, d, dtype, k, v, q, scale=0.0, page=16):
    """Attention of the rows q [rows][hq][d] over the tokens k, v [tokens][d] of one kv-head: (out, lse) and
    what ref.attention gives for the stored values."""
    n, rows = k.shape[0], q.shape[0]
    blocks = -(-n // page)
    nb = ops(hq, 1, d, page, blocks, 1, blocks, dtype, 0, scale)
    pool = torch.zeros(nb.pool_bytes, dtype=torch.uint8, device="cuda")
    nb.append(k[:, None].to(dtype).cuda(), v[:, None].to(dtype).cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), pool)
    q = q.to(dtype)
    out, lse = nb.attention(q.cuda(), i32([0, rows]), i32([n]), i32([list(range(blocks))]), pool, rows, want_lse=True)
    nb.sync()
    want = ref.attention(q, [0, rows], [n], [list(range(blocks))], pool.cpu().numpy(), 1, page, 0, scale)
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), want


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("hq,rows", [(4, 1), (4, 2), (4, 4), (4, 7), (4, 10), (40, 2)])
@pytest.mark.parametrize("tokens", [1, 2, 3])
def test_an_infinite_query_over_few_tokens(d, bad, hq, rows, tokens):
    """Whatever the sign of the scores, the row is NaN if it sees a token, and 0 (lse -inf) if it sees none."""
    g = torch.Generator().manual_seed(tokens)
    for sign in (1.0, -1.0):
        k = torch.randn(tokens, d, generator=g)
        k[:, 7] = 3 * sign
        q = torch.randn(rows, hq, d, generator=g)
        q[:, 1, 7] = bad
        out, lse, _ = one_request(hq, d, BF, k, torch.ones(tokens, d), q)
        sees = tokens - rows + np.arange(rows) >= 0
        assert np.isnan(out[sees, 1]).all() and np.isnan(lse[sees, 1]).all()
        assert (out[~sees, 1] == 0).all() and np.isneginf(lse[~sees, 1]).all()
        rest = np.arange(hq) != 1
        assert np.isfinite(out[:, rest]).all() and np.isfinite(lse[sees][:, rest]).all()


def exact_query_tolerances(o, lse, mag, span, d, dtype):
    """ref.tolerances without its term for query channels that lose their tail."""
    es = span * (d * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
    half = torch.finfo(dtype).eps / 2
    to = mag * (2.0 ** -11 + 2.0 ** -20 + 2 * es[..., None]) + half * np.abs(o) * (1 + 2.0 ** -8) + 2.0 ** -25
    return to, es + 2.0 ** -20 + np.abs(lse) * 2.0 ** -22


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,small", [(BF, 10), (BF, 17), (BF, 20), (BF, 24), (BF, 31), (FP, 10), (FP, 14), (FP, 16), (FP, 22)])
@pytest.mark.parametrize("hq,rows", [(4, 1), (4, 2), (4, 4), (4, 8), (4, 40)])
def test_small_channels_of_a_query_count(d, dtype, small, hq, rows):
    """16 channels of the queries far below the others, with keys as far above theirs: their products are the
    larger ones, and no bit of the 16-bit queries is lost.  (fp16 queries reach down to 2^-24; bf16 magnitudes
    from 1 to 2 times 2^-small, all within 2^-32 of the row's largest, 1.)"""
    g = torch.Generator().manual_seed(small)
    n = 70
    k, v = torch.randn(n, d, generator=g) * 2.0 ** -10, torch.randn(n, d, generator=g)
    k[:, 16:32] = torch.randn(n, 16, generator=g).clamp(-4, 4) * 2.0 ** 13
    sign = torch.randint(0, 2, (rows, hq, d), generator=g) * 2.0 - 1
    q = torch.rand(rows, hq, d, generator=g) * sign
    q[:, :, 0] = 1
    q[:, :, 16:32] = (1 + torch.rand(rows, hq, 16, generator=g)) * sign[:, :, 16:32] * 2.0 ** -small
    out, lse, (o, l, mag, span) = one_request(hq, d, dtype, k, v, q)
    sees = np.isfinite(l)
    to, tl = exact_query_tolerances(o, np.where(sees, l, 0), mag, span, d, dtype)
    assert (np.abs(lse - l)[sees] <= tl[sees]).all(), (np.abs(lse - l)[sees] / tl[sees]).max()
    assert (np.abs(out - o) <= to).all(), (np.abs(out - o) / to).max()


@pytest.mark.parametrize("rows", [1, 2, 4, 8, 40])
@pytest.mark.parametrize("largest", [2.0 ** 127, 2.0 ** 60, 2.0 ** -100, 2.0 ** -126, 2.0 ** -133])
def test_queries_of_any_magnitude(rows, largest):
    """Rows whose largest channel is at either end of bf16: scores from the smallest keys."""
    g = torch.Generator().manual_seed(rows)
    n, d, hq = 40, 128, 4
    k, v = torch.randn(n, d, generator=g) * 2.0 ** -14, torch.randn(n, d, generator=g)
    q = (torch.rand(rows, hq, d, generator=g) * 2 - 1) * largest
    q[:, :, 0] = largest
    scale = min(2.0 ** 10 / largest, 2.0 ** 100)
    out, lse, (o, l, mag, span) = one_request(hq, d, BF, k, v, q, scale)
    sees = np.isfinite(l)
    to, tl = exact_query_tolerances(o, np.where(sees, l, 0), mag, span, d, BF)
    assert (np.abs(lse - l)[sees] <= tl[sees]).all() and (np.abs(out - o) <= to).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,size", [(BF, 1e2), (BF, 3e3), (BF, 1e5), (BF, 1e7), (BF, 1e30), (FP, 3e3), (FP, 1.5e4)])
@pytest.mark.parametrize("hq,rows,n", [(4, 1, 70), (4, 2, 70), (16, 1, 70), (4, 8, 70), (4, 40, 70), (4, 1, 4000), (4, 8, 4000), (4, 70, 4000)])
def test_scores_of_any_magnitude(d, dtype, size, hq, rows, n):
    """Scores of 10^5 to 10^34, of either sign.  A score errs by at most span (d 2^-23 + 2^-21), so that only tokens
    within twice that of the largest one (and 40 below it, whose weights are below 2^-57) have a weight: each output
    lies between their smallest and largest value, give or take the rounding of weights (2^-11 of the largest value)
    and of the output.  Odd heads see negative scores only."""
    g = torch.Generator().manual_seed(n + rows)
    k, v = torch.randn(n, d, generator=g), torch.randn(n, d, generator=g)
    k = k * torch.linspace(0.2, 1, n)[:, None] * 6000             # the maximum moves along the tokens
    k[:, 0] = 20000 + 100 * torch.randn(n, generator=g)
    q = torch.randn(rows, hq, d, generator=g).clamp(-4, 4) * size
    q[:, 1::2] *= 0.01
    q[:, 1::2, 0] = -size
    out, lse, (o, l, mag, span) = one_request(hq, d, dtype, k, v, q)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    x, keys, vals = q.to(dtype).double().numpy(), *(ref.values(*ref.quantise(y.to(dtype).double().numpy())) for y in (k, v))
    es = span * (d * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
    off, half = [], torch.finfo(dtype).eps / 2
    for r in range(rows):
        upto = n - rows + r + 1
        s = x[r] @ keys[:upto].T / d ** 0.5
        for h in range(hq):
            alive = vals[:upto][s[h] >= s[h].max() - 2 * es[r, h] - 40]
            lo, hi = alive.min(0), alive.max(0)
            slack = (2.0 ** -11 + 2.0 ** -15) * np.abs(alive).max() + half * np.abs(out[r, h]) * (1 + 2.0 ** -8)
            off.append(max(((lo - slack) - out[r, h]).max(), (out[r, h] - (hi + slack)).max()))
    assert max(off) <= 0
    assert (np.abs(lse - l) <= es + 2.0 ** -20 + np.abs(l) * 2.0 ** -22).all()


@pytest.mark.parametrize("n", [1, 2, 40])
def test_rows_beside_a_max_q_of_zero_are_recorded(n):
    r = base.Requests(81, 4, 1, 128, 64, BF, [20] * n, [1] + [0] * (n - 1))
    out = torch.full((1, 4, 128), 7.0, dtype=BF, device="cuda")
    r.run(out=out, max_q=0)
    with pytest.raises(dw.DwkvError, match="do not fit"):
        r.nb.sync()
    assert out.eq(7).all()
    r.cu = [0] * (n + 1)                                          # no request has rows: nothing to record
    r.run(out=out, max_q=0)
    r.nb.sync()
    assert out.eq(7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,rows", [(1, 1), (4, 1), (2, 2), (1, 4)])
def test_fp16_outputs_of_up_to_4_rows_take_weights_of_22_bits(d, hq, rows):
    """Weights whose rounding to 11 bits all errs the same way against values that all but cancel.  24 tokens are
    one warp's first unit: a weight is 2^(s - max + 7), in two fp16 parts.  Each errs by at most 2^-22 of itself
    (both parts above 2^-14 here); ref.tolerances with that in place of 2^-11 is a bound that 11 bits fail."""
    g = torch.Generator().manual_seed(d + hq)
    n, h, r = 24, hq - 1, rows - 1                                # the row that the values are made for sees all tokens
    k = torch.randn(n, d, generator=g)
    q = (torch.randn(rows, hq, d, generator=g) * 0.01).to(FP)
    stored = ref.values(*ref.quantise(k.to(FP).double().numpy()))
    s = q[r, h].double().numpy() @ stored.T / d ** 0.5 * np.log2(np.e)
    p = np.exp2(s - s.max() + 7)
    err = p.astype(np.float16).astype(np.float64) - p
    v = np.where(err > 0, 1.0, -1.0)
    for t in np.argsort(np.abs(err)):                             # turn the least wrong ones until the values cancel
        if abs((p * v).sum() - 2 * p[t] * v[t]) < abs((p * v).sum()):
            v[t] = -v[t]
    v = torch.from_numpy(np.repeat(v[:, None], d, 1))
    out, lse, (o, l, mag, span) = one_request(hq, d, FP, k, v, q)
    to, _ = ref.tolerances(o, np.where(np.isfinite(l), l, 0), mag, span, d, FP)
    to = to - mag * (2.0 ** -11 - 2.0 ** -22)
    rounded = (p + err) @ ref.values(*ref.quantise(v.numpy())) / p.sum()
    assert (np.abs(rounded - o[r, h]) > 2 * to[r, h]).all()       # what 11 bits would give is outside the bound
    assert (np.abs(out - o) <= to).all(), (np.abs(out - o) / to).max()


# ------------------------------------------------------------------------------ append and read
@pytest.mark.parametrize("d,hkv,dtype", [(128, 8, FP), (128, 9, BF), (128, 17, FP), (64, 16, BF), (64, 17, FP), (64, 33, BF)])
def test_append_and_read_of_more_heads_than_a_warp_takes_at_once(d, hkv, dtype):
    rng = np.random.default_rng(hkv)
    page, pages, n = 16, 3, 9
    nb = ops(hkv, hkv, d, page, pages, dtype=dtype)
    want = rng.integers(0, 256, nb.pool_bytes, dtype=np.uint8)
    pool = torch.from_numpy(want.copy()).cuda()
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    slots[4] = -1
    x = torch.from_numpy(rng.standard_normal((2, n, hkv, d)) * np.exp(rng.uniform(-4, 4, (2, n, hkv, 1)))).to(dtype)
    nb.append(x[0].cuda(), x[1].cuda(), torch.from_numpy(slots).cuda(), pool)
    got = nb.read(torch.from_numpy(slots).cuda(), pool)
    nb.sync()
    for z in range(2):
        c, b = ref.quantise(x[z].double().numpy())
        val = ref.values(c, b)
        val[slots < 0] = 0
        assert np.array_equal(got[z].double().cpu().numpy(), val)
        for i, s in enumerate(slots):
            for h in range(hkv):
                if s >= 0:
                    ref.put(want, hkv, page, d, int(s), h, z, c[i, h], b[i, h])
    assert np.array_equal(pool.cpu().numpy(), want)

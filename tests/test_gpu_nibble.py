"""The 4-bit cache on the GPU against its plain restatement in 64 bits: tables, append, read,
attention, and the four together."""
import numpy as np
import pytest
import torch

import nibble_ref as ref

pytestmark = pytest.mark.gpu

dw = pytest.importorskip("decode_attention_depthweave_b200")

BF, FP = torch.bfloat16, torch.float16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ops(hq=8, hkv=2, d=128, page=64, pages=8, seqs=4, blocks=8, dtype=BF, window=0, scale=0.0):
    return dw.Nibble(dw.nibble_config_from(hq, hkv, d, page, pages, seqs, blocks, dtype, window, scale))


def random_pool(rng, n_bytes, d, low=90, high=118):
    """Random valid blocks: any codes -7..7, scales 2^-3.75 .. 1.75 (numpy)."""
    un, sc = ref._maps(d)
    blocks = n_bytes // (18 * d)
    pool = np.zeros((blocks, 18 * d), np.uint8)
    c = np.clip(np.rint(rng.standard_normal((blocks, un.size, 4)) * 2.8), -7, 7).astype(np.int64) + 8
    w = c[..., 0] | c[..., 1] << 4 | c[..., 2] << 8 | c[..., 3] << 12
    w = ((w << 2) | (w >> 14)) & 0xFFFF
    pool[:, un.ravel()], pool[:, un.ravel() + 1] = w & 255, w >> 8
    pool[:, sc.ravel()] = rng.integers(low, high, (blocks, sc.size))
    return pool.ravel()


class Requests:
    """Random cached requests: a pool whose unused tokens hold 0xFF (NaN scales), tables, queries."""

    def __init__(self, seed, hq, hkv, d, page, dtype, lens, qs, window=0, scale=0.0, extra_blocks=1, temperature=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.page, self.dtype, self.window, self.scale = hq, hkv, d, page, dtype, window, scale
        self.lens, self.cu = list(lens), np.concatenate([[0], np.cumsum(qs)]).tolist()
        held = [-(-x // page) for x in lens]
        pages, width = sum(held) + 2, max(held + [1]) + extra_blocks
        self.nb = ops(hq, hkv, d, page, pages, len(lens), width, dtype, window, scale)
        ids = rng.permutation(pages)
        self.table = np.full((len(lens), width), -5, np.int64)
        self.pool = random_pool(rng, self.nb.pool_bytes, d)
        un, sc = ref._maps(d)
        blocks = self.pool.reshape(pages, hkv, page // 16, 18 * d)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = ids[at:at + h]
            at += h
            for t in range(lens[b], h * page):                # every token behind the last holds NaN scales
                tt = t % page
                for z in range(2):
                    blocks[self.table[b, t // page], :, tt // 16, sc[z][tt % 16][:, None]] = 255
        for i in ids[at:]:
            blocks[i] = 255
        g = torch.Generator().manual_seed(seed)
        self.q = (torch.randn(self.cu[-1], hq, d, generator=g) * temperature * (128 / d) ** 0.5).to(dtype)
        self.max_q = max(list(qs) + [0])

    def run(self, q=None, out=None, lse=None, max_q=None, stream=None):
        dev = [x if isinstance(x, torch.Tensor) else i32(x) for x in (self.cu, self.lens, self.table.tolist())]
        self.dev_pool = torch.from_numpy(self.pool).cuda()
        q = self.q.cuda() if q is None else q
        return self.nb.attention(q, *dev, self.dev_pool, self.max_q if max_q is None else max_q, out=out, lse=lse,
                                 want_lse=True, stream=stream)

    def want(self):
        return ref.attention(self.q, self.cu, self.lens, self.table, self.pool, self.hkv, self.page, self.window, self.scale)

    def check(self, out, lse):
        o, l, mag, span = (x[:self.cu[-1]] for x in self.want())
        to, tl = ref.tolerances(o, l, mag, span, self.d, self.dtype)
        rows = self.cu[-1]
        out, lse = out[:rows].double().cpu().numpy(), lse[:rows].double().cpu().numpy()
        assert np.array_equal(np.isinf(lse), np.isinf(l))
        fin = np.isfinite(l)
        worst = (np.abs(lse[fin] - l[fin]) / tl[fin]).max(initial=0)
        assert worst <= 1, f"lse off by {worst} of its bound"
        off = np.abs(out - o) / to
        assert np.isfinite(out).all() and off.max(initial=0) <= 1, \
            f"out off by {off.max()} of its bound at {np.unravel_index(off.argmax(), off.shape)}"


# ------------------------------------------------------------------------------ append and read
@pytest.mark.parametrize("d,page,hkv,dtype", [(128, 64, 2, BF), (64, 16, 3, FP), (128, 16, 1, FP), (64, 128, 5, BF), (128, 32, 8, BF)])
def test_append_stores_the_bytes_of_the_definition(d, page, hkv, dtype):
    rng = np.random.default_rng(11)
    pages, n = 5, 37
    nb = ops(hkv, hkv, d, page, pages, dtype=dtype)
    before = rng.integers(0, 256, nb.pool_bytes, dtype=np.uint8)
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    slots[[3, 20]] = -1
    x = torch.from_numpy(rng.standard_normal((2, n, hkv, d)) * np.exp(rng.uniform(-9, 6, (2, n, hkv, 1)))).to(dtype)
    x[0, 0] = 0
    x[1, 1, 0, 16:32] = 0
    x[0, 2, 0, :16] = torch.arange(16) * 0.5 - 3.5                # exact ties
    x[1, 2, 0, :16] = torch.arange(16) * 2.0 ** -20               # below the smallest scale's half
    x[0, 4, 0, :16] = torch.arange(16) * 2.0 ** -16
    x[0, 5, 0, 3] = torch.finfo(torch.float16).max if dtype == FP else 53760.0
    clean = dtype == BF
    pool = torch.from_numpy(before.copy()).cuda()
    nb.append(x[0].cuda(), x[1].cuda(), torch.from_numpy(slots).cuda(), pool)
    if clean:
        nb.sync()
    else:
        with pytest.raises(dw.DwkvError, match="53760"):          # fp16's largest is beyond the codec's
            nb.sync()
    want = before.copy()
    for z in range(2):
        c, b = ref.quantise(x[z].double().numpy())
        for i, s in enumerate(slots):
            for h in range(hkv):
                if s >= 0:
                    ref.put(want, hkv, page, d, int(s), h, z, c[i, h], b[i, h])
    assert np.array_equal(pool.cpu().numpy(), want)
    k, v = nb.read(torch.from_numpy(slots).cuda(), pool)
    nb.sync()
    for z, got in enumerate((k, v)):
        c, b = ref.quantise(x[z].double().numpy())
        val = ref.values(c, b)
        val[slots < 0] = 0
        assert np.array_equal(got.double().cpu().numpy(), val)


def test_append_takes_views_of_a_fused_projection():
    nb = ops(hkv=2, page=16)
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(50, 8, 128, generator=g).to(BF).cuda()
    slots = torch.arange(50, dtype=torch.int32, device="cuda") + 7
    a, b = (torch.zeros(nb.pool_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    nb.append(qkv[:, 4:6], qkv[:, 6:], slots, a)
    nb.append(qkv[:, 4:6].contiguous(), qkv[:, 6:].contiguous(), slots, b)
    assert torch.equal(a, b) and a.any()
    nb.append(qkv[:0, 4:6], qkv[:0, 6:], slots[:0], a)            # nothing to do
    assert nb.read(slots[:0], a)[0].shape == (0, 2, 128)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_the_codec_cannot_hold_are_recorded(bad):
    nb = ops(hq=1, hkv=1, page=16)
    x = torch.ones(1, 1, 128, dtype=BF)
    x[0, 0, 5] = bad
    pool = torch.zeros(nb.pool_bytes, dtype=torch.uint8, device="cuda")
    nb.append(x.cuda(), x.cuda(), i32([0]), pool)
    with pytest.raises(dw.DwkvError, match="NaN, infinite"):
        nb.sync()
    nb.sync()                                                     # the word was cleared
    k, _ = nb.read(i32([0]), pool)
    c, b = ref.quantise(x.double().numpy())
    assert np.array_equal(k.double().cpu().numpy(), ref.values(c, b))


@pytest.mark.parametrize("slot", [-2, 8 * 64, 2**31 - 1, -2**31])
def test_slots_outside_the_pool_are_skipped_and_recorded(slot):
    nb = ops()
    x = torch.ones(3, 2, 128, dtype=BF, device="cuda")
    pool = torch.zeros(nb.pool_bytes, dtype=torch.uint8, device="cuda")
    nb.append(x, x, i32([0, slot, 5]), pool)
    with pytest.raises(dw.DwkvError, match="slot is outside"):
        nb.sync()
    k, v = nb.read(i32([0, slot, 5]), pool)
    with pytest.raises(dw.DwkvError, match="slot is outside"):
        nb.sync()
    one = ref.values(*ref.quantise(np.ones(16)))[0]               # 7 e5m3(1/7)
    assert k[0].eq(one).all() and v[2].eq(one).all() and not k[1].any()


# ------------------------------------------------------------------------------ tables
def run_tables(nb, st, new, rel, max_rows, in_place, with_release=True):
    dev = {k: i32(v) for k, v in st.items()}
    n = len(new)
    cu, pos, slots = (torch.full((m,), -77, dtype=torch.int32, device="cuda") for m in (n + 1, max_rows, max_rows))
    outs = {} if in_place else dict(seq_lens_out=torch.empty_like(dev["seq_lens"]), free_count_out=torch.empty_like(dev["free_count"]))
    nb.tables(i32(new), dev["seq_lens"], dev["block_tables"], dev["free_list"], dev["free_count"], cu, slots, positions=pos,
              release=i32(rel) if with_release else None, **outs)
    got = dict(seq_lens=outs.get("seq_lens_out", dev["seq_lens"]), free_count=outs.get("free_count_out", dev["free_count"]),
               block_tables=dev["block_tables"], free_list=dev["free_list"], cu_rows=cu, positions=pos, slots=slots)
    return {k: v.cpu().tolist() for k, v in got.items()}


def step(nb, st, new, rel, page, max_rows, in_place=True):
    want = ref.tables(st["seq_lens"], new, rel, st["block_tables"], st["free_list"], st["free_count"][0], page, max_rows)
    got = run_tables(nb, st, new, rel, max_rows, in_place)
    for k in want:
        assert got[k] == want[k], k
    return {k: want[k] for k in st}


@pytest.mark.parametrize("n,page,pages,width,max_rows,seed", [
    (1, 64, 40, 40, 3000, 0), (5, 16, 30, 20, 200, 1), (33, 32, 100, 9, 300, 2), (700, 16, 4000, 30, 4000, 3),
    (1500, 128, 3000, 5, 9000, 4)])
def test_tables_over_random_steps(n, page, pages, width, max_rows, seed):
    """Growth, release, release with a new request in the same slot, refusals of each kind."""
    rng = np.random.default_rng(seed)
    nb = ops(page=page, pages=pages, seqs=n, blocks=width)
    st = dict(seq_lens=[0] * n, block_tables=[[0] * width for _ in range(n)], free_list=list(rng.permutation(pages).tolist()),
              free_count=[pages])
    for i in range(6):
        new = np.where(rng.random(n) < 0.5, 1, rng.integers(0, 2 * max_rows // n + 2, n)).tolist()
        rel = (rng.random(n) < 0.25).astype(int).tolist()
        st = step(nb, st, new, rel, page, max_rows, in_place=i % 2 == 0)
        try:
            nb.sync()
        except dw.DwkvError as e:                                  # a refusal was recorded
            assert e.status == 4
    held = [x for b in range(n) for x in st["block_tables"][b][:-(-st["seq_lens"][b] // page)]]
    assert sorted(held + st["free_list"][:st["free_count"][0]]) == list(range(pages))


def test_tables_refusals_are_recorded_by_kind():
    def fresh(lens=(0, 0)):
        held = -(-lens[0] // 16)
        return dict(seq_lens=list(lens), block_tables=[[0, 1, 2, 3], [0] * 4], free_list=[5, 6, 7, 4] + [-1] * 4, free_count=[4 - max(0, held - 4)])
    nb = ops(page=16, pages=8, seqs=2, blocks=4)
    for st, new, rel, rows, what in [
            (fresh(), [65, 1], [0, 0], 100, "length or count"), (fresh(), [60, 50], [0, 0], 200, "no free page"),
            (fresh(), [20, 20], [0, 0], 39, "do not fit"), (fresh((-1, 3)), [1, 1], [0, 0], 10, "length or count"),
            (fresh((70, 0)), [1, 1], [1, 0], 10, "length or count"), (fresh(), [-1, 2], [0, 0], 10, "length or count")]:
        step(nb, st, new, rel, 16, rows)
        with pytest.raises(dw.DwkvError, match=what):
            nb.sync()
    step(nb, fresh(), [0, 0], [1, 1], 16, 0)                       # nothing held, nothing added
    nb.sync()


def test_tables_without_release_or_positions():
    nb = ops(page=16, pages=8, seqs=2, blocks=4)
    st = dict(seq_lens=[3, 0], block_tables=[[2, 0, 0, 0], [0] * 4], free_list=[0, 1, 3, 4, 5, 6, 7, 0], free_count=[7])
    got = run_tables(nb, st, [20, 1], [0, 0], 30, True, with_release=False)
    want = ref.tables(st["seq_lens"], [20, 1], [0, 0], st["block_tables"], st["free_list"], 7, 16, 30)
    assert got == want
    dev = {k: i32(v) for k, v in st.items()}
    slots, cu = torch.zeros(30, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    nb.tables(i32([20, 1]), dev["seq_lens"], dev["block_tables"], dev["free_list"], dev["free_count"], cu, slots)
    assert slots.tolist() == want["slots"]


# ------------------------------------------------------------------------------ attention
CASES = [
    # hq, hkv, d, page, dtype, window, lens, query rows
    (4, 1, 128, 64, BF, 0, [1], [1]),
    (4, 1, 128, 64, BF, 0, [16], [1]),
    (4, 1, 128, 64, BF, 0, [17], [1]),
    (32, 8, 128, 64, BF, 0, [300], [1]),
    (8, 2, 128, 64, FP, 0, [63, 64, 65, 1, 0, 500], [1, 1, 1, 1, 0, 1]),
    (8, 2, 128, 16, BF, 0, [129, 15, 16, 1000], [1, 1, 1, 1]),
    (16, 2, 64, 16, FP, 0, [777, 0, 3, 64, 31], [1, 1, 1, 1, 1]),
    (16, 1, 64, 128, BF, 0, [1025, 127], [1, 1]),
    (3, 3, 128, 32, BF, 0, [200, 47], [1, 1]),
    (10, 2, 64, 32, FP, 0, [90, 301, 5], [1, 1, 1]),
    (14, 2, 128, 64, BF, 0, [333, 128], [1, 1]),
    (4, 1, 128, 64, BF, 0, [5000], [1]),
    (2, 2, 64, 16, BF, 0, [3001, 2999], [1, 1]),
    # a few rows a request
    (8, 2, 128, 64, BF, 0, [100, 259, 4], [4, 4, 4]),
    (8, 2, 128, 32, FP, 0, [640, 33, 900], [2, 3, 1]),
    (16, 4, 64, 16, BF, 0, [515, 8], [4, 8]),
    (4, 4, 128, 64, BF, 0, [300], [7]),
    # more rows than tokens: the first rows see nothing
    (8, 2, 128, 64, BF, 0, [2, 0, 5], [4, 3, 1]),
    (4, 2, 64, 64, FP, 0, [3, 200], [40, 64]),
    # windows
    (8, 2, 128, 64, BF, 100, [1000, 50, 101, 100], [1, 1, 1, 1]),
    (8, 2, 128, 16, BF, 1, [1000, 1, 64], [1, 1, 2]),
    (8, 2, 128, 32, FP, 333, [1000, 700, 40], [4, 2, 4]),
    (4, 1, 128, 64, BF, 65, [700], [130]),
    # chunks, ragged, among decodes
    (8, 2, 128, 64, BF, 0, [64], [64]),
    (4, 1, 128, 64, BF, 0, [1100], [257]),
    (32, 8, 128, 64, BF, 0, [200, 333, 1, 64, 500], [100, 1, 1, 33, 1]),
    (10, 2, 64, 16, FP, 0, [300, 129, 400], [129, 17, 1]),
    (14, 2, 128, 32, BF, 200, [513, 700], [300, 40]),
    (64, 1, 64, 64, BF, 0, [150, 90], [1, 5]),
    (48, 1, 128, 128, FP, 0, [290], [33]),
    (2, 2, 64, 16, BF, 0, [2500], [1000]),
]


@pytest.mark.parametrize("hq,hkv,d,page,dtype,window,lens,qs", CASES)
def test_attention(hq, hkv, d, page, dtype, window, lens, qs):
    r = Requests(hash((hq, d, len(lens), lens[0])) % 1000, hq, hkv, d, page, dtype, lens, qs, window)
    out, lse = r.run()
    r.nb.sync()
    r.check(out, lse)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hq,hkv,d,page,window,lens,qs", [
    (17, 1, 128, 64, 0, [300], [1]),
    (64, 2, 128, 16, 0, [777, 31, 0, 1, 448], [1, 1, 0, 1, 1]),
    (8, 2, 128, 32, 90, [500, 225, 224, 5], [8, 5, 7, 6]),
    (20, 1, 64, 64, 0, [2000, 449], [1, 1]),
    (32, 1, 64, 16, 40, [333, 90], [1, 1]),
    (6, 2, 64, 128, 0, [700, 3], [10, 9]),
    (32, 1, 128, 64, 0, [600, 90, 450], [1, 20, 1]),
])
def test_attention_of_17_to_32_rows_a_kv_head(hq, hkv, d, page, window, lens, qs, dtype):
    r = Requests(sum(lens), hq, hkv, d, page, dtype, lens, qs, window)
    out, lse = r.run()
    r.nb.sync()
    r.check(out, lse)


@pytest.mark.parametrize("longest", [1, 6, 40])
@pytest.mark.parametrize("n", [33, 300])
def test_attention_over_many_requests(n, longest):
    """More requests than a warp has lanes, and than a block has threads; some idle."""
    rng = np.random.default_rng(n + longest)
    lens = rng.integers(0, 400, n).tolist()
    qs = [0 if rng.random() < 0.2 else 1 if rng.random() < 0.7 else int(rng.integers(1, longest + 1)) for _ in range(n)]
    r = Requests(n, 4, 1, 64, 16, BF, lens, qs)
    out, lse = r.run(max_q=longest)
    r.nb.sync()
    r.check(out, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("qs", [[1, 1], [4, 3], [8, 5], [60, 33]])
def test_a_query_that_is_no_number_spoils_its_own_row_only(qs, bad):
    r = Requests(41, 8, 2, 128, 64, BF, [100, 300], qs)
    clean, clean_lse = r.run()
    spoilt = r.q.clone()
    spoilt[0, 1, 7] = bad
    out, lse = r.run(q=spoilt.cuda())
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    r.nb.sync()
    assert torch.isfinite(out[keep]).all()
    # the other rows' running maxima may be taken at other units: equal up to what rounding allows
    out[0, 1], lse[0, 1] = clean[0, 1], clean_lse[0, 1]
    r.check(out, lse)


def test_two_handles_at_once_on_two_streams():
    """A handle each: their launches share no tickets and no records."""
    r = [Requests(51 + i, 8, 2, 128, 64, BF, [3000, 900], qs) for i, qs in enumerate([[1, 1], [40, 3]])]
    alone = [x.run() for x in r]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in r]
    for _ in range(10):
        outs = []
        for x, s in zip(r, streams):
            with torch.cuda.stream(s):
                outs.append(x.run())
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("qs", [[1, 1, 1], [3, 1, 2], [40, 1, 90]])
@pytest.mark.parametrize("temperature,scale", [(30.0, 0.0), (1.0, 0.7), (1e-3, 0.0), (3e4, 1e-4), (1e-5, 40.0)])
def test_attention_over_query_sizes_and_scales(qs, temperature, scale):
    """Peaked and flat softmax; queries far above and below 1."""
    r = Requests(21, 8, 2, 128, 64, BF, [700, 65, 300], qs, scale=scale, temperature=temperature)
    out, lse = r.run()
    r.check(out, lse)


@pytest.mark.parametrize("qs", [[1, 1], [2, 2], [30, 70]])
def test_attention_at_the_ends_of_the_scales_range(qs):
    """Stored scales from the smallest subnormal to the largest: values up to 53760."""
    r = Requests(22, 8, 2, 128, 32, BF, [150, 90], qs, temperature=1e-4)
    rng = np.random.default_rng(5)
    _, sc = ref._maps(128)
    live = r.pool.reshape(-1, 18 * 128)
    vals = live[:, sc.ravel()]
    live[:, sc.ravel()] = np.where(vals == 255, 255, rng.integers(0, 224, vals.shape))
    out, lse = r.run()
    r.check(out, lse)


def test_scores_that_rise_and_fall_along_the_tokens():
    """The running maximum moves by far more than one rescaling step, up and down."""
    r = Requests(23, 4, 1, 128, 16, BF, [2000, 2000], [1, 50], temperature=3.0)
    _, sc = ref._maps(128)
    for b in range(2):
        for t in range(2000):
            blk = r.pool.reshape(-1, 1, 1, 18 * 128)[r.table[b, t // 16], 0, 0]
            blk[sc[0][t % 16]] = 96 + int(16 * abs(np.sin(t / (40 if b else 300))))
    out, lse = r.run()
    r.check(out, lse)


@pytest.mark.parametrize("qs", [[1, 2, 1], [40, 2, 50]])
def test_rows_behind_the_last_request_and_idle_slots_are_left_alone(qs):
    r = Requests(31, 8, 2, 128, 64, BF, [100, 80, 300], qs)
    r.cu = [0, qs[0], qs[0], qs[0] + qs[2]]                        # slot 1 idles
    r.q = r.q[:r.cu[-1] + 5] if len(r.q) >= r.cu[-1] + 5 else torch.cat([r.q[:r.cu[-1]], torch.ones(5, 8, 128, dtype=BF)])
    out = torch.full((r.q.shape[0], 8, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((r.q.shape[0], 8), 7.0, device="cuda")
    r.run(out=out, lse=lse)
    r.nb.sync()
    r.check(out, lse)
    assert out[r.cu[-1]:].eq(7).all() and lse[r.cu[-1]:].eq(7).all()


@pytest.mark.parametrize("qs", [[1, 1], [60, 33]])
def test_queries_as_views_of_a_fused_projection(qs):
    r = Requests(32, 8, 2, 128, 64, BF, [100, 300], qs)
    wide = torch.randn(r.q.shape[0], 12, 128, dtype=torch.float32).to(BF).cuda()
    wide[:, :8] = r.q.cuda()
    out, lse = r.run(q=wide[:, :8])
    r.check(out, lse)


@pytest.mark.parametrize("qs", [[1, 1], [60, 33]])
def test_pages_outside_the_pool_are_left_out_and_recorded(qs):
    """Page ids -1 and num_pages, as the first, a middle and the last page of a request: the call
    gives the attention over the tokens that remain."""
    for bad in (-1, 9999):
        for at in (0, 2, 4):
            r = Requests(33, 4, 1, 128, 16, BF, [75, 64], qs)
            keep = [t for t in range(75) if t // 16 != at]
            r.table[0, at] = bad
            out, lse = r.run()
            with pytest.raises(dw.DwkvError, match="page outside"):
                r.nb.sync()
            slots = np.array([r.table[0, t // 16] * 16 + t % 16 for t in keep])
            k, v = (ref.get(r.pool, 1, 16, 128, slots, 0, z) for z in (0, 1))
            pos = 75 - qs[0] + np.arange(qs[0])
            s = np.einsum("rhd,td->rht", r.q[:qs[0]].double().numpy(), k) / 128 ** 0.5
            s = np.where((np.array(keep)[None] <= pos[:, None])[:, None], s, -np.inf)
            none = np.isinf(s).all(-1)
            w = np.where(none[..., None], 0, np.exp(s - np.where(none, 0, s.max(-1))[..., None]))
            o = (w / np.where(none, 1, w.sum(-1))[..., None]) @ v
            got = out[:qs[0]].double().cpu().numpy()
            # the general bound with the mean magnitude of v, a few times its share
            assert np.abs(got - o).max() <= 2.0 ** -7 * np.abs(v).max()
            assert torch.isfinite(out).all()


def test_bad_lengths_and_rows_skip_their_request_and_are_recorded():
    for what, change in [("length", lambda r: r.lens.__setitem__(1, -3)), ("length", lambda r: r.lens.__setitem__(1, 10**6)),
                         ("rows", None)]:
        for qs in ([1, 2, 1], [40, 50, 1]):
            r = Requests(34, 4, 1, 128, 64, BF, [100, 90, 70], qs)
            o, l, mag, span = r.want()
            if change:
                change(r)
            out = torch.full((r.cu[-1], 4, 128), 7.0, dtype=BF, device="cuda")
            r.run(out=out, max_q=None if change else r.max_q - 1)
            with pytest.raises(dw.DwkvError, match=what):
                r.nb.sync()
            a, b = r.cu[1:3]
            skip = np.argmax(qs) if not change else 1
            got = out.double().cpu().numpy()
            for i in range(3):
                rows = slice(r.cu[i], r.cu[i + 1])
                if i == skip:
                    assert (got[rows] == 7).all()
                else:
                    assert np.abs(got[rows] - o[rows]).max() < 0.05


def test_same_inputs_same_bits_and_nothing_is_kept_between_calls():
    for qs in ([1, 1, 1], [50, 200, 1]):
        r = Requests(35, 8, 2, 128, 64, BF, [5000, 900, 64], qs)
        a, la = r.run()
        b, lb = r.run()
        assert torch.equal(a, b) and torch.equal(la, lb)
        r.q = -r.q
        c, lc = r.run()
        r.check(c, lc)


def test_another_stream_than_the_current_one():
    r = Requests(36, 8, 2, 128, 64, BF, [2000, 900, 64], [1, 1, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = r.run(stream=s)
    s.synchronize()
    r.check(out, lse)


@pytest.mark.parametrize("qs", [[1, 1], [1, 70]])
def test_pool_offsets_beyond_32_bits(qs):
    """A pool of over 4 GiB whose last pages are the ones in use."""
    hkv, d, page = 8, 128, 128
    pages = (1 << 32) // (hkv * page * 144) + 40
    nb = ops(32, hkv, d, page, pages, 2, 8)
    assert nb.pool_bytes > 1 << 32
    pool = torch.empty(nb.pool_bytes, dtype=torch.uint8, device="cuda")
    ids = [pages - 1 - 2 * i for i in range(8)]
    table = i32([ids[:4] + [0] * 4, ids[4:] + [0] * 4])
    lens = [500, 300]
    g = torch.Generator().manual_seed(1)
    slots = torch.tensor([ids[4 * b + t // page] * page + t % page for b in range(2) for t in range(lens[b])], dtype=torch.int32).cuda()
    k, v = (torch.randn(800, hkv, d, generator=g).to(BF).cuda() for _ in range(2))
    nb.append(k, v, slots, pool)
    rk, rv = nb.read(slots, pool)
    q = torch.randn(sum(qs), 32, d, generator=g).to(BF).cuda()
    out = nb.attention(q, i32([0, qs[0], sum(qs)]), i32(lens), table, pool, max(qs))
    nb.sync()
    c, b = ref.quantise(k[:3].double().cpu().numpy())
    assert np.array_equal(rk[:3].double().cpu().numpy(), ref.values(c, b))
    # the same rows in a small pool give the same bits
    small = ops(32, hkv, d, page, 8, 2, 8)
    sp = torch.empty(small.pool_bytes, dtype=torch.uint8, device="cuda")
    ss = torch.tensor([(4 * b + t // page) * page + t % page for b in range(2) for t in range(lens[b])], dtype=torch.int32).cuda()
    small.append(k, v, ss, sp)
    st = i32([[0, 1, 2, 3] + [0] * 4, [4, 5, 6, 7] + [0] * 4])
    assert torch.equal(out, small.attention(q, i32([0, qs[0], sum(qs)]), i32(lens), st, sp, max(qs)))


# ------------------------------------------------------------------------------ refusals
def test_the_wrapper_refuses_what_the_library_cannot_see():
    nb = ops()
    pool = torch.zeros(nb.pool_bytes, dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 8, 128, dtype=BF, device="cuda")
    kv = torch.zeros(1, 2, 128, dtype=BF, device="cuda")
    t = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    ok = dict(q=q, cu_rows=i32([0, 1]), seq_lens=i32([1]), block_tables=t, pool=pool, max_q=1)
    nb.attention(**ok)
    for bad in (dict(q=q.half()), dict(q=q[:, :4]), dict(q=q.cpu()), dict(q=q.transpose(1, 2)), dict(cu_rows=i32([0, 1]).long()),
                dict(cu_rows=i32([0])), dict(seq_lens=torch.zeros(1, dtype=torch.int32)), dict(block_tables=t[:, :4]),
                dict(pool=pool[:-1]), dict(out=torch.zeros(1, 8, 128, device="cuda")), dict(lse=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            nb.attention(**{**ok, **bad})
    for bad in (dict(k=kv.half()), dict(v=kv.expand(2, 2, 128)), dict(slots=i32([0, 1])), dict(slots=torch.zeros(1, device="cuda")),
                dict(k=torch.zeros(1, 128, 2, dtype=BF, device="cuda").transpose(1, 2))):
        with pytest.raises(ValueError):
            nb.append(**{**dict(k=kv, v=kv, slots=i32([0]), pool=pool), **bad})
    with pytest.raises(dw.DwkvError, match="multiples of 8"):
        nb.append(torch.zeros(2, 257, dtype=BF, device="cuda")[:, :256].view(2, 2, 128), kv.expand(2, 2, 128).contiguous(), i32([0, 1]), pool)
    with pytest.raises(dw.DwkvError, match="aligned"):
        nb.attention(**{**ok, "q": torch.zeros(1025, dtype=BF, device="cuda")[1:].view(1, 8, 128)})
    with pytest.raises(ValueError):
        nb.tables(i32([1]), i32([0, 0]), t, i32([0] * 8), i32([8]), i32([0, 0]), i32([0]))
    with pytest.raises(dw.DwkvError, match="n_seqs"):
        nb.attention(q, i32([0] * 6), i32([0] * 5), torch.zeros(5, 8, dtype=torch.int32, device="cuda"), pool, 1)
    nb.sync()


# ------------------------------------------------------------------------------ together
def test_steps_of_a_cache_as_a_server_makes_them():
    """Prompts, decode steps, a drafted step, a finished request replaced in its slot: every step's
    attention against the plain form over the values that the cache says it holds."""
    torch.manual_seed(3)
    hq, hkv, d, layers, seqs = 8, 2, 128, 2, 3
    c = dw.NibbleCache(layers, hq, hkv, d, num_pages=30, max_seqs=seqs, max_context=320, page_tokens=32, max_rows=400)
    lens = [0] * seqs
    for new, rel in [([70, 0, 33], [0, 0, 0]), ([1, 200, 1], [0, 0, 0]), ([1, 1, 1], [0, 0, 0]), ([3, 4, 2], [0, 0, 0]),
                     ([50, 1, 0], [1, 0, 1]), ([1, 1, 0], [0, 0, 0])]:
        c.step(i32(new), i32(rel))
        lens = [(0 if r else x) + n for x, n, r in zip(lens, new, rel)]
        rows = sum(new)
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        assert c.seq_lens.tolist() == lens and c.cu_rows.tolist() == cu
        pos = [lens[b] - new[b] + i for b in range(seqs) for i in range(new[b])]
        assert c.positions.tolist() == pos + [-1] * (400 - rows)
        for layer in range(layers):
            qkv = torch.randn(rows, hq + 2 * hkv, d, device="cuda").to(BF)
            c.append(layer, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:])
            out, lse = c.attention(layer, qkv[:, :hq], max(new), want_lse=True)
            pool = c.pools[layer].cpu().numpy()
            o, l, mag, span = ref.attention(qkv[:, :hq].cpu(), cu, lens, c.block_tables.tolist(), pool, hkv, 32)
            to, tl = ref.tolerances(o, l, mag, span, d, BF)
            assert (np.abs(out.double().cpu().numpy() - o) <= to).all()
            assert (np.abs(lse.double().cpu().numpy() - l) <= tl).all()
            b = int(np.argmax(new))
            k, v = c.read(layer, b, lens[b])
            want = ref.values(*ref.quantise(qkv[cu[b]:cu[b + 1], hq:hq + hkv].double().cpu().numpy()))
            assert np.array_equal(k[lens[b] - new[b]:].double().cpu().numpy(), want)
    c.sync()
    held = [x for b in range(seqs) for x in c.block_tables[b, :-(-lens[b] // 32)].tolist()]
    assert sorted(held + c.free_list[:int(c.free_count)].tolist()) == list(range(30))


def test_a_captured_step_replays_over_growing_lengths():
    """Two graphs of one cache (one row a slot; four rows in one slot), replayed in turn: lengths and
    tables advance on the GPU, and every replay equals the same step run eagerly on another cache."""
    hq, hkv, d, seqs = 16, 4, 64, 4

    def new_cache():
        return dw.NibbleCache(1, hq, hkv, d, num_pages=200, max_seqs=seqs, max_context=1024, page_tokens=16, max_rows=700, dtype=FP)
    g = torch.Generator().manual_seed(9)
    prompt = torch.randn(600, hq + 2 * hkv, d, generator=g).half().cuda()
    caches = [new_cache(), new_cache()]
    for c in caches:
        c.step(i32([15, 300, 0, 285]))
        c.append(0, prompt[:, hq:hq + hkv], prompt[:, hq + hkv:])
        c.sync()
    a, b = caches
    plans = {}
    for name, new in (("decode", [1, 1, 1, 1]), ("draft", [0, 4, 0, 1])):
        rows = sum(new)
        x = torch.zeros(rows, hq + 2 * hkv, d, dtype=FP, device="cuda")
        n = i32(new)
        out = torch.zeros(rows, hq, d, dtype=FP, device="cuda")
        state = [t.clone() for t in (a.seq_lens, a.block_tables, a.free_list, a.free_count, a.pools)]

        def run(c, x, out, n=n, most=max(new)):
            c.step(n)
            c.append(0, x[:, hq:hq + hkv], x[:, hq + hkv:])
            c.attention(0, x[:, :hq], most, out=out)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run(a, x, out)                                        # warm-up; its effects are undone below
        torch.cuda.current_stream().wait_stream(s)
        for t, o in zip((a.seq_lens, a.block_tables, a.free_list, a.free_count, a.pools), state):
            t.copy_(o)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(a, x, out)
        plans[name] = (graph, x, out, run)
    for i in range(40):
        graph, x, out, run = plans["draft" if i % 5 == 3 else "decode"]
        x.copy_(torch.randn(*x.shape, generator=g).half())
        graph.replay()
        other = torch.zeros_like(out)
        run(b, x, other)
        assert torch.equal(out, other), i
        assert torch.equal(a.seq_lens, b.seq_lens) and torch.equal(a.pools, b.pools)
    a.sync()
    b.sync()
    del plans, graph

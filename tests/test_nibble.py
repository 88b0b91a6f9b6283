"""The 4-bit cache without a GPU: its codec and layout (of the plain restatement that the GPU tests
compare with) and the calls that the host refuses."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import decode_attention_depthweave_b200 as dw
import nibble_ref as ref


def _cfg(**over):
    kw = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, page_tokens=64, num_pages=100, max_seqs=8, max_blocks=16)
    kw.update(over)
    return dw.nibble_config_from(**kw)


# ------------------------------------------------------------------------------ codec and layout
def test_every_stored_value_is_exact_in_16_bits():
    s = ref.byte_scale(np.arange(224))                     # every scale byte that append writes
    assert s[223] == 7680.0 and s[8] == 2.0 ** -14 and s[1] == 2.0 ** -17
    v = torch.from_numpy(np.outer(np.arange(-8, 8), s))
    for t in (torch.bfloat16, torch.float16):
        fits = v.abs() <= torch.finfo(t).max
        assert fits[1:].all()                              # codes -7 .. 7
        assert torch.equal(v.to(t).double()[fits], v[fits])


def test_scale_is_the_nearest_and_clamping_costs_less_than_half_a_step():
    rng = np.random.default_rng(1)
    a = np.exp(rng.uniform(np.log(1e-6), np.log(5e4), 4000))
    s = ref.scale_of(a)
    grid = np.unique(ref.byte_scale(np.arange(224)))
    near = np.abs(grid[None] - (a / 7)[:, None]).min(1)
    assert np.all(np.abs(s - a / 7) <= near * (1 + 1e-12))
    normal = a / 7 >= 2.0 ** -14
    assert np.all(a[normal] / s[normal] - 7 <= 0.4375 + 1e-12)   # 7 (1 + 1/16): 7 is the nearest code


@pytest.mark.parametrize("d", [64, 128])
def test_a_block_is_a_permutation_of_its_bytes(d):
    un, sc = ref._maps(d)
    at = np.concatenate([un.ravel(), un.ravel() + 1, sc.ravel()])
    assert sorted(at) == list(range(18 * d))


def test_units_round_trip():
    rng = np.random.default_rng(2)
    for _ in range(200):
        c = rng.integers(-8, 8, 4).tolist()
        assert ref.codes_of(ref.unit_of(c)) == c


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (128, 128)])
def test_put_and_get_agree(d, page):
    rng = np.random.default_rng(3)
    pool = rng.integers(0, 256, 3 * 2 * page // 16 * 18 * d, dtype=np.uint8)
    x = rng.standard_normal((2, 5, 2, d))
    slots = rng.permutation(3 * page)[:5]
    for z in range(2):
        for i, s in enumerate(slots):
            for h in range(2):
                c, b = ref.quantise(x[z, i, h])
                ref.put(pool, 2, page, d, s, h, z, c, b)
    for z in range(2):
        for h in range(2):
            c, b = ref.quantise(x[z, :, h])
            assert np.array_equal(ref.get(pool, 2, page, d, slots, h, z), ref.values(c, b))


def test_tables_walk_conserves_pages():
    """The restatement itself: no page is ever held twice, whatever happens in the steps."""
    rng = np.random.default_rng(4)
    p, n, width, pages = 16, 6, 7, 20
    lens, table = [0] * n, [[0] * width for _ in range(n)]
    free, count = list(range(pages)), pages
    for _ in range(200):
        new = [int(rng.integers(0, 40)) for _ in range(n)]
        rel = [int(rng.random() < 0.3) for _ in range(n)]
        r = ref.tables(lens, new, rel, table, free, count, p, 100)
        lens, table, free, count = r["seq_lens"], r["block_tables"], r["free_list"], r["free_count"][0]
        held = [x for b in range(n) for x in table[b][:-(-lens[b] // p)]]
        assert sorted(held + free[:count]) == list(range(pages))


# ------------------------------------------------------------------------------ refusals
def test_sizes():
    cfg = _cfg()
    assert dw.dwkv_nibble_config_check(cfg) == 0
    assert dw.dwkv_nibble_page_bytes(cfg) == 8 * 64 * 2 * (64 + 8)      # 4.5 bits a value
    assert dw.dwkv_nibble_pool_bytes(cfg) == 100 * dw.dwkv_nibble_page_bytes(cfg)
    assert dw.dwkv_nibble_page_bytes(_cfg(head_dim=64, page_tokens=16)) == 8 * 16 * 2 * (32 + 4)
    assert dw.dwkv_nibble_arena_bytes(cfg) > 0


@pytest.mark.parametrize("over,status", [
    (dict(num_q_heads=30), 1), (dict(num_kv_heads=0), 1), (dict(page_tokens=48), 1), (dict(page_tokens=256), 1),
    (dict(num_pages=0), 1), (dict(num_pages=1 << 25), 1), (dict(max_seqs=0), 1), (dict(max_seqs=8193), 1),
    (dict(max_blocks=0), 1), (dict(max_blocks=1 << 24), 1), (dict(window=-1), 1), (dict(head_dim=0), 1),
    (dict(head_dim=96), 5), (dict(head_dim=256), 5), (dict(num_q_heads=130, num_kv_heads=2), 5),
    (dict(softmax_scale=math.inf), 1), (dict(softmax_scale=math.nan), 1),
])
def test_bad_configs_are_refused(over, status):
    cfg = _cfg(**over)
    assert dw.dwkv_nibble_config_check(cfg) == status and dw.dwkv_last_error()
    assert dw.dwkv_nibble_pool_bytes(cfg) == dw.dwkv_nibble_arena_bytes(cfg) == dw.dwkv_nibble_page_bytes(cfg) == 0


def test_bad_dtypes_are_refused():
    with pytest.raises(ValueError, match="dtype"):
        _cfg(dtype=torch.float32)
    cfg = _cfg()
    cfg.dtype = 2
    assert dw.dwkv_nibble_config_check(cfg) == 1


def test_create_and_null_handles_are_refused_without_a_gpu():
    L, cfg, h = dw.lib(), _cfg(), C.c_void_p()
    assert L.dwkv_nibble_create(C.byref(cfg), None, 0, None, C.byref(h)) == 1 and "arena" in dw.dwkv_last_error()
    assert L.dwkv_nibble_create(C.byref(cfg), 257, 1 << 30, None, C.byref(h)) == 1 and "aligned" in dw.dwkv_last_error()
    assert L.dwkv_nibble_create(C.byref(cfg), 256, 16, None, C.byref(h)) == 2
    assert L.dwkv_nibble_create(C.byref(cfg), 256, 1 << 30, None, None) == 1
    assert h.value is None
    assert L.dwkv_nibble_destroy(None) == 1 and L.dwkv_nibble_sync_status(None, None) == 1
    assert L.dwkv_nibble_tables(None, 0, *[None] * 8, 0, *[None] * 4) == 1
    assert L.dwkv_nibble_append(None, 0, None, 0, None, 0, None, None, None) == 1
    assert L.dwkv_nibble_read(None, 0, *[None] * 5) == 1
    assert L.dwkv_nibble_attention(None, 0, 0, 0, None, 0, *[None] * 7) == 1
    assert "handle" in dw.dwkv_last_error()

"""cache_plan, cache_release and cache_store against token-by-token plain forms."""
import numpy as np
import pytest
import torch

import lm_ref
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def held_tables(lengths, width, page, pool):
    tables = np.full((len(lengths), width), -7, np.int32)
    taken = 0
    for r, n in enumerate(lengths):
        k = min(-(-max(int(n), 0) // page), width)
        tables[r, :k] = pool[taken:taken + k]
        taken += k
    return tables, taken


def run_plan(lengths, counts, page, width, pool_extra, total=None, seed=0, pad=0):
    rng = np.random.default_rng(seed)
    lengths, counts = np.asarray(lengths, np.int32), np.asarray(counts, np.int32)
    need = int(sum(min(-(-max(int(n), 0) // page), width) for n in lengths))
    pool = rng.permutation(need + pool_extra + 3).astype(np.int32)[:need + pool_extra]
    tables, taken = held_tables(lengths, width, page, pool)
    if total is None:
        total = int(np.maximum(counts, 0).sum())
    want = lm_ref.plan(lengths, counts, tables, pool, taken, page, total)
    store = torch.full((len(lengths), width + pad), -7, dtype=torch.int32, device="cuda")
    t = store[:, :width]
    t.copy_(dev(tables))
    args = (dev(lengths), dev(counts), t, dev(pool), dev(np.array([taken], np.int32)), page, total)
    for _ in range(2):   # the same inputs again: the same result
        got = lm.cache_plan(*args)
        torch.cuda.synchronize()
        for name in ("slots", "positions", "starts", "lengths", "taken", "status"):
            assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
        assert np.array_equal(t.cpu().numpy(), want["tables"])
    if pad:
        assert (store[:, width:] == -7).all()
    return got, want


@pytest.mark.parametrize("page", [4, 16, 64, 256])
@pytest.mark.parametrize("rows", [1, 7, 256, 300, 1025, 3000])
def test_plan_ragged(rows, page):
    rng = np.random.default_rng(rows * 1000 + page)
    lengths = rng.integers(0, 100, rows)
    counts = rng.integers(0, 40, rows) * (rng.random(rows) < 0.7)
    run_plan(lengths, counts, page, -(-140 // page), rows * 40, seed=rows, pad=3)


@pytest.mark.parametrize("case", ["one_token", "empty", "long", "no_counts", "negative"])
def test_plan_shapes(case):
    lengths, counts, width = {
        "one_token": ([15, 16, 17, 0], [1, 1, 1, 1], 4),
        "empty": ([], [], 4),
        "long": ([5, 0], [40000, 3], 2600),
        "no_counts": ([5, 0, 64], [0, 0, 0], 4),
        "negative": ([-3, 5], [2, -9], 4),
    }[case]
    run_plan(lengths, counts, 16, width, 2700)


@pytest.mark.parametrize("extra", [0, 1, 5, 17])
def test_plan_pool_runs_dry(extra):
    rng = np.random.default_rng(extra)
    got, want = run_plan(rng.integers(0, 40, 50), rng.integers(0, 40, 50), 8, 10, extra)
    assert (want["status"] & 1).any()


def test_plan_table_and_slot_map_full():
    # a table too narrow for some rows, and a slot map that ends inside a row
    got, want = run_plan([60, 64, 3, 10], [10, 5, 2, 4], 16, 4, 50)
    assert want["status"].tolist() == [2, 2, 0, 0]
    got, want = run_plan([3, 10, 7, 1], [5, 6, 5, 2], 4, 8, 50, total=13)
    assert want["status"].tolist() == [0, 0, 4, 4]
    run_plan([3, 10], [5, 6], 4, 8, 50, total=40)   # a longer one than needed


def test_release_then_append_reuses_pages():
    c = lm.PagedCache(5, 64, 1, 8, page_size=8, num_pages=20)
    cnt = torch.tensor([10, 0, 33, 8, 17], dtype=torch.int32, device="cuda")
    a = c.append(cnt, 68)
    assert c.lengths.tolist() == [10, 0, 33, 8, 17] and int(c.taken) == 11
    before = c.tables.clone()
    c.release(torch.tensor([0, 1, 1, 0, 1], dtype=torch.uint8, device="cuda"))
    assert c.lengths.tolist() == [10, 0, 0, 8, 0] and int(c.taken) == 3
    # the released rows' pages, rows and pages in order, then what was never taken
    freed = before[2, :5].tolist() + before[4, :3].tolist()
    assert c.pool[3:11].tolist() == freed
    b = c.append(torch.tensor([0, 30, 0, 0, 9], dtype=torch.int32, device="cuda"), 39)
    assert c.tables[1, :4].tolist() == freed[:4] and c.tables[4, :2].tolist() == freed[4:6]
    live = [c.tables[r, :-(-n // 8)].tolist() for r, n in enumerate(c.lengths.tolist())]
    flat = sum(live, [])
    assert len(set(flat)) == len(flat) and a.status.sum() == 0 and b.status.sum() == 0


def test_release_many_rows_and_twice():
    rows, page = 2500, 4
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 30, rows).astype(np.int32)
    pool = rng.permutation(20000).astype(np.int32)
    tables, taken = held_tables(lengths, 8, page, pool)
    fin = (rng.random(rows) < 0.5).astype(np.uint8)
    args = [dev(fin), dev(lengths), dev(tables), dev(pool), dev(np.array([taken], np.int32)), page]
    back = [p for r in range(rows) if fin[r] for p in tables[r, :-(-int(lengths[r]) // page)]]
    for _ in range(2):
        n, t = lm.cache_release(*args)
        assert int(t) == taken - len(back)
        assert np.array_equal(n.cpu().numpy(), np.where(fin, 0, lengths))
        assert args[3][taken - len(back):taken].tolist() == back
    # more pages than were taken: nothing outside the pool is touched
    small = dev(np.array([7], np.int32))
    n, t = lm.cache_release(*args[:4], small, page)
    assert int(t) == 0 and args[3][:7].tolist() == back[:7]


@pytest.mark.parametrize("rows", [1, 15, 17, 4097])
def test_release_by_a_bool_mask(rows):
    page, width = 4, 70
    rng = np.random.default_rng(rows)
    lengths = rng.integers(0, page * width + 1, rows).astype(np.int32)
    pool = rng.permutation(rows * width).astype(np.int32)
    tables, taken = held_tables(lengths, width, page, pool)
    fin = rng.random(rows) < 0.7
    back = [p for r in range(rows) if fin[r] for p in tables[r, :-(-int(lengths[r]) // page)]]
    p = dev(pool)
    n, t = lm.cache_release(torch.from_numpy(fin).cuda(), dev(lengths), dev(tables), p,
                            dev(np.array([taken], np.int32)), page)
    assert int(t) == taken - len(back)
    assert np.array_equal(n.cpu().numpy(), np.where(fin, 0, lengths))
    want = pool.copy()
    want[taken - len(back):taken] = back
    assert np.array_equal(p.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,D,page,order,odd", [
    (1, 1, 8, 4, "thd", False), (37, 8, 128, 16, "thd", False), (500, 3, 80, 64, "htd", False),
    (33, 2, 7, 16, "thd", False), (64, 4, 64, 8, "htd", True)])
def test_store(dtype, T, H, D, page, order, odd):
    g = torch.Generator().manual_seed(T)
    pages = -(-T // page) + 2
    kv = torch.randn((T, 2, H, D + 1), generator=g).to(dtype).cuda()
    k, v = (kv[:, i, :, 1:] if odd else kv[:, i, :, :D] for i in (0, 1))   # odd: not aligned
    if not odd:
        k, v = k.contiguous(), v.contiguous()

    def cache():
        c = torch.full((pages, page, H, D) if order == "thd" else (pages, H, page, D), 5.0).to(dtype)
        return (c if order == "thd" else c.transpose(1, 2)).cuda()
    kc, vc = cache(), cache()
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    drop = torch.rand(T, generator=g) < 0.2
    slots[drop] = -1
    if T > 30:
        slots[3], slots[4] = pages * page, 2 ** 31 - 1   # outside the cache: left out
    wk, wv = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            wk[s // page, s % page], wv[s // page, s % page] = k[t], v[t]
    lm.cache_store(k, v, slots.cuda(), kc, vc)
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_store_past_32_bits():
    # element offsets above 2^32: only the last page of a large cache is written
    pages, page, H, D = 40000, 64, 8, 256
    kc = torch.empty((pages, page, H, D), dtype=torch.bfloat16, device="cuda")
    assert kc.numel() > 2 ** 32
    vc = torch.empty_like(kc)
    kc[-1], vc[-1] = 0, 0
    kc[0], vc[0] = 0, 0
    k = torch.randn((2, H, D), device="cuda").bfloat16()
    slots = torch.tensor([pages * page - 1, pages * page - 64], dtype=torch.int32, device="cuda")
    lm.cache_store(k, -k, slots, kc, vc)
    assert torch.equal(kc[-1, 63], k[0]) and torch.equal(vc[-1, 0], -k[1])
    assert not kc[-1, 1:63].any() and not kc[0].any() and not vc[0].any()


def test_refusals():
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="page_size"):
        lm.cache_plan(i, i, tab, i, one, 3, 4)
    with pytest.raises(ValueError, match="page_size"):
        lm.cache_plan(i, i, tab, i, one, 512, 4)
    with pytest.raises(ValueError, match="counts"):
        lm.cache_plan(i, i.long(), tab, i, one, 4, 4)
    with pytest.raises(ValueError, match="counts"):
        lm.cache_plan(i, i[:3], tab, i, one, 4, 4)
    with pytest.raises(ValueError, match="taken"):
        lm.cache_plan(i, i, tab, i, one.cpu(), 4, 4)
    with pytest.raises(ValueError, match="tables"):
        lm.cache_plan(i, i, tab.t().contiguous().t(), i, one, 4, 4)
    with pytest.raises(ValueError, match="total"):
        lm.cache_plan(i, i, tab, i, one, 4, -1)
    with pytest.raises(ValueError, match="finished"):
        lm.cache_release(i, i, tab, i, one, 4)
    c = torch.zeros((3, 4, 2, 8), device="cuda")
    k = torch.zeros((4, 2, 8), device="cuda")
    with pytest.raises(ValueError, match="heads"):
        lm.cache_store(k[:, :1], k[:, :1], i, c, c)
    with pytest.raises(ValueError, match="bfloat16"):
        lm.cache_store(k.double(), k.double(), i, c.double(), c.double())
    with pytest.raises(ValueError, match="v_cache"):
        lm.cache_store(k, k, i, c, c[:2])
    with pytest.raises(ValueError, match="slots"):
        lm.cache_store(k, k, i[:3], c, c)
    with pytest.raises(ValueError, match="GPU"):
        lm.cache_store(k.cpu(), k, i, c, c)

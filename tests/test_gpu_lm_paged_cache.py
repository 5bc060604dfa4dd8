"""PagedCache: its calls on other streams, and the bound of its lengths."""
import pytest
import torch

from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("call", ["append", "release"])
def test_calls_on_a_late_stream_read_what_they_were_given(call):
    """The stream is held back while the current one takes new small tensors, which
    would be given the memory of the old lengths and `taken` if they were let go."""
    def cache():
        c = lm.PagedCache(5, 64, 1, 8, page_size=8, num_pages=20)
        c.append(i32(10, 0, 33, 8, 17), 68)
        return c

    def run(c, stream=None):
        if call == "append":
            p = c.append(more, 30, stream=stream)
            return [p.slots, p.positions, p.starts, p.lengths, p.taken, p.status, c.tables]
        c.release(gone, stream=stream)
        return [c.lengths, c.taken, c.pool]
    more, gone = i32(3, 20, 1, 0, 6), torch.tensor([1, 0, 0, 1, 0], dtype=torch.uint8, device="cuda")
    want = [t.clone() for t in run(cache())]
    c = cache()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = run(c, side)
    taken = [torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (1, 5, 16, 29) * 20]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert len(taken) == 80


@pytest.mark.parametrize("max_len,page", [(100, 16), (65, 64), (128, 16), (1, 4)])
@pytest.mark.parametrize("window", [0, 20])
def test_rows_up_to_the_last_place_of_their_last_page(max_len, page, window):
    """The tables hold max_len tokens rounded up to whole pages: as many are taken, all of
    them are attended to, and what goes past them is flagged."""
    n = -(-max_len // page) * page
    g = torch.Generator().manual_seed(max_len)
    c = lm.PagedCache(2, max_len, 1, 64, torch.float32, page)
    k, v = torch.randn((2, n, 1, 64), generator=g), torch.randn((2, n, 1, 64), generator=g)
    for first, more in ((0, n - 1), (n - 1, 1)):   # row 1 stays one behind at first
        plan = c.append(i32(more, more), 2 * more)
        assert not plan.status.any()
        c.store(k[:, first:first + more].flatten(0, 1).cuda(),
                v[:, first:first + more].flatten(0, 1).cuda(), plan.slots)
    assert c.lengths.tolist() == [n, n]
    q = 2 * torch.randn((2, 1, 64), generator=g)
    out, lse = c.attend(q.cuda(), window=window)
    lo = max(0, n - window) if window else 0
    for r in range(2):
        s = k[r, lo:, 0].double() @ q[r, 0].double() / 8
        want = torch.softmax(s, 0) @ v[r, lo:, 0].double()
        assert torch.allclose(out[r, 0].cpu().double(), want, atol=1e-5, rtol=0)
        assert abs(float(lse[r, 0]) - float(torch.logsumexp(s, 0))) < 1e-5
    assert c.append(i32(1, 0), 1).status.tolist() == [lm.NO_ENTRY, 0]


def test_numbers_that_no_call_can_take_are_refused_as_values():
    i, one, tab = i32(0, 0), i32(0), torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    for kw in (dict(page_size=1 << 31), dict(page_size=16.0), dict(total=1 << 31),
               dict(total=(1 << 30) + 1), dict(page_size="16")):
        with pytest.raises(ValueError):
            lm.cache_plan(i, i, tab, i, one, **{**dict(page_size=16, total=2), **kw})
    with pytest.raises(ValueError):
        lm.cache_release(i.to(torch.uint8), i, tab, i, one, 1 << 40)
    for pool in (None, [0, 1]):
        with pytest.raises(ValueError, match="pool"):
            lm.cache_plan(i, i, tab, pool, one, 16, 2)
        with pytest.raises(ValueError, match="pool"):
            lm.cache_release(i.to(torch.uint8), i, tab, pool, one, 16)
    c = lm.PagedCache(2, 64, 1, 64)
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(max_len=1 << 31), dict(window=1 << 31), dict(window=-(1 << 40)),
               dict(window=2.5), dict(scale="1")):
        with pytest.raises(ValueError):
            c.attend(q, **kw)
    with pytest.raises(ValueError):
        lm.PagedCache(2, 64, 1, 64, page_size=0)
    with pytest.raises(ValueError):
        lm.PagedCache(2, -1, 1, 64)


def step_inputs(rows, heads, D, steps):
    g = torch.Generator(device="cuda").manual_seed(4)
    return [[torch.randn((rows, heads, D), generator=g, device="cuda") for _ in range(3)]
            for _ in range(steps)]


def test_a_captured_step_is_replayed_for_one_token_after_another():
    """Plan, store and attention in a graph: the plan's lengths and counter are copied back
    to the buffers that it reads, so each replay appends the next token."""
    rows, heads, D, steps = 3, 2, 64, 40
    inputs = step_inputs(rows, heads, D, steps)
    ones = i32(1, 1, 1)
    want = lm.PagedCache(rows, 64, heads, D, torch.float32)
    c = lm.PagedCache(rows, 64, heads, D, torch.float32)
    for x in (want, c):
        x.append(i32(0, 3, 7), 10)
        x.k.zero_()
        x.v.zero_()
    q, k, v = (torch.empty_like(t) for t in inputs[0])

    def step():
        plan = lm.cache_plan(c.lengths, ones, c.tables, c.pool, c.taken, c.page_size, rows)
        lm.cache_store(k, v, plan.slots, c.k[0], c.v[0])
        out, lse = lm.attention(q, c.k[0], c.v[0], c.tables, plan.lengths)
        c.lengths.copy_(plan.lengths)
        c.taken.copy_(plan.taken)
        return out, lse, plan.status
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(steps):
        for a, b in zip((q, k, v), inputs[i]):
            a.copy_(b)
        graph.replay()
        plan = want.append(ones, rows)
        want.store(inputs[i][1], inputs[i][2], plan.slots)
        out, lse = want.attend(inputs[i][0])
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i
        assert torch.equal(got[2], plan.status) and torch.equal(c.lengths, want.lengths), i
        assert torch.equal(c.tables, want.tables) and torch.equal(c.taken, want.taken), i
    assert c.lengths.tolist() == [steps, steps + 3, steps + 7]


def test_a_captured_append_repeats_itself():
    """PagedCache goes on to new lengths with each append; what was captured reads the old."""
    c = lm.PagedCache(3, 64, 1, 64, torch.float32)
    c.append(i32(2, 0, 5), 7)
    (q, k, v), = step_inputs(3, 1, 64, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = c.append(c.lengths.clone(), 7)   # as many again
        c.store(k[:1].expand(7, 1, 64), v[:1].expand(7, 1, 64), plan.slots)
        out, _ = c.attend(q)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert plan.lengths.tolist() == [4, 0, 10] and not plan.status.any(), i
        assert plan.positions.tolist() == [2, 3, 5, 6, 7, 8, 9], i
        torch.ones(1000, device="cuda").cumsum(0)


def test_expanded_tensors_are_not_written():
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    c = torch.zeros((3, 16, 2, 64), dtype=q.dtype, device="cuda")
    tab, lens = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), i32(3, 4)
    for out in (q[:1].expand(2, 4, 64), q[:, :1].expand(2, 4, 64)):
        with pytest.raises(ValueError, match="out is written"):
            lm.attention(q, c, c, tab, lens, out=out)
    lm.attention(q[:1], c, c, tab[:1], lens[:1], out=q[1:].expand(1, 4, 64))
    for wide in (c[:1].expand(3, 16, 2, 64), c[:, :1].expand(3, 16, 2, 64),
                 c[:, :, :1].expand(3, 16, 2, 64)):
        for kc, vc, name in ((wide, c, "k_cache"), (c, wide, "v_cache")):
            with pytest.raises(ValueError, match=name + " is written"):
                lm.cache_store(q[:, :2], q[:, :2], i32(0, 1), kc, vc)
        lm.attention(q, wide, wide, tab, lens)   # read, they may be

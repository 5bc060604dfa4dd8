"""Calls of two threads at once, each on a stream of its own, whose kernels take different amounts
of LDS; and such calls in graphs."""
import threading

import pytest
import torch

from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu


def calls():
    """Functions whose results are known, with more than 64 KB of LDS each but the last ones."""
    g = torch.Generator(device="cuda").manual_seed(0)
    got = []
    for rows, hidden in ((8, 8192), (15, 8192), (20, 4096), (30, 4096), (4, 512)):
        w = torch.randint(-127, 128, (200, hidden), generator=g, device="cuda").to(torch.int8)
        ws = torch.rand(200, generator=g, device="cuda") / 100
        x = torch.randn((rows, hidden), generator=g, device="cuda").to(torch.bfloat16)
        got.append(lambda x=x, w=w, ws=ws: lm.linear8(x, w, ws))
    for D, n, rows in ((128, 400, 4), (256, 5000, 1), (64, 40, 3)):
        pages = -(-n // 16)
        c = [torch.randint(-127, 128, (pages, 16, 1, D), generator=g, device="cuda").to(torch.int8)
             for _ in range(2)]
        s = [torch.full((pages, 1), 2.0 ** -6, device="cuda") for _ in range(2)]
        tables = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(rows, 1)
        lens = torch.full((rows,), n, dtype=torch.int32, device="cuda")
        q = torch.randn((rows, 16, D), generator=g, device="cuda").to(torch.float16)
        got.append(lambda q=q, c=c, s=s, t=tables, n=lens: lm.attention8(q, *c, *s, t, n)[0])
    k = torch.randn((40, 4, 64), generator=g, device="cuda")
    slots = torch.arange(40, dtype=torch.int32, device="cuda")

    def store():
        cache = [torch.zeros((3, 16, 4, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
        cache += [torch.zeros((3, 4), device="cuda") for _ in range(2)]
        lm.cache_store8(k, -k, slots, *cache)
        return lm.cache_load8(slots, *cache)[0]
    got.append(store)
    return got


def test_two_threads():
    each = calls()
    want = [f() for f in each]
    torch.cuda.synchronize()
    wrong, ended = [], []

    def work(seed):
        order = torch.randperm(len(each) * 20, generator=torch.Generator().manual_seed(seed)) % len(each)
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in order.tolist():
                    out = each[i]()
                    if not torch.equal(out, want[i]):
                        wrong.append((seed, i))
        except Exception as e:   # shown below, in the test's own thread
            wrong.append((seed, repr(e)))
        ended.append(seed)
    threads = [threading.Thread(target=work, args=(s,)) for s in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and len(ended) == 2


def test_in_graphs():
    each = calls()
    want = [f() for f in each]
    graphs = []
    for f in each:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), f, w in zip(graphs, each, want):
            out.fill_(3.0)
            g.replay()
            assert torch.equal(f(), w)
            torch.cuda.synchronize()
            assert torch.equal(out, w)

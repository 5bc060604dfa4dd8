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

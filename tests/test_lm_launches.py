"""What the language-model operators ask of the HIP runtime, without a GPU: a stand-in for its
launches is loaded in front of it, in a process of its own."""
import json
import os
import subprocess
import sys

import pytest

from code_object import kernels
from ctc_prefix_beam_amd import lm

HERE = os.path.dirname(os.path.abspath(__file__))

CALLS = """
import ctypes, json, sys
standin = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
standin.standin_notes.restype = ctypes.c_char_p
from ctc_prefix_beam_amd import lm
L, P = lm.lib(), 1 << 20

def linear(rows, hidden, features=64, dtype=0):
    return L.ctcpb_lm_linear8(lm._LINEAR8.pack(P, P, P, P, 0, P, hidden, hidden, features, 3, dtype,
                                               rows, features, hidden, 0), P, 1 << 40, None)

def store(tokens, heads=1, D=1, page=16, name="cache_store8"):
    cache = (P, page * D * heads, D * heads, D)
    return getattr(L, "ctcpb_lm_" + name)(lm._CACHE8.pack(
        P, P, P, 0, 0, 0, 0, *cache, *cache, P, 1, 1, P, 1, 1, 0, 0, tokens, (1 << 30) // page, page,
        heads, D), None)

def attend(rows, n, D, group, eight, dtype=0):
    width = n // 16
    args = (P, P, P, P, 0, group * D, D, group * D, D, width, *(P, 16 * D, D, 16 * D) * 2, dtype, rows,
            group, 1, D, 64, 16, width, 0, 0, 1.0)
    if eight:
        return L.ctcpb_lm_attention8(lm._ATTENTION8.pack(*args, P, 1, 1, P, 1, 1, 0), P, 1 << 40, None)
    return L.ctcpb_lm_attention(lm._ATTENTION.pack(*args), P, 1 << 40, None)

got = []
for refuse, call, args in json.loads(sys.argv[2]):
    standin.standin_refuse(refuse)
    rc = globals()[call](*args)
    notes = [l.split() for l in standin.standin_notes().decode().splitlines()]
    got.append([rc, L.ctcpb_lm_last_error().decode(), notes])
print(json.dumps(got))
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    if not os.path.exists(lm.LIB_PATH):
        from ctc_prefix_beam_amd import build
        build.build_lm()
    so = str(tmp_path_factory.mktemp("standin") / "standin.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", os.path.join(HERE, "hip_standin.c"), "-o", so,
                    "-ldl"], check=True)

    def run(*calls):
        p = subprocess.run([sys.executable, "-c", CALLS, so, json.dumps(calls)], capture_output=True,
                           text=True, cwd=os.path.dirname(HERE), timeout=300)
        assert p.returncode == 0, p.stderr
        return json.loads(p.stdout.splitlines()[-1])
    return run


# calls whose kernels take more than 64 KB of LDS, in different amounts
LARGE = [("linear", (8, 8192)), ("linear", (15, 8192)), ("linear", (12, 8192)),
         ("linear", (20, 4096)), ("linear", (30, 4096)),
         ("attend", (4, 512, 128, 16, True)), ("attend", (1, 60000, 256, 16, True)),
         ("attend", (4, 512, 128, 16, False)), ("attend", (1, 60000, 256, 16, False))]


def test_calls_do_not_lower_each_others_lds(run):
    """Whatever a call needs itself, it leaves its kernel the same limit, enough for any other."""
    own = kernels(lm.LIB_PATH)
    limits, most = {}, {}
    for rc, error, notes in run(*[(0, *c) for c in LARGE]):
        assert rc == 0, error
        for what, name, value, *rest in notes:
            if what == "set":
                assert own[name][".group_segment_fixed_size"] == 0
                limits.setdefault(name, set()).add(int(rest[0]))
            else:
                most[name] = max(most.get(name, 0), int(value))
    large = {n for n, size in most.items() if size > 65536}
    assert large == set(limits) and len(large) >= 5
    assert all(len(v) == 1 and min(v) == 160 * 1024 >= most[n] for n, v in limits.items())


def test_a_kernel_that_cannot_have_its_lds_is_not_launched(run):
    """Nor what follows it; the call says so, and the next one is as ever."""
    calls = [c for call in LARGE for c in ((1, *call), (0, *call))]
    got = run(*calls)
    for (rc, error, notes), (again, none, after) in zip(got[::2], got[1::2]):
        assert rc == 4 and "invalid" in error
        assert [n[0] for n in notes] == ["set"]
        assert again == 0 and none == "" and any(n[0] == "launch" for n in after)


def test_a_store_counts_its_tokens_in_32_bits(run):
    """The search for the end of a page's tokens looks up to 64 + 63 past the last one of a chunk:
    as cache_plan, a store takes 2^30 tokens at most."""
    most = 1 << 30
    got = run(*[(0, "store", (n, 1, 1, 64)) for n in (most, most + 1, 2 ** 31 - 1)],
              (0, "store", (2 ** 31 - 1, 1, 1, 64, "cache_load8")))
    assert [g[0] for g in got] == [0, 3, 3, 0]
    assert [len(g[2]) for g in got] == [1, 0, 0, 1]
    assert "too many tokens" in got[1][1]

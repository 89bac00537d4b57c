"""How prompt attention lays its grid out: the kernel's own search (csrc/prompt_items.cuh), compiled for
the host with 32 fibers as a warp's lanes.  A grid's places are taken as its CTAs take them, each
CTA a rising or arbitrary sequence of places with a search of its own: every query tile of every head
is then found exactly once, and places past the last item hold none."""
import collections
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RESIDENT = 304


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("prompt_items") / "prompt_items")
    r = subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-Wno-unknown-pragmas",
                        "-I", os.path.join(ROOT, "paged_kv_cache_73_gb300", "csrc"), "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "host_warp", "prompt_items.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def run(program, heads, max_len, qs, ks, ctas, total_q=None, total_k=None):
    text = [heads, max_len, qs[-1] if total_q is None else total_q, ks[-1] if total_k is None else total_k, len(qs) - 1,
            *qs, *ks, len(ctas)]
    for places in ctas:
        text += [len(places), *places]
    r = subprocess.run([program], input=" ".join(map(str, text)), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.splitlines()
    return (int(lines[0].split()[1]), [tuple(map(int, x.split())) for x in lines[1:-1]],
            int(lines[-1].split()[1]))


def starts(lens):
    return [0] + np.cumsum(lens).tolist()


def tiles_of(heads, news, past):
    """Every (head, q_row, rows, first_pos, k_row, keys)."""
    qs, ks = starts(news), starts([a + b for a, b in zip(news, past)])
    return {(h, qs[s] + i, min(n - i, 128), past[s] + i, ks[s], n + past[s])
            for h in range(heads) for s, n in enumerate(news) for i in range(0, n, 128)}


def check(program, heads, news, past, ctas_of, max_len=None):
    qs, ks = starts(news), starts([a + b for a, b in zip(news, past)])
    max_len = max(news) if max_len is None else max_len
    tiles, _, _ = run(program, heads, max_len, qs, ks, [])
    _, items, codes = run(program, heads, max_len, qs, ks, ctas_of(tiles * heads))
    assert codes == 0
    got = collections.Counter(x[1:7] for x in items)
    want = tiles_of(heads, news, past)
    again = sum(got.values()) - len(got)
    assert set(got) == want and again == 0, f"{again} items found again, of {len(want)} {len(want - set(got))} not found"
    for _, _, _, rows, first_pos, _, keys, n_tiles, edge in items:
        assert n_tiles == (first_pos + rows - 1) // 64 + 1 and edge == min((first_pos + 1) // 64, keys // 64)


def in_order(resident):
    """Each of `resident` CTAs starts at its own place and takes every `resident`-th further one."""
    return lambda places: [list(range(c, places, resident)) for c in range(min(resident, places))]


@pytest.mark.parametrize("heads,news", [(40, [4096] + [500] * 30 + [400]), (32, [16384] + [2000] * 31),
                                        (40, [2048] + [64] * 31), (2, [130] * 3 + [0] * 40 + [900])])
def test_one_long_prompt_among_short_ones(program, heads, news):
    check(program, heads, news, [0] * len(news), in_order(RESIDENT))
    check(program, heads, news, [0] * len(news), in_order(5))


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(program, seed):
    # CTAs take places in any order and number
    rng = np.random.default_rng(seed)
    S = int(rng.integers(1, 80))
    news = [int(x) for x in rng.choice([0, 1, 64, 128, 129, 500, 3000], S)]
    past = [int(x) for x in rng.choice([0, 1, 63, 64, 1000], S)]
    if sum(news) == 0:
        news[0] = 1

    def ctas(places):
        order = rng.permutation(places) if seed % 2 else np.arange(places)
        owner = rng.integers(0, max(1, min(60, places)), places)
        return [order[owner == c].tolist() for c in range(owner.max() + 1)]

    check(program, int(rng.integers(1, 12)), news, past, ctas, max(news) + int(rng.choice([0, 0, 700])))


def test_places_past_the_end(program):
    # a CTA that keeps asking far past the last item gets none, and still finds earlier ones after that
    news = [700] + [20] * 9
    qs = starts(news)
    tiles, _, _ = run(program, 3, 700, qs, qs, [])
    every = list(range(tiles * 3))
    _, items, _ = run(program, 3, 700, qs, qs, [every + [10 ** 6, 10 ** 6 + 1, 2 * 10 ** 6] + every[::-1]])
    counts = collections.Counter(x[1:7] for x in items)
    assert set(counts) == tiles_of(3, news, [0] * 10) and set(counts.values()) == {2}


def test_bad_ranges_are_reported(program):
    # rows outside q or key, more queries than keys; the other sequences' tiles are there
    _, items, codes = run(program, 1, 300, [0, 100, 400, 500], [0, 100, 390, 500], [[0, 1, 2, 3, 4, 5]])
    assert codes > 0 and sorted(x[2] for x in items) == [0, 400]
    _, items, codes = run(program, 1, 300, [0, 100, 400], [0, 100, 400], [[0, 1, 2, 3, 4]], total_k=399)
    assert codes > 0 and [x[2] for x in items] == [0]


@pytest.mark.parametrize("max_len", [10, 59, 99, 100])
def test_more_queries_than_announced_are_reported(program, max_len):
    qs = starts([100, 60, 5])
    _, items, codes = run(program, 1, max_len, qs, qs, [[0, 1, 2, 3]])
    assert (codes > 0) == (max_len < 100) and sorted(x[3] for x in items) == [5, 60, 100]

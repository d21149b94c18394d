"""The split of the paged attention's work, as compiled: csrc/kvpop_paged_split.cuh
is the kernel's own code, built here as plain C++ (paged_split_host.cpp) with
loops for the lanes of a warp."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fixed_budget_kv_kvpop_b200", "csrc")
WARPS, RANGES, MOST = 4, 1024, 1 << 30


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("split") / "split.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", "-ftrapv", "-I" + CSRC,
                    os.path.join(HERE, "paged_split_host.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.split_items.restype = lib.split_slot.restype = ctypes.c_int64
    return lib


def items(lib, lens, hkv, kb, most, tokens, window=0, f32=False):
    """Rows (cta, warp, b, h, j, jend, first, parts, slot, at) and what the split chose."""
    lens = np.ascontiguousarray(lens, np.int32)
    room = 400000
    out, how = np.zeros((room, 10), np.int64), np.zeros(7, np.int64)
    P64, P32 = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32)
    n = lib.split_items(kb, int(f32), lens.ctypes.data_as(P32), len(lens), hkv, window, ctypes.c_int64(tokens), most, WARPS,
                        out.ctypes.data_as(P64), ctypes.c_int64(room), how.ctypes.data_as(P64))
    assert 0 <= n <= room
    return out[:n], dict(zip(("grid", "fixed", "groups", "share", "total", "aligned", "solo"), map(int, how)))


def check(lib, lens, hkv, kb, most, tokens, window=0, f32=False):
    """Every attended block of every sequence and head in one item; the parts of
    a sequence know each other; a partial has a slot of its own inside the
    scratch, the one that the join reads; no more than two of a CTA."""
    rows, how = items(lib, lens, hkv, kb, most, tokens, window, f32)
    n = np.clip(np.asarray(lens, np.int64), 0, min(tokens, MOST))
    lo = np.where((window > 0) & (n > window), n - window, 0)
    begin, end = lo // kb, -(-n // kb)
    if not how["fixed"]:
        assert how["total"] == int((end - begin).sum())
    cover, used, open_items = {}, {}, {}
    for cta, warp, b, h, j, jend, first, parts, slot, at in rows.tolist():
        assert begin[b] <= j < jend <= end[b] and 0 <= h < hkv
        cover.setdefault((b, h), []).append((j, jend, parts, slot, cta, first))
        if parts > 1:
            assert 0 <= slot < 2 * RANGES and slot not in used, (slot, used.get(slot))
            used[slot] = (b, h)
            open_items[cta] = open_items.get(cta, 0) + 1
    assert not open_items or max(open_items.values()) <= 2
    for b in range(len(lens)):
        for h in range(hkv):
            got = sorted(cover.pop((b, h), []))
            want = [begin[b]] + [x[1] for x in got]
            assert [x[0] for x in got] == want[:-1] and want[-1] == end[b], (b, h, got, begin[b], end[b])
            assert all(x[2] == len(got) and x[5] == got[0][5] for x in got)
            if len(got) > 1:
                # the slots that the join of any part reads, in order
                second = got[0][3] != lib.split_slot(got[0][5], 0, h, 0, hkv)
                assert [x[3] for x in got] == [lib.split_slot(got[0][5], int(second), h, i, hkv) for i in range(len(got))]
    assert not cover
    return rows, how


@pytest.mark.parametrize("seed", range(60))
def test_every_block_has_one_item(lib, seed):
    rng = np.random.default_rng(seed)
    hkv, most = int(rng.choice([1, 2, 3, 8, 40, 700])), int(rng.choice([4, 296, 444, 592]))
    kb, window = int(rng.choice([8, 16, 32, 64])), int(rng.choice([0, 0, 1, 100, 5000]))
    lens = rng.integers(-2, kb * int(rng.choice([2, 17, 40, 700])), size=rng.integers(1, 90))
    if seed % 3 == 0:
        lens[0] *= 50
    if seed % 4 == 0:
        lens[:] = max(lens[0], 1)
    check(lib, lens, hkv, kb, most, int(rng.choice([max(lens.max(), 16), 100000])), window, f32=kb == 8)


@pytest.mark.parametrize("hkv,batch,most,fixed", [(1, 1, 444, 4), (8, 2, 444, 20), (3, 70, 444, 1)])
def test_fixed_parts(lib, hkv, batch, most, fixed):
    tokens = fixed * 8 * 16
    lens = np.random.default_rng(batch).integers(0, tokens + 1, size=batch)
    lens[0] = tokens
    _, how = check(lib, lens, hkv, 16, most, tokens)
    assert how["fixed"] == fixed and how["grid"] == hkv * batch * fixed


@pytest.mark.parametrize("hkv,batch,kb,f32", [(8, 512, 16, False), (3, 300, 32, False), (40, 1024, 8, True), (700, 5, 16, False)])
def test_short_sequences_go_to_single_warps(lib, hkv, batch, kb, f32):
    """One item for each sequence and head that has tokens, the warps' counts even to one where none is empty."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(1, 65 if f32 else 257, size=batch)
    rows, how = check(lib, lens, hkv, kb, 444, 4096, f32=f32)
    assert how["solo"] and len(rows) == hkv * batch
    per = np.bincount(rows[:, 0] * WARPS + rows[:, 1], minlength=how["grid"] * WARPS)
    assert per.max() - per.min() <= 1
    lens[rng.random(batch) < 0.3] = 0
    check(lib, lens, hkv, kb, 444, 4096, f32=f32)


@pytest.mark.parametrize("kb,batch,hkv,most", [(8, 32, 8, 444), (8, 64, 1, 296), (16, 64, 1, 296), (8, 1024, 8, 444), (16, 1024, 8, 444),
                                               (64, 1024, 300, 444), (16, 40, 300, 444), (8, 33, 8, 444)])
def test_the_longest_sequences(lib, kb, batch, hkv, most):
    """2^30 tokens in every sequence (their tables may share pages): 2^27 blocks of 8 tokens each, 2^32 of 32 sequences."""
    rows, how = check(lib, [MOST] * batch, hkv, kb, most, MOST, f32=kb == 8)
    assert how["total"] == batch * (MOST // kb)
    assert how["groups"] * how["share"] >= how["total"] or how["aligned"]
    lens = np.full(batch, MOST)
    lens[::3] = np.arange(len(lens[::3])) * 1000
    check(lib, lens, hkv, kb, most, MOST, f32=kb == 8)


def test_the_longest_window(lib):
    for kb in (8, 16, 32, 64):
        check(lib, [MOST, 5, MOST - 7], 2, kb, 444, MOST, window=2 ** 31 - 1)
        check(lib, [MOST] * 40, 8, kb, 444, MOST, window=MOST // 2 + 1, f32=kb == 8)

"""Paged cache and heads: the oracle's own checks, and every refusal that needs no GPU."""
import ctypes
import importlib.util
import os
import struct
import subprocess
import sys

import numpy as np
import pytest
import torch

import fixed_budget_kv_kvpop_b200 as kp
from oracle import paged_oracle as po

ROWS = struct.Struct("@Pqqq")     # kvpop_rows
CFG = dict(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=10, max_batch=4)


def _bytes(**kw):
    cfg = kp.make_paged_config(**{**CFG, **kw})
    n = ctypes.c_size_t(0)
    return kp.lib.kvpop_paged_bytes(ctypes.byref(cfg), ctypes.byref(n)), n.value


# ---- oracle ----

def test_e4m3_rounding_matches_torch():
    x = np.concatenate([np.linspace(-460, 460, 40001), np.random.default_rng(0).normal(size=20000) * 0.02,
                        po.e4m3_grid(), -po.e4m3_grid()])
    x = x.astype(np.float32)
    got = po.round_e4m3(x.astype(np.float64))
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(got, want)


def test_held_rows():
    """The largest magnitude of a row stands for 448, half of it for 224; tiny and zero rows are zeros; bad rows are NaN."""
    x = np.array([[1.0, -0.5, 0.25, 0.0], [0, 0, 0, 0], [1e-37, 0, 0, 0], [np.inf, 1, 1, 1], [1, np.nan, 1, 1]])
    h, s = po.hold_e4m3(x)
    np.testing.assert_array_equal(h[0], [448, -224, 112, 0])
    assert s[0] == np.float32(1.0) / np.float32(448)
    assert (h[1] == 0).all() and s[1] == 0 and (h[2] == 0).all() and s[2] == 0
    assert np.isnan(h[3:]).all() and np.isnan(s[3:]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_keep_norm_and_relative_angle(interleaved):
    """A rotation keeps lengths, and q . k depends on the distance of the two positions alone."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(6, 2, 64))
    f = 1e4 ** (-np.arange(0, 64, 2) / 64)
    y = po.heads(x, None, 0.0, np.arange(6) * 1000, f, interleaved=interleaved)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    q, k = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    dots = [float((po.heads(q, None, 0, [p + 5], f, interleaved=interleaved)
                   * po.heads(k, None, 0, [p], f, interleaved=interleaved)).sum()) for p in (0, 77, 123456)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-8)


def test_heads_hand_example():
    """Weights 2, one pair turned by a right angle: (a, b) -> (-b, a); the rest stays."""
    x = np.array([[[3.0, 0, 0, 0, 4.0, 0, 0, 0] + [0.0] * 8]])
    y = po.heads(x, np.full(16, 2.0), 0.0, [1], [np.pi / 2, 0, 0, 0])
    rms = 5.0 / 4.0
    np.testing.assert_allclose(y[0, 0, :8], np.array([-4.0, 0, 0, 0, 3.0, 0, 0, 0]) * 2 / rms, atol=1e-14)


def test_attend_matches_softmax():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(6, 64)), rng.normal(size=(9, 2, 64)), rng.normal(size=(9, 2, 64))
    out, lse = po.attend(q, k, v)
    for h in range(6):
        s = torch.from_numpy(k[:, h // 3] @ q[h]) / 8.0
        np.testing.assert_allclose(out[h], (torch.softmax(s, 0) @ torch.from_numpy(v[:, h // 3])).numpy(), rtol=1e-12)
        np.testing.assert_allclose(lse[h], torch.logsumexp(s, 0).item(), rtol=1e-12)
    wide, _ = po.attend(q, k, v, window=9)
    np.testing.assert_array_equal(wide, out)
    one, l1 = po.attend(q, k, v, window=1)
    np.testing.assert_allclose(one[0], v[-1, 0], rtol=1e-12)
    none, l0 = po.attend(q, k[:0], v[:0])
    assert (none == 0).all() and (l0 == -np.inf).all()


# ---- refusals ----

@pytest.mark.parametrize("kw,code", [
    (dict(n_layers=0), kp.KVPOP_ERR_BAD_SHAPE), (dict(n_pages=0), kp.KVPOP_ERR_BAD_SHAPE),
    (dict(max_batch=0), kp.KVPOP_ERR_BAD_SHAPE), (dict(max_batch=1025), kp.KVPOP_ERR_BAD_SHAPE),
    (dict(n_q_heads=7), kp.KVPOP_ERR_BAD_SHAPE), (dict(n_q_heads=34), kp.KVPOP_ERR_BAD_SHAPE),   # 17 heads per KV head
    (dict(head_dim=96), kp.KVPOP_ERR_BAD_SHAPE), (dict(page_size=8), kp.KVPOP_ERR_BAD_SHAPE),
    (dict(page_size=48), kp.KVPOP_ERR_BAD_SHAPE), (dict(page_size=512), kp.KVPOP_ERR_BAD_SHAPE),
    (dict(n_pages=1 << 27), kp.KVPOP_ERR_BAD_SHAPE),                                             # 2^31 rows
    (dict(n_kv_heads=1025, n_q_heads=1025), kp.KVPOP_ERR_BAD_SHAPE),
    (dict(dtype="f32", cache="e4m3"), kp.KVPOP_ERR_INVALID_ARG),
])
def test_bad_paged_configs_are_refused(kw, code):
    assert _bytes(**kw)[0] == code


def test_paged_bytes_count_rows_and_scales():
    rows = 2 * 10 * 2 * 2 * 16        # layers, pages, heads, key and value, page_size
    st, n = _bytes()
    assert st == kp.KVPOP_OK and n >= rows * 256
    st, n8 = _bytes(cache="e4m3")
    assert st == kp.KVPOP_OK and rows * (128 + 4) <= n8 < n
    st, big = _bytes(n_layers=80, n_pages=1 << 20, page_size=256, n_kv_heads=64, n_q_heads=64)
    assert st == kp.KVPOP_OK and big > 80 * (1 << 20) * 256 * 64 * 2 * 256


def test_unknown_codes_are_refused():
    cfg = kp.make_paged_config(**CFG)
    n = ctypes.c_size_t(0)
    cfg.dtype = 7
    assert kp.lib.kvpop_paged_bytes(ctypes.byref(cfg), ctypes.byref(n)) == kp.KVPOP_ERR_INVALID_ARG
    cfg.dtype, cfg.cache_format = kp.KVPOP_DTYPE_BF16, 2
    assert kp.lib.kvpop_paged_bytes(ctypes.byref(cfg), ctypes.byref(n)) == kp.KVPOP_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="cache format"):
        kp.make_paged_config(**CFG, cache="int8")


def test_null_handles_and_host_memory_are_refused():
    bad = kp.KVPOP_ERR_INVALID_ARG
    L = kp.lib
    assert L.kvpop_paged_bytes(None, None) == bad
    assert L.kvpop_paged_append(None, 0, None, None, None, 1, 1, None) == bad
    assert L.kvpop_paged_append_qkv(None, 0, None, None, None, None, None, None, None, 1, 1, None) == bad
    assert L.kvpop_paged_gather(None, 0, None, 1, 1, None, 1, 1, None, None, None) == bad
    assert L.kvpop_paged_attend(None, 0, None, None, 1, 1, None, 1, None, None, None, None) == bad
    assert L.kvpop_paged_get_layout(None, None) == bad
    assert L.kvpop_paged_get_error(None, None) == bad
    assert L.kvpop_paged_clear_error(None, None) == bad
    assert L.kvpop_paged_destroy(None) == bad
    cfg = kp.make_paged_config(**CFG)
    n = kp.paged_bytes(cfg)
    buf = ctypes.create_string_buffer(n + 256)
    h = ctypes.c_void_p()
    addr = (ctypes.addressof(buf) + 255) // 256 * 256
    assert L.kvpop_paged_create(ctypes.byref(cfg), ctypes.c_void_p(addr), n, ctypes.byref(h)) == bad
    assert not h.value
    assert L.kvpop_paged_create(ctypes.byref(cfg), None, n, ctypes.byref(h)) == bad


def _heads_call(dtype=kp.KVPOP_DTYPE_BF16, d=128, hq=4, hkv=2, rope=None, batch=1, n=1, addr=None, strides=(0, 0, 128),
                pos=64):
    """kvpop_qk_norm_rope on host memory: every argument but that is in order."""
    buf = ctypes.create_string_buffer(8192)
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    r = ROWS.pack(base if addr is None else addr, *strides)
    rope = kp._pack_rope(0, 0, base, 1e-6, 1.0, 128, 0) if rope is None else rope
    return kp.lib.kvpop_qk_norm_rope(dtype, d, hq, hkv, rope, batch, n, r, r, base + pos if pos else None, r, r, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), kp.KVPOP_ERR_INVALID_ARG), (dict(d=80), kp.KVPOP_ERR_BAD_SHAPE),
    (dict(hq=0), kp.KVPOP_ERR_BAD_SHAPE), (dict(hkv=2000), kp.KVPOP_ERR_BAD_SHAPE),
    (dict(batch=-1), kp.KVPOP_ERR_INVALID_ARG), (dict(n=-1), kp.KVPOP_ERR_INVALID_ARG),
    (dict(rope=kp._pack_rope(0, 0, 4096, 1e-6, 1.0, 132, 0)), kp.KVPOP_ERR_BAD_SHAPE),    # rot_dim past head_dim
    (dict(rope=kp._pack_rope(0, 0, 4096, 1e-6, 1.0, 20, 0)), kp.KVPOP_ERR_BAD_SHAPE),     # not a multiple of 8
    (dict(rope=kp._pack_rope(0, 0, 0, 1e-6, 1.0, 64, 0)), kp.KVPOP_ERR_INVALID_ARG),      # no frequencies
    (dict(rope=kp._pack_rope(8, 0, 4096, 1e-6, 1.0, 64, 0)), kp.KVPOP_ERR_INVALID_ARG),   # misaligned weights
    (dict(rope=kp._pack_rope(0, 0, 4096, -1.0, 1.0, 64, 0)), kp.KVPOP_ERR_INVALID_ARG),
    (dict(rope=kp._pack_rope(0, 0, 4096, float("nan"), 1.0, 64, 0)), kp.KVPOP_ERR_INVALID_ARG),
    (dict(rope=kp._pack_rope(0, 0, 4096, 1e-6, float("inf"), 64, 0)), kp.KVPOP_ERR_INVALID_ARG),
    (dict(rope=kp._pack_rope(0, 0, 4096, 1e-6, 1.0, 64, 2)), kp.KVPOP_ERR_INVALID_ARG),
    (dict(addr=0), kp.KVPOP_ERR_INVALID_ARG), (dict(addr=4104), kp.KVPOP_ERR_INVALID_ARG),
    (dict(strides=(0, 0, -128)), kp.KVPOP_ERR_INVALID_ARG), (dict(strides=(0, 0, 129)), kp.KVPOP_ERR_INVALID_ARG),
    (dict(strides=(0, 0, 0)), kp.KVPOP_ERR_INVALID_ARG),                                   # an output expanded over heads
    (dict(pos=0), kp.KVPOP_ERR_INVALID_ARG), (dict(pos=66), kp.KVPOP_ERR_INVALID_ARG),
    (dict(), kp.KVPOP_ERR_INVALID_ARG),                                                    # host memory
    (dict(batch=0), kp.KVPOP_OK), (dict(n=0), kp.KVPOP_OK),
])
def test_heads_refusals(kw, code):
    assert _heads_call(**kw) == code


def test_binding_refuses_what_is_not_a_cuda_tensor():
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="cuda"):
        kp.make_rope(f)
    q, pos = torch.zeros(1, 1, 4, 64), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="Rope"):
        kp.qk_norm_rope(None, q, q, pos, q, q)
    rope = (bytes(40), 0, 64)
    with pytest.raises(ValueError, match="cuda"):
        kp._binding.qk_norm_rope(kp._FN["kvpop_qk_norm_rope"], rope, q, q, pos, q, q, None)
    with pytest.raises(ValueError, match="torch.Tensor"):
        kp._binding.qk_norm_rope(kp._FN["kvpop_qk_norm_rope"], rope, [1.0], q, pos, q, q, None)
    with pytest.raises(ValueError, match="batch"):
        kp._binding.qk_norm_rope(kp._FN["kvpop_qk_norm_rope"], rope, q[0], q, pos, q, q, None)
    with pytest.raises(TypeError):
        kp._binding.qk_norm_rope(kp._FN["kvpop_qk_norm_rope"], rope)
    cache = (0, 4, 4, 64, kp.KVPOP_DTYPE_F32, 0)
    with pytest.raises(ValueError, match="k: on cpu, expected the cuda device 0"):
        kp._binding.append(kp._FN["kvpop_paged_append"], cache, 0, q, q, pos, None)
    with pytest.raises(ValueError, match="q: on cpu"):
        kp._binding.attend(kp._FN["kvpop_paged_attend"], cache, 0, q[0], pos, pos, q[0], None, 0.0, 0.0, 0, None)
    with pytest.raises(ValueError, match="32 bits"):
        kp._binding.append(kp._FN["kvpop_paged_append"], cache, 1 << 40, q, q, pos, None)
    with pytest.raises(ValueError, match="six"):
        kp._binding.append(kp._FN["kvpop_paged_append"], (0, 4), 0, q, q, pos, None)


# ---- the attention's work split, restated from kvpop_paged_attn.cu ----

NW, MIN_SHARE, RANGES = 4, 8, 1024


def _split(blocks, hkv, n_cta):
    """(share, groups, aligned)"""
    total, longest, seqs = sum(blocks), max(blocks), sum(n > 0 for n in blocks)
    groups = max(1, n_cta // hkv)
    share = min(max(-(-total // groups), MIN_SHARE), 1 << 30)
    if not 0 < seqs <= groups:
        return share, groups, False

    def fits(s):
        return sum(min(-(-n // s), groups + 1) for n in blocks) <= groups

    lo, hi = share, -(-longest // (groups // seqs))
    if hi <= lo or fits(lo):
        hi = lo
    else:
        while hi - lo > 1 + lo // 32:
            mid = lo + (hi - lo) // 2
            lo, hi = (lo, mid) if fits(mid) else (mid, hi)
    return (hi, groups, True) if hi <= share + share // 5 + 16 else (share, groups, False)


def _items(cta, blocks, hkv, n_cta, share, groups, aligned):
    """A CTA's items: (b, h, j, jend, first, parts, second)."""
    many = hkv > n_cta
    grp = 0 if many else cta // hkv
    out = []
    for h in range(cta if many else cta - grp * hkv, hkv, n_cta):
        if grp >= groups:
            return out
        target = grp if aligned else grp * share
        before = 0
        for b, n in enumerate(blocks):
            own = -(-n // share) if aligned else n
            if before + own > target:
                break
            before += own
        else:
            return out
        skip = target - before
        if aligned:
            out.append((b, h, skip * share, min((skip + 1) * share, n), grp - skip, own, 0))
            continue
        pos, left = target, min(share, sum(blocks) - target)
        while True:
            n, beg = blocks[b], pos - skip
            jend = min(n, skip + left)
            first = beg // share
            out.append((b, h, skip, jend, first, (beg + n - 1) // share - first + 1, int(beg != first * share)))
            left -= jend - skip
            pos += jend - skip
            if left <= 0:
                break
            b, skip = b + 1, 0
            while blocks[b] == 0:
                b += 1
    return out


@pytest.mark.parametrize("seed", range(40))
def test_attention_work_split(seed):
    """Every block of every head is covered once; no range is larger than the
    share; the partials that the last arriver reads are the ones that were
    written, each in a slot of its own inside the scratch."""
    rng = np.random.default_rng(seed)
    hkv, n_cta = int(rng.choice([1, 2, 3, 8, 700])), int(rng.choice([4, 296, 592]))
    blocks = [int(x) for x in rng.integers(0, rng.choice([5, 17, 40, 700]), size=rng.integers(1, 90))]
    if seed % 3 == 0:
        blocks[0] *= 50
    if seed % 4 == 0:
        blocks = [max(blocks[0], 1)] * len(blocks)
    share, groups, aligned = _split(blocks, hkv, n_cta)
    cover, written, read, used = {}, {}, {}, set()
    for cta in range(n_cta):
        items = _items(cta, blocks, hkv, n_cta, share, groups, aligned)
        assert sum(x[3] - x[2] for x in items) <= share * -(-hkv // n_cta)
        for b, h, j, jend, first, parts, second in items:
            assert j < jend
            cover.setdefault((b, h), []).append((j, jend, parts))
            own = [list(range(j + ((w - j) & (NW - 1)), jend, NW)) for w in range(NW)]
            assert sorted(sum(own, [])) == list(range(j, jend))
            if parts > 1:
                def slot_of(i):
                    return (2 * (first + i) + (second if i == 0 else 0)) * hkv + h
                mine = slot_of(cta // hkv - first)
                assert mine not in used and mine < 2 * n_cta <= 2 * RANGES
                used.add(mine)
                written.setdefault((b, h), set()).add(mine)
                if (b, h) not in read:
                    read[b, h] = {slot_of(i) for i in range(parts)}
    for b, n in enumerate(blocks):
        for h in range(hkv):
            got = sorted(cover.get((b, h), []))
            assert [x[0] for x in got] == ([0] + [x[1] for x in got[:-1]])[:len(got)]
            assert (got[-1][1] if got else 0) == n
            assert all(x[2] == len(got) for x in got)
    assert read == written


@pytest.mark.parametrize("seed", range(20))
def test_attention_fixed_parts(seed):
    """Narrow tables: parts of MIN_SHARE blocks, as many groups for each sequence as its longest would need."""
    rng = np.random.default_rng(seed)
    hkv, fixed, batch = int(rng.choice([1, 2, 8])), int(rng.integers(1, 9)), int(rng.integers(1, 9))
    blocks = [int(x) for x in rng.integers(0, fixed * MIN_SHARE + 1, size=batch)]
    n_cta = hkv * batch * fixed
    cover, used = {}, set()
    for cta in range(n_cta):
        grp, h = divmod(cta, hkv)
        b, part = divmod(grp, fixed)
        if part * MIN_SHARE >= blocks[b]:
            continue
        parts, first = -(-blocks[b] // MIN_SHARE), grp - part
        cover.setdefault((b, h), []).append((part * MIN_SHARE, min((part + 1) * MIN_SHARE, blocks[b])))
        slot = 2 * (first + part) * hkv + h
        assert slot not in used and slot < 2 * n_cta and len(cover[b, h]) <= parts
        used.add(slot)
    for b, n in enumerate(blocks):
        for h in range(hkv):
            got = sorted(cover.get((b, h), []))
            assert [x[0] for x in got] == ([0] + [x[1] for x in got[:-1]])[:len(got)] and (got[-1][1] if got else 0) == n


@pytest.mark.parametrize("kb", [8, 16, 32, 64])
def test_blocks_of_a_window(kb):
    """A window of w tokens touches at most w / kb + 2 blocks, wherever it ends."""
    for w in range(1, 300):
        assert max((n + kb - 1) // kb - max(n - w, 0) // kb for n in range(1, 400)) <= w // kb + 2


# ---- what the package needs to load ----

@pytest.mark.parametrize("without", ["torch", "binding", "broken binding"])
def test_the_fixed_budget_calls_need_neither_torch_nor_the_binding(tmp_path, without):
    """_binding.so is built for one torch and one Python: without it, or without
    torch, the package loads and its ctypes calls work; the paged ones say what is missing."""
    package = tmp_path / "fixed_budget_kv_kvpop_b200"
    package.mkdir()
    (package / "__init__.py").write_text(open(kp.__file__).read())
    if without == "broken binding":
        (package / "_binding.so").write_bytes(b"built for another Python")
    code = """
import sys
if WITHOUT == "torch":
    sys.modules["torch"] = None
import fixed_budget_kv_kvpop_b200 as kp
cfg = kp.make_config(batch=1, n_layers=1, n_q_heads=8, n_kv_heads=2, head_dim=128, sinks=4, window=16, topk=16,
                     external_scores=True)
assert kp.cache_bytes(cfg) > 0
paged = kp.make_paged_config(n_layers=1, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=4, max_batch=1)
assert kp.paged_bytes(paged) > 0
for make in (lambda: kp.KVPopPagedCache(paged), lambda: kp.Rope(None, None, None, 0.0, 1.0, False), lambda: kp._binding):
    try:
        make()
    except ImportError as e:
        assert "torch" in str(e) if WITHOUT == "torch" else "build.py" in str(e), e
    else:
        raise AssertionError("made without its binding")
try:
    kp.qk_norm_rope(None, None, None, None, None, None)
except ValueError as e:
    assert "make_rope" in str(e)
try:
    kp.nothing
except AttributeError as e:
    assert "nothing" in str(e)
print("ok")
"""
    env = {**os.environ, "KVPOP_LIBRARY": kp.LIB_PATH, "PYTHONPATH": str(tmp_path)}
    r = subprocess.run([sys.executable, "-c", f"WITHOUT = {without!r}" + code], capture_output=True, text=True, env=env, cwd=tmp_path)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


@pytest.mark.parametrize("change", ["nothing", "torch", "python", "compiler", "source"])
def test_the_binding_is_built_again_for_another_torch_or_python(tmp_path, monkeypatch, change):
    """_binding.so reads torch's and Python's structures as they were when it was compiled."""
    spec = importlib.util.spec_from_file_location("kvpop_build", os.path.join(os.path.dirname(kp.__file__), "csrc", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    monkeypatch.setattr(build, "BINDING_OUT", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "_binding.txt"), raising=False)
    runs = []

    def compiler(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build_binding()
    build.build_binding()
    assert len(runs) == 1
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0")
    elif change == "python":
        monkeypatch.setattr(sys, "version", "0.0")
    elif change == "compiler":
        monkeypatch.setenv("CXX", "another")
    elif change == "source":
        os.utime(build.BINDING_OUT, (0, 0))
    build.build_binding()
    assert len(runs) == (1 if change == "nothing" else 2)
    build.build_binding()
    assert len(runs) == (1 if change == "nothing" else 2)


@pytest.mark.parametrize("what,value", [("TORCH", "1.0.0"), ("PYTHON", 0x0301)])
def test_a_binding_of_another_torch_or_python_is_refused(monkeypatch, what, value):
    monkeypatch.setattr(kp._binding, what, value)
    with pytest.raises(ImportError, match="built for .* 1.0.0|built for .*Python 3.1.*build.py"):
        kp.Rope(None, None, None, 0.0, 1.0, False)

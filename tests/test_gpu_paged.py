"""Heads and paged cache on the GPU against the float64 oracle.

Tolerances, fixed before the first run.  u = 2^-24 (fp32), half a step of the
output type relative to the value (`eps / 2`).
  heads   x / rms * w: 64 u relative (a sum of d squares, a root, three
          products); a turned value is a sum of two products of such terms with
          cosine and sine off by 4 u: 128 u (|a| + |b|) |rot_scale|, then one rounding.
  held    of bf16 rows: equal (amax, one product for the scale and one division
          per element are exact operations or single roundings).
  attend  oracle.paged_oracle.attend_slack, then one rounding.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import fixed_budget_kv_kvpop_b200 as kp
from oracle import paged_oracle as po

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(TORCH[dtype]).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TORCH[dtype]).cuda()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def cache_of(hq, hkv, d, page, n_pages, dtype="bf16", cache="native", max_batch=64, n_layers=1):
    return kp.KVPopPagedCache(kp.make_paged_config(n_layers=n_layers, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                                                   page_size=page, n_pages=n_pages, max_batch=max_batch, dtype=dtype,
                                                   cache=cache))


def tables(lens, page, seed=0, spare=2):
    """Pages in a random order: table (one column more than needed, -1 behind the last page) and the pool's size."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    order = np.random.default_rng(seed).permutation(n_pages)
    t = np.full((len(lens), max(need) + 1), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        t[i, :m] = order[at:at + m]
        at += m
    return t, n_pages


def slots_of(table, lens, page, width):
    s = np.full((len(lens), width), -1, np.int32)
    for i, n in enumerate(lens):
        j = np.arange(n)
        s[i, :n] = table[i, j // page] * page + j % page
    return s


def held_rows(c, layer, table, n, page, b):
    """Tokens 0..n-1 of sequence b as the cache holds them, float64 [n][Hkv][2][d]."""
    p = f64(c.pages(layer).float())
    j = np.arange(n)
    x = p[table[b, j // page], :, :, j % page]
    if c.scales(layer) is not None:
        x = x * f64(c.scales(layer))[table[b, j // page], :, :, j % page][..., None]
    return x


# ---- heads ----

def heads_bound(x, w, eps, pos, freq, scale, inter, dtype):
    want = po.heads(x, w, eps, pos, freq, scale, inter)
    y = po.heads(x, w, eps, pos, np.zeros(0))
    size = np.abs(y)
    half = len(freq)
    ia, ib = (np.arange(half) * 2, np.arange(half) * 2 + 1) if inter else (np.arange(half), np.arange(half) + half)
    both = size[..., ia] + size[..., ib]
    size[..., ia], size[..., ib] = both * abs(scale), both * abs(scale)
    return want, half_step(dtype) * np.abs(want) + (128 * U) * size * 1.01 + 1e-38


@pytest.mark.parametrize("dtype,d,hq,hkv,rot,inter,norm,scale", [
    ("bf16", 128, 32, 8, 128, False, True, 1.0),
    ("bf16", 128, 5, 1, 64, False, True, 1.25),
    ("bf16", 64, 8, 8, 64, True, True, 1.0),
    ("bf16", 64, 3, 3, 24, False, True, 1.0),
    ("f32", 128, 7, 1, 128, True, True, 1.0),
    ("f32", 64, 4, 2, 64, False, True, 1.0),
    ("f32", 64, 6, 2, 8, True, False, 0.5),
    ("f32", 128, 2, 2, 0, False, True, 1.0),
    ("bf16", 128, 4, 4, 40, True, False, 1.0),
])
@pytest.mark.parametrize("b,n", [(1, 1), (3, 1), (2, 37), (1, 700)])
def test_heads(dtype, d, hq, hkv, rot, inter, norm, scale, b, n):
    """Views of a projection's rows in, head-major buffers out; positions far apart."""
    x = rows((b, n, hq + 2 * hkv, d), dtype, 5 + n)
    rng = np.random.default_rng(3)
    freq = 1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))
    w = [1 + 0.2 * rng.normal(size=d).astype(np.float32) for _ in range(2)] if norm else [None, None]
    rope = kp.make_rope(torch.from_numpy(freq).cuda(), interleaved=inter, scale=scale,
                        **({} if not norm else dict(q_weight=torch.from_numpy(w[0].astype(np.float32)).cuda(),
                                                    k_weight=torch.from_numpy(w[1].astype(np.float32)).cuda())))
    pos = rng.integers(0, 1 << 20, size=(b, n)).astype(np.int32)
    pos[0, 0] = 0
    pos[-1, -1] = 2 ** 31 - 1
    q, k = x[:, :, :hq], x[:, :, hq:hq + hkv]
    qo = torch.full((b, hq, n, d), 7.0, dtype=TORCH[dtype], device="cuda")
    ko = torch.full((b, hkv, n, d), 7.0, dtype=TORCH[dtype], device="cuda")
    kp.qk_norm_rope(rope, q, k, ints(pos), qo.transpose(1, 2), ko.transpose(1, 2))
    for got, src, weight in ((qo, q, w[0]), (ko, k, w[1])):
        for i in range(b):
            want, bound = heads_bound(f64(src[i]), weight, 1e-6, pos[i], freq, scale, inter, dtype)
            err = np.abs(f64(got[i]).transpose(1, 0, 2) - want)
            assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype,d,rot,inter", [("bf16", 128, 64, False), ("bf16", 128, 40, True), ("f32", 64, 24, False),
                                               ("f32", 64, 0, False), ("bf16", 64, 8, False), ("f32", 128, 120, True)])
def test_heads_nonfinite_elements_that_are_not_turned(dtype, d, rot, inter, norm):
    """An infinity or a NaN behind rot_dim reaches no other element but through the row's norm."""
    x = rows((1, 5, 4, d), dtype, 9)
    for t, (e, bad) in enumerate([(rot, math.inf), (d - 1, -math.inf), (d // 2 + 1 if d // 2 >= rot else d - 3, math.nan), (d - 2, math.inf)]):
        x[0, t, :, e] = bad
    freq = 1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))
    w = 1 + 0.2 * np.random.default_rng(2).normal(size=d).astype(np.float32)
    wt = torch.from_numpy(w).cuda()
    rope = kp.make_rope(torch.from_numpy(freq).cuda(), interleaved=inter, **(dict(q_weight=wt, k_weight=wt) if norm else {}))
    pos = np.array([[3, 1000, 77, 0, 9]], np.int32)
    qo, ko = torch.empty_like(x[:, :, :3]), torch.empty_like(x[:, :, 3:])
    kp.qk_norm_rope(rope, x[:, :, :3], x[:, :, 3:], ints(pos), qo, ko)
    with np.errstate(invalid="ignore"):
        for got, src in ((qo, x[:, :, :3]), (ko, x[:, :, 3:])):
            want, bound = heads_bound(f64(src[0]), w if norm else None, 1e-6, pos[0], freq, 1.0, inter, dtype)
            got = f64(got[0])
            assert (np.isnan(got) == np.isnan(want)).all()
            sure = np.isfinite(want)
            assert (got[~sure & ~np.isnan(want)] == want[~sure & ~np.isnan(want)]).all()
            assert (np.abs(got - want)[sure] <= bound[sure]).all()


@pytest.mark.parametrize("inter", [False, True])
def test_heads_at_negative_positions(inter):
    """Angles of positions below zero, down to the lowest."""
    x = rows((1, 6, 3, 64), "f32", 8)
    freq = 1e5 ** (-np.arange(0, 64, 2) / 64)
    # More than a turn per position; backwards.  At 2^31 the angle 9.5 pos is off by 2^31 ulp(1.5) / 2 = 2^-22 turns
    # (1.5e-6) here and by ulp(2e10) / 2 = 1.9e-6 in the formula: with the 4 U of the rest below the 128 U of the bound.
    freq[3], freq[5] = 9.5, -0.25
    rope = kp.make_rope(torch.from_numpy(freq).cuda(), interleaved=inter, eps=1e-6)
    pos = np.array([[-1, -2, -4097, 5, -2 ** 31, -2 ** 31 + 1]], np.int32)
    qo, ko = torch.empty_like(x[:, :, :2]), torch.empty_like(x[:, :, 2:])
    kp.qk_norm_rope(rope, x[:, :, :2], x[:, :, 2:], ints(pos), qo, ko)
    for got, src in ((qo, x[:, :, :2]), (ko, x[:, :, 2:])):
        want, bound = heads_bound(f64(src[0]), None, 1e-6, pos[0], freq, 1.0, inter, "f32")
        assert (np.abs(f64(got[0]) - want) <= bound).all()


def test_heads_in_place_and_broadcast_input():
    """q_out = q, k_out = k; and one key head expanded over four."""
    x = rows((2, 9, 6, 64), "bf16", 1)
    f = torch.from_numpy(1e4 ** (-np.arange(0, 64, 2) / 64)).cuda()
    rope = kp.make_rope(f, q_weight=torch.ones(64, device="cuda"))
    pos = ints(np.arange(18).reshape(2, 9))
    q, k = x[:, :, :4], x[:, :, 4:]
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kp.qk_norm_rope(rope, q, k, pos, qo, ko)
    wide = k[:, :, :1].expand(2, 9, 4, 64)
    wo = torch.empty(2, 9, 4, 64, dtype=x.dtype, device="cuda")
    kp.qk_norm_rope(rope, q, wide, pos, torch.empty_like(q), wo)
    for h in range(4):
        assert torch.equal(wo[:, :, h], ko[:, :, 0])
    kp.qk_norm_rope(rope, q, k, pos, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_heads_bad_rows_stay_in_their_row():
    """A row with a NaN, one with an infinity, one of zeros and huge ones do not touch others."""
    x = rows((1, 4, 3, 128), "f32", 2)
    good = x.clone()
    x[0, 1, 0, 5] = math.nan
    x[0, 2, 1, 9] = math.inf
    x[0, 3, 0] = 0
    x[0, 0, 2] *= 1e15
    rope = kp.make_rope(torch.ones(64, dtype=torch.float64, device="cuda"), q_weight=torch.ones(128, device="cuda"),
                        k_weight=torch.ones(128, device="cuda"))
    pos = ints([[0, 1, 2, 3]])
    out, ref = (torch.empty_like(x) for _ in range(2))
    kp.qk_norm_rope(rope, x[:, :, :2], x[:, :, 2:], pos, out[:, :, :2], out[:, :, 2:])
    kp.qk_norm_rope(rope, good[:, :, :2], good[:, :, 2:], pos, ref[:, :, :2], ref[:, :, 2:])
    assert out[0, 1, 0].isnan().all() and out[0, 2, 1].isnan().any() and (out[0, 3, 0] == 0).all()
    assert torch.isfinite(out[0, 0, 2]).all()
    keep = torch.ones(1, 4, 3, dtype=torch.bool)
    for t, h in ((1, 0), (2, 1), (3, 0), (0, 2)):
        keep[0, t, h] = False
    assert torch.equal(out[keep.cuda()], ref[keep.cuda()])


# ---- write and read ----

def check_held(c, layer, table, lens, page, k, v, slots, dtype, cache):
    """Every row that a slot names is held as the definition says; every other row is as created (zero)."""
    pages, scales = f64(c.pages(layer).float()), None if c.scales(layer) is None else f64(c.scales(layer))
    seen = np.zeros((pages.shape[0], page), bool)
    for b in range(slots.shape[0]):
        t = np.nonzero(slots[b] >= 0)[0]
        pg, r = slots[b, t] // page, slots[b, t] % page
        seen[pg, r] = True
        for i, x in enumerate((k[b, t], v[b, t])):
            got = pages[pg, :, i, r]
            if cache == "native":
                np.testing.assert_array_equal(got, x)
                continue
            want, s = po.hold_e4m3(x)
            np.testing.assert_array_equal(scales[pg, :, i, r], s)
            assert ((got == want) | np.isnan(s)[..., None]).all()
    assert (pages.transpose(0, 3, 1, 2, 4)[~seen] == 0).all()
    if scales is not None:
        assert (scales.transpose(0, 3, 1, 2)[~seen] == 0).all()


@pytest.mark.parametrize("dtype,cache,d,hkv,page", [
    ("bf16", "native", 128, 8, 16), ("bf16", "native", 64, 3, 64), ("bf16", "e4m3", 128, 8, 64),
    ("bf16", "e4m3", 64, 1, 16), ("bf16", "e4m3", 128, 5, 256), ("f32", "native", 64, 2, 32), ("f32", "native", 128, 1, 128),
])
@pytest.mark.parametrize("lens", [[1], [0, 1, 17, 40], [333, 64]])
def test_append_and_gather(dtype, cache, d, hkv, page, lens):
    b, n = len(lens), max(lens)
    table, n_pages = tables(lens, page, seed=n)
    slots = slots_of(table, lens, page, n)
    x = rows((b, n, 4 * hkv, d), dtype, 11)
    x[:, :, :hkv] *= 3
    k, v = x[:, :, :hkv], x[:, :, 2 * hkv:3 * hkv]
    c = cache_of(2 * hkv, hkv, d, page, n_pages, dtype, cache, n_layers=2)
    c.append(1, k, v, ints(slots))
    assert (c.pages(0).float() == 0).all()
    check_held(c, 1, table, lens, page, f64(k), f64(v), slots, dtype, cache)
    # read back into head-major buffers with room behind
    ko, vo = (torch.full((b, hkv, n + 3, d), 5.0, dtype=TORCH[dtype], device="cuda") for _ in range(2))
    c.gather(1, ints(table), ints(lens), ko.transpose(1, 2), vo.transpose(1, 2))
    for i, m in enumerate(lens):
        want = held_rows(c, 1, table, m, page, i)
        for got, w in ((ko, want[:, :, 0]), (vo, want[:, :, 1])):
            got = f64(got[i]).transpose(1, 0, 2)
            assert (np.abs(got[:m] - w) <= (half_step(dtype) + U) * np.abs(w) + 1e-38).all()
            assert (got[m:] == 5.0).all()
    assert c.get_error() == (kp.KVPOP_OK, 0)


def test_e4m3_special_rows():
    """Zero, tiny, huge, infinite and NaN rows."""
    x = rows((1, 6, 1, 64), "bf16", 4)
    x[0, 0] = 0
    x[0, 1] *= 1e-38
    x[0, 2] = 3e38
    x[0, 3, 0, 7] = math.inf
    x[0, 4, 0, 63] = math.nan
    c = cache_of(1, 1, 64, 16, 2, cache="e4m3")
    c.append(0, x, x, ints([[16, 17, 18, 19, 20, 21]]))
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    c.gather(0, ints([[1]]), ints([6]), ko, vo)
    assert torch.equal(ko.nan_to_num(9), vo.nan_to_num(9))
    assert (ko[0, :2] == 0).all() and ko[0, 3:5].isnan().all() and torch.isfinite(ko[0, 5]).all()
    assert (ko[0, 2].float() / x[0, 2].float() - 1).abs().max() <= 2.0 ** -8 + 2.0 ** -20
    assert (c.scales(0)[1, 0, 0, :2] == 0).all()


def rows_of_every_quotient(exponent, rng):
    """bf16 rows of 128: every significand as a row's largest element, 2^exponent
    times, over every significand of the 19 exponents from there down (what the
    scale brings below 2^-10 is held as zero), in float32."""
    sig = np.arange(128, 256) / 128.0
    small = (sig[None, :] * 2.0 ** -np.arange(0, 20)[:, None]).reshape(-1)
    out = []
    for m in sig:
        x = rng.permutation(np.concatenate([small[small <= m], small[: -(small <= m).sum() % 127]]))
        x = x.reshape(-1, 127) * rng.choice([-1, 1], size=(len(x) // 127, 127))
        out.append(np.concatenate([x, np.full((len(x), 1), m)], 1))
    return (np.concatenate(out) * 2.0 ** exponent).astype(np.float32)


@pytest.mark.parametrize("exponent", [0, -82, -90, -100, 120])
def test_e4m3_quotients_of_bf16_rows(exponent):
    """Every pair of a row's largest element and an element that is not held as
    zero, on both sides of 2^-90, where the quotients are formed differently."""
    x = rows_of_every_quotient(exponent, np.random.default_rng(1))
    n, d, page = len(x), 128, 256
    t = torch.from_numpy(x).to(torch.bfloat16).cuda().view(1, n, 1, d)
    assert np.array_equal(f64(t.float()).reshape(n, d), x.astype(np.float64))       # exact in bf16
    held, scale = po.hold_e4m3(x)
    slots, pos = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n), torch.zeros(1, n, dtype=torch.int32, device="cuda")
    rope = kp.make_rope(torch.empty(0, dtype=torch.float64, device="cuda"))
    for step in (False, True):
        c = cache_of(1, 1, d, page, -(-n // page), cache="e4m3")
        if step:
            c.append_qkv(0, rope, t, t, t, pos, slots, torch.empty_like(t))
        else:
            c.append(0, t, t, slots)
        got = f64(c.pages(0).float())[:, 0].transpose(1, 0, 2, 3).reshape(2, -1, d)[:, :n]
        gs = f64(c.scales(0))[:, 0].transpose(1, 0, 2).reshape(2, -1)[:, :n]
        for kv in range(2):
            assert np.array_equal(gs[kv], scale) and np.array_equal(got[kv], held)


def test_e4m3_quotients_of_fp32_rows():
    """Keys that append_qkv quantises from fp32: at position 0 without a norm they
    are x times the rotation's scale, rounded to fp32 once."""
    rng = np.random.default_rng(2)
    x = rows_of_every_quotient(0, rng)
    n, d, page = len(x), 128, 256
    t = torch.from_numpy(x).to(torch.bfloat16).cuda().view(1, n, 1, d)
    slots, pos = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n), torch.zeros(1, n, dtype=torch.int32, device="cuda")
    c = cache_of(1, 1, d, page, -(-n // page), cache="e4m3")
    freq, qo = torch.ones(d // 2, dtype=torch.float64, device="cuda"), torch.empty_like(t)
    for factor in rng.uniform(1, 2, size=25).astype(np.float32):
        c.append_qkv(0, kp.make_rope(freq, scale=float(factor)), t, t, t, pos, slots, qo)
        held, scale = po.hold_e4m3(x * factor)
        got = f64(c.pages(0).float())[:, 0, 0].reshape(-1, d)[:n]
        assert np.array_equal(f64(c.scales(0))[:, 0, 0].reshape(-1)[:n], scale) and np.array_equal(got, held)


@pytest.mark.parametrize("dtype,cache,d,hq,hkv,rot,inter,b,n", [
    ("bf16", "native", 128, 8, 2, 128, False, 3, 21), ("bf16", "e4m3", 128, 8, 2, 128, False, 3, 21),
    ("bf16", "e4m3", 64, 5, 5, 24, False, 2, 17), ("bf16", "e4m3", 128, 3, 1, 64, True, 1, 16),
    ("bf16", "native", 64, 32, 8, 40, False, 16, 1), ("f32", "native", 128, 6, 3, 128, True, 2, 40),
    ("f32", "native", 64, 4, 2, 24, False, 1, 900), ("bf16", "e4m3", 128, 64, 8, 96, False, 64, 1),
])
def test_append_qkv_is_heads_then_append(dtype, cache, d, hq, hkv, rot, inter, b, n):
    """Queries equal qk_norm_rope's bit for bit; native keys equal its keys; e4m3 keys are within half a step of the oracle's."""
    page = 16
    x = rows((b, n, hq + 2 * hkv, d), dtype, 8)
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    freq = 1e6 ** (-np.arange(0, rot, 2) / rot)
    kw = (1 + 0.1 * np.random.default_rng(0).normal(size=d)).astype(np.float32)
    rope = kp.make_rope(torch.from_numpy(freq).cuda(), q_weight=torch.ones(d, device="cuda"), k_weight=torch.from_numpy(kw).cuda(),
                        interleaved=inter)
    pos = np.arange(b * n, dtype=np.int32).reshape(b, n) * 1001
    table, n_pages = tables([n] * b, page)
    slots = slots_of(table, [n] * b, page, n)
    if n > 1:
        slots[b // 2, n - 6:] = -1
    c = cache_of(hq, hkv, d, page, n_pages, dtype=dtype, cache=cache)
    qo = torch.empty(b, n, hq, d, dtype=TORCH[dtype], device="cuda")
    c.append_qkv(0, rope, q, k, v, ints(pos), ints(slots), qo)
    q1, k1 = torch.empty_like(qo), torch.empty(b, n, hkv, d, dtype=TORCH[dtype], device="cuda")
    kp.qk_norm_rope(rope, q, k, ints(pos), q1, k1)
    assert torch.equal(qo, q1)
    if cache == "native":
        check_held(c, 0, table, [n] * b, page, f64(k1), f64(v), slots, dtype, cache)
        return
    pages, scales = f64(c.pages(0).float()), f64(c.scales(0))
    for i in range(b):
        t = np.nonzero(slots[i] >= 0)[0]
        pg, r = slots[i, t] // page, slots[i, t] % page
        want = po.heads(f64(k[i]), kw, 1e-6, pos[i], freq, interleaved=inter)[t]
        got = pages[pg, :, 0, r] * scales[pg, :, 0, r][..., None]
        top = np.abs(want).max(-1, keepdims=True)
        # half a step of e4m3 (relative 2^-4; 2^-10 of the scale where values are below 2^-6), keys off by 256 u of the row
        bound = 2.0 ** -4 * np.abs(want) + (2.0 ** -10 / 448 + 512 * U) * top
        assert (np.abs(got - want) <= bound).all()
        wv, sv = po.hold_e4m3(f64(v[i])[t])
        np.testing.assert_array_equal(scales[pg, :, 1, r], sv)
        np.testing.assert_array_equal(pages[pg, :, 1, r], wv)
    for i in range(b):                                              # padding wrote nothing
        for t in np.nonzero(slots[i] < 0)[0]:
            assert (scales[table[i, t // page], :, :, t % page] == 0).all()


def test_bad_slots_and_pages_are_recorded():
    """A slot past the pool writes nothing; a page outside it is read as nothing; lengths are cut."""
    c = cache_of(2, 1, 64, 16, 3)
    x = rows((1, 4, 1, 64), "bf16", 3)
    c.append(0, x, x, ints([[0, 48, 2 ** 31 - 1, -5]]))
    assert c.get_error() == (kp.KVPOP_ERR_DEVICE, kp.KVPOP_DEVERR_BAD_INDEX)
    assert torch.equal(c.pages(0)[0, 0, 0, 0], x[0, 0, 0]) and (c.pages(0)[0, 0, :, 1:] == 0).all()
    assert (c.pages(0)[1:] == 0).all()
    c.clear_error()
    assert c.get_error() == (kp.KVPOP_OK, 0)
    q = rows((4, 2, 64), "bf16", 5)
    out, lse = torch.empty_like(q), torch.empty(4, 2, device="cuda")
    k = rows((1, 48, 1, 64), "bf16", 6)
    c.append(0, k, k, ints(np.arange(48)[None]))
    table = ints([[0, 3], [0, -1], [0, 1], [0, 1]])
    lens = ints([32, 17, -4, 1000])
    c.attend(0, q, table, lens, out, lse)
    assert c.get_error() == (kp.KVPOP_ERR_DEVICE, kp.KVPOP_DEVERR_BAD_INDEX)
    c.clear_error()
    for b, n in ((0, 16), (1, 16), (2, 0), (3, 32)):
        check_attend(out[b], lse[b], q[b], f64(k[0, :n]), f64(k[0, :n]), "bf16")
    ko, vo = (torch.full((4, 32, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.gather(0, table, lens, ko, vo)
    assert c.get_error() == (kp.KVPOP_ERR_DEVICE, kp.KVPOP_DEVERR_BAD_INDEX)
    for b, n in ((0, 16), (1, 16), (2, 0), (3, 32)):
        assert torch.equal(ko[b, :n], k[0, :n]) and (ko[b, n:] == 2).all() and (vo[b, n:] == 2).all()


@pytest.mark.parametrize("bad", [-1, -2, -2 ** 31, 7, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,cache,page", [("bf16", "native", 16), ("bf16", "e4m3", 16), ("f32", "native", 32)])
def test_every_bad_page_is_recorded(bad, dtype, cache, page):
    """One bad entry among good ones: recorded, its tokens left out of the sum and of what is read back."""
    n = 5 * page - 3
    c = cache_of(4, 2, 64, page, 7, dtype, cache)
    k = rows((1, n, 2, 64), dtype, 1)
    table = np.array([[6, 0, 4, 2, 5]], np.int32)
    c.append(0, k, k, ints(slots_of(table, [n], page, n)))
    q = rows((1, 4, 64), dtype, 2)
    x = held_rows(c, 0, table, n, page, 0)
    for at in (0, 2, 4):
        t = table.copy()
        t[0, at] = bad
        out = torch.empty_like(q)
        c.attend(0, q, ints(t), ints([n]), out)
        assert c.get_error() == (kp.KVPOP_ERR_DEVICE, kp.KVPOP_DEVERR_BAD_INDEX)
        c.clear_error()
        keep = np.r_[0:at * page, min((at + 1) * page, n):n]
        check_attend(out[0], None, q[0], x[keep, :, 0], x[keep, :, 1], dtype)
        ko, vo = (torch.full((1, n, 2, 64), 9.0, dtype=TORCH[dtype], device="cuda") for _ in range(2))
        c.gather(0, ints(t), ints([n]), ko, vo)
        assert c.get_error() == (kp.KVPOP_ERR_DEVICE, kp.KVPOP_DEVERR_BAD_INDEX)
        c.clear_error()
        gone = slice(at * page, min((at + 1) * page, n))
        assert (ko[0, gone] == 9).all() and (vo[0, gone] == 9).all() and not (ko[0, keep] == 9).all(-1).any()


# ---- attend ----

def check_attend(out, lse, q, k, v, dtype, scale=None, softcap=0.0, window=0):
    want, wl = po.attend(f64(q), k, v, scale, softcap, window)
    slack, ls = po.attend_slack(f64(q), k, v, scale, window)
    err = np.abs(f64(out) - want)
    bound = half_step(dtype) * np.abs(want) + slack * (1 + half_step(dtype)) + 1e-38
    assert (err <= bound).all(), float((err / bound).max())
    if lse is not None:
        got = f64(lse)
        assert np.array_equal(np.isinf(got), np.isinf(wl))
        ok = np.isfinite(wl)
        assert (np.abs(got[ok] - wl[ok]) <= (ls + 4 * U * np.abs(wl) + 4 * U)[ok]).all()


def filled(lens, hq, hkv, d, page, dtype, cache, seed=0, **kw):
    b, n = len(lens), max(max(lens), 1)
    table, n_pages = tables(lens, page, seed)
    k, v = rows((b, n, hkv, d), dtype, seed + 1), rows((b, n, hkv, d), dtype, seed + 2)
    c = cache_of(hq, hkv, d, page, n_pages, dtype, cache, **kw)
    c.append(0, k, v, ints(slots_of(table, lens, page, n)))
    return c, table, rows((b, hq, d), dtype, seed + 3)


SHAPES = [("bf16", "native", 128, 4, 2, 16), ("bf16", "native", 128, 1, 1, 64), ("bf16", "native", 64, 8, 2, 32),
          ("bf16", "native", 128, 16, 1, 16), ("bf16", "native", 64, 3, 4, 256), ("bf16", "e4m3", 128, 4, 8, 64),
          ("bf16", "e4m3", 64, 7, 1, 16), ("bf16", "e4m3", 128, 12, 2, 128), ("f32", "native", 64, 2, 2, 32),
          ("f32", "native", 128, 4, 3, 16), ("f32", "native", 64, 16, 1, 64), ("f32", "native", 128, 5, 1, 128),
          ("bf16", "native", 128, 6, 2, 32), ("bf16", "e4m3", 64, 2, 2, 32)]


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", SHAPES)
@pytest.mark.parametrize("lens", [[1], [5], [17, 0, 1, 16], [1000, 31, 257, 64, 2, 0, 700], [2900]])
def test_attend(dtype, cache, d, g, hkv, page, lens):
    c, table, q = filled(lens, g * hkv, hkv, d, page, dtype, cache, seed=len(lens) * 10 + d)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    c.attend(0, q, ints(table), ints(lens), out, lse)
    again = torch.empty_like(q)
    c.attend(0, q, ints(table), ints(lens), again)
    assert torch.equal(out, again)
    assert c.get_error() == (kp.KVPOP_OK, 0)
    for b, n in enumerate(lens):
        x = held_rows(c, 0, table, n, page, b)
        check_attend(out[b], lse[b], q[b], x[:, :, 0], x[:, :, 1], dtype)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[9]])
@pytest.mark.parametrize("lens,width", [([40, 0, 3], 0), ([2900, 17], 0), ([2900, 700, 64], 4000), ([33] * 300, 0), ([900, 20] * 120, 0)])
def test_attend_in_place(dtype, cache, d, g, hkv, page, lens, width):
    """out = q, for each way of splitting the work: the bits of a call with a separate out."""
    c, table, q = filled(lens, g * hkv, hkv, d, page, dtype, cache, seed=12, max_batch=512)
    wide = np.zeros((len(lens), max(width, table.shape[1])), np.int32)
    wide[:, :table.shape[1]] = table
    want = torch.empty_like(q)
    c.attend(0, q, ints(wide), ints(lens), want)
    c.attend(0, q, ints(wide), ints(lens), q)
    assert torch.equal(q, want) and c.get_error() == (kp.KVPOP_OK, 0)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[8], SHAPES[6], SHAPES[3]])
@pytest.mark.parametrize("scale,softcap,window", [(0.3, 0.0, 0), (0.0, 5.0, 0), (0.0, 0.0, 1), (0.0, 0.0, 100), (0.2, 30.0, 16),
                                                  (0.0, 0.0, 5000)])
def test_attend_options(dtype, cache, d, g, hkv, page, scale, softcap, window):
    lens = [333, 16, 0, 1, 100, 117]
    c, table, q = filled(lens, g * hkv, hkv, d, page, dtype, cache, seed=77)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    c.attend(0, q, ints(table), ints(lens), out, lse, scale=scale, softcap=softcap, window=window)
    for b, n in enumerate(lens):
        x = held_rows(c, 0, table, n, page, b)
        check_attend(out[b], lse[b], q[b], x[:, :, 0], x[:, :, 1], dtype, scale or None, softcap, window)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[8]])
def test_attend_sharp_and_growing_scores(dtype, cache, d, g, hkv, page):
    """Scores that rise along the sequence (the running maximum moves at every
    step) and weights that fall on one key."""
    n = 700
    c, table, q = filled([n, n], g * hkv, hkv, d, page, dtype, cache, seed=5)
    k = (q[:, ::g].float().unsqueeze(1) * torch.linspace(-2, 2, n, device="cuda").view(1, n, 1, 1)).to(q.dtype)
    v = rows((2, n, hkv, d), dtype, 9)
    s = slots_of(table, [n, n], page, n)
    c.append(0, k, v, ints(s))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    for order in (table, table[:, ::-1].copy()):
        t = order if order is table else np.roll(order, -1, 1).copy()   # pages reversed: falling scores
        t = t if (t[:, :-(-n // page)] >= 0).all() else table
        c.attend(0, q, ints(t), ints([n, n]), out, lse)
        for b in range(2):
            x = held_rows(c, 0, t, n, page, b)
            check_attend(out[b], lse[b], q[b], x[:, :, 0], x[:, :, 1], dtype)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[8], SHAPES[2]])
def test_attend_ignores_what_is_not_attended(dtype, cache, d, g, hkv, page):
    """NaN and infinities behind the last token, before the window and in other pages change no bit."""
    lens = [45, 100, 16 * 5]
    c, table, q = filled(lens, g * hkv, hkv, d, page, dtype, cache, seed=21)
    out, ref = torch.empty_like(q), torch.empty_like(q)
    c.attend(0, q, ints(table), ints(lens), ref, window=33)
    bad = torch.full((1, 1, hkv, d), math.nan, dtype=q.dtype, device="cuda")
    bad[..., ::2] = math.inf
    spots = [int(table[b, n // page]) * page + n % page for b, n in ((0, 45), (1, 100)) if n % page]
    spots += [int(table[b, (n - 34) // page]) * page + (n - 34) % page for b, n in enumerate(lens)]
    spots += [int(table[0, 0]) * page]
    m = len(spots)
    c.append(0, bad.expand(1, m, hkv, d), bad.expand(1, m, hkv, d), ints([spots]))
    c.attend(0, q, ints(table), ints(lens), out, window=33)
    assert torch.equal(out, ref) and torch.isfinite(out).all()


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[8]])
def test_attend_nonfinite_scores(dtype, cache, d, g, hkv, page):
    """A NaN key makes its sequence's heads NaN and no other's; keys of -inf scores have no weight; all -inf gives NaN."""
    lens = [40, 40, 40, 40]
    c, table, q = filled(lens, g * hkv, hkv, d, page, dtype, cache, seed=31)
    q.abs_()
    k, v = rows((4, 40, hkv, d), dtype, 1), rows((4, 40, hkv, d), dtype, 2)
    k[0, 7, 0, 3] = math.nan
    v[1, 3, 0, 2] = math.nan
    if cache == "native":
        k[2, 5:9] = -math.inf       # scores of -inf: no weight
        k[3] = -math.inf            # every score -inf: 0 / 0
    c.append(0, k, v, ints(slots_of(table, lens, page, 40)))
    out = torch.empty_like(q)
    c.attend(0, q, ints(table), ints(lens), out)
    assert out[0, :g].isnan().all() and torch.isfinite(out[0, g:]).all()
    if cache == "native":
        assert out[1, :g, 2].isnan().all() and torch.isfinite(out[1, :, 3:]).all()
        kk = f64(k[2])
        keep = np.r_[0:5, 9:40]
        check_attend(out[2], None, q[2], kk[keep], f64(v[2])[keep], dtype)
        assert out[3].isnan().all()
    else:
        assert out[1, :g].isnan().all() and torch.isfinite(out[1, g:]).all()   # the whole row is NaN in 8 bits
        assert torch.isfinite(out[2:]).all()


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[8], SHAPES[3]])
def test_attend_long_and_many(dtype, cache, d, g, hkv, page):
    """One long sequence over many blocks of the GPU, and many short ones."""
    for lens in ([30011], [20000, 3], list(np.random.default_rng(0).integers(0, 90, size=200))):
        lens = [int(x) for x in lens]
        b, n = len(lens), max(lens)
        table, n_pages = tables(lens, page, 3)
        k, v = rows((b, n, hkv, d), dtype, 4), rows((b, n, hkv, d), dtype, 5)
        c = cache_of(g * hkv, hkv, d, page, n_pages, dtype, cache, max_batch=256)
        c.append(0, k, v, ints(slots_of(table, lens, page, n)))
        q = rows((b, g * hkv, d), dtype, 6)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        for _ in range(2):
            c.attend(0, q, ints(table), ints(lens), out, lse)
        for i in range(0, b, max(1, b // 23)):
            x = held_rows(c, 0, table, lens[i], page, i)
            check_attend(out[i], lse[i], q[i], x[:, :, 0], x[:, :, 1], dtype)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [("bf16", "e4m3", 128, 4, 2, 16), ("bf16", "e4m3", 128, 8, 1, 64),
                                                      ("bf16", "e4m3", 128, 16, 1, 16), ("bf16", "e4m3", 64, 3, 2, 32),
                                                      ("bf16", "e4m3", 64, 16, 1, 32), ("bf16", "native", 128, 4, 2, 16)])
@pytest.mark.parametrize("exponent,below", [(20, 35.0), (28, 45.0), (40, 80.0), (40, 10.0), (-40, -20.0)])
@pytest.mark.parametrize("n", [30, 2900])
def test_attend_values_of_unlike_magnitudes(dtype, cache, d, g, hkv, page, exponent, below, n):
    """One value row 2^exponent times the others, half of it zeros, whose score
    lies `below` the others' (far below: no weight; a little below: most of the
    output; above them and small: none of it): first, in the middle and last."""
    spots = [0, n // 2, n - 1]
    c, table, q = filled([n] * 3, g * hkv, hkv, d, page, dtype, cache, seed=n + abs(exponent))
    base = torch.ones(d, device="cuda")
    q = (base * (1 + torch.arange(g * hkv, device="cuda").view(1, -1, 1) / 32)).expand(3, -1, -1).to(q.dtype).contiguous()
    k, v = rows((3, n, hkv, d), dtype, 5, 0.25), rows((3, n, hkv, d), dtype, 6)
    for b, at in enumerate(spots):
        k[b, at] = (k[b, at].float() - base * (below / d ** 0.5)).to(k.dtype)
        v[b, at] *= 2.0 ** exponent
        v[b, at, :, 1::2] = 0
    c.append(0, k, v, ints(slots_of(table, [n] * 3, page, n)))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    c.attend(0, q, ints(table), ints([n] * 3), out, lse)
    for b in range(3):
        x = held_rows(c, 0, table, n, page, b)
        check_attend(out[b], lse[b], q[b], x[:, :, 0], x[:, :, 1], dtype)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[6], SHAPES[7], SHAPES[9]])
@pytest.mark.parametrize("ek,eq,scale", [(-90, 90, 0.25), (20, -20, 0.25), (110, -110, 0.25), (118, -98, 2.0 ** -22), (-60, -20, 2.0 ** 78)])
def test_attend_large_keys_and_small_queries(dtype, cache, d, g, hkv, page, ek, eq, scale):
    """Keys of 2^ek and queries of 2^eq times the ordinary have ordinary scores under a scale that makes up for them."""
    n = 300
    c, table, q = filled([n], g * hkv, hkv, d, page, dtype, cache, seed=4)
    q *= 2.0 ** eq
    c.append(0, rows((1, n, hkv, d), dtype, 5, 2.0 ** ek), rows((1, n, hkv, d), dtype, 6), ints(slots_of(table, [n], page, n)))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    c.attend(0, q, ints(table), ints([n]), out, lse, scale=scale)
    x = held_rows(c, 0, table, n, page, 0)
    check_attend(out[0], lse[0], q[0], x[:, :, 0], x[:, :, 1], dtype, scale)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[3], SHAPES[5], SHAPES[7], SHAPES[8], SHAPES[9]])
@pytest.mark.parametrize("n", [300, 2900])
def test_attend_values_near_the_end_of_the_range(dtype, cache, d, g, hkv, page, n):
    """Values of 2^116 whose scores lie 2^7.8 above those before them: their sum stays in fp32's range, 2^7.8 times it would not."""
    c, table, q = filled([n], g * hkv, hkv, d, page, dtype, cache, seed=8)
    q = (1 + torch.arange(g * hkv, device="cuda").view(1, -1, 1) / 1024).expand(1, -1, d).to(q.dtype).contiguous()
    k, v = rows((1, n, hkv, d), dtype, 5, 0.01), rows((1, n, hkv, d), dtype, 6).abs() * 2.0 ** 116
    k[:, n // 2:] += 5.4 / d ** 0.5
    c.append(0, k, v, ints(slots_of(table, [n], page, n)))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    c.attend(0, q, ints(table), ints([n]), out, lse)
    x = held_rows(c, 0, table, n, page, 0)
    check_attend(out[0], lse[0], q[0], x[:, :, 0], x[:, :, 1], dtype)


@pytest.mark.parametrize("dtype,cache,hq,hkv", [("bf16", "native", 600, 600), ("bf16", "e4m3", 460, 460), ("f32", "native", 500, 500),
                                                 ("bf16", "native", 96, 6)])
def test_attend_more_heads_than_the_gpu_has_blocks(dtype, cache, hq, hkv):
    lens = [40, 0, 500, 17]
    c, table, q = filled(lens, hq, hkv, 64, 16, dtype, cache, seed=2)
    wide = np.full((4, 700), -1, np.int32)          # a wide table: nothing is known of the lengths beforehand
    wide[:, :table.shape[1]] = table
    out, lse, narrow = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), torch.empty_like(q)
    c.attend(0, q, ints(wide), ints(lens), out, lse)
    c.attend(0, q, ints(table), ints(lens), narrow)
    for b, n in enumerate(lens):
        x = held_rows(c, 0, table, n, 16, b)
        check_attend(out[b], lse[b], q[b], x[:, :, 0], x[:, :, 1], dtype)
        check_attend(narrow[b], None, q[b], x[:, :, 0], x[:, :, 1], dtype)
    assert c.get_error() == (kp.KVPOP_OK, 0)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [SHAPES[0], SHAPES[5], SHAPES[9], SHAPES[12]])
@pytest.mark.parametrize("lens", [[1], [0], [3, 200, 0, 129], [700] * 20, [1, 2, 3] * 20, [5000, 4000, 3000, 10]])
def test_attend_does_not_depend_on_the_table_s_width(dtype, cache, d, g, hkv, page, lens):
    """Narrow tables fix the split beforehand, wide ones leave it to the lengths."""
    c, table, q = filled(lens, g * hkv, hkv, d, page, dtype, cache, seed=13)
    wide = np.full((len(lens), 4000), -1, np.int32)
    wide[:, :table.shape[1]] = table
    for t in (table[:, :max(1, -(-max(lens) // page))].copy(), wide):
        for window in (0, 40):
            out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
            if max(lens) == 0:
                out.fill_(7), lse.fill_(7)
            c.attend(0, q, ints(t), ints(lens), out, lse, window=window)
            for b in range(0, len(lens), max(1, len(lens) // 7)):
                x = held_rows(c, 0, table, lens[b], page, b)
                check_attend(out[b], lse[b], q[b], x[:, :, 0], x[:, :, 1], dtype, window=window)


@pytest.mark.parametrize("dtype,cache,d,g,hkv,page", [("bf16", "native", 128, 4, 4, 16), ("bf16", "native", 64, 8, 6, 32),
                                                      ("bf16", "e4m3", 128, 2, 8, 16), ("bf16", "e4m3", 64, 16, 5, 64),
                                                      ("f32", "native", 128, 3, 4, 16), ("f32", "native", 64, 9, 4, 16)])
@pytest.mark.parametrize("most,window", [(17, 0), (60, 0), (90, 33), (257, 0)])
def test_attend_many_short_sequences(dtype, cache, d, g, hkv, page, most, window):
    """More short sequences than blocks of the GPU: each head of each goes to a warp of its own."""
    lens = [int(x) for x in np.random.default_rng(most).integers(0, most, size=250)]
    b, n = len(lens), max(lens)
    table, n_pages = tables(lens, page, 3)
    wide = np.full((b, 600), -1, np.int32)
    wide[:, :table.shape[1]] = table
    k, v = rows((b, n, hkv, d), dtype, 4), rows((b, n, hkv, d), dtype, 5)
    c = cache_of(g * hkv, hkv, d, page, n_pages, dtype, cache, max_batch=256)
    c.append(0, k, v, ints(slots_of(table, lens, page, n)))
    q = rows((b, g * hkv, d), dtype, 6)
    out, lse = torch.full_like(q, 7), torch.full(q.shape[:2], 7.0, device="cuda")
    for _ in range(2):
        c.attend(0, q, ints(wide), ints(lens), out, lse, window=window)
    for i in range(0, b, 9):
        x = held_rows(c, 0, table, lens[i], page, i)
        check_attend(out[i], lse[i], q[i], x[:, :, 0], x[:, :, 1], dtype, window=window)
    assert torch.isfinite(out).all() and c.get_error() == (kp.KVPOP_OK, 0)


def test_offsets_past_32_bits():
    """The last pages of a pool of more than 2^31 elements and 2^32 bytes."""
    page, hkv, d = 256, 8, 128
    n_pages = 4200                       # 4200 * 8 * 2 * 256 * 128 = 2.2e9 elements
    c = cache_of(32, hkv, d, page, n_pages)
    k, v = rows((1, 300, hkv, d), "bf16", 1), rows((1, 300, hkv, d), "bf16", 2)
    table = np.array([[n_pages - 1, n_pages - 2]], np.int32)
    c.append(0, k, v, ints(slots_of(table, [300], page, 300)))
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    c.gather(0, ints(table), ints([300]), ko, vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    q = rows((1, 32, d), "bf16", 3)
    out = torch.empty_like(q)
    c.attend(0, q, ints(table), ints([300]), out)
    check_attend(out[0], None, q[0], f64(k[0]), f64(v[0]), "bf16")


def test_shared_pages_and_wide_tables():
    """Sequences that share a prefix's pages, one sequence twice, tables far wider than needed."""
    page, hkv, d, g = 16, 2, 128, 4
    c, table, q = filled([64, 50], g * hkv, hkv, d, page, "bf16", "native", seed=3)
    wide = np.full((4, 40), -1, np.int32)
    wide[0, :4] = table[0, :4]
    wide[1, :4] = table[0, :4]
    wide[2, :2], wide[2, 2:5] = table[0, :2], table[1, :3]
    wide[3, :3] = table[0, 0]
    lens = [64, 64, 70, 48]
    qq = q[[0, 0, 1, 1]].contiguous()
    out = torch.empty_like(qq)
    c.attend(0, qq, ints(wide), ints(lens), out)
    assert torch.equal(out[0], out[1])
    for b in range(4):
        x = held_rows(c, 0, wide, lens[b], page, b)
        check_attend(out[b], None, qq[b], x[:, :, 0], x[:, :, 1], "bf16")


# ---- streams, graphs, refusals ----

def test_a_step_in_a_graph_with_growing_lengths():
    """append_qkv and attend captured once and replayed while lengths, slots
    and inputs change in place equal eager calls on another cache, on another stream."""
    b, hq, hkv, d, page, steps = 3, 8, 2, 128, 16, 20
    freq = torch.from_numpy(1e6 ** (-np.arange(0, d, 2) / d)).cuda()
    rope = kp.make_rope(freq, q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda"))
    table, n_pages = tables([64] * b, page, 1)
    tab = ints(table)
    start = np.array([0, 13, 31])
    xs = rows((steps, b, 1, hq + 2 * hkv, d), "bf16", 1)
    caches = [cache_of(hq, hkv, d, page, n_pages, cache="e4m3") for _ in range(2)]
    for c in caches:
        k = rows((b, 31, hkv, d), "bf16", 2)
        c.append(0, k, k, ints(slots_of(table, list(start), page, 31)))
    x, pos, slot, lens = xs[0].clone(), ints(np.zeros((b, 1))), ints(np.zeros((b, 1))), ints(np.zeros(b))
    bufs = [(torch.empty(b, 1, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(b, hq, d, dtype=torch.bfloat16, device="cuda"))
            for _ in range(2)]

    def step(c, qo, out):
        c.append_qkv(0, rope, x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], pos, slot, qo)
        c.attend(0, qo[:, 0], tab, lens, out)

    def feed(i):
        p = start + i
        x.copy_(xs[i])
        pos.copy_(ints(p[:, None]))
        slot.copy_(ints((table[np.arange(b), p // page] * page + p % page)[:, None]))
        lens.copy_(ints(p + 1))

    feed(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(caches[0], *bufs[0])
    for i in range(steps):
        feed(i)
        g.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step(caches[1], *bufs[1])
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][1], bufs[1][1]) and torch.equal(bufs[0][0], bufs[1][0])
    assert caches[0].get_error() == caches[1].get_error() == (kp.KVPOP_OK, 0)
    assert torch.equal(caches[0].pages(0).view(torch.uint8), caches[1].pages(0).view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "budget"])
def test_a_cache_made_in_memory_that_a_stream_still_writes(kind):
    """On a side stream torch hands a freed block on while work queued there may
    still write to it: a cache made in it begins empty all the same."""
    if kind == "budget":
        cfg = kp.make_config(batch=2, n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=128, sinks=4, window=32, topk=64,
                             max_prefill_chunk=256, external_scores=True)
        make, nbytes = (lambda: kp.KVPopCache(cfg)), kp.cache_bytes(cfg)
    else:
        lens, page, hkv, d = [2900, 40], 16, 2, 128
        table, n_pages = tables(lens, page, 1)
        cfg = kp.make_paged_config(n_layers=1, n_q_heads=8, n_kv_heads=hkv, head_dim=d, page_size=page, n_pages=n_pages,
                                   max_batch=64, cache="native" if kind == "bf16" else kind)
        make, nbytes = (lambda: kp.KVPopPagedCache(cfg)), kp.paged_bytes(cfg)
        x = [rows((2, 2900, hkv, d), "bf16", i) for i in (2, 3)]
        slots, q = ints(slots_of(table, lens, page, 2900)), rows((2, 8, d), "bf16", 4)
        tab, n = ints(table), ints(lens)
    quiet = make()
    side = torch.cuda.Stream()
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        block = torch.empty(nbytes + 256, dtype=torch.uint8, device="cuda")
        at = block.data_ptr()
        for i in range(60):          # 10 ms or more of work before the block is written
            big.fill_(i)
        block.fill_(0x55)
        del block
        late = make()
        assert late.buffer.data_ptr() == at      # the same memory
    for c in (quiet, late):
        start = (-c.buffer.data_ptr()) % 256
        c.held = c.buffer[start:start + nbytes]
    torch.cuda.synchronize()
    assert torch.equal(quiet.held, late.held)
    if kind != "budget":
        assert not late.held.any()
        outs = []
        for c in (quiet, late):
            c.append(0, *x, slots)
            outs.append(torch.empty_like(q))
            c.attend(0, q, tab, n, outs[-1])
        assert torch.equal(*outs)


def test_two_caches_on_two_streams():
    """Calls of two objects overlap on two streams and keep their results."""
    args = [filled([3000, 500], 8, 2, 128, 64, "bf16", "native", seed=s) for s in (1, 2)]
    want = []
    for c, t, q in args:
        o = torch.empty_like(q)
        c.attend(0, q, ints(t), ints([3000, 500]), o)
        want.append(o)
    torch.cuda.synchronize()
    tabs, lens = [ints(t) for _, t, _ in args], ints([3000, 500])
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (c, _, q), t, o, s in zip(args, tabs, outs, streams):
            c.attend(0, q, t, lens, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("captured", [False, True])
def test_two_caches_fork_and_join(captured):
    """A step of two layers in two caches whose writes fork to a second stream and join again, captured and eager, ten times."""
    b, hq, hkv, d, page = 5, 8, 2, 128, 16
    freq = torch.from_numpy(1e4 ** (-np.arange(0, d, 2) / d)).cuda()
    rope = kp.make_rope(freq, q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda"))
    start = np.array([0, 13, 500, 31, 64])
    table, n_pages = tables([600] * b, page, 1)
    tab, steps = ints(table), 10
    xs = rows((steps, b, 1, hq + 2 * hkv, d), "bf16", 1)

    def caches():
        cs = [cache_of(hq, hkv, d, page, n_pages, cache=f) for f in ("native", "e4m3")]
        for c in cs:
            k = rows((b, 500, hkv, d), "bf16", 2)
            c.append(0, k, k, ints(slots_of(table, list(start), page, 500)))
        return cs

    side = torch.cuda.Stream()

    def step(cs, x, pos, slot, lens, qo, out, fork):
        here = torch.cuda.current_stream()
        if fork:
            side.wait_stream(here)
        cs[0].append_qkv(0, rope, x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], pos, slot, qo[0])
        with torch.cuda.stream(side if fork else here):
            cs[1].append_qkv(0, rope, x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], pos, slot, qo[1])
            cs[1].attend(0, qo[1][:, 0], tab, lens, out[1])
        cs[0].attend(0, qo[0][:, 0], tab, lens, out[0])
        if fork:
            here.wait_stream(side)
        kp.qk_norm_rope(rope, out[0].unsqueeze(1), out[1][:, :hkv].unsqueeze(1), pos, out[2].unsqueeze(1), out[3][:, :hkv].unsqueeze(1))

    one, two = caches(), caches()
    x, pos, slot, lens = xs[0].clone(), ints(np.zeros((b, 1))), ints(np.zeros((b, 1))), ints(np.zeros(b))
    bufs = [([torch.zeros(b, 1, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)],
             [torch.zeros(b, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]) for _ in range(2)]
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            step(one, x, pos, slot, lens, *bufs[0], True)
    for i in range(steps):
        at = start + i
        x.copy_(xs[i])
        pos.copy_(ints(at[:, None]))
        slot.copy_(ints((table[np.arange(b), at // page] * page + at % page)[:, None]))
        lens.copy_(ints(at + 1))
        torch.cuda.synchronize()
        if captured:
            g.replay()
        else:
            with torch.cuda.stream(main):
                step(one, x, pos, slot, lens, *bufs[0], True)
        torch.cuda.synchronize()
        step(two, x, pos, slot, lens, *bufs[1], False)
        torch.cuda.synchronize()
        for p, q in zip(bufs[0][1], bufs[1][1]):
            assert torch.equal(p, q)
    for c in one + two:
        assert c.get_error() == (kp.KVPOP_OK, 0)


def test_calls_from_two_threads():
    """Two host threads, each with its own stream and cache, at once."""
    from concurrent.futures import ThreadPoolExecutor
    lens = [300, 17, 0, 64]
    made = [filled(lens, 8, 2, 128, 16, "bf16", f, seed=3) for f in ("native", "e4m3")]
    want = []
    for c, table, q in made:
        out = torch.empty_like(q)
        c.attend(0, q, ints(table), ints(lens), out)
        want.append(out)
    torch.cuda.synchronize()

    def work(i):
        c, table, q = made[i]
        s, t, n = torch.cuda.Stream(), ints(table), ints(lens)
        outs = [torch.empty_like(q) for _ in range(200)]
        torch.cuda.synchronize()
        for o in outs:
            c.attend(0, q, t, n, o, stream=s)
        s.synchronize()
        return all(torch.equal(o, want[i]) for o in outs)

    with ThreadPoolExecutor(2) as pool:
        assert all(pool.map(work, range(2)))


def test_a_failed_paged_call_leaves_no_error_behind():
    """A paged call that CUDA refuses (here: a clearing while a stream captures)
    reports it, and the next calls, paged and fixed-budget, do not."""
    hq, hkv, d = 8, 2, 128
    budget = kp.KVPopCache(kp.make_config(batch=1, n_layers=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, sinks=4, window=32,
                                          topk=32, external_scores=True))
    c, table, q = filled([40], hq, hkv, d, 16, "bf16", "native")
    out, tab, lens = torch.empty_like(q), ints(table), ints([40])
    k, score = rows((1, hkv, d), "bf16", 1), torch.ones(1, hkv, device="cuda")
    cfg = kp.make_paged_config(n_layers=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=16, n_pages=4, max_batch=1)
    mem = torch.empty(kp.paged_bytes(cfg), dtype=torch.uint8, device="cuda")
    rt = ctypes.CDLL("libcudart.so.12")
    side, graph, handle = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(ctypes.c_void_p(side.cuda_stream), 0) == 0
    status = kp.lib.kvpop_paged_create(ctypes.byref(cfg), mem.data_ptr(), mem.numel(), ctypes.byref(handle))
    rt.cudaStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph))
    rt.cudaGetLastError()
    assert status == kp.KVPOP_ERR_CUDA and not handle.value
    budget.decode_append(0, k, k, ext_score=score)
    budget.decode_attend(0, q, out)
    c.attend(0, q, tab, lens, out)
    assert budget.get_error() == c.get_error() == (kp.KVPOP_OK, 0)


def test_refusals_on_the_gpu():
    c = cache_of(4, 2, 64, 16, 4, max_batch=2)
    k = rows((1, 3, 2, 64), "bf16", 1)
    s = ints([[0, 1, 2]])
    before = c.pages(0).clone()
    with pytest.raises(ValueError, match="dtype"):
        c.append(0, k.float(), k.float(), s)
    with pytest.raises(ValueError, match="shape"):
        c.append(0, k[:, :, :1], k, s)
    with pytest.raises(ValueError, match="strides"):
        c.append(0, rows((1, 3, 2, 128), "bf16", 1)[..., ::2], k, s)
    with pytest.raises(ValueError, match="strides"):
        c.append(0, rows((1, 3, 2, 68), "bf16", 1)[..., 4:], k, s)
    with pytest.raises(ValueError, match="slots"):
        c.append(0, k, k, s.long())
    with pytest.raises(kp.KVPopError):
        c.append(1, k, k, s)
    with pytest.raises(ValueError, match="expanded"):
        c.gather(0, ints([[0]]), ints([3]), k[:, :1].expand(1, 3, 2, 64), k)
    q = rows((3, 4, 64), "bf16", 2)
    t, n = ints(np.zeros((3, 1))), ints([1, 1, 1])
    with pytest.raises(kp.KVPopError) as e:
        c.attend(0, q, t, n, torch.empty_like(q))                    # three sequences, max_batch two
    assert e.value.status == kp.KVPOP_ERR_BAD_SHAPE
    for kw in (dict(scale=-1.0), dict(softcap=-1.0), dict(window=-1), dict(scale=math.nan), dict(softcap=math.inf),
               dict(scale=1e-40), dict(softcap=1e-40), dict(scale=3e38), dict(softcap=3e38), dict(scale=1e-60), dict(softcap=1e-60)):
        with pytest.raises(kp.KVPopError) as e:
            c.attend(0, q[:2], t[:2], n[:2], torch.empty_like(q[:2]), **kw)
        assert e.value.status == kp.KVPOP_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="contiguous"):
        c.attend(0, q[:2].transpose(0, 1).contiguous().transpose(0, 1), t[:2], n[:2], torch.empty_like(q[:2]))
    rope = kp.make_rope(torch.ones(32, dtype=torch.float64, device="cuda"), k_weight=torch.ones(128, device="cuda"))
    with pytest.raises(ValueError, match="head_dim"):
        kp.qk_norm_rope(rope, k, k, s, torch.empty_like(k), torch.empty_like(k))
    out = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    c.attend(0, out, ints(np.zeros((0, 1))), ints(np.zeros(0)), out)   # no sequence: nothing to do
    c.append(0, k[:, :0], k[:, :0], s[:, :0])
    none = torch.full((2, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    c.attend(0, q[:2], ints(np.zeros((2, 0))), ints([0, 0]), none)     # no page at all: empty sequences
    assert (none == 0).all()
    assert torch.equal(c.pages(0), before) and c.get_error() == (kp.KVPOP_OK, 0)


@pytest.mark.parametrize("name", ["q_weight", "k_weight"])
def test_empty_norm_weights_are_refused(name):
    """An empty tensor has no address: it would be taken for heads that are not normalised."""
    with pytest.raises(ValueError, match=f"{name}: empty"):
        kp.make_rope(torch.ones(32, dtype=torch.float64, device="cuda"), **{name: torch.empty(0, device="cuda")})


# ---- together, and beside the fixed-budget cache ----

def test_paged_decode_equals_a_budget_that_evicts_nothing():
    """Heads, write, attend against the fixed-budget cache whose budget covers
    the context; then the paged prompt is read back and prefilled into a
    second fixed-budget cache, which holds the same rows as the first."""
    b, hq, hkv, d, page, prompt, steps = 2, 8, 2, 128, 16, 50, 6
    freq = torch.from_numpy(1e6 ** (-np.arange(0, d, 2) / d)).cuda()
    rope = kp.make_rope(freq, q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda"))
    x = rows((b, prompt + steps, hq + 2 * hkv, d), "bf16", 1)
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    pos = ints(np.arange(prompt + steps)[None].repeat(b, 0))
    qo, ko = torch.empty(b, prompt + steps, hq, d, dtype=x.dtype, device="cuda"), torch.empty(b, prompt + steps, hkv, d, dtype=x.dtype, device="cuda")
    kp.qk_norm_rope(rope, q, k, pos, qo, ko)
    table, n_pages = tables([prompt + steps] * b, page)
    slots = slots_of(table, [prompt + steps] * b, page, prompt + steps)
    paged = cache_of(hq, hkv, d, page, n_pages)
    paged.append_qkv(0, rope, *(t[:, :prompt] for t in (q, k, v)), pos[:, :prompt].contiguous(), ints(slots[:, :prompt]),
                     torch.empty(b, prompt, hq, d, dtype=x.dtype, device="cuda"))

    def budget_cache():
        return kp.KVPopCache(kp.make_config(batch=b, n_layers=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, sinks=4, window=16,
                                            topk=108, max_prefill_chunk=prompt, external_scores=True))

    first, second = budget_cache(), budget_cache()
    score = torch.zeros(b, hkv, prompt, device="cuda")
    kh, vh = (t[:, :prompt].transpose(1, 2).contiguous() for t in (ko, v))
    first.prefill(0, kh, vh, ext_scores=score)
    k2, v2 = torch.empty_like(kh), torch.empty_like(vh)
    paged.gather(0, ints(table), ints([prompt] * b), k2.transpose(1, 2), v2.transpose(1, 2))
    assert torch.equal(k2, kh) and torch.equal(v2, vh)
    second.prefill(0, k2, v2, ext_scores=score)
    assert torch.equal(first.kv_rows(0), second.kv_rows(0))
    for i in range(prompt, prompt + steps):
        o1, o2, qi = (torch.empty(b, hq, d, dtype=x.dtype, device="cuda") for _ in range(3))
        first.decode_step(0, qo[:, i].contiguous(), ko[:, i].contiguous(), v[:, i].contiguous(), o1,
                          ext_score=torch.zeros(b, hkv, device="cuda"))
        paged.append_qkv(0, rope, *(t[:, i:i + 1] for t in (q, k, v)), pos[:, i:i + 1].contiguous(), ints(slots[:, i:i + 1]), qi[:, None])
        paged.attend(0, qi, ints(table), ints([i + 1] * b), o2)
        for s in range(b):
            kk, vv = f64(ko[s, :i + 1]), f64(v[s, :i + 1])
            check_attend(o2[s], None, qi[s], kk, vv, "bf16")
            # the fixed-budget kernel holds weights in bf16: 2^-8 of sum p |v| more
            want, _ = po.attend(f64(qi[s]), kk, vv)
            amount, _ = po.attend(f64(qi[s]), kk, np.abs(vv))
            assert (np.abs(f64(o1[s]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * amount).all()
    assert paged.get_error() == (kp.KVPOP_OK, 0) and first.get_error() == (kp.KVPOP_OK, 0)

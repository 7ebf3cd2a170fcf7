"""K/V insert and block operations against plain models, their refusals, and a server's life of them."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import paged_block_sparse_gb300 as pbs
from oracle import window_attend as ow
from window_cases import page_bytes

FMT = ("bf16", "fp8_e4m3", "nvfp4")
gpu = pytest.mark.gpu
A, N, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0), ctypes.c_void_p(0x10008)


def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def L():
    from paged_block_sparse_gb300 import _build
    _build.build()
    return pbs.lib()


# ---- refusals (no GPU) ------------------------------------------------------------------------------

@pytest.mark.parametrize("want,kw", [
    (0, dict(n=0)), (1, dict(n=-1)), (1, dict(k=N)), (1, dict(v=N)), (1, dict(kv=N)), (1, dict(sm=N)),
    (1, dict(fmt=5)), (1, dict(ks=0.0)), (1, dict(vs=float("nan"))), (1, dict(h=0)), (3, dict(d=64)),
    (2, dict(bps=4)), (2, dict(ps=100 * 16)), (2, dict(kr=-1)), (2, dict(np=0)), (4, dict(kv=ODD)),
    (4, dict(sm=ctypes.c_void_p(0x10004))), (4, dict(k=ctypes.c_void_p(0x10001)))])
def test_insert_refusals(L, want, kw):
    a = dict(k=A, kr=1024, kh=128, kd=1, v=A, vr=1024, vh=128, vd=1, n=4, h=8, d=128, kv=A, ps=65536, np=64, fmt=0,
             bps=8, sm=A, ss=1, ks=1.0, vs=1.0)
    a.update(kw)
    assert L.pbs_insert_kv_cache(*a.values(), N, N) == want


@pytest.mark.parametrize("want,kw", [(1, dict(ks=1e-39)), (1, dict(vs=-1e-39)), (3, dict(n=2 ** 31 - 1, h=65535))])
def test_insert_refuses_scales_without_a_reciprocal_and_grids_past_31_bits(L, want, kw):
    test_insert_refusals(L, want, kw)


POOL = dict(kv=A, ls=0, nl=1, ps=64, pb=64, np=64, bps=8)
ROWS = dict(pt=A, pts=4, nr=3, mb=4)


@pytest.mark.parametrize("want,kw", [
    (1, dict(kv=N)), (1, dict(nl=0)), (1, dict(np=0)), (1, dict(pb=0)), (2, dict(bps=7)), (2, dict(pb=80)),
    (2, dict(nl=2, ls=16)), (4, dict(ps=72)), (4, dict(kv=ODD)), (4, dict(nl=2, ls=72)), (4, dict(pb=56))])
def test_pool_refusals(L, want, kw):
    p = {**POOL, **kw}
    assert L.pbs_copy_cache_blocks(*p.values(), A, A, 1, N, N) == want
    assert L.pbs_fork_cache(*p.values(), *ROWS.values(), A, A, 8, A, A, 1, A, A, N, N) == want
    assert L.pbs_compact_cache(*p.values(), *ROWS.values(), A, 8, A, A, A, N, N) == want


@pytest.mark.parametrize("want,kw,nb", [
    (1, dict(pt=N), 8), (1, dict(nr=0), 8), (1, dict(mb=0), 8), (1, {}, 0), (2, dict(pts=3), 8),
    (4, dict(pt=ctypes.c_void_p(0x10002)), 8)])
def test_row_refusals(L, want, kw, nb):
    r = {**ROWS, **kw}
    assert L.pbs_reserve_cache_blocks(*r.values(), A, A, nb, A, A, 1, N, N) == want
    assert L.pbs_release_cache_blocks(*r.values(), A, A, nb, A, 1, 0, 0, N, N) == want
    assert L.pbs_fork_cache(*POOL.values(), *r.values(), A, A, nb, A, A, 1, A, A, N, N) == want
    assert L.pbs_compact_cache(*POOL.values(), *r.values(), A, nb, A, A, A, N, N) == want


def test_other_refusals(L):
    r, p = ROWS.values(), POOL.values()
    assert L.pbs_copy_cache_blocks(*p, N, A, 1, N, N) == 1 and L.pbs_copy_cache_blocks(*p, A, A, -1, N, N) == 1
    assert L.pbs_copy_cache_blocks(*p, N, N, 0, N, N) == 0
    assert L.pbs_reserve_cache_blocks(*r, N, A, 8, A, A, 1, N, N) == 1
    assert L.pbs_reserve_cache_blocks(*r, A, A, 8, N, A, 1, N, N) == 1
    assert L.pbs_reserve_cache_blocks(*r, A, A, 8, A, A, 0, N, N) == 0
    assert L.pbs_release_cache_blocks(*r, A, A, 8, A, 1, -1, 0, N, N) == 1
    assert L.pbs_release_cache_blocks(*r, A, A, 8, A, 1, 0, -1, N, N) == 1
    assert L.pbs_release_cache_blocks(*r, A, A, 8, N, 1, 0, 0, N, N) == 1
    assert L.pbs_fork_cache(*p, *r, A, A, 9, A, A, 1, A, A, N, N) == 2  # more blocks than the cache holds
    assert L.pbs_fork_cache(*p, *r, A, A, 8, A, A, 1, N, A, N, N) == 1
    assert L.pbs_compact_cache(*p, *r, A, 9, A, A, A, N, N) == 2
    assert L.pbs_compact_cache(*p, *r, A, 8, A, N, A, N, N) == 1


# ---- insert -----------------------------------------------------------------------------------------

def stored(cache, kv, hkv, page, row):
    """(K, V) [Hkv, 128] values at a page row, and NVFP4's scales and codes."""
    k, v = ow.rows_of({0: cache[page].cpu().numpy()}, kv, hkv, [0], [row])
    return np.stack([k[0], v[0]], 1)


@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("layout", ["rows", "slices", "odd"])
def test_insert(kv, hkv, layout):
    rng = np.random.default_rng(hkv)
    n, bps = 37, 9
    x = rng.standard_normal((n, 2, hkv, 128)).astype(np.float32) * np.exp2(rng.integers(-9, 10, (n, 2, hkv, 1)))
    x[0] = 0
    x[1, :, :, 5] = 1e30                      # saturates
    x[2] *= 1e-20                             # too small for e4m3
    x[3, 0, 0, 17] = np.inf
    kvt = torch.from_numpy(x).to(torch.bfloat16)
    if layout == "rows":
        k, v = kvt[:, 0].contiguous().cuda(), kvt[:, 1].contiguous().cuda()
    elif layout == "slices":
        big = kvt.cuda()
        k, v = big[:, 0], big[:, 1]
    else:
        big = torch.zeros(n, hkv, 2, 130, dtype=torch.bfloat16, device="cuda")
        big[:, :, 0, 1:129], big[:, :, 1, 2:130] = kvt[:, 0].cuda(), kvt[:, 1].cuda()
        k, v = big[:, :, 0, 1:129], big[:, :, 1, 2:130]
        v = v.transpose(1, 2).contiguous().transpose(1, 2)  # strided dims
    pb = page_bytes(kv, hkv)
    cache = torch.full((6 * bps, pb + 16), 0xA5, dtype=torch.uint8, device="cuda")
    slots = torch.from_numpy(rng.permutation(6 * 128)[:n]).long()
    slots[5], slots[6] = -1, -(1 << 40)
    before = cache.clone()
    ks, vs = 0.5, 2.0  # powers of two: x / scale is exact, so the stored codes have one right answer
    e = err()
    pbs.insert_kv_cache(k, v, cache[:, :pb], kv, slots.cuda(), ks, vs, block_page_stride=bps, err_word=e)
    assert int(e) == 0
    untouched = torch.ones_like(cache, dtype=torch.bool)
    e4, e2 = ow.e4m3_values(), ow.e2m1_values()
    for i in range(n):
        s = int(slots[i])
        if s < 0:
            continue
        page, row = s // 128 * bps + s % 128 // 16, s % 16
        got = stored(cache[:, :pb], kv, hkv, page, row)                       # [hkv, 2, 128]
        y = kvt[i].double().numpy().transpose(1, 0, 2)                        # [hkv, 2, 128]
        if kv == "bf16":
            want = y
        else:
            y = np.clip(y / np.array([ks, vs])[None, :, None], -1e38, 1e38)
            if kv == "fp8_e4m3":
                want = np.sign(y) * e4[ow.nearest(np.abs(y), e4)]
            else:
                z = y.reshape(hkv, 2, 8, 16)
                # max / 6 in fp32 as the definition's single rounding next to e4m3's 3 bits
                m = (np.abs(z).max(-1).astype(np.float32) * np.float32(1 / 6)).astype(np.float64)
                sc = e4[ow.nearest(m, e4)][..., None]
                with np.errstate(divide="ignore", invalid="ignore"):
                    w = np.where(sc > 0, np.sign(z) * e2[ow.nearest(np.abs(z / sc), e2)] * sc, 0)
                want = w.reshape(hkv, 2, 128)
        assert np.array_equal(got, want), (i, np.argwhere(got != want)[:4], got[got != want][:4], want[got != want][:4])
        if kv == "nvfp4":
            for t in range(2 * hkv):
                untouched[page, t * 1152 + row * 64:t * 1152 + row * 64 + 64] = False
                untouched[page, t * 1152 + 1024 + row * 8:t * 1152 + 1024 + row * 8 + 8] = False
        else:
            w = 512 if kv == "bf16" else 256
            for g in range(hkv):
                untouched[page, (g * 16 + row) * w:(g * 16 + row + 1) * w] = False
    assert torch.equal(cache[untouched], before[untouched])


@gpu
@pytest.mark.parametrize("kv", FMT[1:])
def test_insert_scales_and_nan(kv):
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((64, 2, 128)).astype(np.float32)).to(torch.bfloat16)
    x[3, 0, 20] = float("nan")
    pb = page_bytes(kv, 2)
    cache = torch.zeros(8, pb, dtype=torch.uint8, device="cuda")
    pbs.insert_kv_cache(x.cuda(), x.cuda(), cache, kv, torch.arange(64, device="cuda"), 0.3, 0.7)
    for i in range(64):
        got = stored(cache, kv, 2, i // 16, i % 16)
        y = x[i].double().numpy()[:, None] / np.array([np.float32(0.3), np.float32(0.7)], np.float64)[None, :, None]
        nan = np.isnan(got)
        if i == 3:  # an fp8 NaN is itself, an NVFP4 NaN its group of 16
            want = np.zeros_like(nan)
            want[0, :, slice(20, 21) if kv == "fp8_e4m3" else slice(16, 32)] = True
            assert np.array_equal(nan, want)
        else:
            assert not nan.any()
        y = np.where(nan, 0, y)
        got = np.where(nan, 0, got)
        if kv == "fp8_e4m3":
            tol = 2.0 ** -4 * np.abs(y) * (1 + 2.0 ** -20) + 2.0 ** -10  # half a step; subnormal steps are 2^-9
        else:
            # half an e2m1 step is at most 1 (between 4 and 6) scales; the scale is within 2^-4 of
            # max / 6, and max / scale may exceed 6 by that much before it saturates
            m = np.abs(y.reshape(2, 2, 8, 16)).max(-1, keepdims=True) / 6
            tol = np.broadcast_to(m * (1 + 2.0 ** -4) * 1.0 + 2.0 ** -9, (2, 2, 8, 16)).reshape(2, 2, 128)
        assert (np.abs(got - y) <= tol).all()


@gpu
def test_insert_bad_slots():
    x = torch.ones(4, 1, 128, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(16, page_bytes("bf16", 1), dtype=torch.uint8, device="cuda")
    e = err()
    pbs.insert_kv_cache(x, x, cache, "bf16", torch.tensor([0, 256, 1 << 62, -5], device="cuda"), err_word=e)
    assert int(e) == pbs.DEVERR["slot_oob"]
    assert int((cache != 0).sum()) == int((x[0].view(torch.uint8) != 0).sum()) * 2
    with pytest.raises(pbs.PbsError):
        pbs.insert_kv_cache(x, x, cache, "bf16", torch.zeros(4, dtype=torch.int64, device="cuda"), k_scale=0.0)
    for kw in (dict(v=x[:2]), dict(v=x.float()), dict(slots=torch.zeros(4, dtype=torch.int32, device="cuda")),
               dict(slots=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(kv="fp6")):
        with pytest.raises((TypeError, ValueError)):
            pbs.insert_kv_cache(x, kw.get("v", x), cache, kw.get("kv", "bf16"),
                                kw.get("slots", torch.zeros(4, dtype=torch.int64, device="cuda")))


# ---- block operations -------------------------------------------------------------------------------

class Model:
    """Plain model of a pool: page table, lengths, counts, and the cache as one number per block."""

    def __init__(self, table, lens, refs, cache):
        self.t, self.l, self.r, self.c = (x.cpu().numpy().copy() for x in (table, lens, refs, cache))

    def take(self):
        free = np.flatnonzero(self.r == 0)
        if not len(free):
            return -1
        self.r[free[0]] = 1
        return int(free[0])

    def reserve(self, rows, add):
        for r, n in zip(rows, add):
            ok = True
            for b in range(self.l[r] // 128, -(-(self.l[r] + n) // 128)) if n else []:
                if self.t[r, b] < 0:
                    got = self.take()
                    ok &= got >= 0
                    if got >= 0:
                        self.t[r, b] = got
            if ok:
                self.l[r] += n

    def fork(self, src, dst):
        tails = []
        for s in src:
            n = self.l[s]
            tails.append(self.take() if n % 128 and self.t[s, n // 128] >= 0 else None)
        for s, d, tail in zip(src, dst, tails):
            self.t[d] = -1
            if tail == -1:
                self.l[d] = 0
                continue
            n = self.l[s]
            for b in range(n // 128):
                self.t[d, b] = self.t[s, b]
                if self.t[s, b] >= 0:
                    self.r[self.t[s, b]] += 1
            if tail is not None:
                self.t[d, n // 128] = tail
                self.c[:, tail] = self.c[:, self.t[s, n // 128]]
            self.l[d] = n

    def release(self, rows, window=0, sinks=0):
        for r in rows:
            for b in range(self.t.shape[1]):
                if window and (b * 128 < sinks or b * 128 + 127 > self.l[r] - window):
                    continue
                if self.t[r, b] >= 0:
                    self.r[self.t[r, b]] -= 1
                self.t[r, b] = -1
            if not window:
                self.l[r] = 0

    def compact(self):
        live = np.flatnonzero(self.r > 0)
        n = len(live)
        movers, holes = live[live >= n], np.flatnonzero(self.r[:n] == 0)
        remap = np.where(self.r > 0, np.arange(len(self.r)), -1)
        for s, d in zip(movers, holes):
            remap[s] = d
            self.c[:, d] = self.c[:, s]
            self.r[d], self.r[s] = self.r[s], 0
        self.t = np.where(self.t >= 0, remap[self.t], self.t)
        return remap, n

    def same(self, table, lens, refs, cache):
        for name, want, got in (("table", self.t, table), ("lens", self.l, lens), ("refs", self.r, refs), ("cache", self.c, cache)):
            got = got.cpu().numpy()
            assert np.array_equal(want, got), (name, np.argwhere(want != got)[:5])


def pool(seed, num_blocks, rows, width, layers=2, bps=8, page=48, pad=0):
    """An empty pool; the cache holds distinct bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = torch.randint(0, 256, (layers, num_blocks * bps, page + pad), dtype=torch.uint8, device="cuda", generator=g)
    return (torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), i32([0] * rows), i32([0] * num_blocks),
            cache[..., :page])


def by_block(cache, bps=8):
    return cache.unflatten(1, (-1, bps))


@gpu
@pytest.mark.parametrize("n,layers,bps,page,pad", [(1, 1, 8, 16, 0), (5, 3, 8, 48, 0), (40, 2, 9, 2304, 0),
                                                  (7, 2, 16, 4096, 64), (3, 1, 8, 65536, 0)])
def test_copy(n, layers, bps, page, pad):
    t, l, r, cache = pool(n, 100, 1, 1, layers, bps, page, pad)
    perm = torch.randperm(100, generator=torch.Generator().manual_seed(n))
    src, dst = perm[:n].int().cuda(), perm[n:2 * n].int().cuda()
    want = by_block(cache, bps).clone()
    want[:, dst.long()] = want[:, src.long()]
    pbs.copy_cache_blocks(cache, src, dst, block_page_stride=bps)
    assert torch.equal(by_block(cache, bps), want)
    flat = cache[0] if layers == 1 else None
    if flat is not None:  # one layer as [pages, page]
        pbs.copy_cache_blocks(flat, dst, src, block_page_stride=bps)
        assert torch.equal(by_block(cache, bps), want)


@gpu
def test_copy_skips_and_reports():
    _, _, _, cache = pool(0, 10, 1, 1)
    want = by_block(cache).clone()
    e = err()
    pbs.copy_cache_blocks(cache, i32([-1, 3, 5, 2]), i32([4, -7, 5, 6]), err_word=e)
    want[:, 6] = want[:, 2]
    assert torch.equal(by_block(cache), want) and int(e) == 0
    pbs.copy_cache_blocks(cache, i32([10, 2, 2 ** 31 - 1]), i32([1, 10, 7]), err_word=e)
    assert torch.equal(by_block(cache), want) and int(e) == pbs.DEVERR["block_oob"]
    pbs.copy_cache_blocks(cache, i32([]), i32([]))


@gpu
@pytest.mark.parametrize("num_blocks,rows,width", [(64, 6, 8), (5000, 40, 300), (9000, 1500, 4)])
def test_reserve(num_blocks, rows, width):
    rng = np.random.default_rng(rows)
    s = pool(1, num_blocks, rows, width)
    s[2][torch.from_numpy(rng.permutation(num_blocks)[:num_blocks // 3]).cuda()] = 2
    m = Model(s[0], s[1], s[2], by_block(s[3]))
    for _ in range(4):
        n = int(rng.integers(1, rows + 1))
        pick = rng.permutation(rows)[:n]
        room = width * 128 - m.l[pick]
        add = np.minimum(rng.integers(0, 300, n), room) * (rng.random(n) < 0.9)
        e = err()
        pbs.reserve_cache_blocks(s[0], s[1], s[2], i32(pick.tolist()), i32(add.tolist()), err_word=e)
        m.reserve(pick, add)
        m.same(s[0], s[1], s[2], by_block(s[3]))
        short = bool((m.r > 0).all())
        assert int(e) in ((0, pbs.DEVERR["no_block"]) if short else (0,))


@gpu
def test_reserve_reports():
    s = pool(2, 3, 3, 4)
    m = Model(s[0], s[1], s[2], by_block(s[3]))
    e = err()
    pbs.reserve_cache_blocks(s[0], s[1], s[2], i32([-1, 3, 0, 1]), i32([1, 1, 513, -1]), err_word=e)
    m.same(s[0], s[1], s[2], by_block(s[3]))
    assert int(e) == pbs.DEVERR["table"]
    e = err()
    pbs.reserve_cache_blocks(s[0], s[1], s[2], i32([2, 0, 1]), i32([129, 256, 1]), err_word=e)
    m.reserve([2, 0, 1], [129, 256, 1])  # row 0 gets one of its two blocks, row 1 none
    m.same(s[0], s[1], s[2], by_block(s[3]))
    assert int(e) == pbs.DEVERR["no_block"] and m.l.tolist() == [0, 0, 129]


@gpu
@pytest.mark.parametrize("num_blocks,parents,children,width,bps,pad", [(200, 3, 7, 6, 8, 0), (6000, 30, 1100, 12, 9, 16),
                                                                       (40, 2, 2, 3, 8, 0)])
def test_fork_release(num_blocks, parents, children, width, bps, pad):
    rng = np.random.default_rng(children)
    rows = parents + children
    s = pool(3, num_blocks, rows, width, bps=bps, pad=pad)
    lens = rng.integers(0, (width - 1) * 128, parents)
    lens[0] = 256
    pbs.reserve_cache_blocks(s[0], s[1], s[2], i32(list(range(parents))), i32(lens.tolist()))
    pbs.release_cache_blocks(s[0], s[1], s[2], i32([parents - 1]), window=100, num_sinks=1)  # gaps
    m = Model(s[0], s[1], s[2], by_block(s[3], bps))
    src, dst = rng.integers(0, parents, children), parents + rng.permutation(children)
    start = [x.clone() for x in s[:3]]
    e = err()
    cs, cd = pbs.fork_cache(s[3], s[0], s[1], s[2], i32(src.tolist()), i32(dst.tolist()), block_page_stride=bps, err_word=e)
    m.fork(src, dst)
    m.same(s[0], s[1], s[2], by_block(s[3], bps))
    assert int(e) == 0
    tails = [(int(m.t[a, m.l[a] // 128]), int(m.t[b, m.l[b] // 128])) for a, b in zip(src, dst)
             if m.l[a] % 128 and m.t[a, m.l[a] // 128] >= 0]
    assert [(int(a), int(b)) for a, b in zip(cs, cd) if int(b) >= 0] == tails
    pbs.release_cache_blocks(s[0], s[1], s[2], i32(dst.tolist()), err_word=e)
    for a, b in zip(s[:3], start):
        assert torch.equal(a, b)
    assert int(e) == 0


@gpu
def test_fork_reports():
    s = pool(4, 4, 6, 3)
    pbs.reserve_cache_blocks(s[0], s[1], s[2], i32([0]), i32([300]))
    m = Model(s[0], s[1], s[2], by_block(s[3]))
    e = err()
    pbs.fork_cache(s[3], s[0], s[1], s[2], i32([0, 6, 0, -1]), i32([0, 1, 6, 1]), err_word=e)
    m.same(s[0], s[1], s[2], by_block(s[3]))
    assert int(e) == pbs.DEVERR["table"]
    e = err()
    pbs.fork_cache(s[3], s[0], s[1], s[2], i32([0, 0, 0]), i32([1, 2, 3]), err_word=e)  # one free block
    m.fork([0, 0, 0], [1, 2, 3])
    m.same(s[0], s[1], s[2], by_block(s[3]))
    assert int(e) == pbs.DEVERR["no_block"] and m.l.tolist() == [300, 300, 0, 0, 0, 0]


@gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 0), (128, 1), (129, 128), (300, 200), (5000, 3)])
def test_release(window, sinks):
    lens = [0, 1, 127, 128, 129, 255, 256, 257, 700, 1000]
    s = pool(5, 200, 12, 9)
    pbs.reserve_cache_blocks(s[0], s[1], s[2], i32(list(range(10))), i32(lens))
    m = Model(s[0], s[1], s[2], by_block(s[3]))
    e = err()
    rows = [9, 0, 1, 2, 3, 4, 5, 6, 7, 8]
    pbs.release_cache_blocks(s[0], s[1], s[2], i32(rows + [9, 3]), window=window, num_sinks=sinks, err_word=e)
    m.release(rows, window, sinks)  # a row listed twice gives back once
    m.same(s[0], s[1], s[2], by_block(s[3]))
    assert int(e) == 0
    # what is left is what the next queries see
    if window:
        for r, n in enumerate(lens):
            for key in ow.visible(n, window, sinks)[:-1]:
                assert m.t[r, key // 128] >= 0
    pbs.release_cache_blocks(s[0], s[1], s[2], i32([-1, 12]), err_word=e)
    assert int(e) == pbs.DEVERR["table"]
    e = err()
    s[0][11, 0], s[0][11, 1] = 7, 200  # a block already free, and one that is none
    s[2][7] = 0
    pbs.release_cache_blocks(s[0], s[1], s[2], i32([11]), err_word=e)
    assert int(e) == pbs.DEVERR["table"] | pbs.DEVERR["block_oob"] and int(s[2][7]) == 0


@gpu
@pytest.mark.parametrize("num_blocks,live,bps,pad", [(1, 0, 8, 0), (1, 1, 8, 0), (300, 150, 8, 0), (300, 300, 9, 16),
                                                     (300, 0, 8, 0), (9500, 4000, 8, 0), (5001, 5000, 8, 0)])
def test_compact(num_blocks, live, bps, pad):
    rng = np.random.default_rng(num_blocks + live)
    s = pool(6, num_blocks, 7, 40, bps=bps, pad=pad)
    ids = rng.permutation(num_blocks)[:live]
    s[2][torch.from_numpy(ids).cuda()] = torch.from_numpy(rng.integers(1, 5, live)).int().cuda()
    if live:
        t = ids[rng.integers(0, live, (7, 40))]
        t[rng.random((7, 40)) < 0.3] = -1
        s[0].copy_(torch.from_numpy(t).int())
    m = Model(s[0], s[1], s[2], by_block(s[3], bps))
    e = err()
    remap, n = pbs.compact_cache(s[3], s[0], s[2], block_page_stride=bps, err_word=e)
    want, count = m.compact()
    m.same(s[0], s[1], s[2], by_block(s[3], bps))
    assert np.array_equal(remap.cpu().numpy(), want) and int(n) == count == live and int(e) == 0


@gpu
def test_compact_reports():
    s = pool(7, 10, 2, 3)
    s[2][8] = 1
    s[0].copy_(torch.tensor([[8, 3, 10], [-1, 8, -5]], dtype=torch.int32))
    e = err()
    pbs.compact_cache(s[3], s[0], s[2], err_word=e)
    assert s[0].tolist() == [[0, -1, 10], [-1, 0, -5]]
    assert int(e) == pbs.DEVERR["table"] | pbs.DEVERR["block_oob"]


@gpu
def test_python_refusals():
    t, l, r, c = pool(8, 10, 2, 3)
    for f in (lambda: pbs.copy_cache_blocks(c, i32([1]), i32([1, 2])),
              lambda: pbs.copy_cache_blocks(c, torch.tensor([1]).cuda(), i32([1])),
              lambda: pbs.copy_cache_blocks(c.unsqueeze(0), i32([1]), i32([2])),
              lambda: pbs.reserve_cache_blocks(t, l[:1], r, i32([0]), i32([1])),
              lambda: pbs.reserve_cache_blocks(t.long(), l, r, i32([0]), i32([1])),
              lambda: pbs.fork_cache(c, t, l, r, i32([0]), i32([1, 0])),
              lambda: pbs.release_cache_blocks(t, l, r.cpu(), i32([0])),
              lambda: pbs.compact_cache(c, t.t(), r)):
        with pytest.raises((TypeError, ValueError)):
            f()
    with pytest.raises(pbs.PbsError):
        pbs.compact_cache(c, t, i32([0] * 11))


# ---- together -----------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kv", FMT)
def test_a_servers_life(kv):
    """Prompts in, decode steps, a fork, a window's blocks released, the pool packed: at each point the
    attends see what plain attention over the tokens' stored K and V sees."""
    hkv, g, width, nb, window, sinks = 2, 4, 8, 40, 150, 10
    rows = 5
    gen = torch.Generator().manual_seed(3)
    cache = torch.full((nb * 8, page_bytes(kv, hkv)), 0x7F, dtype=torch.uint8, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens, refs = i32([0] * rows), i32([0] * nb)
    scales = (1.0, 1.0) if kv == "bf16" else (0.75, 1.25)
    e = err()
    tokens = {r: [] for r in range(rows)}  # (k, v) of each token

    def append(which, counts):
        old = lens.tolist()
        pbs.reserve_cache_blocks(table, lens, refs, i32(which), i32(counts), err_word=e)
        total = sum(counts)
        k, v = (torch.randn(total, hkv, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
        slots, at = [], 0
        tb = table.cpu()
        for r, n in zip(which, counts):
            for p in range(old[r], old[r] + n):
                slots.append(int(tb[r, p // 128]) * 128 + p % 128)
            tokens[r] += [(k[at + i], v[at + i]) for i in range(n)]
            at += n
        pbs.insert_kv_cache(k, v, cache, kv, torch.tensor(slots, device="cuda"), *scales, err_word=e)

    def look(which):
        """The last token of each row against 64-bit attention over its stored rows."""
        q = torch.randn(len(which), hkv * g, 128, generator=gen).to(torch.bfloat16)
        idx = torch.tensor(which, device="cuda")
        tab, ln = table[idx].contiguous(), lens[idx].contiguous()
        out = pbs.window_decode_attention(q.cuda(), cache, kv, hkv, tab, ln, 1, 0.09, window=window, num_sinks=sinks,
                                          k_scale=scales[0], v_scale=scales[1], err_word=e)
        pre = pbs.window_prefill_attention(q.cuda(), cache, kv, hkv, tab,
                                           torch.arange(len(which) + 1, dtype=torch.int32, device="cuda"), ln, 0.09,
                                           window=window, num_sinks=sinks, k_scale=scales[0], v_scale=scales[1], err_word=e)
        host = cache.cpu().numpy()
        for i, r in enumerate(which):
            n = int(ln[i])
            o, _, mass, z = ow.window_row(q[i].double().numpy(), host, kv, hkv, tab[i].cpu().numpy(), n - 1, window,
                                          sinks, 0.09, *scales)
            tol = 2.0 ** -8 * np.abs(o) + mass * (2.0 ** -10 + 2.0 ** -15 * z[:, None])
            for got in (out, pre):
                assert (np.abs(got[i].double().cpu().numpy() - o) <= tol).all()
            # the stored rows are the tokens' own: the newest and the oldest visible
            for p in (n - 1, max(0, n - window)):
                page = int(tab[i, p // 128]) * 8 + p % 128 // 16
                kk, vv = ow.rows_of(host, kv, hkv, [page], [p % 16])
                want = torch.stack(tokens[r][p]).double().cpu().numpy()
                got = np.stack([kk[0] * scales[0], vv[0] * scales[1]])
                assert np.abs(got - want).max() <= {"bf16": 0, "fp8_e4m3": 2.0 ** -4, "nvfp4": 0.2}[kv] * np.abs(want).max()
        assert int(e) == 0

    append([0, 2], [300, 513])
    look([0, 2])
    for _ in range(3):
        append([0, 2], [1, 1])
    look([0, 2])
    pbs.fork_cache(cache, table, lens, refs, i32([0, 0]), i32([1, 3]), err_word=e)
    tokens[1], tokens[3] = list(tokens[0]), list(tokens[0])
    append([1, 3, 0], [200, 1, 2])
    look([0, 1, 2, 3])
    pbs.release_cache_blocks(table, lens, refs, i32([0, 1, 2, 3]), window=window, num_sinks=sinks, err_word=e)
    append([0, 1, 2, 3], [1, 1, 1, 1])
    look([0, 1, 2, 3])
    pbs.release_cache_blocks(table, lens, refs, i32([0]), err_word=e)
    tokens[0] = []
    _, live = pbs.compact_cache(cache, table, refs, err_word=e)
    assert int(live) == int((refs > 0).sum()) and bool((refs[:int(live)] > 0).all())
    look([1, 2, 3])
    append([0, 1], [130, 140])
    look([0, 1, 2, 3])
    pbs.release_cache_blocks(table, lens, refs, i32([0, 1, 2, 3]), err_word=e)
    assert not bool(refs.any()) and not bool((table >= 0).any()) and int(e) == 0


@gpu
@pytest.mark.parametrize("how", ["stream", "graph"])
def test_cache_operations_on_another_stream_and_in_a_graph(how):
    """Reserve, insert, fork, copy, a window's release and compact as one sequence: the same state as on the
    current stream, each time the graph is replayed."""
    hkv, nb, rows, width = 2, 300, 40, 12
    rng = np.random.default_rng(2)
    first = i32(list(range(8))), i32(rng.integers(100, 1400, 8).tolist())
    grow = i32(list(range(16))), i32(rng.integers(1, 3, 16).tolist())
    src, dst = i32([i % 8 for i in range(16)]), i32(list(range(8, 24)))
    k = torch.randn(64, hkv, 128, device="cuda").to(torch.bfloat16)
    slots = torch.from_numpy(rng.permutation(nb * 128)[:64]).cuda()
    moved = i32([290, 291]), i32([298, 299])

    def state():
        gen = torch.Generator(device="cuda").manual_seed(1)
        cache = torch.randint(0, 256, (nb * 8, page_bytes("fp8_e4m3", hkv)), dtype=torch.uint8, device="cuda", generator=gen)
        return cache, torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), i32([0] * rows), i32([0] * nb)

    def sequence(s, **kw):
        cache, table, lens, refs = s
        pbs.reserve_cache_blocks(table, lens, refs, *first, **kw)
        pbs.insert_kv_cache(k, k, cache, "fp8_e4m3", slots, 0.5, 0.25, **kw)
        pairs = pbs.fork_cache(cache, table, lens, refs, src, dst, **kw)
        pbs.reserve_cache_blocks(table, lens, refs, *grow, **kw)
        pbs.copy_cache_blocks(cache, *moved, **kw)
        pbs.release_cache_blocks(table, lens, refs, first[0], **kw)
        pbs.release_cache_blocks(table, lens, refs, dst, window=200, num_sinks=3, **kw)
        return (*pairs, *pbs.compact_cache(cache, table, refs, **kw))

    want = state()
    out = sequence(want)
    s = state()
    start = [x.clone() for x in s]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if how == "stream":
        got = sequence(s, stream=side)
        side.synchronize()
        runs = 1
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = sequence(s)
        runs = 3
    for _ in range(runs):
        if how == "graph":
            for x, y in zip(s, start):
                x.copy_(y)
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*want, *out), (*s, *got)):
            assert torch.equal(a, b)

"""Window attend with sinks (decode rows and varlen prefill) against the 64-bit oracle, its refusals
and its errors."""
import ctypes

import numpy as np
import pytest
import torch

import paged_block_sparse_gb300 as pbs
from window_cases import Case, check

FMT = ("bf16", "fp8_e4m3", "nvfp4")
gpu = pytest.mark.gpu


def decode(c, d, dql, **kw):
    return pbs.window_decode_attention(d["q"], d["cache"], c.kv, c.hkv, d["table"], d["lens"], dql, c.scale,
                                       window=c.window, num_sinks=c.sinks, k_scale=c.k_scale, v_scale=c.v_scale,
                                       block_page_stride=c.bps, **kw)


def prefill(c, d, **kw):
    return pbs.window_prefill_attention(d["q"], d["cache"], c.kv, c.hkv, d["table"], d["cu"], d["lens"], c.scale,
                                        window=c.window, num_sinks=c.sinks, k_scale=c.k_scale, v_scale=c.v_scale,
                                        block_page_stride=c.bps, **kw)


def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- refusals (no GPU: each call fails a check that runs before the first CUDA call) ---------------

@pytest.fixture(scope="module")
def L():
    from paged_block_sparse_gb300 import _build
    _build.build()
    return pbs.lib()


A, N = ctypes.c_void_p(0x10000), ctypes.c_void_p(0)


def c_decode(L, **kw):
    a = dict(q=A, qr=1024, qh=128, kv=A, ps=65536, np=64, fmt=0, hq=8, hkv=8, d=128, pt=A, pts=4, mb=4, sl=A, b=2,
             dql=1, bps=8, w=16, s=4, sc=1.0, ks=1.0, vs=1.0, out=A, orow=1024, oh=128, lse=N, ls=0, ws=N, wb=0)
    a.update(kw)
    return L.pbs_window_decode_attention(*a.values(), N, N)


def c_prefill(L, **kw):
    a = dict(q=A, qr=1024, qh=128, kv=A, ps=65536, np=64, fmt=0, hq=8, hkv=8, d=128, pt=A, pts=4, mb=4, cu=A, sl=A,
             n=2, tq=5, bps=8, w=16, s=4, sc=1.0, ks=1.0, vs=1.0, out=A, orow=1024, oh=128, lse=N, ls=0, ws=N, wb=0)
    a.update(kw)
    return L.pbs_window_prefill_attention(*a.values(), N, N)


@pytest.mark.parametrize("call", [c_decode, c_prefill])
@pytest.mark.parametrize("want,kw", [
    (1, dict(q=N)), (1, dict(kv=N)), (1, dict(out=N)), (1, dict(pt=N)), (1, dict(sl=N)), (1, dict(fmt=3)),
    (1, dict(w=-1)), (1, dict(s=-1)), (1, dict(sc=float("nan"))), (1, dict(vs=float("inf"))), (1, dict(mb=0)),
    (1, dict(wb=64)), (2, dict(pts=3)), (2, dict(bps=7)), (2, dict(hkv=3)), (2, dict(ps=65520)), (2, dict(np=0)),
    (2, dict(lse=A, ls=7)), (3, dict(d=64)), (3, dict(hq=24)), (3, dict(hq=256)), (4, dict(ps=65540)),
    (4, dict(kv=ctypes.c_void_p(0x10008))), (4, dict(q=ctypes.c_void_p(0x10002))), (4, dict(qr=1023)),
    (4, dict(lse=ctypes.c_void_p(0x10002), ls=8))])
def test_refusals(L, call, want, kw):
    assert call(L, **kw) == want


def test_refusals_of_one_entry(L):
    assert c_decode(L, b=0) == 0 and c_prefill(L, tq=0) == 0
    assert c_decode(L, b=-1) == 1 and c_decode(L, dql=0) == 1 and c_decode(L, b=1 << 30) == 3
    assert c_decode(L, ws=ctypes.c_void_p(0x10008), wb=1 << 40) == 4
    assert c_decode(L, ws=A, wb=1) == 2
    assert c_prefill(L, tq=-1) == 1 and c_prefill(L, n=0) == 2 and c_prefill(L, cu=N) == 1
    assert L.pbs_window_decode_workspace_bytes(0, 1, 8, 8) == 0
    assert L.pbs_window_decode_workspace_bytes(1, 1, 8, 3) == 0
    assert L.pbs_window_prefill_workspace_bytes(1, 1, 1, 1, 3, 0, 0) == 0
    assert L.pbs_window_prefill_workspace_bytes(1, 1, 1, 1, 0, -1, 0) == 0


@gpu
def test_python_refusals():
    c = Case("bf16", 1, 1, [(1, 5)], 4, 0)
    d = c.dev()
    for kw in (dict(q=d["q"].float()), dict(q=d["q"].transpose(1, 2)), dict(table=d["table"].long()),
               dict(table=d["table"].cpu()), dict(lens=d["lens"].long()), dict(lens=d["lens"][:0]),
               dict(cache=d["cache"].cpu()), dict(q=torch.cat([d["q"]] * 2))):
        with pytest.raises((TypeError, ValueError, pbs.PbsError)):
            decode(c, {**d, **kw}, 1)
    with pytest.raises(ValueError):
        decode(c, d, 1, workspace="none")
    with pytest.raises(pbs.PbsError):
        decode(c, d, 1, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        prefill(c, {**d, "cu": d["cu"][:1]})


# ---- decode rows ----------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 2), (3, 4), (2, 8), (1, 16)])
@pytest.mark.parametrize("dql", [1, 2, 3])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_decode(kv, hkv, g, dql, workspace):
    # lengths around page, block and window borders; one request shorter than its rows, one empty
    lens = [0, 1, dql, 15, 16, 17, 127, 128, 129, 300, 391]
    c = Case(kv, hkv, g, [(dql, t) for t in lens], 130, 5, seed=g * 10 + dql)
    d, e = c.dev(), err()
    out, lse = decode(c, d, dql, return_lse=True, workspace=workspace, err_word=e)
    check(out, lse, c.want())
    assert int(e) == 0


@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 16), (128, 128), (129, 127), (100, 400), (37, 3)])
def test_decode_windows(kv, window, sinks):
    c = Case(kv, 2, 4, [(2, t) for t in (2, 40, 128, 257, 515)], window, sinks, seed=window)
    d = c.dev()
    out, lse = decode(c, d, 2, return_lse=True)
    check(out, lse, c.want())


@gpu
@pytest.mark.parametrize("kv", FMT)
def test_decode_long_and_ragged(kv):
    # one long request among short ones: cut between many CTAs, merged in order
    c = Case(kv, 1, 8, [(1, 5000), (1, 3), (1, 0), (1, 700), (1, 1)], 0, 0, seed=5)
    d = c.dev()
    out, lse = decode(c, d, 1, return_lse=True)
    check(out, lse, c.want())
    for _ in range(3):  # the same bits however the CTAs finish, and the workspace is left ready
        again, l2 = decode(c, d, 1, return_lse=True)
        assert torch.equal(again, out) and torch.equal(l2, lse)


@gpu
@pytest.mark.parametrize("kv", FMT)
def test_decode_strides_page_stride_and_streams(kv):
    c = Case(kv, 2, 8, [(2, 200), (2, 77)], 64, 9, seed=3, bps=16, pad=48)
    d = c.dev()
    big = torch.full((c.total_q, c.hq + 3, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros_like(big)
    q[:, 1:c.hq + 1, 2:130] = d["q"]
    d["q"] = q[:, 1:c.hq + 1, 2:130]
    out = big[:, 2:c.hq + 2, 1:129]
    wide = torch.full((2, d["table"].shape[1] + 3), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + d["table"].shape[1]] = d["table"]
    d["table"] = wide[:, 2:2 + d["table"].shape[1]]
    lse = torch.full((c.total_q, c.hq + 5), 3.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    decode(c, d, 2, out=out, lse=lse[:, :c.hq], stream=s)
    s.synchronize()
    check(out, lse[:, :c.hq], c.want())
    keep = torch.ones_like(big, dtype=torch.bool)
    keep[:, 2:c.hq + 2, 1:129] = False
    assert (big[keep] == 7).all() and (lse[:, c.hq:] == 3).all()


@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("workspace", ["auto", None])
def test_decode_masked_values_do_not_leak(kv, workspace):
    # rows 0 and 1 of a request: row 0 must not see what the newest key holds, nor row 1 the oldest
    c = Case(kv, 1, 4, [(2, 200)], 100, 0, seed=1)
    pos = [198, 199]
    o, l, mass, z = c.want()
    for key in (199, 99):  # visible to row 1 only / row 0 only
        b = c.table[0, key // 128]
        page = c.pages[int(b) * 8 + key % 128 // 16]
        saved = page.copy()
        row = key % 16
        if kv == "nvfp4":
            page[1152 + 1024 + row * 8:1152 + 1024 + row * 8 + 8] = 0x7F
        else:
            w = {"bf16": 512, "fp8_e4m3": 256}[kv]
            page[row * w + w // 2:(row + 1) * w] = 0xFF
        out = decode(c, c.dev(), 2, workspace=workspace)
        hidden = 0 if key == 199 else 1
        check(out[hidden:hidden + 1], None, [x[hidden:hidden + 1] for x in (o, l, mass, z)])
        assert torch.isnan(out[1 - hidden]).all()
        c.pages[int(b) * 8 + key % 128 // 16] = saved


@gpu
@pytest.mark.parametrize("workspace", ["auto", None])
def test_decode_bad_tables_are_reported(workspace):
    c = Case("bf16", 1, 2, [(1, 300), (1, 300)], 0, 0, seed=2)
    d = c.dev()
    good = decode(c, d, 1, workspace=workspace)
    for value in (-1, c.num_blocks, 2 ** 31 - 1, -2 ** 31):
        t = d["table"].clone()
        t[0, 1] = value
        e = err()
        out = decode(c, {**d, "table": t}, 1, err_word=e, workspace=workspace)
        assert int(e) == pbs.DEVERR["page_oob"]
        assert torch.equal(out[1], good[1])
        # the row's other keys are attended
        keys = [n for n in range(300) if n // 128 != 1]
        assert torch.isfinite(out[0]).all() and not torch.equal(out[0], good[0]) and keys
    e = err()
    out = decode(c, {**d, "table": d["table"][:, :2].contiguous()}, 1, err_word=e, workspace=workspace)
    assert int(e) == pbs.DEVERR["block_oob"] and torch.isfinite(out).all()


@gpu
@pytest.mark.parametrize("kv", FMT)
def test_decode_offsets_past_32_bits(kv):
    pb = {"bf16": 8192, "fp8_e4m3": 4096, "nvfp4": 2304}[kv]
    c = Case(kv, 1, 8, [(1, 150)], 0, 0, seed=4, first_block=-(-(1 << 32) // (pb * 8)) + 5)
    d = c.dev()
    assert d["cache"].numel() > 1 << 32
    check(decode(c, d, 1), None, c.want())
    check(prefill(c, d), None, c.want())


@gpu
def test_decode_captured_graphs_share_nothing():
    cs = [Case("bf16", 1, 8, [(1, 3000), (1, 900)], 0, 0, seed=s) for s in (6, 7)]
    ds = [c.dev() for c in cs]
    want = [decode(c, d, 1) for c, d in zip(cs, ds)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, d in zip(cs, ds):
        out = torch.empty_like(d["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode(c, d, 1, out=out)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


# ---- prefill --------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 2), (1, 4), (2, 8), (1, 16)])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_prefill(kv, hkv, g, workspace):
    reqs = [(1, 1), (17, 17), (0, 0), (33, 200), (150, 150), (5, 130), (1, 300)]
    c = Case(kv, hkv, g, reqs, 77, 6, seed=g)
    d, e = c.dev(), err()
    out, lse = prefill(c, d, return_lse=True, workspace=workspace, err_word=e)
    check(out, lse, c.want())
    assert int(e) == 0


@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 16), (128, 128), (300, 129), (100, 400), (37, 3)])
def test_prefill_windows(kv, window, sinks):
    c = Case(kv, 1, 8, [(70, 400), (130, 130), (3, 515)], window, sinks, seed=window + 1)
    out, lse = prefill(c, c.dev(), return_lse=True)
    check(out, lse, c.want())


@gpu
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1), (0, 2 ** 31 - 1)])
def test_widest_windows_and_sinks(window, sinks):
    c = Case("bf16", 2, 4, [(2, 2), (2, 300), (2, 129)], 0, 0, seed=3)
    d = c.dev()
    c.window, c.sinks = 0, 0
    want, plain = decode(c, d, 2, return_lse=True), prefill(c, d, return_lse=True)
    check(*want, c.want())
    c.window, c.sinks = window, sinks
    for a, b in zip((*decode(c, d, 2, return_lse=True), *prefill(c, d, return_lse=True)), (*want, *plain)):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("kv", FMT)
def test_prefill_long(kv):
    # sampled rows of prompts that span many key blocks and query tiles
    c = Case(kv, 1, 8, [(700, 1500), (260, 260)], 600, 40, seed=8)
    out, lse = prefill(c, c.dev(), return_lse=True)
    rows = [0, 1, 15, 16, 127, 128, 300, 599, 699, 700, 701, 828, 959]
    check(out, lse, c.want(rows), rows)


@gpu
@pytest.mark.parametrize("workspace", ["auto", None])
def test_prefill_padded_rows_and_strides(workspace):
    c = Case("bf16", 2, 4, [(40, 90), (9, 9)], 33, 2, seed=9, bps=16, pad=32)
    d = c.dev()
    pad = 6
    q = torch.zeros(c.total_q + pad, c.hq + 2, 128, dtype=torch.bfloat16, device="cuda")
    q[:c.total_q, 1:c.hq + 1] = d["q"]
    big = torch.full((c.total_q + pad, c.hq + 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.total_q + pad, c.hq), 3.0, device="cuda")
    d["q"] = q[:, 1:c.hq + 1]
    prefill(c, d, out=big[:, 1:c.hq + 1], lse=lse, workspace=workspace)
    check(big[:c.total_q, 1:c.hq + 1], lse[:c.total_q], c.want())
    assert (big[c.total_q:] == 7).all() and (big[:, 0] == 7).all() and (big[:, -1] == 7).all()
    assert (lse[c.total_q:] == 3).all()
    # rows that start off a 16-byte boundary
    odd = torch.zeros(c.total_q, c.hq, 130, dtype=torch.bfloat16, device="cuda")
    odd[..., 2:] = c.q.cuda()
    out = prefill(c, {**c.dev(), "q": odd[..., 2:]}, workspace=workspace)
    check(out, None, c.want())


@gpu
@pytest.mark.parametrize("workspace", ["auto", None])
def test_prefill_requests_that_start_before_row_0_are_left_out(workspace):
    c = Case("bf16", 2, 4, [(8, 50), (7, 200)], 40, 3, seed=8)
    d = c.dev()
    out = torch.full_like(d["q"], 7.0)
    d["cu"][0] = -3
    prefill(c, d, out=out, workspace=workspace)
    assert (out[:8] == 7.0).all()
    check(out, None, c.want(range(8, 15)), range(8, 15))


@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("workspace", ["auto", None])
def test_prefill_bad_tables_are_reported(kv, workspace):
    c = Case(kv, 1, 8, [(20, 300), (40, 140)], 0, 0, seed=2)
    d = c.dev()
    good = prefill(c, d, workspace=workspace)
    for value in (-1, c.num_blocks, 2 ** 31 - 1, -2 ** 31):
        t = d["table"].clone()
        t[0, 1] = value
        e = err()
        out = prefill(c, {**d, "table": t}, err_word=e, workspace=workspace)
        assert int(e) == pbs.DEVERR["page_oob"]
        assert torch.equal(out[20:], good[20:]) and torch.isfinite(out).all()
        assert not torch.equal(out[:20], good[:20])
    e = err()
    out = prefill(c, {**d, "table": d["table"][:, :2].contiguous()}, err_word=e, workspace=workspace)
    assert int(e) == pbs.DEVERR["block_oob"] and torch.equal(out[20:], good[20:]) and torch.isfinite(out).all()


@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("g", [2, 8])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_prefill_odd_values_reach_the_rows_that_see_them(kv, g, window, sinks, workspace):
    """Infinities and NaN in V of keys that some tokens of a tile see and others do not."""
    c = Case(kv, 2, g, [(200, 200), (77, 390), (1, 140), (33, 33)], window, sinks, seed=g, bps=9)
    rng = np.random.default_rng(5)
    bits = (0x7F80, 0xFF80, 0x7FC0)  # +inf, -inf, NaN
    for r, key in ((0, 3), (0, 60), (0, 127), (0, 128), (0, 199), (1, 10), (1, 300), (1, 389), (2, 130), (3, 32)):
        page, row = int(c.table[r, key // 128]) * c.bps + key % 128 // 16, key % 16
        for head in range(2):
            if page not in c.pages or c.table[r, key // 128] < 0:
                continue
            for d in rng.choice(128, 3, replace=False):
                if kv == "bf16":
                    at = (head * 16 + row) * 512 + 256 + 2 * int(d)
                    c.pages[page][at:at + 2] = np.array([bits[d % 3]], np.uint16).view(np.uint8)
                elif kv == "fp8_e4m3":
                    c.pages[page][(head * 16 + row) * 256 + 128 + int(d)] = 0x7F
                else:
                    c.pages[page][(2 * head + 1) * 1152 + 1024 + row * 8 + int(d) // 16] = 0x7F
    d, e = c.dev(), err()
    out, lse = prefill(c, d, return_lse=True, workspace=workspace, err_word=e)
    with np.errstate(invalid="ignore"):
        want = c.want()
    o = want[0]
    got = out.double().cpu().numpy()
    assert int(e) == 0 and not np.isfinite(o).all() and np.isfinite(o).any()
    assert np.array_equal(np.isnan(got), np.isnan(o))
    assert np.array_equal(got == np.inf, o == np.inf) and np.array_equal(got == -np.inf, o == -np.inf)
    ok = np.isfinite(o)
    want[0], want[2] = np.where(ok, o, 0), np.where(ok, want[2], 0)
    check(torch.where(torch.from_numpy(ok).cuda(), out, torch.zeros_like(out)), lse, want)


@gpu
@pytest.mark.parametrize("kv", FMT)
def test_prefill_values_of_any_size(kv):
    # V blocks whose magnitudes differ by far more than fp16 spans, each the only one some rows see
    c = Case(kv, 1, 8, [(300, 300)], 20, 0, seed=12)
    if kv == "bf16":
        for b, f in ((0, 2.0 ** -60), (1, 2.0 ** 60), (2, 1.0)):
            for p in range(8):
                page = c.pages.get(int(c.table[0, b]) * 8 + p)
                if page is not None:
                    x = torch.from_numpy(page.copy()).view(torch.bfloat16).view(16, 256)
                    x[:, 128:] *= f
                    page[:] = x.view(torch.uint8).numpy().reshape(-1)
    out = prefill(c, c.dev())
    check(out, None, c.want())


@gpu
def test_prefill_values_that_shrink_along_a_long_context():
    """80 blocks of V around 2^50, then smaller and smaller ones, all of one weight (q = 0): sums near 2^63, to
    which the last blocks add nothing."""
    c = Case("bf16", 1, 8, [(3, 10900)], 0, 0, seed=17)
    c.q.zero_()
    shift = {80: 2, 81: -20, 82: -38, 83: -45, 84: -80, 85: -90}
    for b in range(c.max_blocks):
        for page in range(int(c.table[0, b]) * 8, int(c.table[0, b]) * 8 + 8):
            if page in c.pages:
                rows = c.pages[page].reshape(16, 512)[:, 256:]
                v = torch.from_numpy(rows.copy()).view(torch.bfloat16)
                v = torch.where(v.isnan(), v, (v.float() * 2.0 ** shift.get(b, 50)).to(torch.bfloat16))
                rows[:] = v.view(torch.uint8).numpy()
    d = c.dev()
    out, lse = prefill(c, d, return_lse=True)
    check(out, lse, c.want())


@gpu
def test_prefill_captured():
    c = Case("nvfp4", 1, 8, [(60, 500), (1, 9)], 200, 4, seed=11)
    d = c.dev()
    want = prefill(c, d)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prefill(c, d, out=out)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("kv", FMT)
def test_window_and_sparse_attends_agree(kv):
    # every block selected: the sparse decode attend and the full window attend see the same keys
    c = Case(kv, 1, 8, [(1, 500), (1, 77)], 0, 0, seed=13)
    d = c.dev()
    topk = torch.arange(4, dtype=torch.int32, device="cuda").expand(2, 4).contiguous()
    if kv != "nvfp4":
        d["cache"] = d["cache"].contiguous()
    ours, l1 = decode(c, d, 1, return_lse=True)
    theirs, l2 = pbs.sparse_decode_attention(d["q"], d["cache"], kv, 1, topk, d["table"].clamp(min=0), d["lens"], 1,
                                             c.scale, c.k_scale, c.v_scale, return_lse=True)
    check(ours, l1, c.want())
    check(theirs, l2, c.want())


@gpu
@pytest.mark.parametrize("kv", FMT)
def test_prefill_calls_on_two_streams_at_once(kv):
    cases = [Case(kv, 2, 4, [(300, 300), (70, 500)], 130, 20, seed=21), Case(kv, 2, 4, [(520, 700)], 0, 0, seed=22)]
    ds = [c.dev() for c in cases]
    want = [prefill(c, d, return_lse=True) for c, d in zip(cases, ds)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[prefill(c, d, return_lse=True, stream=st) for c, d, st in zip(cases, ds, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("kv", FMT)
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 20)])
def test_prefill_in_parts(kv, window, sinks, monkeypatch):
    """A workspace for one or some of the requests: the same bits as with all of it; for less: the other kernel."""
    c = Case(kv, 2, 4, [(40, 300), (1, 1), (130, 130), (0, 77), (70, 500)], window, sinks, seed=31)
    d, e = c.dev(), err()
    n, mb = len(c.reqs), c.max_blocks
    want = prefill(c, d, return_lse=True, err_word=e)
    check(*want, c.want())
    size = lambda reqs: pbs.window_prefill_workspace_bytes(c.total_q, reqs, c.hkv, mb, kv, window, sinks)
    for reqs in range(1, n):
        assert size(reqs) < size(n)
        ws = torch.empty(size(reqs), dtype=torch.uint8, device="cuda")
        got = prefill(c, d, return_lse=True, err_word=e, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    small = torch.empty(size(1) - 256, dtype=torch.uint8, device="cuda")
    check(*prefill(c, d, return_lse=True, err_word=e, workspace=small), c.want())
    for cap in (size(2), size(1) - 256):
        monkeypatch.setattr(pbs, "WINDOW_WORKSPACE_CAP", cap)
        pbs._window_workspaces.clear()
        got = prefill(c, d, return_lse=True, err_word=e)
        check(*got, c.want())
    pbs._window_workspaces.clear()
    assert int(e) == 0


@gpu
def test_prefill_with_more_images_than_the_conversion_has_blocks():
    """40 blocks x 512 kv heads. Both kernels are within 2^-8 |o| + mass (2^-10 + 2 logit) of the true value (see
    check), mass <= max |V| and logit <= 2^-16 * 16 here: twice that between them."""
    hkv, blocks = 512, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = torch.empty(blocks * 8, hkv * 16 * 256, dtype=torch.uint8, device="cuda")
    for i in range(0, blocks * 8, 8):
        cache[i:i + 8] = torch.randn(8, hkv * 16 * 256, device="cuda", generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(5, hkv, 128, device="cuda", generator=g).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(blocks, device="cuda", generator=g).int()[None]
    cu, lens = torch.tensor([0, 5], **i32), torch.tensor([blocks * 128 - 3], **i32)
    got, want = (pbs.window_prefill_attention(q, cache, "fp8_e4m3", hkv, table, cu, lens, 128 ** -0.5, workspace=w).float()
                 for w in ("auto", None))
    pbs._window_workspaces.clear()
    vmax = cache.view(torch.float8_e4m3fn).float().abs().max()
    assert ((got - want).abs() <= 2 * (2.0 ** -8 * want.abs() + vmax * (2.0 ** -10 + 2.0 ** -11))).all()


@gpu
def test_empty_calls_leave_nothing_behind():
    c = Case("bf16", 2, 4, [(2, 40)], 16, 2)
    d = c.dev()
    none = dict(d, q=d["q"][:0], table=d["table"][:0], lens=d["lens"][:0])
    assert decode(c, none, 2).shape == (0, 8, 128)
    out = prefill(c, dict(d, q=d["q"][:0], cu=torch.zeros(2, dtype=torch.int32, device="cuda")))
    assert out.shape == (0, 8, 128)

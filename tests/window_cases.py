"""Inputs of the window attend's tests: a cache whose bytes are NaN except for the keys that some
row of a request sees, ragged requests, shuffled blocks."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import window_attend as ow

NAN_BYTE = {"bf16": 0xFF, "fp8_e4m3": 0x7F, "nvfp4": 0x7F}


def page_bytes(kv, hkv):
    return hkv * 16 * {"bf16": 512, "fp8_e4m3": 256, "nvfp4": 144}[kv]


def write_row(page, kv, hkv, row, rng):
    """Finite random K and V of one page row."""
    for g in range(hkv):
        if kv == "bf16":
            x = torch.from_numpy(rng.standard_normal(256).astype(np.float32)).to(torch.bfloat16)
            page[(g * 16 + row) * 512:(g * 16 + row + 1) * 512] = x.view(torch.uint8).numpy()
        elif kv == "fp8_e4m3":
            x = torch.from_numpy(rng.standard_normal(256).astype(np.float32)).to(torch.float8_e4m3fn)
            page[(g * 16 + row) * 256:(g * 16 + row + 1) * 256] = x.view(torch.uint8).numpy()
        else:
            for s in (2 * g, 2 * g + 1):
                at = s * 1152
                page[at + row * 64:at + row * 64 + 64] = rng.integers(0, 256, 64, dtype=np.uint8)
                page[at + 1024 + row * 8:at + 1024 + row * 8 + 8] = rng.integers(32, 48, 8, dtype=np.uint8)


class Case:
    """reqs: (query tokens, all tokens) of each request; queries are the last tokens of each."""

    def __init__(self, kv, hkv, g, reqs, window, sinks, seed=0, bps=8, pad=0, spare=3, first_block=0):
        rng = np.random.default_rng(seed)
        self.kv, self.hkv, self.hq, self.reqs, self.window, self.sinks, self.bps = kv, hkv, hkv * g, reqs, window, sinks, bps
        need = [-(-max(t, 0) // 128) for _, t in reqs]
        self.max_blocks = max(1, max(need))
        ids = first_block + rng.permutation(sum(need) + spare)
        self.num_blocks = first_block + sum(need) + spare
        pb = page_bytes(kv, hkv)
        self.pages = {}  # physical page -> its bytes, NaN until a visible row is written
        table = np.full((len(reqs), self.max_blocks), -1, np.int32)
        at = 0
        for r, (n, total) in enumerate(reqs):
            seen = sorted(set().union(*(ow.visible(p, window, sinks).tolist() for p in
                                        (max(total - n, 0), *range(max(total - n, 0), total)))) if n and total > 0 else [])
            if n and total > 0:  # every key between the first row's window and the last row is seen by someone
                low = max(0, total - n - window + 1) if window else 0
                seen = sorted(set(seen) | set(range(low, total)))
            mine = ids[at:at + need[r]]
            at += need[r]
            for key in seen:
                b = key // 128
                table[r, b] = mine[b]
                page = int(mine[b]) * bps + key % 128 // 16
                if page not in self.pages:
                    self.pages[page] = np.full(pb, NAN_BYTE[kv], np.uint8)
                write_row(self.pages[page], kv, hkv, key % 16, rng)
        self.table, self.pb, self.pad = table, pb, pad
        self.total_q = sum(n for n, _ in reqs)
        self.q = torch.from_numpy(rng.standard_normal((self.total_q, self.hq, 128)).astype(np.float32)).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(128)
        self.k_scale, self.v_scale = (1.0, 1.0) if kv == "bf16" else (0.75, 1.25)

    def positions(self):
        return [(r, total - n + i) for r, (n, total) in enumerate(self.reqs) for i in range(n)]

    def want(self, rows=None):
        cache = {p: b for p, b in self.pages.items()}
        pos = self.positions()
        rows = range(self.total_q) if rows is None else rows
        got = [ow.window_row(self.q[i].double().numpy(), cache, self.kv, self.hkv, self.table[pos[i][0]], pos[i][1],
                             self.window, self.sinks, self.scale, self.k_scale, self.v_scale, self.bps) for i in rows]
        return [np.stack([x[j] for x in got]) for j in range(4)]

    def device_cache(self):
        """uint8 [pages, page bytes] on the GPU, pages `pad` bytes apart."""
        full = torch.empty(self.num_blocks * self.bps, self.pb + self.pad, dtype=torch.uint8, device="cuda")
        full.fill_(NAN_BYTE[self.kv])
        ids = torch.tensor(sorted(self.pages), device="cuda")
        if len(ids):
            full[ids, :self.pb] = torch.from_numpy(np.stack([self.pages[int(p)] for p in ids])).cuda()
        return full[:, :self.pb]

    def dev(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        cu = np.concatenate([[0], np.cumsum([n for n, _ in self.reqs])])
        return dict(cache=self.device_cache(), table=torch.from_numpy(self.table).cuda(),
                    lens=torch.tensor([t for _, t in self.reqs], **i32), cu=torch.tensor(cu, **i32),
                    q=self.q.cuda())


def check(out, lse, want, rows=None):
    """Against the oracle. out: half a bf16 step (2^-8 of the value; 2^-133 where it is subnormal), and
    what fp16 p (2^-11 of sum p|v|, twice: p and its share of the sum), the logits' fp32 sums (128 terms,
    2^-23 each at worst, of zabs: as much again relative to p) and ex2 (2^-22) move. lse: the logits' error."""
    o, l, mass, zabs = want
    got = out.double().cpu().numpy() if rows is None else out[list(rows)].double().cpu().numpy()
    logit = 2.0 ** -16 * zabs + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(o) + mass * (2.0 ** -10 + 2 * logit[..., None]) + 1e-30
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), got[bad][:5], o[bad][:5], tol[bad][:5])
    if lse is not None:
        got = lse.double().cpu().numpy() if rows is None else lse[list(rows)].double().cpu().numpy()
        none = np.isneginf(l)
        assert np.array_equal(np.isneginf(got), none)
        d = np.abs(got[~none] - l[~none])
        assert (d <= (logit + 2.0 ** -22 * np.abs(l))[~none] + 2.0 ** -20).all(), d.max()

"""What is measured of the paged cache's dense operators: window attention with sinks (decode rows
and varlen prefill), the K/V insert and the block operations (copy, fork and release, compact).

The cache layouts are the library's: a page holds 16 token rows of every kv head; a 128-token block
is 8 consecutive pages. bf16 and fp8 pages are [kv head][16 rows][K 128 | V 128]; an NVFP4 page is
[kv head][K, V][16 rows x 64 bytes of e2m1 pairs, then 16 rows x 8 e4m3 scales].
"""
import math

import torch

own = False

D = 128
BLOCK = 128
ROWS = 16
SLOT = 1152  # bytes of K (or V) of one page and kv head, NVFP4
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one request's next token on a small model: nothing but latency
        dict(name="decode_one_bf16", op="decode", kv="bf16", batch=1, lo=1000, hi=1000, dql=1, hq=8, hkv=1,
             window=512, sinks=4),
        # a serving step of a windowed layer
        dict(name="decode_b64_bf16", op="decode", kv="bf16", batch=64, lo=16384, hi=32768, dql=1, hq=64, hkv=8,
             window=4096, sinks=128),
        # a dense layer's step over a 4-bit cache, ragged long contexts
        dict(name="decode_b32_nvfp4_full", op="decode", kv="nvfp4", batch=32, lo=8192, hi=65536, dql=1, hq=64,
             hkv=8, window=0, sinks=0),
        # two rows per request (one drafted token), fp8 cache, very long contexts behind a window
        dict(name="mtp_b128_fp8", op="decode", kv="fp8_e4m3", batch=128, lo=65536, hi=131072, dql=2, hq=64, hkv=8,
             window=8191, sinks=64),
        # few short ragged prompts, odd lengths, window not a multiple of anything
        dict(name="prefill_ragged_fp8", op="prefill", kv="fp8_e4m3", q="1,17,333,2049,130", ctx="40,0,5,0,700",
             hq=32, hkv=4, window=333, sinks=7),
        # a step of whole prompts through a windowed layer
        dict(name="prefill_prompts_bf16", op="prefill", kv="bf16", q="2048,4096,8192,8192", ctx="0,0,0,0", hq=64,
             hkv=8, window=1024, sinks=64),
        # chunked prefill after long contexts on the 4-bit cache, 16 query heads per kv head
        dict(name="prefill_chunks_nvfp4", op="prefill", kv="nvfp4", q="4096,4096", ctx="16384,32768", hq=64, hkv=4,
             window=4096, sinks=128),
        # the new tokens of one decode step, quantised into the cache
        dict(name="insert_step_nvfp4", op="insert", kv="nvfp4", tokens=64, hkv=8, pool=64),
        # the tokens of a step of whole prompts
        dict(name="insert_prompts_fp8", op="insert", kv="fp8_e4m3", tokens=22528, hkv=8, pool=256),
        # parallel samples of 16 prompts: children share the full blocks, own their last block, and end
        dict(name="fork_release", op="fork", kv="bf16", layers=4, hkv=8, parents=16, children=64, lo=1000, hi=6000,
             pool=1024),
        # the pool of a drained server packed to the front
        dict(name="compact_pool", op="compact", kv="fp8_e4m3", layers=2, hkv=8, rows=48, max_blocks=64, pool=2048,
             live=0.6),
        # blocks moved by list (a prefix brought back, an evicted one replaced)
        dict(name="copy_blocks", op="copy", kv="bf16", layers=2, hkv=8, pairs=300, pool=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "prefill", "prefill", "insert", "fork", "compact", "copy"])
    kv = rng.choice(["bf16", "fp8_e4m3", "nvfp4"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8, 8, 16])
    window = 0 if rng.random() < 0.25 else _log(rng, 64, 8192)
    sinks = 0 if rng.random() < 0.25 else _log(rng, 1, 256)
    if op == "decode":
        batch = _log(rng, 1, 128)
        hi = _log(rng, 128, min(131072, (1 << 21) // batch))
        return dict(op=op, kv=kv, batch=batch, lo=max(1, hi // rng.choice([1, 2, 4, 50])), hi=hi,
                    dql=rng.choice([1, 1, 2, 3, 5]), hq=g * hkv, hkv=hkv, window=window, sinks=sinks)
    if op == "prefill":
        n = rng.randint(1, 6)
        q = [_log(rng, 1, 4096) for _ in range(n)]
        ctx = [0 if rng.random() < 0.4 else _log(rng, 1, 16384) for _ in range(n)]
        if window == 0:
            ctx = [c % 2048 for c in ctx]
        return dict(op=op, kv=kv, q=",".join(map(str, q)), ctx=",".join(map(str, ctx)), hq=min(64, g * hkv),
                    hkv=hkv if g * hkv <= 64 else 64 // g, window=min(window, 4096), sinks=sinks)
    if op == "insert":
        tokens = _log(rng, 1, 22528)
        return dict(op=op, kv=kv, tokens=tokens, hkv=hkv, pool=max(1, math.ceil(tokens / 128)) + rng.randint(0, 80))
    if op == "fork":
        parents = _log(rng, 1, 32)
        return dict(op=op, kv=kv, layers=rng.randint(1, 4), hkv=hkv, parents=parents,
                    children=parents * rng.randint(1, 4), lo=rng.randint(1, 999), hi=_log(rng, 1000, 6000), pool=2048)
    if op == "compact":
        return dict(op=op, kv=kv, layers=rng.randint(1, 2), hkv=hkv, rows=_log(rng, 1, 64),
                    max_blocks=_log(rng, 2, 64), pool=_log(rng, 256, 2048), live=rng.choice([0.2, 0.5, 0.8]))
    return dict(op=op, kv=kv, layers=rng.randint(1, 2), hkv=hkv, pairs=_log(rng, 1, 300), pool=_log(rng, 700, 1024))


# ---------------------------------------------------------------------------------------------
# what a case's numbers stand for
# ---------------------------------------------------------------------------------------------

def _page_bytes(case):
    per = {"bf16": 2 * D * 2, "fp8_e4m3": 2 * D, "nvfp4": 2 * (SLOT // ROWS)}[case["kv"]]
    return case["hkv"] * ROWS * per


def _block_bytes(case):
    return 8 * _page_bytes(case)


def _lens(n, lo, hi):
    """n lengths spread evenly over [lo, hi], in a fixed mixed order."""
    step = 7 if n % 7 else 5 if n % 5 else 1
    return [lo + (hi - lo) * ((i * step) % n) // max(1, n - 1) for i in range(n)]


def _requests(case):
    """(query tokens, all tokens) of each request."""
    if case["op"] == "decode":
        return [(case["dql"], max(v, case["dql"])) for v in _lens(case["batch"], case["lo"], case["hi"])]
    q, ctx = ([int(x) for x in case[k].split(",")] for k in ("q", "ctx"))
    return [(a, a + b) for a, b in zip(q, ctx)]


def _visible(case, first, last):
    """Keys that a query at first or last, or between them, sees: [0, head) and [low, last]."""
    w = case["window"]
    low = max(0, first - w + 1) if w else 0
    return min(case["sinks"], low), low


def _seen(case, p):
    head, low = _visible(case, p, p)
    return head + p - low + 1


def work(case):
    op = case["op"]
    if op in ("decode", "prefill"):
        keys = pairs = toks = blocks = 0
        w, s = case["window"], case["sinks"]
        for n, total in _requests(case):
            first = total - n
            head, low = _visible(case, first, total - 1)
            keys += head + total - low
            blocks += (head + BLOCK - 1) // BLOCK + (total - 1) // BLOCK - low // BLOCK + 1
            toks += n
            if n <= 8:
                pairs += sum(_seen(case, p) for p in range(first, total))
            else:  # the sum over positions of _seen, with seen constant once window and sinks are full
                full = max(first, min(total, w + s)) if w else total
                pairs += sum(_seen(case, p) for p in range(first, full)) + (total - full) * (w + s)
        row = _page_bytes(case) // ROWS
        return {"bytes": keys * row + 4 * blocks + 2 * 2 * toks * case["hq"] * D, "flops": 4 * D * case["hq"] * pairs}
    if op == "insert":
        return {"bytes": case["tokens"] * (case["hkv"] * 2 * D * 2 + _page_bytes(case) // ROWS + 8), "flops": 0}
    if op == "fork":
        lens = _lens(case["parents"], case["lo"], case["hi"])
        per = [lens[i % case["parents"]] for i in range(case["children"])]
        tails = sum(1 for n in per if n % BLOCK)
        entries = sum((n + BLOCK - 1) // BLOCK for n in per)
        return {"bytes": 2 * tails * case["layers"] * _block_bytes(case) + 4 * 6 * entries, "flops": 0}
    if op == "compact":
        live = int(case["pool"] * case["live"])
        moves = live * (case["pool"] - live) // case["pool"]
        return {"bytes": 2 * moves * case["layers"] * _block_bytes(case) + 8 * case["rows"] * case["max_blocks"]
                + 8 * case["pool"], "flops": 0}
    return {"bytes": 2 * case["pairs"] * case["layers"] * _block_bytes(case) + 8 * case["pairs"], "flops": 0}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _bytes_of_cache(case, pages, gen, layers=None):
    """Random cache content: values as K and V have them after projection (about unit normal)."""
    hkv, dev = case["hkv"], "cuda"
    shape = (pages,) if layers is None else (layers, pages)
    if case["kv"] == "bf16":
        x = torch.empty(*shape, hkv * ROWS * 2 * D, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        return x.view(torch.uint8)
    if case["kv"] == "fp8_e4m3":
        out = torch.empty(*shape, hkv * ROWS * 2 * D, dtype=torch.float8_e4m3fn, device=dev)
        flat = out.view(-1)
        for a in range(0, flat.numel(), 1 << 28):
            part = flat[a:a + (1 << 28)]
            part.copy_(torch.empty(part.numel(), dtype=torch.bfloat16, device=dev).normal_(generator=gen))
        return out.view(torch.uint8)
    out = torch.empty(*shape, hkv * 2, SLOT, dtype=torch.uint8, device=dev)
    out.random_(0, 256, generator=gen)  # codes: every e2m1 value
    # scales between 2^-3 and 0.47: e4m3 codes 32 .. 47
    out[..., ROWS * 64:].random_(32, 48, generator=gen)
    return out.flatten(-2)


def _table(need, max_blocks, gen, dev="cuda"):
    """Each request's blocks at random places of the pool."""
    total = sum(need)
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(need), max_blocks), -1, dtype=torch.int32, device=dev)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], {"case": dict(case)}
    dev = "cuda"
    i32 = dict(dtype=torch.int32, device=dev)
    if op in ("decode", "prefill"):
        reqs = _requests(case)
        need = [(t + BLOCK - 1) // BLOCK for _, t in reqs]
        s["table"] = _table(need, max(need), gen)
        s["cache"] = _bytes_of_cache(case, sum(need) * 8, gen)
        total_q = sum(n for n, _ in reqs)
        s["q"] = torch.empty(total_q, case["hq"], D, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        s["lens"] = torch.tensor([t for _, t in reqs], **i32)
        cu = [0]
        for n, _ in reqs:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, **i32)
        s["scale"] = 1.0 / math.sqrt(D)
        s["k_scale"], s["v_scale"] = (1.0, 1.0) if case["kv"] == "bf16" else (0.75, 1.25)
        # the plain form's plan: query groups of one request (at most 128 tokens) and the keys each group sees
        groups = []
        for r, (n, t) in enumerate(reqs):
            for a in range(0, n, 128):
                m = min(128, n - a)
                first = t - n + a
                head, low = _visible(case, first, first + m - 1)
                groups.append((r, cu[r] + a, m, first, head, low, head + first + m - low))
        s["groups"] = torch.tensor(groups, dtype=torch.int64, device=dev)
        s["most"] = (max(g[2] for g in groups), max(g[6] for g in groups))
        return s
    pool = case["pool"]
    if op == "insert":
        s["cache"] = _bytes_of_cache(case, pool * 8, gen)
        # K and V as slices of one projection's output
        kv = torch.empty(case["tokens"], 2, case["hkv"], D, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["slots"] = torch.randperm(pool * BLOCK, generator=gen, device=dev)[:case["tokens"]].contiguous()
        s["k_scale"], s["v_scale"] = (1.0, 1.0) if case["kv"] == "bf16" else (0.75, 1.25)
        if case["kv"] == "nvfp4":
            s["e2m1"] = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)
        return s
    s["cache"] = _bytes_of_cache(case, pool * 8, gen, case["layers"])
    perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    if op == "copy":
        n = case["pairs"]
        s["src"], s["dst"] = perm[:n].contiguous(), perm[n:2 * n].contiguous()
        return s
    s["refs"] = torch.zeros(pool, **i32)
    if op == "fork":
        lens = _lens(case["parents"], case["lo"], case["hi"])
        need = [(n + BLOCK - 1) // BLOCK for n in lens]
        rows = case["parents"] + case["children"]
        s["table"] = torch.full((rows, max(need) + 1), -1, **i32)
        at = 0
        for r, n in enumerate(need):
            s["table"][r, :n] = perm[at:at + n]
            at += n
        s["refs"][perm[:at].long()] = 1
        s["lens"] = torch.tensor(lens + [0] * case["children"], **i32)
        s["src"] = torch.arange(case["children"], **i32) % case["parents"]
        s["dst"] = torch.arange(case["children"], **i32) + case["parents"]
        return s
    live = int(pool * case["live"])
    rows, width = case["rows"], case["max_blocks"]
    # the tables name live blocks, some of them more than once (shared prefixes), and hold gaps
    pick = torch.randint(0, max(1, live), (rows, width), generator=gen, device=dev)
    table = perm[pick]
    table[torch.rand(rows, width, generator=gen, device=dev) < 0.2] = -1
    s["refs"][perm[:live].long()] = 1
    s["refs"].index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
    s["table"] = table
    s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------

def _rows_of(cache, kv, hkv, page, row):
    """K and V [..., hkv, 128] in fp32 of the token rows (page, row), any index shape."""
    if kv == "bf16":
        x = cache.view(torch.bfloat16).view(-1, hkv, ROWS, 2 * D)
        x = x.permute(0, 2, 1, 3)[page, row].float()
        return x[..., :D], x[..., D:]
    if kv == "fp8_e4m3":
        x = cache.view(-1, hkv, ROWS, 2 * D).permute(0, 2, 1, 3)[page, row]
        x = x.view(torch.float8_e4m3fn).float()
        return x[..., :D], x[..., D:]
    slots = cache.view(-1, hkv, 2, SLOT)
    codes = slots[..., :ROWS * 64].unflatten(-1, (ROWS, 64)).permute(0, 3, 1, 2, 4)[page, row]
    scales = slots[..., ROWS * 64:].unflatten(-1, (ROWS, 8)).permute(0, 3, 1, 2, 4)[page, row]
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=cache.device)
    x = lut[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(-2)
    x = (x.unflatten(-1, (8, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)
    return x[..., 0, :], x[..., 1, :]


def _attend(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    tokens, keys = s["most"]
    r, t0, m, first, head, low, count = (x.unsqueeze(1) for x in s["groups"].unbind(1))
    i = torch.arange(keys, device=s["q"].device).unsqueeze(0)
    key = torch.where(i < head, i, low + i - head)                     # [groups, keys]
    here = i < count
    key = torch.where(here, key, 0)
    block = s["table"][r, key // BLOCK].long()
    block = torch.where(here, block, 0)
    k, v = _rows_of(s["cache"], c["kv"], hkv, block * 8 + key % BLOCK // ROWS, key % ROWS)
    j = torch.arange(tokens, device=s["q"].device).unsqueeze(0)
    q = s["q"][torch.where(j < m, t0 + j, t0)].float()                 # [groups, tokens, hq, 128]
    q = q.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    logits = torch.matmul(q, k.permute(0, 2, 3, 1)) * (s["scale"] * s["k_scale"])
    pos = (first + j).unsqueeze(2)                                     # [groups, tokens, 1]
    key = key.unsqueeze(1)
    seen = here.unsqueeze(1) & (key <= pos)
    if c["window"]:
        seen = seen & ((key > pos - c["window"]) | (key < c["sinks"]))
    seen = seen.repeat_interleave(hq // hkv, 1).unsqueeze(1)           # row = token * G + head
    logits = torch.where(seen, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1) * s["v_scale"]
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.unflatten(2, (tokens, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.unflatten(2, (tokens, hq // hkv)).permute(0, 2, 1, 3).flatten(2, 3)
    # the groups' tokens are in the order of q's rows
    g_of = torch.repeat_interleave(torch.arange(r.shape[0], device=r.device), m.squeeze(1), output_size=s["q"].shape[0])
    j_of = torch.arange(s["q"].shape[0], device=r.device) - t0.squeeze(1)[g_of]
    return out[g_of, j_of].to(torch.bfloat16), lse[g_of, j_of]


def _insert(s):
    c = s["case"]
    hkv, kv = c["hkv"], c["kv"]
    page, row = s["slots"] // ROWS, s["slots"] % ROWS
    k, v = s["k"], s["v"]
    if kv == "bf16":
        s["cache"].view(torch.bfloat16).view(-1, hkv, ROWS, 2 * D).permute(0, 2, 1, 3)[page, row] = torch.cat([k, v], -1)
        return s["cache"].view(torch.bfloat16)
    x = torch.stack([k.float() * (1.0 / s["k_scale"]), v.float() * (1.0 / s["v_scale"])], 2)  # [n, hkv, 2, 128]
    if kv == "fp8_e4m3":
        x = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
        s["cache"].view(-1, hkv, ROWS, 2 * D).permute(0, 2, 1, 3)[page, row] = x
        return s["cache"].view(torch.float8_e4m3fn)
    x = x.unflatten(-1, (8, 16))
    sc = (x.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    scf = sc.float().unsqueeze(-1)
    y = torch.where(scf > 0, x / scf, 0)
    a = y.abs()  # to the nearest e2m1 value, ties to the even code
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code | (torch.signbit(y).int() << 3)).flatten(-2)
    code = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    slots = s["cache"].view(-1, hkv, 2, SLOT)
    slots[..., :ROWS * 64].unflatten(-1, (ROWS, 64)).permute(0, 3, 1, 2, 4)[page, row] = code
    slots[..., ROWS * 64:].unflatten(-1, (ROWS, 8)).permute(0, 3, 1, 2, 4)[page, row] = sc.view(torch.uint8)
    return _written(s)


def _written(s):
    """The inserted rows of an NVFP4 cache as the values they stand for."""
    return _rows_of(s["cache"], "nvfp4", s["case"]["hkv"], s["slots"] // ROWS, s["slots"] % ROWS)


def _move_blocks(cache, src, dst):
    """Blocks src of every layer to dst."""
    blocks = cache.unflatten(1, (-1, 8))
    blocks[:, dst.long()] = blocks[:, src.long()]


def _fork(s):
    table, refs, lens, src, dst = s["table"], s["refs"], s["lens"], s["src"].long(), s["dst"].long()
    width = table.shape[1]
    n = lens[src]
    full, tail = n // BLOCK, n % BLOCK > 0
    free = torch.argsort((refs > 0).to(torch.int8), stable=True).to(torch.int32)  # the free ids first, ascending
    fresh = free[torch.cumsum(tail, 0) - 1]
    at = torch.arange(width, device=table.device).unsqueeze(0)
    parent = table[src]
    last = parent.gather(1, full.long().clamp(max=width - 1).unsqueeze(1)).squeeze(1)
    shared = (at < full.unsqueeze(1)) & (parent >= 0)
    child = torch.where(shared, parent, -1)
    child = torch.where((at == full.unsqueeze(1)) & tail.unsqueeze(1), fresh.unsqueeze(1), child)
    refs.index_add_(0, child.clamp(min=0).flatten().long(), (child >= 0).flatten().to(torch.int32))
    table[dst] = child
    lens[dst] = n
    keep = torch.where(tail, last, 0)
    _move_blocks(s["cache"], keep, torch.where(tail, fresh, 0))


def _release(s):
    rows = s["dst"].long()
    old = s["table"][rows]
    s["refs"].index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().to(torch.int32))
    s["table"][rows] = -1
    s["lens"][rows] = 0


def _compact(s):
    table, refs = s["table"], s["refs"]
    ids = torch.arange(refs.shape[0], device=refs.device)
    live = refs > 0
    n = live.sum()
    src = torch.nonzero(live & (ids >= n)).squeeze(1)
    dst = torch.nonzero(~live & (ids < n)).squeeze(1)
    remap = torch.where(live, ids, -1).to(torch.int32)
    remap[src] = dst.to(torch.int32)
    table.copy_(torch.where(table >= 0, remap[table.long().clamp(min=0)], table))
    refs[dst] = refs[src]
    refs[src] = 0
    _move_blocks(s["cache"], src, dst)
    return remap, n.to(torch.int32)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import paged_block_sparse_gb300 as pbs
    if op == "decode":
        if own:
            return pbs.window_decode_attention(
                s["q"], s["cache"], c["kv"], c["hkv"], s["table"], s["lens"], c["dql"], s["scale"],
                window=c["window"], num_sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
        return _attend(s)
    if op == "prefill":
        if own:
            return pbs.window_prefill_attention(
                s["q"], s["cache"], c["kv"], c["hkv"], s["table"], s["cu"], s["lens"], s["scale"],
                window=c["window"], num_sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return _attend(s)[0]
    if op == "insert":
        if own:
            pbs.insert_kv_cache(s["k"], s["v"], s["cache"], c["kv"], s["slots"], k_scale=s["k_scale"],
                                v_scale=s["v_scale"])
            if c["kv"] == "nvfp4":
                return _written(s)
            return s["cache"].view(torch.bfloat16 if c["kv"] == "bf16" else torch.float8_e4m3fn)
        return _insert(s)
    if op == "fork":
        if own:
            pbs.fork_cache(s["cache"], s["table"], s["lens"], s["refs"], s["src"], s["dst"])
        else:
            _fork(s)
        forked = s["table"].clone(), s["refs"].clone(), s["lens"].clone()
        if own:
            pbs.release_cache_blocks(s["table"], s["lens"], s["refs"], s["dst"])
        else:
            _release(s)
        return (*forked, s["table"], s["refs"], s["lens"], s["cache"].view(torch.int32))
    if op == "compact":
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        remap, n = pbs.compact_cache(s["cache"], s["table"], s["refs"]) if own else _compact(s)
        return remap, n, s["table"], s["refs"], s["cache"].view(torch.int32)
    if own:
        pbs.copy_cache_blocks(s["cache"], s["src"], s["dst"])
    else:
        _move_blocks(s["cache"], s["src"], s["dst"])
    return s["cache"].view(torch.int32)


# ---------------------------------------------------------------------------------------------
# from the definition, in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_kv(s, r, keys):
    """K and V [keys, hkv, 128] of request r in 64 bits, decoded field by field."""
    c = s["case"]
    hkv = c["hkv"]
    phys = s["table"][r].long()[keys // BLOCK]
    page, row = phys * 8 + (keys % BLOCK) // ROWS, keys % ROWS
    raw = s["cache"][page]
    n = raw.shape[0]
    at = torch.arange(n, device=raw.device)
    if c["kv"] != "nvfp4":
        width = 4 * D if c["kv"] == "bf16" else 2 * D
        x = raw.view(n, hkv, ROWS, width)[at, :, row].contiguous()
        x = x.view(torch.bfloat16 if c["kv"] == "bf16" else torch.float8_e4m3fn).double()
        return x[..., :D], x[..., D:]
    x = raw.view(n, hkv, 2, SLOT)
    codes = x[..., :ROWS * 64].reshape(n, hkv, 2, ROWS, 64)[at, :, :, row].long()
    sc = x[..., ROWS * 64:].reshape(n, hkv, 2, ROWS, 8)[at, :, :, row].long()
    both = torch.empty(n, hkv, 2, D, dtype=torch.int64, device=raw.device)
    both[..., 0::2], both[..., 1::2] = codes % 16, codes // 16
    e, m = both // 2 % 4, both % 2
    mag = torch.where(e > 0, (1 + m * 0.5) * torch.exp2(e.double() - 1), m * 0.5)
    val = torch.where(both >= 8, -mag, mag)
    e, m = sc // 8 % 16, (sc % 8).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6)
    val = val * torch.where(sc >= 128, -mag, mag).repeat_interleave(16, -1)
    return val[:, :, 0], val[:, :, 1]


def _nearest(x, values):
    """x >= 0 at the nearest of the ascending values, ties to the even index, the last where x is beyond it."""
    i = (torch.searchsorted(values, x, right=True) - 1).clamp(max=len(values) - 2)
    below, above = x - values[i], values[i + 1] - x
    return values[i + ((below > above) | ((below == above) & (i % 2 == 1))).long()]


def _exact_nvfp4(x):
    """What an NVFP4 cache holds for x [..., 128]: per 16 elements an e4m3 scale of amax / 6 and e2m1 values."""
    code = torch.arange(127, device=x.device)
    e4m3 = torch.where(code < 8, code / 8 * 2.0 ** -6, (1 + code % 8 / 8) * torch.exp2(code // 8 - 7.0)).double()
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    x = x.unflatten(-1, (8, 16))
    scale = _nearest(x.abs().amax(-1, keepdim=True) / 6, e4m3)
    y = torch.where(scale > 0, x / scale, 0)
    return (torch.sign(y) * _nearest(y.abs().contiguous(), e2m1) * scale).flatten(-2)


def exact(case, seed):
    op = case["op"]
    if op == "insert":
        s = prepare(case, seed)
        x = s["k"].double() / s["k_scale"], s["v"].double() / s["v_scale"]
        if case["kv"] == "nvfp4":
            return tuple(_exact_nvfp4(v) for v in x)
        kind = torch.bfloat16 if case["kv"] == "bf16" else torch.float8_e4m3fn
        cache = s["cache"].view(kind).double()
        by = cache.view(-1, case["hkv"], ROWS, 2, D)
        for i, part in enumerate(x):
            by[s["slots"] // ROWS, :, s["slots"] % ROWS, i] = part
        return cache
    if op not in ("decode", "prefill") or work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    hq, hkv, w = case["hq"], case["hkv"], case["window"]
    g = hq // hkv
    outs, lses = [], []
    at = 0
    for r, (n, total) in enumerate(_requests(case)):
        for a in range(0, n, 256):
            b = min(n, a + 256)
            pos = torch.arange(total - n + a, total - n + b, device="cuda")
            keys = torch.arange(total - n + b, device="cuda")
            if w:
                keys = keys[(keys > int(pos[0]) - w) | (keys < case["sinks"])]
            k, v = _exact_kv(s, r, keys)
            q = s["q"][at + a:at + b].double().view(b - a, hkv, g, D)
            z = torch.einsum("tkgd,nkd->kgtn", q, k) * (s["scale"] * s["k_scale"])
            hidden = keys[None, :] > pos[:, None]
            if w:
                hidden |= (keys[None, :] <= pos[:, None] - w) & (keys[None, :] >= case["sinks"])
            z.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(z, -1)
            o = torch.einsum("kgtn,nkd->tkgd", torch.exp(z - lse.unsqueeze(-1)), v) * s["v_scale"]
            outs.append(o.reshape(b - a, hq, D))
            lses.append(lse.permute(2, 0, 1).reshape(b - a, hq))
        at += n
    out = torch.cat(outs)
    return (out, torch.cat(lses)) if op == "decode" else out

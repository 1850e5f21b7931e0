"""Cases for the attention operators over a 4-bit paged key/value cache.

Four operators: block tables and slot maps from request lengths, per-head
query/key norms with the rotary rotation, quantising keys and values into the
paged cache, and attention that reads it.  ``run`` computes them with
elementary torch operations in 32 bits (``own`` false) or through the
package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
#: bit of dim 8w + i inside 32-bit word w of a row of codes (even dims in the low half, odd dims in the high half)
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's bookkeeping: eight running requests, one token each
        dict(name="tables-step", op="tables", B=8, new_lo=1, new_hi=1, cached_hi=4000, page=16, pad=0),
        # admission of a batch of prompts behind running requests
        dict(name="tables-prompts", op="tables", B=257, new_lo=0, new_hi=2047, cached_hi=8191, page=64, pad=100),
        # one decode step of the 2048-wide layer: 16 heads of 128
        dict(name="rope-step", op="rope", T=8, hq=16, hkv=16, D=128, rot=128, inter=False, norm=True),
        # a prompt batch with grouped heads
        dict(name="rope-prompt", op="rope", T=16383, hq=32, hkv=8, D=128, rot=128, inter=False, norm=True),
        # one decode step of 64 requests into the cache
        dict(name="append-step", op="append", T=64, hkv=8, D=64, page=16),
        # a prompt batch into the cache of the 2048-wide layer
        dict(name="append-prompt", op="append", T=16384, hkv=16, D=128, page=64),
        # latency of one request's decode step
        dict(name="decode-one", op="attention", B=1, q_lo=1, q_hi=1, kv_lo=511, kv_hi=511, hq=16, hkv=16, D=128,
             page=16, window=0, causal=True),
        # ordinary serving: 64 requests of ragged lengths, grouped heads
        dict(name="decode-batch", op="attention", B=64, q_lo=1, q_hi=1, kv_lo=1, kv_hi=16384, hq=32, hkv=8, D=128,
             page=64, window=0, causal=True),
        # few requests with very long contexts and one key head for all query heads
        dict(name="decode-long", op="attention", B=4, q_lo=1, q_hi=1, kv_lo=100000, kv_hi=131072, hq=16, hkv=1, D=64,
             page=32, window=0, causal=True),
        # verification of drafted tokens, sliding window
        dict(name="draft-window", op="attention", B=32, q_lo=1, q_hi=5, kv_lo=5, kv_hi=8192, hq=16, hkv=4, D=128,
             page=16, window=1024, causal=True),
        # fresh prompts of the 2048-wide layer
        dict(name="prompt", op="attention", B=4, q_lo=777, q_hi=2048, kv_lo=0, kv_hi=0, hq=16, hkv=16, D=128, page=64,
             window=0, causal=True),
        # one chunk of a long prompt against what is cached already
        dict(name="chunk-long", op="attention", B=1, q_lo=2048, q_hi=2048, kv_lo=30011, kv_hi=30011, hq=32, hkv=4,
             D=128, page=64, window=0, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "append", "attention", "attention", "attention"])
    if op == "tables":
        B = _log(rng, 1, 600)
        lo = rng.choice([0, 1])
        hi = max(lo, 1, _log(rng, 1, max(1, min(2047, 250000 // B))))
        return dict(op=op, B=B, new_lo=lo, new_hi=hi, cached_hi=_log(rng, 1, 16384), page=rng.choice([16, 32, 64]),
                    pad=rng.choice([0, 0, rng.randrange(1, 200)]))
    D = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "rope":
        T = _log(rng, 1, 16000)
        hq = hkv * rng.choice([1, 2, 4]) if hkv < 16 else 16
        return dict(op=op, T=T, hq=hq, hkv=hkv, D=D, rot=rng.choice([D, D, D // 2]), inter=rng.random() < 0.3,
                    norm=rng.random() < 0.8)
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 16000), hkv=hkv, D=D, page=rng.choice([16, 32, 64]))
    G = rng.choice([1, 2, 4, 5, 8])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64])
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    kind = rng.choice(["decode", "draft", "prompt"])
    if kind == "prompt":
        B = _log(rng, 1, 6)
        q_hi = _log(rng, 16, 2048)
        kv = rng.choice([0, 0, _log(rng, 1, 16000)])
        room = 2048 * 30000 * 32 / (B * hkv * G * D / 128)       # no dearer than the long chunk
        q_hi = max(1, min(q_hi, int(room / (kv + q_hi))))
        return dict(op=op, B=B, q_lo=max(1, q_hi // 3), q_hi=q_hi, kv_lo=kv // 2, kv_hi=kv, hq=hkv * G, hkv=hkv, D=D,
                    page=page, window=window, causal=rng.random() < 0.85)
    kv = _log(rng, 2, 60000)
    B = _log(rng, 1, max(1.01, min(128, 1.5e6 / (kv * hkv))))
    return dict(op=op, B=B, q_lo=1, q_hi=1 if kind == "decode" else rng.randrange(2, 7), kv_lo=rng.choice([0, kv // 3]),
                kv_hi=kv, hq=hkv * G, hkv=hkv, D=D, page=page, window=window, causal=True)


def _lengths(case, seed):
    """Host-side request lengths of a case: (cached before, new tokens).  The new tokens' lengths are the case's own, in
    an order that the seed gives, so that every seed has as many tokens."""
    r = np.random.RandomState((seed * 7919 + 17) % (1 << 31))
    B, tables = case["B"], case["op"] == "tables"
    lo, hi = (case["new_lo"], case["new_hi"]) if tables else (case["q_lo"], case["q_hi"])
    new = np.random.RandomState(1000 * B + hi).randint(lo, hi + 1, B)
    new[0] = hi
    r.shuffle(new)
    if tables:
        return r.randint(0, case["cached_hi"] + 1, B), new
    old = r.randint(case["kv_lo"], case["kv_hi"] + 1, B)
    old[-1] = case["kv_hi"]
    return old, new


def _mean_lengths(case):
    """Expected lengths of a case, for work()."""
    B = case["B"]
    if case["op"] == "tables":
        return B * case["cached_hi"] / 2, B * (case["new_lo"] + case["new_hi"]) / 2
    q = case["q_hi"] + (B - 1) * (case["q_lo"] + case["q_hi"]) / 2
    kv = case["kv_hi"] + (B - 1) * (case["kv_lo"] + case["kv_hi"]) / 2
    return kv, q


def work(case):
    op = case["op"]
    if op == "tables":
        B = case["B"]
        tokens = _mean_lengths(case)[1]
        pages = tokens / case["page"]
        # lengths in, q_start and kv_len out, free pages read and table entries written, slot and position of each token
        return {"bytes": 16 * B + 4 + 8 * pages + 8 * (tokens + case["pad"]), "flops": 0}
    if op == "rope":
        row = (case["hq"] + case["hkv"]) * case["D"]
        return {"bytes": case["T"] * (4 * row + 4 * case["rot"] + 4) + 4 * case["D"],
                "flops": case["T"] * row * (7 if case["norm"] else 3)}
    if op == "append":
        return {"bytes": case["T"] * case["hkv"] * (4 * case["D"] + case["D"] + 8) + 4 * case["T"],
                "flops": case["T"] * case["hkv"] * case["D"] * 8}
    B, w = case["B"], case["window"]
    kv, q = _mean_lengths(case)
    kv_b, q_b = kv / B, q / B
    pos = kv_b + (q_b / 2 if case["causal"] else q_b)          # keys that the middle query sees
    seen = min(pos, w) if w else pos
    span = min(kv_b + q_b, w + q_b) if w else kv_b + q_b       # keys that some query of the request sees
    return {"bytes": B * (span * case["hkv"] * (case["D"] + 8) + 4 * q_b * case["hq"] * case["D"]),
            "flops": 4 * q * seen * case["hq"] * case["D"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(torch.bfloat16)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _random_pages(g, n_pages, P, hkv, D):
    """A cache as appends leave it: codes of bell-shaped values over each row's own range, fp16 scale and minimum."""
    pages = torch.empty((n_pages, hkv, P * (D + 8)), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (hkv * P * D))
    for a in range(0, n_pages, step):
        n = min(step, n_pages - a)
        u = torch.randn((n, hkv, 2 * P * D // 2, 2), generator=g, device=DEV, dtype=torch.bfloat16)
        u = u.mul_(2.8).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        pages[a:a + n, :, :P * D] = u[..., 0] | (u[..., 1] << 4)
        del u
    s = torch.rand((n_pages, hkv, 2 * P, 1), generator=g, device=DEV) * 0.25 + 0.2
    z = -s * (7.5 + 0.7 * torch.randn((n_pages, hkv, 2 * P, 1), generator=g, device=DEV))
    pages[:, :, P * D:] = torch.cat([s, z], dim=-1).to(torch.float16).view(torch.uint8).reshape(n_pages, hkv, P * 8)
    return pages.reshape(n_pages, hkv * P * (D + 8))


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    s = dict(case=dict(case))
    if op == "tables":
        old, new = _lengths(case, seed)
        P = case["page"]
        have = -(-old // P)
        need = -(-(old + new) // P) - have
        spare = 7
        total = int(have.sum() + need.sum()) + spare
        perm = np.random.RandomState(seed % (1 << 31)).permutation(total).astype(np.int32)
        width = -(-(case["cached_hi"] + case["new_hi"]) // P) + 1
        table = np.full((case["B"], width), -1, dtype=np.int32)
        at = np.concatenate([[0], np.cumsum(have)])
        for b in range(case["B"]):
            table[b, :have[b]] = perm[at[b]:at[b + 1]]
        free = perm[at[-1]:]
        n = int(new.sum()) + case["pad"]
        s.update(cached=_ints(old), new=_ints(new), free=_ints(free), n_free=_ints([len(free)]), table=_ints(table),
                 n=n, page=P)
        return s
    if op == "rope":
        T, hq, hkv, D, rot = case["T"], case["hq"], case["hkv"], case["D"], case["rot"]
        n_pos = 8192
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * inv[None]
        s.update(qkv=_bf16(g, T, (hq + 2 * hkv) * D, scale=1.7),
                 wq=(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16),
                 wk=(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16), eps=1e-5,
                 cos_sin=torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32).contiguous(),
                 pos=torch.randint(0, n_pos, (T,), generator=g, device=DEV, dtype=torch.int32))
        return s
    if op == "append":
        T, hkv, D, P = case["T"], case["hkv"], case["D"], case["page"]
        n_pages = -(-T // P) + 3
        kv = _bf16(g, T, 2 * hkv * D)
        kv[:, ::37] *= 6                                     # channels with larger values, as keys have
        slots = torch.randperm(n_pages * P, generator=g, device=DEV)[:T].to(torch.int32)
        s.update(kv=kv, slots=slots,
                 pages=torch.zeros((n_pages, hkv * P * (D + 8)), dtype=torch.uint8, device=DEV))
        return s
    old, new = _lengths(case, seed)
    hq, hkv, D, P = case["hq"], case["hkv"], case["D"], case["page"]
    kv = old + new
    blocks = -(-kv // P)
    n_pages = int(blocks.sum()) + 3
    perm = np.random.RandomState(seed % (1 << 31)).permutation(n_pages).astype(np.int32)
    at = np.concatenate([[0], np.cumsum(blocks)])
    table = np.full((case["B"], int(blocks.max())), -1, dtype=np.int32)
    for b in range(case["B"]):
        table[b, :blocks[b]] = perm[at[b]:at[b + 1]]
    q_start = np.concatenate([[0], np.cumsum(new)])
    s.update(pages=_random_pages(g, n_pages, P, hkv, D), q=_bf16(g, int(new.sum()), hq, D, scale=1.5),
             q_start=_ints(q_start), kv_len=_ints(kv), table=_ints(table), max_q=int(new.max()), max_kv=int(kv.max()),
             scale=D ** -0.5)
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_tables(s):
    cached, new, P, n = s["cached"].long(), s["new"].long(), s["page"], s["n"]
    kv = cached + new
    have = torch.div(cached + P - 1, P, rounding_mode="floor")
    need = torch.div(kv + P - 1, P, rounding_mode="floor") - have
    q_start = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    page_start = torch.cumsum(need, 0) - need
    table = s["table"].clone()
    col = torch.arange(table.shape[1], device=DEV)[None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    rank = page_start[:, None] + col - have[:, None]
    n_free = s["n_free"].long()
    at = n_free - 1 - rank
    page = s["free"][at.clamp(0, s["free"].numel() - 1)]
    table = torch.where(fresh, torch.where(at >= 0, page, torch.full_like(page, -1)), table)
    tok = torch.arange(n, device=DEV)
    b = torch.searchsorted(q_start[1:], tok, right=True).clamp(max=new.numel() - 1)
    live = tok < q_start[-1]
    pos = torch.where(live, cached[b] + tok - q_start[b], torch.zeros_like(tok))
    blk = table[b, torch.div(pos, P, rounding_mode="floor").clamp(max=table.shape[1] - 1)].long()
    slot = torch.where(live & (blk >= 0), blk * P + pos % P, torch.full_like(tok, -1))
    left = (n_free - need.sum()).clamp(min=0)
    return dict(table=table, q_start=q_start.int(), kv_len=kv.int(), slots=slot.int(), positions=pos.int(),
                n_free=left.int())


def _plain_rope(s):
    c = s["case"]
    T, hq, hkv, D, rot = c["T"], c["hq"], c["hkv"], c["D"], c["rot"]
    x = s["qkv"][:, :(hq + hkv) * D].reshape(T, hq + hkv, D).float()
    if c["norm"]:
        w = torch.cat([s["wq"].float()[None].expand(hq, D), s["wk"].float()[None].expand(hkv, D)])
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :rot // 2], r[..., rot // 2:])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], -1).reshape(T, hq + hkv, rot) if c["inter"] else torch.cat([ya, yb], -1)
    y = torch.cat([y, rest], -1).to(torch.bfloat16)
    return dict(q=y[:, :hq].contiguous(), k=y[:, hq:].contiguous())


def _plain_quantise(x):
    """The values that a row of keys or values stands for once it is held in 4 bits."""
    x = torch.nan_to_num(x.float(), nan=0.0).clamp(-32768, 32768)
    z = x.amin(-1, keepdim=True).to(torch.float16).float()
    sc = ((x.amax(-1, keepdim=True) - z) / 15).to(torch.float16).float()
    u = torch.where(sc > 0, torch.round((x - z) / sc).clamp(0, 15), torch.zeros_like(x))
    return (u * sc + z).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    y = _plain_quantise(s["kv"].reshape(c["T"], 2, c["hkv"], c["D"]))
    return dict(k=y[:, 0].contiguous(), v=y[:, 1].contiguous())


def _plain_unpack(pages, table, P, hkv, D):
    """fp32 keys and values [B, hkv, tokens, D] of the pages that a block table names."""
    B, nb = table.shape
    pg = pages[table.clamp(min=0).long()].reshape(B, nb, hkv, P * (D + 8))
    codes = pg[..., :P * D].contiguous().view(torch.int32).reshape(B, nb, hkv, 2, P, D // 8, 1)
    sh = torch.tensor(SHIFTS, dtype=torch.int32, device=DEV)
    u = ((codes >> sh) & 15).reshape(B, nb, hkv, 2, P, D).float()
    par = pg[..., P * D:].contiguous().view(torch.float16).reshape(B, nb, hkv, 2, P, 2).float()
    x = u * par[..., 0:1] + par[..., 1:2]
    x = x.permute(3, 0, 2, 1, 4, 5).reshape(2, B, hkv, nb * P, D)
    return x[0], x[1]


def _plain_attention(s):
    c = s["case"]
    B, hq, hkv, D, P, w = c["B"], c["hq"], c["hkv"], c["D"], c["page"], c["window"]
    G, mq = hq // hkv, s["max_q"]
    k, v = _plain_unpack(s["pages"], s["table"], P, hkv, D)
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    q_len = q_start[1:] - q_start[:-1]
    i = torch.arange(mq, device=DEV)
    at = (q_start[:-1, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))
    qp = s["q"][at].float().reshape(B, mq, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, mq * G, D)
    sc = torch.matmul(qp, k.transpose(-1, -2)) * s["scale"]
    j = torch.arange(k.shape[2], device=DEV)
    pos = kv_len[:, None] - q_len[:, None] + i if c["causal"] else (kv_len[:, None] - 1).expand(B, mq)
    seen = (j < kv_len[:, None, None]) & (j <= pos[..., None])
    if w:
        seen &= j > (pos - w)[..., None]
    seen = seen.repeat_interleave(G, dim=1)[:, None]
    sc = sc.masked_fill_(~seen, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(sc.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.reshape(B, hkv, mq, G, D).permute(0, 2, 1, 3, 4).reshape(B, mq, hq, D)
    return o[(i < q_len[:, None])].to(torch.bfloat16)


# ------------------------------------------------------------------ the framework's kernels
def _handle(s):
    """What a user's program makes once and keeps: outputs, the cache handle, the workspace."""
    import decode_matvec_gb300 as Q
    c, h = s["case"], {"Q": Q}
    bf = dict(dtype=torch.bfloat16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    if c["op"] == "tables":
        h.update(table=s["table"].clone(), q_start=torch.empty(c["B"] + 1, **i32), kv_len=torch.empty(c["B"], **i32),
                 slots=torch.empty(s["n"], **i32), positions=torch.empty(s["n"], **i32), n_free=torch.empty(1, **i32))
    elif c["op"] == "rope":
        h.update(q=torch.empty((c["T"], c["hq"], c["D"]), **bf), k=torch.empty((c["T"], c["hkv"], c["D"]), **bf))
    elif c["op"] == "append":
        h.update(cache=Q.Kv4Cache(s["pages"], c["page"], c["hkv"], c["D"]),
                 k=torch.empty((c["T"], c["hkv"], c["D"]), **bf), v=torch.empty((c["T"], c["hkv"], c["D"]), **bf))
    else:
        n = Q.kv4_attention_ws_size(c["B"], c["hq"], c["hkv"], c["D"], s["q"].shape[0], s["max_q"], s["max_kv"])
        h.update(cache=Q.Kv4Cache(s["pages"], c["page"], c["hkv"], c["D"]), out=torch.empty_like(s["q"]),
                 ws=torch.empty(max(n, 1), dtype=torch.uint8, device=DEV))
    return h


def _own(s):
    h = s.get("handle") or s.setdefault("handle", _handle(s))
    Q, c = h["Q"], s["case"]
    if c["op"] == "tables":
        Q.kv4_block_tables(s["cached"], s["new"], s["free"], s["n_free"], s["page"], h["table"], h["q_start"],
                           h["kv_len"], h["slots"], h["positions"], h["n_free"])
        return {k: h[k] for k in ("table", "q_start", "kv_len", "slots", "positions", "n_free")}
    if c["op"] == "rope":
        w = (s["wq"], s["wk"]) if c["norm"] else (None, None)
        Q.qk_norm_rope(s["qkv"], c["hq"], c["hkv"], c["D"], w[0], w[1], s["eps"], s["cos_sin"], s["pos"], h["q"],
                       h["k"], interleaved=c["inter"])
        return dict(q=h["q"], k=h["k"])
    if c["op"] == "append":
        kv = s["kv"].view(c["T"], 2, c["hkv"], c["D"])
        Q.kv4_append(h["cache"], kv[:, 0], kv[:, 1], s["slots"])
        Q.kv4_gather(h["cache"], s["slots"], h["k"], h["v"])
        return dict(k=h["k"], v=h["v"])
    return Q.kv4_attention(h["cache"], s["q"], s["q_start"], s["kv_len"], s["table"], h["out"], h["ws"], s["max_q"],
                           s["max_kv"], s["scale"], causal=c["causal"], window=c["window"])


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "rope": _plain_rope, "append": _plain_append,
            "attention": _plain_attention}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    op, s = case["op"], prepare(case, seed)
    if op == "tables":
        return None
    if op == "rope":
        hq, hkv, D, rot = case["hq"], case["hkv"], case["D"], case["rot"]
        half = rot // 2
        cs = s["cos_sin"].double()[s["pos"].long()]
        i = torch.arange(half, device=DEV)
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
        out = {}
        for name, h0, h1, w in (("q", 0, hq, s["wq"]), ("k", hq, hq + hkv, s["wk"])):
            x = s["qkv"][:, h0 * D:h1 * D].double().reshape(-1, h1 - h0, D)
            if case["norm"]:
                x = x * w.double() * (x.pow(2).sum(-1, keepdim=True) / D + s["eps"]).pow(-0.5)
            z = torch.complex(x[..., first], x[..., second]) * torch.complex(cs[:, :half], cs[:, half:])[:, None]
            x[..., first], x[..., second] = z.real, z.imag
            out[name] = x
        return out
    if op == "append":
        kv = s["kv"].double().cpu().numpy().reshape(case["T"], 2, case["hkv"], case["D"])
        lo = kv.min(-1, keepdims=True).astype(np.float16).astype(np.float64)
        step = ((kv.max(-1, keepdims=True) - lo) / 15).astype(np.float16).astype(np.float64)
        with np.errstate(divide="ignore", invalid="ignore"):
            u = np.where(step > 0, np.clip(np.rint((kv - lo) / step), 0, 15), 0)
        y = torch.from_numpy(u * step + lo)
        return dict(k=y[:, 0].contiguous(), v=y[:, 1].contiguous())
    hq, hkv, D, P, w = case["hq"], case["hkv"], case["D"], case["page"], case["window"]
    G = hq // hkv
    out = torch.zeros((s["q"].shape[0], hq, D), dtype=torch.float64, device=DEV)
    starts, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].long()
    bits = [[4 * (i // 2) + 16 * (i % 2) for i in range(8)]]
    for b in range(case["B"]):
        n, kv = starts[b + 1] - starts[b], lens[b]
        if not n or not kv:
            continue
        nb = -(-kv // P)
        pg = s["pages"][table[b, :nb]].reshape(nb, hkv, P * (D + 8))
        pos = torch.arange(kv - n, kv, device=DEV) if case["causal"] else torch.full((n,), kv - 1, device=DEV)
        lo = max(0, int(pos[0]) + 1 - w) if w else 0
        keys = torch.arange(lo, kv, device=DEV)
        hide = keys[None] > pos[:, None]
        if w:
            hide |= keys[None] <= pos[:, None] - w
        for h in range(hkv):
            part = []
            for x in (0, 1):
                word = pg[:, h, x * P * D // 2:(x + 1) * P * D // 2].contiguous().view(torch.int32).reshape(nb * P, D // 8)
                sz = pg[:, h, P * D + 4 * P * x:P * D + 4 * P * (x + 1)].contiguous().view(torch.float16).reshape(nb * P, 2)
                word, sz = word[lo:kv], sz[lo:kv].double()
                u = torch.stack([(word >> t) & 15 for t in bits[0]], -1).reshape(kv - lo, D).double()
                part.append(u * sz[:, :1] + sz[:, 1:])
            for a in range(0, n, 256):
                q = s["q"][starts[b] + a:starts[b] + min(n, a + 256), h * G:(h + 1) * G].double()
                t = torch.einsum("igd,jd->gij", q, part[0]) * s["scale"]
                t = t.masked_fill(hide[a:a + 256][None], float("-inf"))
                p = torch.softmax(t, -1)
                p = torch.nan_to_num(p, nan=0.0)
                out[starts[b] + a:starts[b] + min(n, a + 256), h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", p, part[1])
    return out

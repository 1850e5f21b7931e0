"""Cases for what a decoder layer's step needs around its attention and its experts, and for attention over chosen blocks.

Five operators: the root-mean-square norm of whole rows with the residual's addition (and an output in 8 bits with
scales), the choice of experts from scores with a bias and groups, the bounds of each cached block's keys, the choice of
the blocks that a query attends to, and attention over the chosen blocks of the 4-bit cache.  ``run`` computes them with
elementary torch operations (``own`` false) or through the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
#: bit of dim 8w + i inside 32-bit word w of a row of codes (even dims in the low half, odd dims in the high half)
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)
#: largest value of the 8-bit float with 4 exponent and 3 fraction bits
E4M3_MAX = 448.0
#: a row's 8-bit scales: one for each run of so many values
GROUP = 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # between the experts' fp32 sums and the next layer, one decode step of the 2048-wide layer
        dict(name="norm-step", op="norm", T=32, n=2048, f32=True, add=True, q8=0),
        # a prompt batch behind the attention's projection, the normed rows also in 8 bits for the next projection
        dict(name="norm-prompt", op="norm", T=16384, n=2048, f32=False, add=True, q8=GROUP),
        # rows of the 2080-wide layer, one 8-bit scale a row
        dict(name="norm-odd", op="norm", T=4095, n=2080, f32=True, add=True, q8=1),
        # one decode step: 256 experts in 8 groups of which a token may use 4, sigmoid scores with a balancing bias
        dict(name="route-step", op="route", T=32, E=256, k=8, sigmoid=True, bias=True, groups=8, top_groups=4, best=2,
             renorm=True, f32=True),
        # the same router over a prompt batch, logits as a bf16 projection leaves them
        dict(name="route-prompt", op="route", T=16383, E=256, k=8, sigmoid=True, bias=True, groups=8, top_groups=4, best=2,
             renorm=True, f32=False),
        # the 2048-expert layer's 4096 tokens with two experts each
        dict(name="route-wide", op="route", T=4096, E=2048, k=2, sigmoid=False, bias=True, groups=1, top_groups=1, best=1,
             renorm=True, f32=True),
        # the bounds of the blocks that a decode step of 64 requests writes to
        dict(name="bounds-step", op="bounds", B=64, q_lo=1, q_hi=1, kv_lo=1, kv_hi=32768, hkv=8, D=128, page=64),
        # ... and that a prompt batch fills
        dict(name="bounds-prompt", op="bounds", B=16, q_lo=777, q_hi=2048, kv_lo=0, kv_hi=0, hkv=8, D=128, page=64),
        # 64 ragged requests choose 64 of their blocks for a decode step
        dict(name="select-batch", op="select", B=64, q_lo=1, q_hi=1, kv_lo=1, kv_hi=32768, hq=32, hkv=8, D=128, page=64,
             top=64),
        # few requests with very long contexts, one key head
        dict(name="select-long", op="select", B=4, q_lo=1, q_hi=1, kv_lo=100000, kv_hi=131072, hq=16, hkv=1, D=64, page=16,
             top=128),
        # attention of the batch over its chosen blocks
        dict(name="blocks-batch", op="blocks", B=64, q_lo=1, q_hi=1, kv_lo=1, kv_hi=32768, hq=32, hkv=8, D=128, page=64,
             top=64),
        # one request with a very long context
        dict(name="blocks-one", op="blocks", B=1, q_lo=1, q_hi=1, kv_lo=131071, kv_hi=131071, hq=16, hkv=16, D=128, page=16,
             top=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "bounds", "select", "blocks"])
    if op == "norm":
        n = rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 2, 1024), 128 * _log(rng, 1, 64)])
        q8 = rng.choice([0, 0, 1, GROUP])
        if q8:
            n = -(-n // 8) * 8
        return dict(op=op, T=_log(rng, 1, max(2, min(20000, (1 << 25) // n))), n=n, f32=rng.random() < 0.5,
                    add=rng.random() < 0.7, q8=q8)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.choice([_log(rng, 2, 64), 8, 16, 32])
        if rng.random() < 0.2:
            groups, E = 1, _log(rng, 256, 8192)
        top_groups = rng.randrange(1, groups + 1)
        k = min(rng.randrange(1, 11), top_groups * (E // groups))
        return dict(op=op, T=_log(rng, 1, max(2, min(16000, (1 << 22) // E))), E=E, k=k, sigmoid=rng.random() < 0.6,
                    bias=rng.random() < 0.6, groups=groups, top_groups=top_groups, best=rng.choice([1, 2]) if E // groups > 1 else 1,
                    renorm=rng.random() < 0.7, f32=rng.random() < 0.5)
    D, page, hkv = rng.choice([64, 128]), rng.choice([16, 32, 64]), rng.choice([1, 2, 3, 4, 8])
    if op == "bounds":
        kind = rng.choice(["step", "draft", "prompt"])
        q_hi = 1 if kind == "step" else rng.randrange(2, 7) if kind == "draft" else _log(rng, 16, 2048)
        kv = _log(rng, 1, 32768) if kind != "prompt" else rng.choice([0, _log(rng, 1, 2000)])
        B = _log(rng, 1, max(2, min(96, 24000 // q_hi, 2500000 // (hkv * (kv + q_hi)))))
        return dict(op=op, B=B, q_lo=1 if kind != "prompt" else max(1, q_hi // 3), q_hi=q_hi, kv_lo=kv // 4, kv_hi=kv, hkv=hkv,
                    D=D, page=page)
    G = rng.choice([1, 2, 4, 5, 8])
    kv = _log(rng, 2, 100000)
    top = rng.choice([4, 8, 16, 33, 64, 128])
    B = _log(rng, 1, max(1.01, min(96, 2.0e6 / (kv * hkv))))
    q_hi = rng.choice([1, 1, 1, rng.randrange(2, 6)])
    return dict(op=op, B=B, q_lo=1, q_hi=q_hi, kv_lo=rng.choice([0, kv // 3]), kv_hi=kv, hq=hkv * G, hkv=hkv, D=D, page=page,
                top=top if op == "select" else min(top, max(4, 2000000 // (B * q_hi * hkv * page))))


def _lengths(case, seed):
    """Host-side request lengths of a case: (cached before, new tokens).  The lengths are the case's own, in an order that
    the seed gives, so that every seed has as many tokens."""
    r = np.random.RandomState((seed * 7919 + 17) % (1 << 31))
    B = case["B"]
    fixed = np.random.RandomState(1000 * B + case["q_hi"])
    new = fixed.randint(case["q_lo"], case["q_hi"] + 1, B)
    old = fixed.randint(case["kv_lo"], case["kv_hi"] + 1, B)
    new[0], old[-1] = case["q_hi"], case["kv_hi"]
    r.shuffle(new)
    r.shuffle(old)
    return old, new


def work(case):
    op = case["op"]
    if op == "norm":
        T, n = case["T"], case["n"]
        size = (4 if case["f32"] else 2) + 2 + (4 if case["add"] else 0)
        if case["q8"]:
            size += 1
        scales = 4 * T * (-(-n // GROUP) if case["q8"] == GROUP else 1 if case["q8"] else 0)
        return {"bytes": T * n * size + 2 * n + scales, "flops": T * n * (5 + (3 if case["q8"] else 0))}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (4 if case["f32"] else 2) + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": T * E * 6}
    old, new = _lengths(case, 0)
    kv, P, hkv, D = old + new, case["page"], case["hkv"], case["D"]
    if op == "bounds":
        first = old // P
        tokens = int((kv - first * P).sum())                   # of the blocks that new tokens went to
        blocks = int((-(-kv // P) - first).sum())
        return {"bytes": tokens * hkv * (D // 2 + 4) + blocks * hkv * (2 * D + 4) + 4 * int(new.sum()),
                "flops": tokens * hkv * D * 4}
    hq, top = case["hq"], case["top"]
    blocks = -(-kv // P)
    rows = int(new.sum())
    if op == "select":
        return {"bytes": int(blocks.sum()) * (hkv * (2 * D + 4) + 4) + rows * (2 * hq * D + 4 * hkv * top) + 8 * case["B"],
                "flops": 4 * int((new * blocks).sum()) * hkv * D}
    seen = int((new * np.minimum(blocks, top)).sum()) * P
    return {"bytes": seen * hkv * (D + 8) + rows * (4 * hq * D + 4 * hkv * top) + 4 * int(np.minimum(blocks, top).sum()),
            "flops": 4 * seen * hq * D}


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


def _random_bounds(g, n_pages, hkv, D):
    """Bounds of blocks of keys: a centre and a spread for each channel, as 8-bit codes of a power-of-two step."""
    mid = torch.randn((n_pages, hkv, D), generator=g, device=DEV) * 0.6
    off = torch.rand((n_pages, hkv, D), generator=g, device=DEV) + 0.7
    top = torch.maximum((mid + off).abs(), (mid - off).abs()).amax(-1)
    step = torch.exp2(torch.ceil(torch.log2(top / 127)))
    code = torch.stack([((mid + off) / step[..., None]).ceil(), ((mid - off) / step[..., None]).floor()], 2)
    return code.clamp_(-127, 127).to(torch.int8).contiguous(), step.contiguous()


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    s = dict(case=dict(case))
    if op == "norm":
        T, n = case["T"], case["n"]
        x = torch.randn((T, n), generator=g, device=DEV) * (0.5 + torch.rand((T, 1), generator=g, device=DEV))
        x[:, ::61] *= 8                                       # channels with larger values, as a residual stream has
        s.update(x=x if case["f32"] else x.to(torch.bfloat16), eps=1e-5,
                 weight=(1 + 0.2 * torch.randn(n, generator=g, device=DEV)).to(torch.bfloat16),
                 residual=_bf16(g, T, n, scale=2.0) if case["add"] else None)
        return s
    if op == "route":
        T, E = case["T"], case["E"]
        x = 1.5 * torch.randn((T, E), generator=g, device=DEV) + 0.7 * torch.randn((1, E), generator=g, device=DEV)
        s.update(logits=x if case["f32"] else x.to(torch.bfloat16), scale=2.5 if case["renorm"] else 1.0,
                 bias=(0.05 if case["sigmoid"] else 0.2 / E) * torch.randn(E, generator=g, device=DEV) if case["bias"] else None)
        return s
    old, new = _lengths(case, seed)
    P, hkv, D = case["page"], case["hkv"], case["D"]
    kv = old + new
    blocks = -(-kv // P)
    n_pages = int(blocks.sum()) + 3
    perm = np.random.RandomState(seed % (1 << 31)).permutation(n_pages).astype(np.int32)
    at = np.concatenate([[0], np.cumsum(blocks)])
    table = np.full((case["B"], int(blocks.max())), -1, dtype=np.int32)
    for b in range(case["B"]):
        table[b, :blocks[b]] = perm[at[b]:at[b + 1]]
    if op == "bounds":
        slots = np.concatenate([table[b, pos // P] * P + pos % P for b in range(case["B"])
                                for pos in [np.arange(old[b], kv[b])]])
        s.update(pages=_random_pages(g, n_pages, P, hkv, D), slots=_ints(slots),
                 codes=torch.zeros((n_pages, hkv, 2, D), dtype=torch.int8, device=DEV),
                 steps=torch.zeros((n_pages, hkv), device=DEV))
        return s
    hq, top = case["hq"], case["top"]
    n = int(new.sum())
    s.update(q=_bf16(g, n, hq, D, scale=1.5), q_start=_ints(np.concatenate([[0], np.cumsum(new)])), kv_len=_ints(kv),
             table=_ints(table), max_q=int(new.max()), max_kv=int(kv.max()))
    if op == "select":
        s["codes"], s["steps"] = _random_bounds(g, n_pages, hkv, D)
        s["page_size"] = P
        return s
    # chosen blocks: the first and the last one, and others at random, ascending, -1 behind them
    seen = _ints(np.concatenate([(old[b] + np.arange(new[b])) // P + 1 for b in range(case["B"])]))[:, None, None]
    col = torch.arange(table.shape[1], device=DEV)
    key = torch.rand((n, hkv, table.shape[1]), generator=g, device=DEV)
    key = torch.where((col == 0) | (col == seen - 1), -1.0, torch.where(col < seen, key, 2.0))
    far = 1 << 30
    pick = torch.argsort(key, dim=-1)[..., :top]
    pick = torch.sort(torch.where(torch.gather(key, 2, pick) < 2, pick, far), dim=-1).values
    sel = torch.full((n, hkv, top), far, dtype=torch.int64, device=DEV)
    sel[..., :pick.shape[2]] = pick
    s.update(pages=_random_pages(g, n_pages, P, hkv, D), scale=D ** -0.5,
             sel=torch.where(sel == far, -1, sel).to(torch.int32).contiguous())
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["residual"] = h.to(torch.bfloat16)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    out["y"] = y.to(torch.bfloat16)
    if c["q8"]:
        T, n = y.shape
        size = GROUP if c["q8"] == GROUP else n
        pad = torch.nn.functional.pad(y, (0, -n % size)).reshape(T, -1, size)
        scale = pad.abs().amax(-1, keepdim=True) / E4M3_MAX
        q = torch.where(scale > 0, pad / scale, torch.zeros_like(pad)).clamp(-E4M3_MAX, E4M3_MAX)
        out["codes"] = q.reshape(T, -1)[:, :n].to(torch.float8_e4m3fn)
        out["scales"] = scale[..., 0]
    return out


def _plain_route(s):
    """In 64 bits: which expert is the better one is decided by values next to each other."""
    c = s["case"]
    x = s["logits"].double()
    x = torch.where(torch.isnan(x), float("-inf"), x).clamp(max=3.4028234663852886e38)
    T, E = x.shape
    if c["sigmoid"]:
        score = 1 / (1 + torch.exp(-x))
    else:
        m = x.amax(-1, keepdim=True)
        e = torch.where(x > float("-inf"), torch.exp(x - m), torch.zeros_like(x))
        score = e / e.sum(-1, keepdim=True).clamp(min=1)
    by = x if s["bias"] is None else score + s["bias"].double()      # the scores' own order is that of the logits
    if c["groups"] > 1:
        value = by if c["best"] == 1 else score if s["bias"] is None else by
        value = torch.sort(value.reshape(T, c["groups"], -1), dim=-1, descending=True).values[..., :c["best"]].sum(-1)
        kept = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        on = torch.zeros((T, c["groups"]), dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        on = on.repeat_interleave(E // c["groups"], dim=1)
        # experts of other groups stand behind all of the kept ones, whatever their values
        order = torch.sort(by, dim=-1, descending=True, stable=True).indices
        order = torch.gather(order, 1, torch.sort((~torch.gather(on, 1, order)).to(torch.uint8), dim=-1, stable=True).indices)
    else:
        order = torch.sort(by, dim=-1, descending=True, stable=True).indices
    ids = order[:, :c["k"]]
    gates = torch.gather(score, 1, ids)
    if c["renorm"]:
        total = gates.sum(-1, keepdim=True)
        gates = torch.where(total > 0, gates / total, torch.zeros_like(gates))
    return dict(ids=ids.to(torch.int32), gates=(gates * s["scale"]).float())


def _plain_rows(pages, P, hkv, D, side):
    """Values [n, hkv, P, D] of pages [n, page_bytes], rounded once to 32 bits."""
    n = pages.shape[0]
    pg = pages.reshape(n, hkv, P * (D + 8))
    codes = pg[..., side * P * D // 2:(side + 1) * P * D // 2].contiguous().view(torch.int32).reshape(n, hkv, P, D // 8, 1)
    sh = torch.tensor(SHIFTS, dtype=torch.int32, device=DEV)
    u = ((codes >> sh) & 15).reshape(n, hkv, P, D).double()
    par = pg[..., P * D + 4 * P * side:P * D + 4 * P * (side + 1)].contiguous().view(torch.float16).reshape(n, hkv, P, 2).double()
    return (u * par[..., :1] + par[..., 1:]).float()


def _plain_bounds(s):
    c = s["case"]
    P, hkv, D = c["page"], c["hkv"], c["D"]
    slot = s["slots"].long()
    nxt = torch.cat([slot[1:], slot.new_full((1,), -1)])
    last = (nxt != slot + 1) | (nxt % P == 0)                        # a block's last new token
    slot = slot[last]
    page, size = torch.div(slot, P, rounding_mode="floor"), slot % P + 1
    k = _plain_rows(s["pages"][page], P, hkv, D, 0)
    off = (torch.arange(P, device=DEV) >= size[:, None])[:, None, :, None]
    hi = k.masked_fill(off, float("-inf")).amax(2)
    lo = k.masked_fill(off, float("inf")).amin(2)
    big = torch.maximum(hi.abs(), lo.abs()).amax(-1).double()
    e = torch.frexp(big).exponent - 7                                # big = m 2^e with m in [64, 128)
    e = e + (big > 127 * torch.exp2(e.double())).to(e.dtype)
    step = torch.where(big > 0, torch.exp2(e.double()), torch.zeros_like(big))
    div = torch.where(step > 0, step, torch.ones_like(step))[..., None]
    codes, steps = s["codes"].clone(), s["steps"].clone()
    codes[page] = torch.stack([torch.ceil(hi / div), torch.floor(lo / div)], 2).to(torch.int8)
    steps[page] = step.float()
    return dict(codes=codes, steps=steps)


def _plain_select(s):
    """Sums of whole numbers (in 64 bits, exactly), rounded once to 32 bits, times the blocks' steps."""
    c = s["case"]
    B, hq, hkv, D, P, top = c["B"], c["hq"], c["hkv"], c["D"], c["page"], c["top"]
    G, n = hq // hkv, s["q"].shape[0]
    bits = 15 - math.ceil(math.log2(G))
    q = s["q"].double().reshape(n, hkv, G, D)
    big = q.abs().amax((-1, -2), keepdim=True)
    q = torch.round(q * torch.exp2((bits - torch.frexp(big).exponent).double())).clamp(-2 ** bits + 1, 2 ** bits - 1)
    q = torch.cat([q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)], -1)                       # [n, hkv, 2 D]
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    tok = torch.arange(n, device=DEV)
    b = torch.searchsorted(q_start[1:], tok, right=True)
    pos = kv_len[b] - (q_start[b + 1] - tok)
    mq = s["max_q"]
    i = torch.arange(mq, device=DEV)
    at = (q_start[:-1, None] + i).clamp(max=n - 1)
    page = s["table"].clamp(min=0).long()
    bounds = s["codes"].reshape(-1, hkv, 2 * D)[page].double()                               # [B, nb, hkv, 2 D]
    dot = torch.einsum("bmhd,bnhd->bmhn", q[at], bounds)[b, tok - q_start[b]]               # [n, hkv, nb]
    score = dot.float() * s["steps"][page].permute(0, 2, 1)[b]
    blk = torch.arange(score.shape[2], device=DEV)
    own_blk = torch.div(pos, P, rounding_mode="floor")[:, None, None]
    score = torch.where((blk == 0) | (blk == own_blk), float("inf"), torch.where(blk <= own_blk, score, float("-inf")))
    pick = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    far = 1 << 30
    pick = torch.sort(torch.where(pick <= own_blk, pick, far), dim=-1).values
    sel = torch.full((n, hkv, top), far, dtype=torch.int64, device=DEV)
    sel[..., :pick.shape[2]] = pick
    return torch.where(sel == far, -1, sel).to(torch.int32)


def _plain_blocks(s):
    c = s["case"]
    hq, hkv, D, P = c["hq"], c["hkv"], c["D"], c["page"]
    G, n = hq // hkv, s["q"].shape[0]
    q_start, kv_len, sel = s["q_start"].long(), s["kv_len"].long(), s["sel"].long()
    tok = torch.arange(n, device=DEV)
    b = torch.searchsorted(q_start[1:], tok, right=True)
    pos = (kv_len[b] - (q_start[b + 1] - tok))[:, None, None, None]
    page = s["table"].long()[b[:, None, None], sel.clamp(min=0)]                             # [n, hkv, top]
    head = torch.arange(hkv, device=DEV)[:, None]
    pg = s["pages"].reshape(-1, hkv, P * (D + 8))[page, head].reshape(-1, P * (D + 8))       # [n hkv top, bytes]
    k, v = (_plain_rows(pg, P, 1, D, x).reshape(n, hkv, -1, D) for x in (0, 1))
    at = (sel * P)[..., None] + torch.arange(P, device=DEV)
    seen = ((sel >= 0)[..., None] & (at <= pos)).reshape(n, hkv, 1, -1)
    sc = torch.matmul(s["q"].float().reshape(n, hkv, G, D), k.transpose(-1, -2)) * s["scale"]
    sc = sc.masked_fill_(~seen, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o.reshape(n, hq, D).to(torch.bfloat16)


# ------------------------------------------------------------------ the framework's kernels
def _handle(s):
    """What a user's program makes once and keeps: outputs, the cache's handles, the workspace."""
    import decode_matvec_gb300 as Q
    c, h = s["case"], {"Q": Q}
    if c["op"] == "norm":
        T, n = c["T"], c["n"]
        h.update(y=torch.empty((T, n), dtype=torch.bfloat16, device=DEV), codes=None, scales=None,
                 out=None if s["residual"] is None else torch.empty_like(s["residual"]))
        if c["q8"]:
            h.update(codes=torch.empty((T, n), dtype=torch.float8_e4m3fn, device=DEV),
                     scales=torch.empty((T, -(-n // GROUP) if c["q8"] == GROUP else 1), device=DEV))
    elif c["op"] == "route":
        h.update(ids=torch.empty((c["T"], c["k"]), dtype=torch.int32, device=DEV),
                 gates=torch.empty((c["T"], c["k"]), device=DEV))
    elif c["op"] == "bounds":
        h.update(cache=Q.Kv4Cache(s["pages"], c["page"], c["hkv"], c["D"]),
                 bounds=Q.Kv4Bounds(s["codes"].clone(), s["steps"].clone(), c["page"]))
    else:
        n = s["q"].shape[0]
        if c["op"] == "select":
            size = Q.kv4_select_blocks_ws_size(n, c["hkv"], c["page"], s["max_kv"])
            h.update(bounds=Q.Kv4Bounds(s["codes"], s["steps"], c["page"]),
                     sel=torch.empty((n, c["hkv"], c["top"]), dtype=torch.int32, device=DEV))
        else:
            size = Q.kv4_attention_blocks_ws_size(n, c["hq"], c["hkv"], c["D"], c["page"], c["top"])
            h.update(cache=Q.Kv4Cache(s["pages"], c["page"], c["hkv"], c["D"]), out=torch.empty_like(s["q"]))
        h["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=DEV)
    return h


def _own(s):
    h = s.get("handle") or s.setdefault("handle", _handle(s))
    Q, c = h["Q"], s["case"]
    if c["op"] == "norm":
        Q.add_rms_norm(s["x"], s["weight"], s["eps"], h["y"], residual=s["residual"], residual_out=h["out"], codes=h["codes"],
                       scales=h["scales"])
        out = {} if h["out"] is None else {"residual": h["out"]}
        return {**out, "y": h["y"]} if h["codes"] is None else {**out, "y": h["y"], "codes": h["codes"], "scales": h["scales"]}
    if c["op"] == "route":
        Q.qmoe_route_scored(s["logits"], c["k"], h["ids"], h["gates"], sigmoid=c["sigmoid"], bias=s["bias"],
                            n_groups=c["groups"], top_groups=c["top_groups"], group_best=c["best"], renormalise=c["renorm"],
                            scale=s["scale"])
        return dict(ids=h["ids"], gates=h["gates"])
    if c["op"] == "bounds":
        Q.kv4_block_bounds(h["cache"], h["bounds"], s["slots"])
        return dict(codes=h["bounds"].codes, steps=h["bounds"].steps)
    if c["op"] == "select":
        return Q.kv4_select_blocks(h["bounds"], s["q"], s["q_start"], s["kv_len"], s["table"], h["sel"], h["ws"], s["max_kv"],
                                   first=1, last=1)
    return Q.kv4_attention_blocks(h["cache"], s["q"], s["q_start"], s["kv_len"], s["table"], s["sel"], h["out"], h["ws"],
                                  s["scale"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "route": _plain_route, "bounds": _plain_bounds, "select": _plain_select,
            "blocks": _plain_blocks}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_codes(y, scale):
    """The 8-bit floats nearest to y / scale: 3 fraction bits, exponents from -6."""
    q = np.divide(y, scale, out=np.zeros_like(y), where=scale > 0)
    unit = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 1e-300))), -6) - 3)
    return np.clip(np.rint(q / unit) * unit, -E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    op, s = case["op"], prepare(case, seed)
    if op == "norm":
        h = s["x"].double().cpu().numpy()
        w = s["weight"].double().cpu().numpy()
        out = {}
        if case["add"]:
            h = h + s["residual"].double().cpu().numpy()
            out["residual"] = torch.from_numpy(h)
        y = h * ((np.einsum("ij,ij->i", h, h) / h.shape[1] + s["eps"]) ** -0.5)[:, None] * w
        out["y"] = torch.from_numpy(y)
        if case["q8"]:
            size = GROUP if case["q8"] == GROUP else case["n"]
            starts = np.arange(0, case["n"], size)
            scale = np.maximum.reduceat(np.abs(y), starts, axis=1) / E4M3_MAX
            out["codes"] = torch.from_numpy(_exact_codes(y, np.repeat(scale, size, axis=1)[:, :case["n"]]))
            out["scales"] = torch.from_numpy(scale)
        return out
    if op == "route":
        x = s["logits"].double().cpu().numpy()
        T, E = x.shape
        p = np.reciprocal(1 + np.exp(-x)) if case["sigmoid"] else np.exp(x - x.max(1, keepdims=True))
        if not case["sigmoid"]:
            p /= p.sum(1, keepdims=True)
        v = p + (0 if s["bias"] is None else s["bias"].double().cpu().numpy())
        if case["groups"] > 1:
            rank = np.sort(v.reshape(T, case["groups"], -1), axis=2)[:, :, -case["best"]:].sum(2)
            keep = np.argsort(-rank, axis=1, kind="stable")[:, :case["top_groups"]]
            on = np.zeros((T, case["groups"]), bool)
            np.put_along_axis(on, keep, True, axis=1)
            v = np.where(np.repeat(on, E // case["groups"], axis=1), v, -np.inf)
        ids = np.argsort(-v, axis=1, kind="stable")[:, :case["k"]]
        w = np.take_along_axis(p, ids, 1)
        if case["renorm"]:
            w /= w.sum(1, keepdims=True)
        return dict(ids=None, gates=torch.from_numpy(w * s["scale"]))
    if op == "select":
        return None
    if op == "bounds":
        P, hkv, D = case["page"], case["hkv"], case["D"]
        slots = s["slots"].cpu().numpy()
        page, size = np.unique(slots // P, return_inverse=True)
        fill = np.zeros(len(page), np.int64)
        np.maximum.at(fill, size, slots % P + 1)
        pg = s["pages"].cpu().numpy()[page].reshape(len(page), hkv, -1)
        word = np.ascontiguousarray(pg[:, :, :P * D // 2]).view("<u4").reshape(len(page), hkv, P, D // 8, 1)
        u = (word >> np.array(SHIFTS, np.uint32)[None]) & 15
        sz = np.ascontiguousarray(pg[:, :, P * D:P * D + 4 * P]).view("<f2").reshape(len(page), hkv, P, 2).astype(np.float64)
        k = u.reshape(len(page), hkv, P, D) * sz[..., :1] + sz[..., 1:]
        k[np.broadcast_to((np.arange(P) >= fill[:, None])[:, None, :, None], k.shape)] = 0
        steps = np.zeros(s["steps"].shape)
        steps[page] = np.exp2(np.ceil(np.log2(np.abs(k).max((2, 3)) / 127)))
        return dict(codes=None, steps=torch.from_numpy(steps))
    hq, hkv, D, P = case["hq"], case["hkv"], case["D"], case["page"]
    G = hq // hkv
    out = torch.zeros((s["q"].shape[0], hq, D), dtype=torch.float64, device=DEV)
    starts, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].long()
    shift = torch.tensor([4 * (i // 2) + 16 * (i % 2) for i in range(8)], dtype=torch.int32, device=DEV)
    within = torch.arange(P, device=DEV)
    for b in range(case["B"]):
        for t in range(starts[b], starts[b + 1]):
            pos = lens[b] - (starts[b + 1] - t)
            for h in range(hkv):
                blk = s["sel"][t, h].long()
                blk = blk[blk >= 0]
                where = (blk[:, None] * P + within).reshape(-1)
                pg = s["pages"][table[b, blk], h * P * (D + 8):(h + 1) * P * (D + 8)]
                part = []
                for x in (0, 1):
                    word = pg[:, x * P * D // 2:(x + 1) * P * D // 2].contiguous().view(torch.int32).reshape(-1, D // 8, 1)
                    sz = pg[:, P * D + 4 * P * x:P * D + 4 * P * (x + 1)].contiguous().view(torch.float16).reshape(-1, 2).double()
                    part.append((((word >> shift) & 15).reshape(-1, D).double() * sz[:, :1] + sz[:, 1:])[where <= pos])
                w = torch.softmax(s["q"][t, h * G:(h + 1) * G].double() @ part[0].T * s["scale"], -1)
                out[t, h * G:(h + 1) * G] = w @ part[1]
    return out

"""Cases of the paged-cache operators: append with rotation, chunk attention, single-token attention.

A cache holds keys and values in pages of `page` slots that sequences own through a table:
position p of sequence b lives in page table[b, p // page], slot p % page.  Pages that no query
can see any more (behind the window and behind the sinks) have the table entry -1.  A query at
position p sees key j iff j <= p and (j > p - W or j < sinks).

Lengths and start positions of a case come from its "mix" number, tensors from the seed.
"""

import math
import random

import torch

own = False


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 sequences: rotate q and k, write one slot each (latency counts)
        dict(name="append_step64", op="append", n_seq=64, len_lo=1, len_hi=1, ctx_lo=4096,
             ctx_hi=131072, H=32, Hkv=8, d=128, page=16, layout="hnd", rot=128, axes=1,
             inter=False, mix=1),
        # a packed prefill of images and text: three position axes, half of the dims rotated,
        # token-major pages
        dict(name="append_image", op="append", n_seq=16, len_lo=256, len_hi=1021, ctx_lo=0,
             ctx_hi=5000, H=32, Hkv=8, d=128, page=32, layout="nhd", rot=64, axes=3, inter=False,
             mix=2),
        # a long prefill of one sequence, interleaved pairs, own key/value heads per query head
        dict(name="append_long", op="append", n_seq=1, len_lo=16384, len_hi=16384, ctx_lo=0,
             ctx_hi=0, H=32, Hkv=32, d=128, page=64, layout="hnd", rot=128, axes=1, inter=True,
             mix=3),
        # five drafted tokens verified over a short context, small heads (latency counts)
        dict(name="chunk_draft", op="chunk", n_seq=2, len_lo=5, len_hi=5, ctx_lo=300, ctx_hi=1000,
             H=8, Hkv=2, d=64, page=16, layout="hnd", W=512, sinks=0, mix=4),
        # chunked prefill: 512 new tokens per sequence over a full window
        dict(name="chunk_512", op="chunk", n_seq=4, len_lo=512, len_hi=512, ctx_lo=12288,
             ctx_hi=12288, H=32, Hkv=8, d=128, page=16, layout="hnd", W=4096, sinks=0, mix=5),
        # a mixed batch: chunks of 1 to 512 tokens, four sinks, token-major pages
        dict(name="chunk_mixed", op="chunk", n_seq=16, len_lo=1, len_hi=512, ctx_lo=0, ctx_hi=20000,
             H=32, Hkv=8, d=128, page=128, layout="nhd", W=4096, sinks=4, mix=6),
        # narrow window, own key/value heads per query head, odd length
        dict(name="chunk_narrow", op="chunk", n_seq=1, len_lo=8191, len_hi=8191, ctx_lo=0,
             ctx_hi=0, H=32, Hkv=32, d=128, page=64, layout="hnd", W=512, sinks=0, mix=7),
        # a whole prompt through a layer whose window covers it
        dict(name="chunk_prompt", op="chunk", n_seq=1, len_lo=8192, len_hi=8192, ctx_lo=0,
             ctx_hi=0, H=32, Hkv=8, d=128, page=64, layout="hnd", W=1 << 20, sinks=0, mix=8),
        # a short turn over a long context without a window: few rows, many keys
        dict(name="chunk_turn", op="chunk", n_seq=1, len_lo=61, len_hi=61, ctx_lo=130000,
             ctx_hi=130000, H=32, Hkv=8, d=128, page=32, layout="hnd", W=1 << 20, sinks=0, mix=9),
        # one token of one sequence (latency counts)
        dict(name="decode_one", op="decode", n_seq=1, ctx_lo=1000, ctx_hi=1000, H=32, Hkv=8, d=128,
             page=16, layout="hnd", W=4096, sinks=0, mix=10),
        # batched decode with full windows
        dict(name="decode_64", op="decode", n_seq=64, ctx_lo=4096, ctx_hi=131072, H=32, Hkv=8,
             d=128, page=16, layout="hnd", W=4096, sinks=4, mix=11),
        # batched decode without a window: lengths of very different sizes, eight heads a group
        dict(name="decode_mixed", op="decode", n_seq=24, ctx_lo=1, ctx_hi=100000, H=64, Hkv=8,
             d=128, page=64, layout="nhd", W=1 << 20, sinks=0, mix=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, int(round(lo * (hi / lo) ** rng.random())))

    H, Hkv = rng.choice([(32, 8), (8, 2), (16, 2), (4, 4), (32, 32), (12, 4), (7, 1), (64, 8)])
    case = dict(op=rng.choice(["append", "chunk", "decode"]), H=H, Hkv=Hkv,
                d=rng.choice([64, 128]), page=rng.choice([8, 16, 32, 48, 64, 128, 256]),
                layout=rng.choice(["hnd", "nhd"]), mix=rng.randrange(1 << 30))
    if case["op"] == "append":
        case["n_seq"] = log_int(1, 64)
        top = log_int(1, max(1, 16384 // case["n_seq"]))
        case |= dict(len_lo=rng.choice([0, 1, max(1, top // 2), top]), len_hi=top, ctx_lo=0,
                     ctx_hi=log_int(1, 100000), axes=rng.choice([1, 1, 3]),
                     rot=rng.choice([case["d"], case["d"] // 2, 16, 0]),
                     inter=rng.random() < 0.5)
        return case
    case |= dict(W=log_int(1, 20000) if rng.random() < 0.7 else 1 << 20,
                 sinks=rng.choice([0, 0, 1, 4, 128]))
    if case["op"] == "decode":
        case["n_seq"] = log_int(1, 128)
        case |= dict(ctx_lo=1, ctx_hi=log_int(1, 100000))
        largest = next(c for c in listed() if c["name"] == "decode_mixed")
    else:
        case["n_seq"] = log_int(1, 32)
        top = log_int(1, max(1, 8192 // case["n_seq"]))
        case |= dict(len_lo=rng.choice([0, 1, max(1, top // 2), top]), len_hi=top, ctx_lo=0,
                     ctx_hi=log_int(1, 100000))
        largest = next(c for c in listed() if c["name"] == "chunk_prompt")
    kind = "bytes" if case["op"] == "decode" else "flops"
    while (work(case)[kind] > work(largest)[kind] or _padded(case) > 2.2e9
           or _gathered(case) > 2.6e9):
        case["ctx_hi"] = max(1, case["ctx_hi"] // 2)
        if "len_hi" in case:
            case["len_hi"] = max(1, case["len_hi"] * 2 // 3)
            case["len_lo"] = min(case["len_lo"], case["len_hi"])
    return case


def _spans(case):
    """New tokens and positions of the first of them, per sequence."""
    r = random.Random(case["mix"])
    if case["op"] == "decode":
        starts = [r.randint(case["ctx_lo"], case["ctx_hi"]) - 1 for _ in range(case["n_seq"])]
        return [1] * case["n_seq"], starts
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["n_seq"])]
    lens[0] = max(1, lens[0])
    return lens, [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n_seq"])]


def _padded(case):
    """Score entries of the batch padded to its longest sequence."""
    lens, starts = _spans(case)
    span = max(n + min(s, case["W"]) for n, s in zip(lens, starts))
    return case["n_seq"] * case["H"] * max(lens) * span


def _gathered(case):
    """Key entries of the batch padded to its longest span."""
    lens, starts = _spans(case)
    span = case["sinks"] + max(n + min(s, case["W"]) for n, s in zip(lens, starts))
    return case["n_seq"] * span * case["Hkv"] * case["d"]


def work(case):
    lens, starts = _spans(case)
    total, H, Hkv, d = sum(lens), case["H"], case["Hkv"], case["d"]
    if case["op"] == "append":
        rows = total * (H + 2 * Hkv)
        return {"bytes": 2 * rows * d * 2 + total * 8 * case["axes"] * (case["rot"] > 0),
                "flops": total * (H + Hkv) * case["rot"] * 3}
    W, S = case["W"], case["sinks"]
    pairs = rows = 0
    for n, s in zip(lens, starts):
        if n == 0:
            continue
        first = max(0, s - W + 1)  # lowest position in any window of the chunk
        rows += s + n - first + min(S, first)
        # sum over p = s .. s+n-1 of min(p + 1, W) + min(S, max(0, p + 1 - W))
        grow = max(0, min(s + n, W) - s)  # queries whose window is not full yet
        pairs += grow * (s + 1) + grow * (grow - 1) // 2 + (n - grow) * W
        a = s + grow + 1 - W  # keys behind the window of the first full query
        few = max(0, min(n - grow, S - a))
        pairs += few * a + few * (few - 1) // 2 + (n - grow - few) * S
    return {"bytes": 2 * total * H * d * 2 + 4 * total * H + rows * Hkv * d * 2 * 2,
            "flops": 4 * d * H * pairs}


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, starts = _spans(case)
    H, Hkv, d, ps = case["H"], case["Hkv"], case["d"], case["page"]
    total = sum(lens)
    n_len = torch.tensor(lens, dtype=torch.int64)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n_len.cumsum(0)]).to(dev)
    first = torch.tensor(starts, dtype=torch.int64, device=dev)
    end = first + n_len.to(dev)
    longest = max(n + s for n, s in zip(lens, starts))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    # the table: live pages are those that a query of this call can see (append: writes)
    page0 = torch.arange((longest + ps - 1) // ps, device=dev) * ps
    low = first if case["op"] == "append" else (first - case["W"] + 1).clamp(min=0)
    live = (page0 + ps > low[:, None]) & (page0 < end[:, None])
    if case.get("sinks"):
        live |= (page0 < case["sinks"]) & (page0 < end[:, None])
    n_pages = int(live.sum()) + 3
    ids = torch.randperm(n_pages, generator=g, device=dev)
    table = torch.where(live, ids[(live.flatten().cumsum(0) - 1).view_as(live).clamp(min=0)], -1)

    def cache():
        if case["layout"] == "hnd":
            return normal(n_pages, Hkv, ps, d)
        return normal(n_pages, ps, Hkv, d).transpose(1, 2)

    s = dict(case=case, table=table.to(torch.int32), k_cache=cache(), v_cache=cache(), cu=cu,
             first=first, max_len=max(lens), total=total)
    if case["op"] == "append":
        # views of one fused projection's output
        qkv = normal(total, H + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64)
                                     / max(1, half))).float()
        s["positions"] = s["pair_axis"] = None
        if case["axes"] > 1 and half:
            s["positions"] = torch.randint(0, 200000, (case["axes"], total), generator=g,
                                           device=dev)
            s["pair_axis"] = (torch.arange(half, device=dev) * case["axes"] // half).int()
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    s["q"] = normal(total, H, d)
    # keys between the lowest position any query sees and the last one, at most
    s["span"] = max(n + min(a, case["W"]) for n, a in zip(lens, starts))
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        return _call(s)
    return _append(s) if case["op"] == "append" else _attend(s)


def _call(s):
    import sliding_window_sparse_b200 as swa

    case = s["case"]
    if case["op"] == "append":
        rope = dict(inv_freq=s["inv_freq"], interleaved=case["inter"], positions=s["positions"],
                    pair_axis=s["pair_axis"]) if case["rot"] else {}
        q = swa.swa_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"],
                                 s["first"], q=s["q"], **rope)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] == "decode":
        out, lse = swa.swa_attn_decode_paged(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                             s["first"], case["W"], s["scale"],
                                             n_sink=case["sinks"], return_lse=True)
    else:
        out, lse = swa.swa_attn_chunk_paged(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                            s["cu"], s["first"], case["W"], s["scale"],
                                            n_sink=case["sinks"], return_lse=True)
    return {"out": out, "lse": lse}


def _tokens(s):
    """Sequence and index within it, of every packed token."""
    t = torch.arange(s["total"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    return b, t - s["cu"][b]


def _append(s):
    case, ps = s["case"], s["case"]["page"]
    b, t = _tokens(s)
    pos = s["first"][b] + t
    page, slot = s["table"][b, pos // ps].long(), pos % ps
    q, k = s["q"].float(), s["k"].float()
    rot = case["rot"]
    if rot:
        half = rot // 2
        if s["positions"] is None:
            at = pos[:, None].double()
        else:
            at = s["positions"][s["pair_axis"].long()].T.double()
        angle = at * s["inv_freq"].double()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turn(x):
            if case["inter"]:
                a, c = x[..., 0:rot:2], x[..., 1:rot:2]
                r = torch.stack([a * cos - c * sin, c * cos + a * sin], dim=-1).flatten(-2)
            else:
                a, c = x[..., :half], x[..., half:rot]
                r = torch.cat([a * cos - c * sin, c * cos + a * sin], dim=-1)
            return torch.cat([r, x[..., rot:]], dim=-1)

        q, k = turn(q), turn(k)
    s["k_cache"][page, :, slot] = k.bfloat16()
    s["v_cache"][page, :, slot] = s["v"]
    return {"q": q.bfloat16(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _rows(s, pos):
    """Keys and values [n_seq, Hkv, n, d] in 32 bits at positions pos [n_seq, n]; what the table
    does not hold reads as zero."""
    ps = s["case"]["page"]
    at = pos.clamp(max=s["table"].shape[1] * ps - 1)
    page = s["table"].gather(1, at // ps)
    held = (page >= 0)[:, None, :, None]
    page, slot = page.clamp(min=0).long(), at % ps
    k, v = (c[page, :, slot].transpose(1, 2).float() for c in (s["k_cache"], s["v_cache"]))
    return torch.where(held, k, 0.0), torch.where(held, v, 0.0)


def _attend(s):
    case = s["case"]
    W, S, H, Hkv, d = case["W"], case["sinks"], case["H"], case["Hkv"], case["d"]
    n_seq, dev, Lq = case["n_seq"], s["q"].device, s["max_len"]
    # queries padded to the longest chunk
    t = torch.arange(Lq, device=dev)
    q = s["q"][(s["cu"][:-1, None] + t).clamp(max=s["total"] - 1)].float()
    q = q.view(n_seq, Lq, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(n_seq, Hkv, -1, d)
    qp = (s["first"][:, None] + t)[:, :, None]
    # the sinks, then the union of the chunk's windows
    low = (s["first"] - W + 1).clamp(min=0)
    win = low[:, None] + torch.arange(s["span"], device=dev)
    sink = torch.arange(S, device=dev).expand(n_seq, S)
    kp = torch.cat([sink, win], dim=1)
    is_sink = torch.arange(kp.shape[1], device=dev) < S
    k, v = _rows(s, kp)
    kp = kp[:, None, :]
    seen = torch.where(is_sink, kp <= qp - W, (kp <= qp) & (kp > qp - W))
    x = (q @ k.transpose(2, 3) * s["scale"]).view(n_seq, Hkv, H // Hkv, Lq, -1)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    del x
    z = p.sum(-1, keepdim=True)
    o = (p.view(n_seq, Hkv, -1, p.shape[-1]) @ v).view(n_seq, H, Lq, d) / z.view(n_seq, H, Lq, 1)
    lse = (m + z.log()).view(n_seq, H, Lq)
    if case["op"] == "decode":
        return {"out": o[:, :, 0].bfloat16(), "lse": lse[:, :, 0]}
    b, t = _tokens(s)
    return {"out": o[b, :, t].bfloat16(), "lse": lse[b, :, t].T.contiguous()}


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lens, starts = _spans(case)
    table, ps = s["table"].long(), case["page"]
    done = 0
    if case["op"] == "append":
        q_out = s["q"].double()
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, (n, a) in enumerate(zip(lens, starts)):
            pos = torch.arange(a, a + n, device="cuda")
            rows = slice(done, done + n)
            done += n
            k = s["k"][rows].double()
            for i in range(case["rot"] // 2):
                x, y = (2 * i, 2 * i + 1) if case["inter"] else (i, i + case["rot"] // 2)
                at = pos if s["positions"] is None else \
                    s["positions"][int(i * case["axes"] // (case["rot"] // 2)), rows]
                angle = at.double() * s["inv_freq"][i].double()
                c, z = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
                for w in (q_out[rows], k):
                    u, v = w[..., x].clone(), w[..., y].clone()
                    w[..., x], w[..., y] = u * c - v * z, u * z + v * c
            page = table[b][pos // ps]
            kc[page, :, pos % ps] = k
            vc[page, :, pos % ps] = s["v"][rows].double()
        return {"q": q_out, "k_cache": kc, "v_cache": vc}
    H, Hkv, W, S, d = case["H"], case["Hkv"], case["W"], case["sinks"], case["d"]
    out = torch.zeros(s["total"], H, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], H, dtype=torch.float64, device="cuda")
    for b, (n, a) in enumerate(zip(lens, starts)):
        for i in range(0, n, 512):  # queries i .. j - 1 of the chunk
            j = min(n, i + 512)
            qp = torch.arange(a + i, a + j, device="cuda")
            low = max(0, a + i - W + 1)
            kp = torch.cat([torch.arange(0, min(S, low), device="cuda"),
                            torch.arange(low, a + j, device="cuda")])
            seen = (kp <= qp[:, None]) & ((kp > qp[:, None] - W) | (kp < S))
            page, slot = table[b][kp // ps], kp % ps
            for h in range(Hkv):
                G = H // Hkv
                q = s["q"][done + i:done + j, h * G:(h + 1) * G].double()
                x = torch.einsum("tgd,kd->tgk", q, s["k_cache"][page, h, slot].double())
                x = torch.where(seen[:, None], x * (1.0 / math.sqrt(d)), -math.inf)
                lse[done + i:done + j, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[done + i:done + j, h * G:(h + 1) * G] = torch.einsum(
                    "tgk,kd->tgd", torch.softmax(x, -1), s["v_cache"][page, h, slot].double())
        done += n
    return {"out": out, "lse": lse if case["op"] == "decode" else lse.T.contiguous()}

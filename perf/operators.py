"""Measured cases of the paged-cache operators.

Four operators serve packed sequences of different lengths over a cache in
pages: the append of new keys and values with the position rotation on the way
(ds_paged_append), rows of the cache read back as values (ds_paged_gather),
attention of a few new tokens per sequence over the pages
(ds_paged_attention), and causal attention of whole prompts
(ds_prompt_attention).  Pages hold 16-bit values, or 4-bit codes with a scale
and a minimum per (token, head) row.

A pass computes the operators in plain torch operations in 32 bits, or, with
``own`` set, through this package's binding.  ``exact`` computes the same
outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
TABLE_POSITIONS = 16384  # rows of the rotation table that the append cases keep


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of eight conversations, full heads: the smallest write, where latency counts
        _append("append step f16", "f16", "16", 32, 32, 128, 16, 8, 1, 1, 17, 1500, 128, False),
        # a batch of prompts of very different lengths entering the cache, grouped heads
        _append("append prompts bf16", "bf16", "16", 32, 8, 128, 64, 24, 97, 2048, 0, 300, 128, False),
        # a decode step of 64 conversations into the 4-bit cache, the new rows read back
        _append("append4 step bf16", "bf16", "4", 40, 8, 128, 16, 64, 1, 1, 40, 2000, 128, False),
        # prompts into the 4-bit cache, neighbouring channels paired and half of them rotated, rows read back
        _append("append4 prompts f16", "f16", "4", 20, 20, 128, 32, 7, 33, 1500, 0, 700, 64, True),
        # one token of one conversation, full heads: the smallest attention call
        _decode("decode one f16", "f16", "16", 32, 32, 128, 16, 1, 1, 545, 545),
        # a busy server's step: 48 conversations of 700 to 8192 tokens, four query heads to a key head
        _decode("decode many bf16", "bf16", "16", 32, 8, 128, 32, 48, 1, 700, 8192),
        # four drafted tokens each for five conversations, small heads, eight query heads to a key head
        _decode("decode drafts bf16", "bf16", "16", 16, 2, 64, 16, 5, 4, 200, 1500),
        # two very long documents in the 4-bit cache, five query heads to a key head
        _decode("decode4 long f16", "f16", "4", 40, 8, 128, 64, 2, 1, 90001, 131072),
        # 96 conversations in the 4-bit cache, eight query heads to a key head
        _decode("decode4 many bf16", "bf16", "4", 32, 4, 128, 16, 96, 1, 300, 6000),
        # six short prompts of a small model in one call: latency
        _prompt("prompt short f16", "f16", 4, 4, 64, 6, 20, 130, 0, 0),
        # a batch of packed prompts, four query heads to a key head: the ordinary prefill
        _prompt("prompt packed bf16", "bf16", 32, 8, 128, 9, 500, 4096, 0, 0),
        # prompt chunks on top of long cached prefixes, full heads
        _prompt("prompt chunk f16", "f16", 40, 40, 128, 2, 384, 701, 6000, 9001),
    ]


def draw(rng):
    dtype = rng.choice(["f16", "bf16"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 5, 8, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt"])
    if op == "append":
        batch = _log_int(rng, 1, 48)
        hi = _log_int(rng, 1, 1024)
        lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
        past = _log_int(rng, 1, 4000)
        r = rng.choice([d, d, d // 2])
        return _append(None, dtype, rng.choice(["16", "4"]), heads, kv, d, page, batch, lo, hi, past // 3, past, r,
                       rng.random() < 0.3)
    if op == "decode":
        new = rng.choice([1, 1, 1, 2, 3, 5])
        hi = _log_int(rng, 16, 60000)
        batch = _log_int(rng, 1, max(1, min(64, 150000 // hi)))
        lo = max(new, int(hi * rng.uniform(0.1, 1.0)))
        return _decode(None, dtype, rng.choice(["16", "4"]), heads, kv, d, page, batch, new, lo, hi)
    hi = _log_int(rng, 8, 3000)
    batch = _log_int(rng, 1, max(1, min(16, 9000 // hi)))
    lo = max(1, int(hi * rng.uniform(0.2, 1.0)))
    past = 0 if rng.random() < 0.6 else _log_int(rng, 1, 3000)
    return _prompt(None, dtype, heads, kv, d, batch, lo, hi, past // 2, past)


def _append(name, dtype, cache, heads, kv, d, page, batch, lo, hi, past_lo, past_hi, rotary, neighbours):
    c = {"op": "append", "dtype": dtype, "cache": cache, "heads": heads, "kv_heads": kv, "head_dim": d, "page": page,
         "batch": batch, "lo": lo, "hi": hi, "past_lo": past_lo, "past_hi": past_hi, "rotary": rotary,
         "neighbours": neighbours}
    return c if name is None else {"name": name, **c}


def _decode(name, dtype, cache, heads, kv, d, page, batch, new, lo, hi):
    c = {"op": "decode", "dtype": dtype, "cache": cache, "heads": heads, "kv_heads": kv, "head_dim": d, "page": page,
         "batch": batch, "new": new, "lo": lo, "hi": hi}
    return c if name is None else {"name": name, **c}


def _prompt(name, dtype, heads, kv, d, batch, lo, hi, past_lo, past_hi):
    c = {"op": "prompt", "dtype": dtype, "heads": heads, "kv_heads": kv, "head_dim": d, "batch": batch, "lo": lo,
         "hi": hi, "past_lo": past_lo, "past_hi": past_hi}
    return c if name is None else {"name": name, **c}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _spread(lo, hi, n, phase=0.0):
    """n lengths from lo to hi, spread over their logarithm, in no order: the longest is hi."""
    if n == 1:
        return [hi]
    at = [((i + 1) * 0.6180339887498949 + phase) % 1.0 for i in range(n)]
    top, low = max(at), min(at)
    span = (top - low) or 1.0
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** ((a - low) / span))) - 1 for a in at]


def _lens(case):
    """New tokens and tokens cached before them, for each sequence."""
    n = case["batch"]
    if case["op"] == "decode":
        total = _spread(case["lo"], case["hi"], n)
        return [case["new"]] * n, [t - case["new"] for t in total]
    return _spread(case["lo"], case["hi"], n), _spread(case["past_lo"], case["past_hi"], n, 0.37)


# ------------------------------------------------------------------ a pass's needs
def work(case):
    new, past = _lens(case)
    nh, nk, d = case["heads"], case["kv_heads"], case["head_dim"]
    tokens = sum(new)
    row16, row4 = 2 * d, d // 2 + 4  # bytes of one (token, head) row
    if case["op"] == "append":
        row = row4 if case["cache"] == "4" else row16
        table = tokens * 4 * case["rotary"]
        moved = tokens * (2 * nh * row16 + 2 * nk * row16 + 2 * nk * row) + table
        if case["cache"] == "4":
            moved += tokens * 2 * nk * (row4 + row16)  # the rows read back
        return {"bytes": moved, "flops": tokens * (3 * (nh + nk) * case["rotary"] + 6 * 2 * nk * d)}
    total = sum(new) + sum(past)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    flops = 4 * d * nh * pairs
    if case["op"] == "decode":
        row = row4 if case["cache"] == "4" else row16
        return {"bytes": 2 * nk * total * row + 2 * tokens * nh * row16, "flops": flops}
    return {"bytes": 2 * nk * total * row16 + 2 * tokens * nh * row16, "flops": flops}


# ------------------------------------------------------------------ inputs
def _starts(lens, device="cuda"):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(device)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    nh, nk, d, n = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    new, past = _lens(case)
    tokens = sum(new)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = {"op": case["op"], "batch": n, "dtype": dt, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "prompt":
        total = tokens + sum(past)
        if sum(past):
            s["q"], s["k"], s["v"] = normal(tokens, nh, d), normal(total, nk, d), normal(total, nk, d)
        else:  # the three parts of a fused projection's rows
            s["q"], s["k"], s["v"] = _parts(normal(tokens, (nh + 2 * nk) * d), nh, nk, d)
        s["cu_q"], s["cu_k"] = _starts(new), _starts([a + b for a, b in zip(new, past)])
        s["longest_q"], s["longest_k"] = max(new), max(a + b for a, b in zip(new, past))
        s["out"] = torch.empty(tokens, nh, d, dtype=dt, device="cuda")
        if own:
            from transformer_layer_gb300 import ds
            s["ws_bytes"] = ds.ds_prompt_attention_workspace_bytes(nh, n, tokens)
            s["ws"] = _workspace(ds, s["ws_bytes"])
        return s

    page = case["page"]
    s["past"] = torch.tensor(past, dtype=torch.int32, device="cuda")
    need = [-(-(a + b) // page) for a, b in zip(new, past)]
    pages = sum(need) + 3  # some pages belong to nobody
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = _starts(need)
    at = first[:-1, None] + torch.arange(max(need), device="cuda")
    owned = torch.arange(max(need), device="cuda") < (first[1:] - first[:-1])[:, None]
    s["table"] = torch.where(owned, order[at.clamp(max=pages - 1).long()], torch.full_like(order[:1], -1)).contiguous()
    s["page"] = page
    if case["cache"] == "16":
        s["k_pages"], s["v_pages"] = normal(pages, nk, page, d), normal(pages, nk, page, d)
        s["k_scale"] = s["v_scale"] = None
    else:
        for x in "kv":
            s[x + "_pages"], s[x + "_scale"] = _to_codes(normal(pages, nk, page, d).float())
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = _parts(normal(tokens, (nh + 2 * nk) * d), nh, nk, d)
        s["q_out"] = torch.empty(tokens, nh, d, dtype=dt, device="cuda")
        s["cu"] = _starts(new)
        half = case["rotary"] // 2
        angle = torch.arange(TABLE_POSITIONS, dtype=torch.float64, device="cuda")[:, None] * torch.exp(
            torch.arange(half, dtype=torch.float64, device="cuda") * (-math.log(10000.0) / half))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["neighbours"] = case["neighbours"]
        if case["cache"] == "4":
            s["k_rows"] = torch.empty(tokens, nk, d, dtype=dt, device="cuda")
            s["v_rows"] = torch.empty(tokens, nk, d, dtype=dt, device="cuda")
    else:
        s["new"], s["longest"] = case["new"], max(a + b for a, b in zip(new, past))
        s["q"] = normal(n * case["new"], nh, d)
        s["out"] = torch.empty(n * case["new"], nh, d, dtype=dt, device="cuda")
    if own:
        from transformer_layer_gb300 import ds
        s["cache"] = ds.paged_cache(s["k_pages"], s["v_pages"], s["table"], dt, s["k_scale"], s["v_scale"])
        if case["op"] == "append":
            s["rotary"] = ds.rotary(s["cos_sin"], s["neighbours"])
            s["ws_bytes"] = 256
        else:
            s["ws_bytes"] = ds.ds_paged_attention_workspace_bytes(s["cache"], nh, n, case["new"])
        s["ws"] = _workspace(ds, s["ws_bytes"])
    return s


def _parts(qkv, nh, nk, d):
    rows = qkv.view(qkv.shape[0], nh + 2 * nk, d)
    return rows[:, :nh], rows[:, nh:nh + nk], rows[:, nh + nk:]


def _workspace(ds, size):
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    ds.ds_workspace_init(ws, size)
    return ws


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"append": _append_plain, "decode": _decode_plain, "prompt": _prompt_plain}[s["op"]](s)


def _run_own(s):
    from transformer_layer_gb300 import ds
    if s["op"] == "append":
        ds.ds_paged_append(s["cache"], s["q"], s["k"], s["v"], s["q_out"], s["cu"], s["past"], s["batch"], s["rotary"],
                           s["ws"])
        if s["k_scale"] is None:
            return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        ds.ds_paged_gather(s["cache"], s["k_rows"], s["v_rows"], s["cu"], s["past"], s["batch"], s["ws"])
        return {"q": s["q_out"], "k": s["k_rows"], "v": s["v_rows"]}
    if s["op"] == "decode":
        ds.ds_paged_attention(s["cache"], s["q"], s["out"], s["past"], s["batch"], s["new"], s["ws"], s["ws_bytes"],
                              s["scale"])
    else:
        ds.ds_prompt_attention(s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["cu_k"], s["batch"], s["ws"],
                               s["ws_bytes"], s["scale"])
    return {"out": s["out"]}


# ------------------------------------------------------------------ plain forms
def _to_codes(x):
    """[..., d] in 32 bits -> codes [..., d / 2] (channel 2i in the low bits of byte i) and [..., 2] (scale, minimum)."""
    low = x.amin(-1, keepdim=True).half()
    step = ((x.amax(-1, keepdim=True) - low.float()) / 15).half()
    code = torch.where(step > 0, ((x - low.float()) / step.float()).round().clamp(0, 15), torch.zeros_like(x)).byte()
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([step, low], -1)


def _from_codes(codes, scale):
    x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return x * scale[..., 0:1].float() + scale[..., 1:2].float()


def _rotate(x, cos, sin, neighbours):
    """x [N, heads, d] in 32 bits; cos, sin [N, r / 2]: the first r channels are rotated in pairs."""
    r = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if neighbours else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if neighbours else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _places(s):
    """Position, page and row in the page of each packed token."""
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = s["past"][b] + (t - s["cu"][b])
    return pos, s["table"][b, pos // s["page"]].long(), pos % s["page"]


def _append_plain(s):
    pos, page, row = _places(s)
    angles = s["cos_sin"][pos]
    cos, sin = angles.chunk(2, -1)
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, s["neighbours"]))
    k, v = _rotate(s["k"].float(), cos, sin, s["neighbours"]), s["v"].float()
    if s["k_scale"] is None:
        s["k_pages"][page, :, row] = k.to(s["dtype"])
        s["v_pages"][page, :, row] = v.to(s["dtype"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    s["k_pages"][page, :, row], s["k_scale"][page, :, row] = _to_codes(k)
    s["v_pages"][page, :, row], s["v_scale"][page, :, row] = _to_codes(v)
    s["k_rows"].copy_(_from_codes(s["k_pages"][page, :, row], s["k_scale"][page, :, row]))
    s["v_rows"].copy_(_from_codes(s["v_pages"][page, :, row], s["v_scale"][page, :, row]))
    return {"q": s["q_out"], "k": s["k_rows"], "v": s["v_rows"]}


def _softmax_sum(scores, seen, v):
    """softmax over the last axis where `seen`, times v; zeros where a row sees nothing."""
    scores = torch.where(seen, scores, torch.full_like(scores[..., :1], -math.inf))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, torch.ones_like(total), total)


def _decode_plain(s):
    B, T, P = s["batch"], s["new"], s["page"]
    nh, d = s["q"].shape[1:]
    table = s["table"][:, :-(-s["longest"] // P)].long().clamp(min=0)
    held = []
    for pages, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])):
        x = pages[table].float() if scale is None else _from_codes(pages[table], scale[table])
        held.append(x.transpose(1, 2).flatten(2, 3))  # [B, kv_heads, positions, d]
    k, v = held
    nk, L = k.shape[1], k.shape[2]
    j = torch.arange(L, device="cuda")
    last = s["past"][:, None] + torch.arange(T, device="cuda")  # [B, T]
    v = torch.where((j <= last[:, -1:])[:, None, :, None], v, torch.zeros_like(v[..., :1]))
    q = s["q"].float().view(B, T, nk, nh // nk, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # rows (group, token)
    seen = (j <= last[..., None]).repeat(1, nh // nk, 1)[:, None]
    o = _softmax_sum((q @ k.transpose(-1, -2)) * s["scale"], seen, v)
    s["out"].copy_(o.view(B, nk, nh // nk, T, d).permute(0, 3, 1, 2, 4).reshape(B * T, nh, d))
    return {"out": s["out"]}


def _prompt_plain(s):
    B = s["batch"]
    nh, d = s["q"].shape[1:]
    nk = s["k"].shape[1]
    lq, lk = s["cu_q"].diff(), s["cu_k"].diff()
    i, j = torch.arange(s["longest_q"], device="cuda"), torch.arange(s["longest_k"], device="cuda")
    row_q = (s["cu_q"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()  # padded to the longest
    row_k = (s["cu_k"][:-1, None] + j).clamp(max=s["k"].shape[0] - 1).long()
    q = s["q"][row_q].float().view(B, -1, nk, nh // nk, d).permute(0, 2, 3, 1, 4)  # [B, nk, group, Lq, d]
    k = s["k"][row_k].float().transpose(1, 2)[:, :, None]
    v = s["v"][row_k].float().transpose(1, 2)[:, :, None]
    seen = (j <= (lk - lq)[:, None, None] + i[:, None])[:, None, None]
    o = _softmax_sum((q @ k.transpose(-1, -2)) * s["scale"], seen, v)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, nh, d)
    s["out"].copy_(o[i < lq[:, None]])
    return {"out": s["out"]}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    new, past = _lens(case)
    if case["op"] == "append":
        return _append_exact(case, s, new, past)
    nh, nk, d = case["heads"], case["kv_heads"], case["head_dim"]
    outs, first_q, first_k = [], 0, 0
    for b in range(case["batch"]):
        n, total = new[b], new[b] + past[b]
        q = s["q"][first_q:first_q + n].double()
        if case["op"] == "prompt":
            k, v = s["k"][first_k:first_k + total].double(), s["v"][first_k:first_k + total].double()
        else:
            k, v = (_held_exact(s, x, b, total) for x in "kv")
        o = torch.empty(n, nh, d, dtype=torch.float64, device="cuda")
        later = torch.ones(n, total, dtype=torch.bool, device="cuda").triu(total - n + 1)
        for h in range(nh):
            of = h // (nh // nk)
            w = torch.softmax((q[:, h] @ k[:, of].T / math.sqrt(d)).masked_fill(later, -math.inf), -1)
            o[:, h] = w @ v[:, of]
        outs.append(o)
        first_q += n
        first_k += total
    return {"out": torch.cat(outs)}


def _held_exact(s, x, b, total):
    """Rows 0 .. total-1 of sequence b, in 64 bits: [total, kv_heads, d]."""
    at = s["table"][b, :-(-total // s["page"])].long()
    rows = s[x + "_pages"][at].transpose(1, 2).flatten(0, 1)[:total]
    if s[x + "_scale"] is None:
        return rows.double()
    sc = s[x + "_scale"][at].transpose(1, 2).flatten(0, 1)[:total].double()
    out = torch.empty(*rows.shape[:2], 2 * rows.shape[2], dtype=torch.float64, device="cuda")
    out[..., 0::2], out[..., 1::2] = (rows % 16).double(), (rows // 16).double()
    return out * sc[..., :1] + sc[..., 1:]


def _append_exact(case, s, new, past):
    at = torch.cat([torch.arange(p, p + n, device="cuda") for n, p in zip(new, past)])
    r = case["rotary"]
    turn = torch.complex(s["cos_sin"][at, :r // 2].double(), s["cos_sin"][at, r // 2:].double())[:, None]

    def rotated(x):
        y = x.double().clone()
        if case["neighbours"]:
            z = torch.view_as_complex(y[..., :r].reshape(*y.shape[:2], r // 2, 2).contiguous()) * turn
            y[..., :r] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * turn
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        return y

    q, k, v = rotated(s["q"]), rotated(s["k"]), s["v"].double()
    if case["cache"] == "4":
        rows = []
        for x in (k, v):
            m = x.amin(-1, keepdim=True).half().double()
            step = ((x.amax(-1, keepdim=True) - m) / 15).half().double()
            rows.append(torch.clamp(torch.round((x - m) / torch.where(step > 0, step, 1.0)), 0, 15) * step + m)
        return {"q": q, "k": rows[0], "v": rows[1]}
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    first = 0
    for b in range(case["batch"]):
        for t in range(0, new[b]):
            p = past[b] + t
            if t == 0 or p % s["page"] == 0:  # the rest of this page in one piece
                n = min(s["page"] - p % s["page"], new[b] - t)
                pg, row = int(s["table"][b, p // s["page"]]), p % s["page"]
                kp[pg, :, row:row + n] = k[first + t:first + t + n].transpose(0, 1)
                vp[pg, :, row:row + n] = v[first + t:first + t + n].transpose(0, 1)
        first += new[b]
    return {"q": q, "k_pages": kp, "v_pages": vp}

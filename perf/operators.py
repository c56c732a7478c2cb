"""Measured cases of the serving operators around the 8-bit KV cache: rotary
positions, page tables from request lengths, placement into and attention over a
cache held in 8 bits with one scale per page of 16 tokens and KV head.

``run`` computes a case either in plain torch operations (``own`` false) or with
the library's calls (``own`` true).  The state of a case holds the buffers a
serving loop keeps: pools in the library's block layout, tables, lengths, inputs,
outputs and workspaces.

Cache layout (d = head dim, page = 16 tokens).  The block of (page, KV head) has
32*d + 16 bytes: key codes, value codes, then the fp32 key scale and value scale
and 8 spare bytes.  Key code (t, c) of an area lies at
  (((c/64)*2 + t%2)*32 + 4*(t/2) + (c/16)%4)*16 + c%16,
value code (t, c) at
  ((c/32)*32 + 4*((c/4)%8) + t/4)*16 + 4*(c%4) + t%4.
int8 codes are stored plus 128, e4m3 codes as they are; a value is code * scale.
The last L % 16 tokens of a sequence lie in its bf16 tail block (keys, values),
in the same order of elements.
"""
import math

import torch

own = False

PAGE = 16
DEV = "cuda"


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one sequence: the smallest call of a decode loop
        dict(name="rope decode 1", op="rope", n=1, hq=32, hkv=8, d=128, rd=128, inter=False,
             parts=False, ctx=32768),
        # a packed prefill of prompts that add up to an odd number of tokens
        dict(name="rope prefill 16411", op="rope", n=16411, hq=32, hkv=8, d=128, rd=128,
             inter=False, parts=False, ctx=32768),
        # half of each head rotated, neighbouring pairs, frequencies scaled for 128k positions
        dict(name="rope part of head 5003", op="rope", n=5003, hq=64, hkv=8, d=128, rd=64,
             inter=True, parts=True, ctx=131072),
        # one decode step of 256 sequences: most get no new page
        dict(name="pages decode 256", op="pages", batch=256, lo=1, hi=1, stored=4096, hold=15),
        # 256 prompts of up to 4096 tokens admitted at once
        dict(name="pages prefill 256x4096", op="pages", batch=256, lo=2048, hi=4096, stored=0,
             hold=0),
        # decode append of 64 sequences (one in 16 completes a page)
        dict(name="place append 64", op="place", batch=64, lo=1, hi=1, stored=6000, hkv=8, d=128,
             e4m3=False),
        # prompts of ragged lengths placed at once, read back for another kernel
        dict(name="place prefill 32x4096", op="place", batch=32, lo=3001, hi=4096, stored=0, hkv=8,
             d=128, e4m3=True),
        # a short context with one KV head: launch latency
        dict(name="attention 512 d64", op="attend", batch=1, rows=1, lo=512, hi=512, hq=4, hkv=1,
             d=64, e4m3=False),
        # Qwen3-8B shape at 32k, batch 1
        dict(name="attention 32k", op="attend", batch=1, rows=1, lo=32768, hi=32768, hq=32, hkv=8,
             d=128, e4m3=False),
        # Qwen3-4B shape, 64 sequences of 4096 to 8192 tokens
        dict(name="attention b64", op="attend", batch=64, rows=1, lo=4096, hi=8192, hq=32, hkv=8,
             d=128, e4m3=True),
        # Qwen3-32B shape at 128k, batch 1
        dict(name="attention 128k", op="attend", batch=1, rows=1, lo=131071, hi=131071, hq=64,
             hkv=8, d=128, e4m3=True),
        # a chunk of 65 rows per sequence after a long prefix (chunked prefill, verification)
        dict(name="attention 65 rows", op="attend", batch=4, rows=65, lo=6000, hi=16385, hq=32,
             hkv=8, d=128, e4m3=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "pages", "place", "attend", "attend"])
    g, hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "rope":
        half = rng.randint(4, d // 2)
        return dict(op=op, n=_log(rng, 1, 16000), hq=g * hkv, hkv=hkv, d=d,
                    rd=rng.choice([d, 2 * half]), inter=rng.random() < 0.5,
                    parts=rng.random() < 0.5, ctx=_log(rng, 20000, 1000000))
    if op == "pages":
        hi = _log(rng, 1, 4096)
        return dict(op=op, batch=_log(rng, 1, 256), lo=rng.randint(0, hi), hi=hi,
                    stored=_log(rng, 1, 20000), hold=rng.choice([0, 15, 128]))
    if op == "place":
        one = rng.random() < 0.4
        hi = 1 if one else _log(rng, 2, 4096)
        return dict(op=op, batch=_log(rng, 1, 32), lo=1 if one else rng.randint(1, hi), hi=hi,
                    stored=_log(rng, 1, 8000) if one else 16 * rng.randint(0, 100), hkv=hkv, d=d,
                    e4m3=rng.random() < 0.5)
    rows = rng.choice([1, 1, 1, rng.randint(2, 9), rng.randint(10, 80)])
    batch = _log(rng, 1, 48)
    hi = _log(rng, 64, max(64, min(100000, 400000 // (batch * (1 if rows == 1 else 6)))))
    return dict(op=op, batch=batch, rows=rows, lo=rng.randint(max(1, hi // 3), hi), hi=hi,
                hq=g * hkv, hkv=hkv, d=d, e4m3=rng.random() < 0.5)


# ------------------------------------------------------------------ the states

def _lens(case, g):
    """Ragged lengths in [lo, hi]: the same ones for every seed (so that packed rows
    number the same), in an order of the seed's."""
    own_rng = _host_rng(case["batch"] * 1000003 + case["lo"] * 8191 + case["hi"])
    n = torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=own_rng,
                      dtype=torch.int32)
    return n[torch.randperm(case["batch"], generator=g)]


def _host_rng(seed):
    g = torch.Generator()
    g.manual_seed(int(seed))
    return g


def _device_rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _keys_values(n, hkv, d, gen):
    """bf16 keys and values [n][hkv][d]: a spread of each channel's own, four strong
    key channels per head with an offset, two strong value channels."""
    out = []
    for outliers, mult, offset in ((4, 15.0, 3.0), (2, 6.0, 0.0)):
        sigma = torch.exp(0.5 * torch.randn(hkv, d, generator=gen, device=DEV))
        shift = torch.zeros(hkv, d, device=DEV)
        strong = torch.rand(hkv, d, generator=gen, device=DEV).argsort(-1)[:, :outliers]
        sigma.scatter_(1, strong, sigma.gather(1, strong) * mult)
        shift.scatter_(1, strong, offset)
        x = torch.randn(n, hkv, d, generator=gen, device=DEV, dtype=torch.bfloat16)
        out.append((x.float() * sigma + shift).bfloat16())
    return out


def _encode(x, e4m3):
    """[pages, 16, hkv, d] bf16 -> codes [pages, hkv, 16, d] uint8, scales [pages, hkv]."""
    x = x.float().permute(0, 2, 1, 3)
    top = 448.0 if e4m3 else 127.0
    amax = x.abs().amax((2, 3))
    live = amax >= 2.0 ** -100
    tops = torch.full_like(amax, top)     # tensor by tensor: correctly rounded quotients
    scale = torch.where(live, amax / tops, 0.0)
    inv = torch.where(live, tops / torch.where(live, amax, 1.0), 0.0)
    y = (x * inv[:, :, None, None]).clamp(-top, top)
    if e4m3:
        return y.to(torch.float8_e4m3fn).view(torch.uint8), scale
    return (torch.round(y) + 128.0).to(torch.uint8), scale


def _key_order(x):
    """[n, hkv, 16, d] -> [n, hkv, 16 * d] in the order of a block's key area."""
    n, h, _, d = x.shape
    return x.view(n, h, 8, 2, d // 64, 4, 16).permute(0, 1, 4, 3, 2, 5, 6).reshape(n, h, 16 * d)


def _value_order(x):
    n, h, _, d = x.shape
    return x.view(n, h, 4, 4, d // 32, 8, 4).permute(0, 1, 4, 5, 2, 6, 3).reshape(n, h, 16 * d)


def _key_tokens(a, d):
    """The inverse of _key_order: [n, hkv, 16 * d] -> [n, hkv, 16, d]."""
    n, h = a.shape[:2]
    return a.view(n, h, d // 64, 2, 8, 4, 16).permute(0, 1, 4, 3, 2, 5, 6).reshape(n, h, 16, d)


def _value_tokens(a, d):
    n, h = a.shape[:2]
    return a.view(n, h, d // 32, 8, 4, 4, 4).permute(0, 1, 4, 6, 2, 3, 5).reshape(n, h, 16, d)


def _fill_pages(k, v, e4m3):
    """Blocks [pages, hkv, 32 * d + 16] uint8 of keys and values [pages, 16, hkv, d]."""
    n, _, h, d = k.shape
    pool = torch.zeros(n, h, 32 * d + 16, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, h, 4, dtype=torch.float32, device=DEV)
    kc, scales[:, :, 0] = _encode(k, e4m3)
    vc, scales[:, :, 1] = _encode(v, e4m3)
    pool[:, :, :16 * d] = _key_order(kc)
    pool[:, :, 16 * d:32 * d] = _value_order(vc)
    pool[:, :, 32 * d:] = scales.view(torch.uint8)
    return pool


def _table(pages_of, max_pages, gen):
    """Page table [batch][max_pages] of shuffled ids, -1 behind a sequence's pages."""
    pages_of = pages_of.to(DEV)
    total = max(1, int(pages_of.sum()))
    ids = torch.randperm(total, generator=gen, device=DEV).int()
    p = torch.arange(max_pages, device=DEV)
    live = p[None, :] < pages_of[:, None]
    first = pages_of.cumsum(0) - pages_of
    return torch.where(live, ids[(first[:, None] + p).clamp(max=total - 1)], -1).int(), total


def prepare(case, seed):
    return {"rope": _prepare_rope, "pages": _prepare_pages, "place": _prepare_place,
            "attend": _prepare_attend}[case["op"]](case, seed)


def _prepare_rope(case, seed):
    gen = _device_rng(seed)
    n, hq, hkv, d, rd = (case[k] for k in ("n", "hq", "hkv", "d", "rd"))
    # queries and keys are columns of the projection's output [n][(hq + 2 hkv) * d]
    qkv = torch.randn(n, hq + 2 * hkv, d, generator=gen, device=DEV).bfloat16()
    i = torch.arange(rd // 2, dtype=torch.float64)
    freq = 1e6 ** (-2.0 * i / rd)
    amplitude = 1.0
    if case["parts"]:   # frequencies of fewer than 1 turn in 32768 tokens divided by 4
        turns = 32768.0 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        freq = (1 - keep) * freq / 4.0 + keep * freq
        amplitude = 0.1 * math.log(4.0) + 1.0
    phases = torch.round(freq / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(DEV)
    pos = torch.randint(0, case["ctx"], (n,), generator=gen, device=DEV, dtype=torch.int32)
    out = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
    kout = torch.empty(n, hkv, d, dtype=torch.bfloat16, device=DEV)
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], pos=pos, phases=phases,
                amplitude=amplitude, q_out=out, k_out=kout)


def _prepare_pages(case, seed):
    g, gen = _host_rng(seed), _device_rng(seed)
    b = case["batch"]
    new = _lens(case, g)
    lens = torch.randint(0, case["stored"] + 1, (b,), generator=g, dtype=torch.int32)
    after = lens + new
    held = lambda n: ((n - case["hold"] + PAGE - 1).clamp(min=0) // PAGE).int()  # noqa: E731
    max_pages = -(-(case["stored"] + case["hi"]) // PAGE) + 1
    table, used = _table(held(lens), max_pages, gen)
    need = int((held(after) - held(lens)).sum())
    free = (used + torch.randperm(need + 17, generator=gen, device=DEV)).int()
    total = int(new.sum())
    rows = total + 3      # a captured loop's row buffers are larger than one step's rows
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(case=case, table=table, lens=lens.to(DEV), new=new.to(DEV), free=free,
                cursor=torch.tensor([5], **i32), lens_after=torch.empty(b, **i32),
                page_starts=torch.empty(b + 1, **i32), row_starts=torch.empty(b + 1, **i32),
                seq_ids=torch.empty(rows, **i32), positions=torch.empty(rows, **i32),
                slots=torch.empty(rows, dtype=torch.int64, device=DEV),
                status=torch.zeros(1, **i32))


def _prepare_place(case, seed):
    g, gen = _host_rng(seed), _device_rng(seed)
    b, hkv, d = case["batch"], case["hkv"], case["d"]
    new = _lens(case, g)
    if case["hi"] == 1:   # a decode step finds sequences at any length
        before = torch.randint(0, case["stored"] + 1, (b,), generator=g, dtype=torch.int32)
    else:                 # a prompt, or a chunk behind whole pages
        before = 16 * torch.randint(0, case["stored"] // 16 + 1, (b,), generator=g, dtype=torch.int32)
    after = before + new
    # read back from the start of the page that the first new token falls in
    first = before // PAGE * PAGE
    starts, back_starts = (torch.zeros(b + 1, dtype=torch.int32) for _ in range(2))
    starts[1:] = new.cumsum(0)
    back_starts[1:] = (after - first).cumsum(0)
    back_rows = PAGE * b if case["hi"] == 1 else int(new.sum())
    k, v = _keys_values(int(new.sum()), hkv, d, gen)
    max_pages = max(1, int(after.max()) // PAGE)
    table, total = _table(after // PAGE, max_pages, gen)
    tk, tv = _keys_values(b * PAGE, hkv, d, gen)
    tail = torch.stack([_key_order(tk.view(b, PAGE, hkv, d).permute(0, 2, 1, 3)),
                        _value_order(tv.view(b, PAGE, hkv, d).permute(0, 2, 1, 3))], 2)
    return dict(case=case, k=k, v=v, before=before.to(DEV), after=after.to(DEV),
                starts=starts.to(DEV), table=table, tail=tail.contiguous(),
                pool=torch.zeros(total, hkv, 32 * d + 16, dtype=torch.uint8, device=DEV),
                first=first.to(DEV), back_starts=back_starts.to(DEV),
                k_back=torch.zeros(back_rows, hkv, d, dtype=torch.bfloat16, device=DEV),
                v_back=torch.zeros(back_rows, hkv, d, dtype=torch.bfloat16, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_attend(case, seed):
    g, gen = _host_rng(seed), _device_rng(seed)
    b, hq, hkv, d, m = (case[k] for k in ("batch", "hq", "hkv", "d", "rows"))
    lens = _lens(case, g)
    max_pages = max(1, -(-int(case["hi"]) // PAGE))
    table, total = _table(lens // PAGE, max_pages, gen)
    k, v = _keys_values(total * PAGE, hkv, d, gen)
    pool = _fill_pages(k.view(total, PAGE, hkv, d), v.view(total, PAGE, hkv, d), case["e4m3"])
    del k, v
    tk, tv = _keys_values(b * PAGE, hkv, d, gen)
    tail = torch.stack([_key_order(tk.view(b, PAGE, hkv, d).permute(0, 2, 1, 3)),
                        _value_order(tv.view(b, PAGE, hkv, d).permute(0, 2, 1, 3))], 2)
    decay = 0.9 ** (0.5 * torch.arange(d, device=DEV))
    q = (torch.randn(b, m, hq, d, generator=gen, device=DEV) * decay).bfloat16()
    # the rows are the sequence's last tokens; rows of sequences that are too short see nothing
    pos = lens[:, None] - m + torch.arange(m, dtype=torch.int32)[None, :]
    pos = torch.where(pos < 0, -1, pos).int()
    ws = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    return dict(case=case, q=q if m > 1 else q[:, 0], lens=lens.to(DEV), pos=pos.to(DEV),
                table=table, pool=pool, tail=tail.contiguous(), out=torch.empty_like(q), ws=ws,
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


# -------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "pages": _own_pages, "place": _own_place,
                "attend": _own_attend}[op](state)
    return {"rope": _plain_rope, "pages": _plain_pages, "place": _plain_place,
            "attend": _plain_attend}[op](state)


def _library():
    from int2_rotated_kv_gb300 import oscar
    return oscar


def _cache(s, hq):
    """The binding's descriptor of a state's cache, kept beside its buffers."""
    c = s.get("cache")
    if c is None:
        oscar = _library()
        case = s["case"]
        c = s["cache"] = oscar.Kv8Cache(
            case["hkv"], hq, case["d"], s["pool"], s["tail"], s["table"],
            fmt=oscar.KV8_E4M3 if case["e4m3"] else oscar.KV8_INT8, status=s["status"])
    return c


def _own_rope(s):
    _library().oscar_rope(s["q"], s["k"], s["pos"], s["phases"], s["q_out"], s["k_out"],
                          interleaved=s["case"]["inter"], amplitude=s["amplitude"])
    return s["q_out"], s["k_out"]


def _own_pages(s):
    _library().oscar_extend_pages(s["table"], s["lens"], s["new"], s["free"], s["cursor"],
                                  s["lens_after"], s["page_starts"], s["row_starts"], s["seq_ids"],
                                  s["positions"], s["slots"], hold_back=s["case"]["hold"],
                                  status=s["status"])
    return (s["table"], s["lens_after"], s["page_starts"], s["row_starts"], s["seq_ids"],
            s["positions"], s["slots"])


def _own_place(s):
    oscar, c = _library(), _cache(s, s["case"]["hkv"])
    oscar.oscar_kv8_place(c, s["k"], s["v"], s["before"], s["starts"], s["case"]["hi"])
    oscar.oscar_kv8_gather(c, s["after"], s["first"], s["back_starts"],
                           max(PAGE, s["case"]["hi"]), s["k_back"], s["v_back"])
    return s["k_back"], s["v_back"]


def _own_attend(s):
    case = s["case"]
    _library().oscar_kv8_attention(_cache(s, case["hq"]), s["q"], s["lens"], case["hi"],
                                   s["out"] if case["rows"] > 1 else s["out"][:, 0], s["ws"],
                                   q_pos=s["pos"] if case["rows"] > 1 else None)
    return s["out"]


def _plain_rope(s):
    case = s["case"]
    rd, half = case["rd"], case["rd"] // 2
    turns = s["phases"].double() * 2.0 ** -64 * s["pos"].double()[:, None]
    angle = (turns - torch.round(turns)) * (2 * math.pi)
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]

    def rotate(x, out):
        y = x.float()
        if case["inter"]:
            a, b = y[..., 0:rd:2], y[..., 1:rd:2]
            pair = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rd]
            pair = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out.copy_(torch.cat([pair, y[..., rd:]], -1))
        return out

    return rotate(s["q"], s["q_out"]), rotate(s["k"], s["k_out"])


def _plain_pages(s):
    hold, b = s["case"]["hold"], s["case"]["batch"]
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"]
    after = lens + new
    old_pages = (lens - hold + PAGE - 1).clamp(min=0) // PAGE
    new_pages = (after - hold + PAGE - 1).clamp(min=0) // PAGE
    page_starts = torch.cat([s["cursor"].long(), s["cursor"].long() + (new_pages - old_pages).cumsum(0)])
    p = torch.arange(table.shape[1], device=DEV)
    fresh = (p[None] >= old_pages[:, None]) & (p[None] < new_pages[:, None])
    at = (page_starts[:-1, None] + p[None] - old_pages[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    row_starts = torch.cat([torch.zeros_like(lens[:1]), new.cumsum(0)])
    row = torch.arange(s["seq_ids"].numel(), device=DEV)
    seq = torch.searchsorted(row_starts[1:], row, right=True)
    live = seq < b
    seq = seq.clamp(max=b - 1)
    pos = lens[seq] + row - row_starts[seq]
    page = (pos // PAGE).clamp(max=table.shape[1] - 1)
    held = live & (pos // PAGE < new_pages[seq])
    slots = torch.where(held, table[seq, page].long() * PAGE + pos % PAGE, -1)
    return (table, after.int(), page_starts.int(), row_starts.int(),
            torch.where(live, seq, -1).int(), torch.where(live, pos, -1).int(), slots)


def _values(area, e4m3):
    return area.view(torch.float8_e4m3fn).float() if e4m3 else area.float() - 128.0


def _plain_place(s):
    case = s["case"]
    hkv, d, e4m3 = case["hkv"], case["d"], case["e4m3"]
    before, after, starts, table = (s[k].long() for k in ("before", "after", "starts", "table"))
    n = s["k"].shape[0]
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(starts[1:], row, right=True)
    pos = before[seq] + row - starts[seq]
    full = (after // PAGE)[seq]
    # every page that these tokens complete, with all of its 16 tokens: from the rows, or from the tail
    last = row[(pos % PAGE == PAGE - 1) & (pos // PAGE < full)]
    b, top = seq[last], pos[last]
    slot = torch.arange(PAGE, device=DEV)
    src = last[:, None] - (PAGE - 1) + slot[None]
    tail_k = _key_tokens(s["tail"][:, :, 0], d).permute(0, 2, 1, 3)
    tail_v = _value_tokens(s["tail"][:, :, 1], d).permute(0, 2, 1, 3)
    old = (top[:, None] - (PAGE - 1) + slot[None] < before[b][:, None])[:, :, None, None]
    src = src.clamp(min=0)
    pages = table[b, top // PAGE]
    s["pool"][pages] = _fill_pages(torch.where(old, tail_k[b], s["k"][src]),
                                   torch.where(old, tail_v[b], s["v"][src]), e4m3)
    # the tokens behind the last whole page
    rest = row[pos // PAGE >= full]
    tail_k = tail_k.clone()
    tail_v = tail_v.clone()
    tail_k[seq[rest], pos[rest] % PAGE] = s["k"][rest]
    tail_v[seq[rest], pos[rest] % PAGE] = s["v"][rest]
    s["tail"][:, :, 0] = _key_order(tail_k.permute(0, 2, 1, 3))
    s["tail"][:, :, 1] = _value_order(tail_v.permute(0, 2, 1, 3))
    # and back: each token from the page that was completed, or from the tail
    block = s["pool"][pages]
    scale = block[:, :, 32 * d:].contiguous().view(torch.float32)
    k_page = _values(_key_tokens(block[:, :, :16 * d].contiguous(), d), e4m3) * scale[:, :, 0, None, None]
    v_page = _values(_value_tokens(block[:, :, 16 * d:32 * d].contiguous(), d), e4m3) * scale[:, :, 1, None, None]
    back = torch.arange(s["k_back"].shape[0], device=DEV)
    seq = torch.searchsorted(s["back_starts"][1:].long(), back, right=True)
    back, seq = back[seq < case["batch"]], seq[seq < case["batch"]]
    pos = s["first"].long()[seq] + back - s["back_starts"].long()[seq]
    paged = pos // PAGE < (after // PAGE)[seq]
    number = torch.zeros_like(table)
    number[b, top // PAGE] = torch.arange(last.numel(), device=DEV)
    at = number[seq[paged], pos[paged] // PAGE]
    s["k_back"][back[paged]] = k_page[at, :, pos[paged] % PAGE].bfloat16()
    s["v_back"][back[paged]] = v_page[at, :, pos[paged] % PAGE].bfloat16()
    s["k_back"][back[~paged]] = tail_k[seq[~paged], pos[~paged] % PAGE]
    s["v_back"][back[~paged]] = tail_v[seq[~paged], pos[~paged] % PAGE]
    return s["k_back"], s["v_back"]


def _plain_attend(s):
    case = s["case"]
    b, m, hq, hkv, d, e4m3 = (case[k] for k in ("batch", "rows", "hq", "hkv", "d", "e4m3"))
    lens, table = s["lens"].long(), s["table"].long()
    pages = table.shape[1]
    block = s["pool"][table.clamp(min=0).view(-1)]
    scale = block[:, :, 32 * d:].contiguous().view(torch.float32)
    t = torch.arange(pages * PAGE, device=DEV)
    whole = (lens // PAGE * PAGE)[:, None]
    slot = torch.arange(PAGE, device=DEV)
    pos = torch.cat([torch.where(t[None] < whole, t[None], 1 << 30),
                     torch.where(whole + slot[None] < lens[:, None], whole + slot[None], 1 << 30)], 1)
    limit = s["pos"].long() if m > 1 else lens[:, None] - 1
    seen = pos[:, None, :] <= limit[:, :, None]                     # [b, m, tokens]

    def tokens(area, scales, order, tail):
        x = _values(order(area.contiguous(), d), e4m3) * scales[:, :, None, None]
        x = x.view(b, pages, hkv, PAGE, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, pages * PAGE, d)
        x = torch.cat([x, order(tail.contiguous(), d).float()], 2)
        return torch.where((pos < (1 << 30))[:, None, :, None], x, 0.0)

    k = tokens(block[:, :, :16 * d], scale[:, :, 0], _key_tokens, s["tail"][:, :, 0])
    q = s["q"].float().view(b, m, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    logits = q @ k.transpose(-1, -2) / math.sqrt(d)
    del k
    logits = logits.view(b, hkv, m, hq // hkv, -1).masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    v = tokens(block[:, :, 16 * d:32 * d], scale[:, :, 1], _value_tokens, s["tail"][:, :, 1])
    o = (p.view(b, hkv, m * (hq // hkv), -1) @ v).view(b, hkv, m, hq // hkv, d)
    o = torch.where(total > 0, o / total, 0.0)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(b, m, hq, d))
    return s["out"]


# ----------------------------------------------------------------------- floors

def work(case):
    op = case["op"]
    if op == "rope":
        heads = case["n"] * (case["hq"] + case["hkv"])
        return {"bytes": heads * case["d"] * 4 + 4 * case["n"] + 4 * case["rd"],
                "flops": heads * case["rd"] * 3}
    if op == "pages":
        b, rows = case["batch"], case["batch"] * (case["lo"] + case["hi"]) / 2
        pages = rows / PAGE
        return {"bytes": 8 * b + 12 * b + pages * 8 + rows * 16, "flops": rows}
    if op == "place":
        tokens = case["batch"] * (case["lo"] + case["hi"]) / 2
        # an append's page is read back whole: half of one, on average
        back = tokens if case["hi"] > 1 else case["batch"] * (PAGE + 1) / 2
        width = case["hkv"] * case["d"] * 2
        # bf16 in, codes out; codes in, bf16 out
        return {"bytes": width * (tokens * (2 + 1) + back * (1 + 2)),
                "flops": width * (tokens * 3 + back)}
    tokens = case["batch"] * (case["lo"] + case["hi"]) / 2
    rows = case["batch"] * case["rows"] * case["hq"]
    return {"bytes": tokens * case["hkv"] * (2 * case["d"] + 1) + rows * case["d"] * 4,
            "flops": 4.0 * tokens * case["rows"] * case["hq"] * case["d"]}


# ------------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "pages": _exact_pages, "place": _exact_place,
            "attend": _exact_attend}[case["op"]](s)


def _exact_rope(s):
    case = s["case"]
    rd, inter = case["rd"], case["inter"]
    i = torch.arange(rd // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    turns = torch.frac(s["pos"].double()[:, None] * (s["phases"].double() / 2.0 ** 64)[None])
    unit = torch.polar(torch.full_like(turns, s["amplitude"]), 2 * math.pi * turns)[:, None]

    def rotate(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return rotate(s["q"]), rotate(s["k"])


def _exact_pages(s):
    """The same lists built sequence by sequence."""
    hold, free = s["case"]["hold"], s["free"].cpu()
    table, lens, new = s["table"].cpu().clone(), s["lens"].tolist(), s["new"].tolist()
    at, row = int(s["cursor"]), 0
    rows = s["seq_ids"].numel()
    seq_ids, positions = (torch.full((rows,), -1, dtype=torch.int32) for _ in range(2))
    slots = torch.full((rows,), -1, dtype=torch.int64)
    page_starts, row_starts = [at], [0]
    for b, (old, more) in enumerate(zip(lens, new)):
        lo, hi = (max(0, -((hold - n) // PAGE)) for n in (old, old + more))
        table[b, lo:hi] = free[at:at + hi - lo]
        at += hi - lo
        pos = torch.arange(old, old + more)
        seq_ids[row:row + more] = b
        positions[row:row + more] = pos.int()
        held = pos < hi * PAGE
        slots[row:row + more][held] = table[b, pos[held] // PAGE].long() * PAGE + pos[held] % PAGE
        row += more
        page_starts.append(at)
        row_starts.append(row)
    after = torch.tensor([a + n for a, n in zip(lens, new)], dtype=torch.int32)
    return (table, after, torch.tensor(page_starts, dtype=torch.int32),
            torch.tensor(row_starts, dtype=torch.int32), seq_ids, positions, slots)


def _nearest_e4m3(y):
    """|y| <= 448 to the nearest multiple of its binade's step, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _element(d, value):
    """Index of (token, channel) in a key or value area, [16, d]."""
    t = torch.arange(PAGE, device=DEV)[:, None]
    c = torch.arange(d, device=DEV)[None, :]
    if value:
        return (c // 32 * 32 + 4 * (c // 4 % 8) + t // 4) * 16 + 4 * (c % 4) + t % 4
    return ((c // 64 * 2 + t % 2) * 32 + 4 * (t // 2) + c // 16 % 4) * 16 + c % 16


def _exact_place(s):
    """Each token's 16-token page worked out on its own: the page's largest value, the
    scale and its reciprocal in 32 bits as the format defines them, the rest in 64."""
    case = s["case"]
    d, top = case["d"], 448.0 if case["e4m3"] else 127.0
    starts, back_starts, before, after = (s[k].tolist() for k in ("starts", "back_starts", "before", "after"))
    out = []
    for which, rows in ((0, s["k"]), (1, s["v"])):
        back = torch.zeros(s["k_back"].shape, dtype=torch.float64, device=DEV)
        el = _element(d, which == 1)
        for b in range(case["batch"]):
            n_old = before[b] % PAGE
            old = s["tail"][b, :, which][:, el[:n_old]].permute(1, 0, 2).double()
            y = torch.cat([old, rows[starts[b]:starts[b + 1]].double()])
            whole = len(y) // PAGE * PAGE
            x = y[:whole].view(-1, PAGE, case["hkv"], d)
            amax = x.abs().amax((1, 3), keepdim=True)
            live = amax >= 2.0 ** -100
            safe = torch.where(live, amax, 1.0)
            tops = torch.full_like(safe, top)
            z = (x * (tops / safe).float().double()).float().double().clamp(-top, top)
            code = _nearest_e4m3(z) if case["e4m3"] else torch.round(z)
            z = torch.where(live, code * (safe / tops).float().double(), 0.0)
            y[:whole] = z.view(whole, case["hkv"], d)
            back[back_starts[b]:back_starts[b + 1]] = y
        out.append(back)
    return tuple(out)


def _exact_attend(s):
    case = s["case"]
    b, m, hq, hkv, d, e4m3 = (case[k] for k in ("batch", "rows", "hq", "hkv", "d", "e4m3"))
    if m * case["hi"] * hq * b > 2 ** 31:
        return None
    q = s["q"].double().view(b, m, hkv, hq // hkv, d)
    out = torch.zeros(b, m, hkv, hq // hkv, d, dtype=torch.float64, device=DEV)
    key_el, value_el = _element(d, False), _element(d, True) + 16 * d

    def codes(area):
        return area.view(torch.float8_e4m3fn).double() if e4m3 else area.double() - 128.0

    for i, n in enumerate(s["lens"].tolist()):
        block = s["pool"][s["table"][i, :n // PAGE].long()]
        scale = block[:, :, 32 * d:].contiguous().view(torch.float32).double()
        limit = s["pos"][i].long() if m > 1 else torch.tensor([n - 1], device=DEV)
        hidden = torch.arange(n, device=DEV)[None] > limit[:, None]
        for h in range(hkv):
            k = (codes(block[:, h][:, key_el]) * scale[:, h, 0, None, None]).view(-1, d)
            v = (codes(block[:, h][:, value_el]) * scale[:, h, 1, None, None]).view(-1, d)
            tail = s["tail"][i, h].double()
            k = torch.cat([k, tail[0][key_el[:n % PAGE]]])
            v = torch.cat([v, tail[1][value_el[:n % PAGE] - 16 * d]])
            w = torch.einsum("mgd,td->gmt", q[i, :, h], k) * d ** -0.5
            w = torch.softmax(w.masked_fill(hidden[None], -math.inf), -1).nan_to_num(0.0)
            out[i, :, h] = torch.einsum("gmt,td->mgd", w, v)
    return out.view(b, m, hq, d)

"""Measured cases of the 4-bit KV cache (place, read back, attend) and of reading the
calibrated INT2/INT4 cache back.

``run`` computes a case either in plain torch operations (``own`` false) or with the
library's calls (``own`` true).  The state of a case holds the buffers a serving loop
keeps: pools in the library's block layouts, tables, lengths, inputs, outputs and
workspaces.

4-bit cache (d = head dim, page = 16 tokens): a value is code * block scale * page scale, code
an e2m1 number, 16 codes to a block with an e4m3 scale.  A block of keys is one channel of
the page's 16 tokens, a block of values 16 channels of one token; the page scale (fp32, one
for keys and one for values of a page and KV head) is max|x| / 2688.  Bytes of (page, KV head):
  [0, 8d) key codes: (t, c) in chunk (c/64)*32 + 4*(t/2) + (c/16)%4 of 16 bytes, byte
    8*(t%2) + (c%16)/2, low nibble for even c;
  [8d, 16d) value codes: (t, c) in chunk (c/64)*32 + 4*((c/4)%8) + t/4, byte
    8*((c/32)%2) + 2*(c%4) + (t%4)/2, low nibble for even t;
  [16d, 17d) key scales by channel;
  [17d, 18d) value scales: (t, b = c/16) at (b/4)*64 + ((b%2)*4 + t/4)*8 + ((b/2)%2)*4 + t%4;
  then the fp32 key scale and value scale and 8 spare bytes.
The last L % 16 tokens of a sequence lie in its bf16 tail block (16*d keys, 16*d values): key
(t, c) at (((c/64)*2 + t%2)*32 + 4*(t/2) + (c/16)%4)*16 + c%16, value (t, c) at
((c/32)*32 + 4*((c/4)%8) + t/4)*16 + 4*(c%4) + t%4.

Calibrated cache: include/oscar.h and csrc/layout.cuh have its blocks; tokens t < sink and t >=
L - window of a sequence of L tokens are bf16 as they came, the others codes of x R.
"""
import math

import torch

own = False

PAGE = 16
DEV = "cuda"
SINK, WINDOW = 4, 128


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # decode append of 64 sequences (one in 16 completes a page), the page read back
        dict(name="place append 64", op="place", batch=64, lo=1, hi=1, stored=9000, hkv=8, d=128),
        # prompts of ragged lengths placed at once, read back for another kernel
        dict(name="place prefill 24x5000", op="place", batch=24, lo=2500, hi=5000, stored=0, hkv=8,
             d=128),
        # a short prefix read back: launch latency
        dict(name="read back 777", op="back", batch=1, lo=777, hi=777, hkv=2, d=64),
        # prefixes moved out of the cache, every other one from its fifth part on
        dict(name="read back 16x8192", op="back", batch=16, lo=4097, hi=8192, hkv=8, d=128),
        # a short context with one KV head: launch latency
        dict(name="attention 600 d64", op="attend", batch=1, rows=1, lo=600, hi=600, hq=4, hkv=1,
             d=64),
        # Qwen3-8B shape at 32k, batch 1
        dict(name="attention 32k", op="attend", batch=1, rows=1, lo=32768, hi=32768, hq=32, hkv=8,
             d=128),
        # Qwen3-4B shape, 64 sequences of 4096 to 8192 tokens
        dict(name="attention b64", op="attend", batch=64, rows=1, lo=4096, hi=8192, hq=32, hkv=8,
             d=128),
        # Qwen3-32B shape at 128k, batch 1
        dict(name="attention 128k", op="attend", batch=1, rows=1, lo=131071, hi=131071, hq=64,
             hkv=8, d=128),
        # five rows of each of 16 sequences at once (verification of drafted tokens)
        dict(name="attention 16x5 rows", op="attend", batch=16, rows=5, lo=2000, hi=9001, hq=32,
             hkv=8, d=128),
        # a chunk of a prompt behind a long prefix (chunked prefill)
        dict(name="attention 1000 rows", op="attend", batch=1, rows=1000, lo=17000, hi=17000, hq=32,
             hkv=8, d=128),
        # one sequence of the calibrated cache read back (INT2), d = 64
        dict(name="uncode 1x2000 int2", op="uncode", batch=1, lo=2000, hi=2000, hkv=4, d=64, bits=2),
        # sequences of the calibrated cache read back (INT4)
        dict(name="uncode 16x4096 int4", op="uncode", batch=16, lo=2048, hi=4096, hkv=8, d=128,
             bits=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["place", "back", "attend", "attend", "uncode"])
    g, hkv, d = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "place":
        one = rng.random() < 0.4
        hi = 1 if one else _log(rng, 2, 3700)
        return dict(op=op, batch=_log(rng, 1, 24), lo=1 if one else rng.randint(1, hi), hi=hi,
                    stored=_log(rng, 1, 8000) if one else 16 * rng.randint(0, 100), hkv=hkv, d=d)
    if op in ("back", "uncode"):
        batch = _log(rng, 1, 32)
        hi = _log(rng, 8, max(8, min(8192, 45000 // batch)))
        case = dict(op=op, batch=batch, lo=rng.randint(max(1, hi // 2), hi), hi=hi, hkv=hkv, d=d)
        return dict(case, bits=rng.choice([2, 4])) if op == "uncode" else case
    rows = rng.choice([1, 1, 1, rng.randint(2, 9), rng.randint(10, 80)])
    batch = _log(rng, 1, 48)
    hi = _log(rng, 64, max(64, min(100000, 400000 // (batch * (1 if rows == 1 else 6)))))
    return dict(op=op, batch=batch, rows=rows, lo=rng.randint(max(1, hi // 3), hi), hi=hi,
                hq=g * hkv, hkv=hkv, d=d)


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


def _e2m1(y):
    """fp32 -> e2m1 codes: nearest, ties to the even code, saturating at 6."""
    a = y.abs()
    code = torch.zeros_like(y, dtype=torch.uint8)
    # a tie at an edge goes up where the code above it is even
    for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if up else (a > edge)
    return code | (torch.signbit(y).to(torch.uint8) << 3)


_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x, block_dims):
    """x [n, h, 16, d] bf16 -> codes [n, h, 16, d] uint8, block scales as e4m3 (keys: [n, h, 1, d, 1],
    values: [n, h, 16, d/16, 1]) and page scales [n, h] fp32."""
    n, h, _, d = x.shape
    x = x.float()
    a = x.abs().amax((2, 3))
    live = a >= 2.0 ** -97
    safe = torch.where(live, a, 1.0)
    tops, mids = torch.full_like(a, 2688.0), torch.full_like(a, 448.0)
    scale = torch.where(live, safe / tops, 0.0)   # tensor by tensor: correctly rounded quotients
    inv, inv7 = torch.where(live, tops / safe, 0.0), torch.where(live, mids / safe, 0.0)
    x = x.view(n, h, 1, 16, d).transpose(-1, -2) if block_dims == "tokens" else x.view(n, h, 16, d // 16, 16)
    m = x.abs().amax(-1, keepdim=True) * inv7[:, :, None, None, None]
    block = m.to(torch.float8_e4m3fn)
    s = block.float()
    r = torch.where(s > 0, inv[:, :, None, None, None] / torch.where(s > 0, s, 1.0), 0.0)
    code = _e2m1(x * r)
    code = code.transpose(-1, -2).reshape(n, h, 16, d) if block_dims == "tokens" else code.view(n, h, 16, d)
    return code, block, scale


def _key_pack(c):
    """codes [n, h, 16, d] -> bytes [n, h, 8d]"""
    n, h, _, d = c.shape
    # t = (t2, 2), c = (c64, c16, 8, 2) -> chunk (c64, t2, c16), byte (t%2, 8)
    c = c.view(n, h, 8, 2, d // 64, 4, 8, 2).permute(0, 1, 4, 2, 5, 3, 6, 7)
    return (c[..., 0] | (c[..., 1] << 4)).reshape(n, h, 8 * d)


def _key_unpack(b):
    n, h, w = b.shape
    d = w // 8
    c = torch.stack([b & 15, b >> 4], -1).view(n, h, d // 64, 8, 4, 2, 8, 2)
    return c.permute(0, 1, 3, 5, 2, 4, 6, 7).reshape(n, h, 16, d)


def _value_pack(c):
    n, h, _, d = c.shape
    # t = (t4, 2, 2), c = (c64, half, c4, 4) -> chunk (c64, c4, t4), byte (half, c%4, (t%4)/2)
    c = c.view(n, h, 4, 2, 2, d // 64, 2, 8, 4).permute(0, 1, 5, 7, 2, 6, 8, 3, 4)
    return (c[..., 0] | (c[..., 1] << 4)).reshape(n, h, 8 * d)


def _value_unpack(b):
    n, h, w = b.shape
    d = w // 8
    c = torch.stack([b & 15, b >> 4], -1).view(n, h, d // 64, 8, 4, 2, 4, 2, 2)
    return c.permute(0, 1, 4, 7, 8, 2, 5, 3, 6).reshape(n, h, 16, d)


def _value_scale_pack(s):
    """[n, h, 16, d/16] -> [n, h, d]"""
    n, h, _, b = s.shape
    # b = (b4, b2, b%2), t = (t4, 4) -> (b4, b%2, t4, b2, t%4)
    return s.view(n, h, 4, 4, b // 4, 2, 2).permute(0, 1, 4, 6, 2, 5, 3).reshape(n, h, 16 * b)


def _value_scale_unpack(s):
    n, h, d = s.shape
    return s.view(n, h, d // 64, 2, 4, 2, 4).permute(0, 1, 4, 6, 2, 5, 3).reshape(n, h, 16, d // 16)


def _fill_pages(k, v):
    """Blocks [pages, hkv, 18 * d + 16] uint8 of keys and values [pages, 16, hkv, d]."""
    n, _, h, d = k.shape
    pool = torch.zeros(n, h, 18 * d + 16, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, h, 4, dtype=torch.float32, device=DEV)
    kc, ks, scales[:, :, 0] = _encode(k.permute(0, 2, 1, 3), "tokens")
    vc, vs, scales[:, :, 1] = _encode(v.permute(0, 2, 1, 3), "channels")
    pool[:, :, :8 * d] = _key_pack(kc)
    pool[:, :, 8 * d:16 * d] = _value_pack(vc)
    pool[:, :, 16 * d:17 * d] = ks.view(torch.uint8).view(n, h, d)
    pool[:, :, 17 * d:18 * d] = _value_scale_pack(vs.view(torch.uint8).view(n, h, 16, d // 16))
    pool[:, :, 18 * d:] = scales.view(torch.uint8)
    return pool


def _page_values(block):
    """Blocks [n, hkv, 18 * d + 16] -> fp32 keys and values [n, hkv, 16, d]."""
    d = (block.shape[-1] - 16) // 18
    mag = torch.tensor(_MAGNITUDES + tuple(-x for x in _MAGNITUDES), device=DEV)
    g = block[:, :, 18 * d:].contiguous().view(torch.float32)[:, :, None, None]
    ks = block[:, :, 16 * d:17 * d].contiguous().view(torch.float8_e4m3fn).float()[:, :, None]
    vs = _value_scale_unpack(block[:, :, 17 * d:18 * d].contiguous()).contiguous()
    vs = vs.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    k = mag[_key_unpack(block[:, :, :8 * d].contiguous()).int()] * ks * g[..., 0]
    v = mag[_value_unpack(block[:, :, 8 * d:16 * d].contiguous()).int()] * vs * g[..., 1]
    return k, v


def _key_order(x):
    """[n, hkv, 16, d] -> [n, hkv, 16 * d] in the order of a tail block's keys."""
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


def _tails(b, hkv, d, gen):
    tk, tv = _keys_values(b * PAGE, hkv, d, gen)
    return torch.stack([_key_order(tk.view(b, PAGE, hkv, d).permute(0, 2, 1, 3)),
                        _value_order(tv.view(b, PAGE, hkv, d).permute(0, 2, 1, 3))], 2).contiguous()


def _table(pages_of, max_pages, gen):
    """Page table [batch][max_pages] of shuffled ids, -1 behind a sequence's pages."""
    return _table_of(torch.arange(max_pages, device=DEV)[None, :] < pages_of.to(DEV)[:, None], gen)


def _table_of(live, gen):
    """Page table with shuffled ids where `live`, -1 elsewhere, and how many there are."""
    total = max(1, int(live.sum()))
    ids = torch.randperm(total, generator=gen, device=DEV).int()
    number = live.flatten().cumsum(0).view(live.shape) - 1
    return torch.where(live, ids[number.clamp(min=0)], -1).int(), total


def prepare(case, seed):
    return {"place": _prepare_place, "back": _prepare_back, "attend": _prepare_attend,
            "uncode": _prepare_uncode}[case["op"]](case, seed)


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
    # keys and values are columns of the projection's output [n][3 * hkv][d] (G = 1 beside them)
    kv = torch.empty(int(new.sum()), 3, hkv, d, dtype=torch.bfloat16, device=DEV)
    kv[:, 1], kv[:, 2] = _keys_values(int(new.sum()), hkv, d, gen)
    kv[:, 0] = 0
    max_pages = max(1, int(after.max()) // PAGE)
    table, total = _table(after // PAGE, max_pages, gen)
    return dict(case=case, k=kv[:, 1], v=kv[:, 2], before=before.to(DEV), after=after.to(DEV),
                starts=starts.to(DEV), table=table, tail=_tails(b, hkv, d, gen),
                pool=torch.zeros(total, hkv, 18 * d + 16, dtype=torch.uint8, device=DEV),
                first=first.to(DEV), back_starts=back_starts.to(DEV),
                k_back=torch.zeros(back_rows, hkv, d, dtype=torch.bfloat16, device=DEV),
                v_back=torch.zeros(back_rows, hkv, d, dtype=torch.bfloat16, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _filled(case, lens, gen):
    """Table, pool and tails of sequences of these lengths."""
    b, hkv, d = case["batch"], case["hkv"], case["d"]
    table, total = _table(lens // PAGE, max(1, -(-case["hi"] // PAGE)), gen)
    pool = torch.empty(total, hkv, 18 * d + 16, dtype=torch.uint8, device=DEV)
    k, v = _keys_values(total * PAGE, hkv, d, gen)
    for at in range(0, total, 4096):
        n = min(4096, total - at)
        pool[at:at + n] = _fill_pages(*(x[at * PAGE:(at + n) * PAGE].view(n, PAGE, hkv, d) for x in (k, v)))
    return table, pool, _tails(b, hkv, d, gen)


def _spans(case, lens):
    """first, back_starts and rows of the outputs (enough for all tokens) of sequences read back,
    every other one from its fifth part on."""
    first = torch.where(torch.arange(len(lens)) % 2 == 1, lens // 5, 0).int()
    starts = torch.zeros(len(lens) + 1, dtype=torch.int32)
    starts[1:] = (lens - first).cumsum(0)
    return first, starts, int(lens.sum())


def _prepare_back(case, seed):
    g, gen = _host_rng(seed), _device_rng(seed)
    lens = _lens(case, g)
    table, pool, tail = _filled(case, lens, gen)
    first, starts, rows = _spans(case, lens)
    out = lambda: torch.zeros(rows, case["hkv"], case["d"], dtype=torch.bfloat16, device=DEV)  # noqa: E731
    return dict(case=case, after=lens.to(DEV), table=table, pool=pool, tail=tail,
                first=first.to(DEV), back_starts=starts.to(DEV), k_back=out(), v_back=out(),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_attend(case, seed):
    g, gen = _host_rng(seed), _device_rng(seed)
    b, hq, hkv, d, m = (case[k] for k in ("batch", "hq", "hkv", "d", "rows"))
    lens = _lens(case, g)
    table, pool, tail = _filled(case, lens, gen)
    decay = 0.9 ** (0.5 * torch.arange(d, device=DEV))
    q = (torch.randn(b, m, hq, d, generator=gen, device=DEV) * decay).bfloat16()
    # the rows are the sequence's last tokens; rows of sequences that are too short see nothing
    pos = lens[:, None] - m + torch.arange(m, dtype=torch.int32)[None, :]
    pos = torch.where(pos < 0, -1, pos).int()
    return dict(case=case, q=q if m > 1 else q[:, 0], lens=lens.to(DEV), pos=pos.to(DEV),
                table=table, pool=pool, tail=tail, out=torch.empty_like(q),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _code_fields(d, value):
    """[4d bytes][4]: the element t * d + j whose 2-bit code lies in bits 2f, 2f + 1 of a byte of
    a code plane."""
    t, j = torch.meshgrid(torch.arange(PAGE), torch.arange(d), indexing="ij")
    if value:
        lane, m, i = 4 * (j & 7) + ((t >> 1) & 3), j >> 5, (j >> 4) & 1
        s, e = ((j >> 3) & 1) + 2 * (t >> 3), t & 1
    else:
        lane, m, i = 4 * (t & 7) + ((j >> 1) & 3), j >> 5, (j >> 4) & 1
        s, e = 2 * (t >> 3) + ((j >> 3) & 1), j & 1
    bit = 16 * e + 4 * s + 2 * i
    at = 4 * (lane * (d // 32) + m) + bit // 8
    out = torch.empty(4 * d, 4, dtype=torch.int64)
    out[at.flatten(), (bit % 8 // 2).flatten()] = (t * d + j).flatten()
    return out.to(DEV)


def _value_groups(d):
    """[16][d/32]: index of a (token, group) among a block's value scales."""
    t, g = torch.meshgrid(torch.arange(PAGE), torch.arange(d // 32), indexing="ij")
    return (((((t >> 1) & 3) * 2 + (t >> 3)) * (d // 32) + g) * 2 + (t & 1)).to(DEV)


def _bf16_elements(d, value):
    """[16][d]: index of (token, channel) in the key or value half of a bf16 block."""
    t, j = torch.meshgrid(torch.arange(PAGE), torch.arange(d), indexing="ij")
    if value:
        lane, r, e = 4 * (j & 7) + ((t >> 1) & 3), ((j >> 3) & 1) + 2 * (t >> 3), t & 1
    else:
        lane, r, e = 4 * (t & 7) + ((j >> 1) & 3), (t >> 3) + 2 * ((j >> 3) & 1), j & 1
    return (2 * (((j >> 4) * 32 + lane) * 4 + r) + e).to(DEV)


def _prepare_uncode(case, seed):
    """Rotated values with a spread of each channel's own, coded in groups of 32 channels; bf16
    tokens beside them."""
    g, gen = _host_rng(seed), _device_rng(seed)
    b, hkv, d, bits = (case[k] for k in ("batch", "hkv", "d", "bits"))
    lens = _lens(case, g)
    max_pages = -(-case["hi"] // PAGE)
    page = torch.arange(max_pages)[None, :] * PAGE
    coded = (page < lens[:, None] - WINDOW) & (page + PAGE > SINK)
    plain = (page < lens[:, None]) & ((page < SINK) | (page + PAGE > lens[:, None] - WINDOW))
    coded_table, coded_total = _table_of(coded.to(DEV), gen)
    plain_table, plain_total = _table_of(plain.to(DEV), gen)
    planes, ng, top = bits // 2, d // 32, 2 ** bits - 1
    pool = torch.empty(coded_total, hkv, (4 * bits + 4) * d, dtype=torch.uint8, device=DEV)
    sigma = torch.exp(0.3 * torch.randn(2, hkv, 1, d, generator=gen, device=DEV))
    for at in range(0, coded_total, 2048):
        n = min(2048, coded_total - at)
        parts = []
        for kv in range(2):
            y = torch.randn(n, hkv, PAGE, d, generator=gen, device=DEV) * sigma[kv]
            y = y.view(n, hkv, PAGE, ng, 32)
            lo = y.amin(-1, keepdim=True).half()
            step = ((y.amax(-1, keepdim=True) - y.amin(-1, keepdim=True)) / top).half()
            code = ((y - lo.float()) / step.float()).round().clamp(0, top).to(torch.uint8)
            code = code.view(n, hkv, PAGE * d)
            for plane in range(planes):
                f = ((code >> (2 * (planes - 1 - plane))) & 3)[:, :, _code_fields(d, kv == 1)]
                parts.append(f[..., 0] | (f[..., 1] << 2) | (f[..., 2] << 4) | (f[..., 3] << 6))
            if kv == 0:
                parts.append(torch.cat([step, lo], -1).contiguous().view(torch.uint8).view(n, hkv, -1))
            else:
                at_group = _value_groups(d).flatten()
                for x in (step, lo):
                    area = torch.empty(n, hkv, PAGE * ng, dtype=torch.float16, device=DEV)
                    area[:, :, at_group] = x.view(n, hkv, PAGE * ng)
                    parts.append(area.view(torch.uint8))
        pool[at:at + n] = torch.cat(parts, -1)
    bf16 = torch.empty(plain_total, hkv, 2, PAGE * d, dtype=torch.bfloat16, device=DEV)
    xk, xv = _keys_values(plain_total * PAGE, hkv, d, gen)
    for kv, x in enumerate((xk, xv)):
        x = x.view(plain_total, PAGE, hkv, d).permute(0, 2, 1, 3).reshape(plain_total, hkv, PAGE * d)
        bf16[:, :, kv][:, :, _bf16_elements(d, kv == 1).flatten()] = x
    r = [torch.linalg.qr(torch.randn(hkv, d, d, generator=gen, device=DEV, dtype=torch.float64))[0].float().contiguous()
         for _ in range(2)]
    first, starts, rows = _spans(case, lens)
    out = lambda: torch.zeros(rows, hkv, d, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    return dict(case=case, after=lens.to(DEV), pool=pool, bf16=bf16, coded=coded_table,
                plain=plain_table, r_k=r[0], r_v=r[1], clip=torch.full((hkv,), 8.0, device=DEV),
                first=first.to(DEV), back_starts=starts.to(DEV), k_back=out(), v_back=out(),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


# -------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"place": _own_place, "back": _own_back, "attend": _own_attend,
                "uncode": _own_uncode}[op](state)
    return {"place": _plain_place, "back": _plain_back, "attend": _plain_attend,
            "uncode": _plain_uncode}[op](state)


def _library():
    from int2_rotated_kv_gb300 import oscar
    return oscar


def _cache(s, hq):
    """The binding's descriptor of a state's cache, kept beside its buffers."""
    c = s.get("cache")
    if c is None:
        case = s["case"]
        c = s["cache"] = _library().Kv4Cache(case["hkv"], hq, case["d"], s["pool"], s["tail"],
                                             s["table"], status=s["status"])
    return c


def _own_place(s):
    oscar, c = _library(), _cache(s, s["case"]["hkv"])
    oscar.oscar_kv4_place(c, s["k"], s["v"], s["before"], s["starts"], s["case"]["hi"])
    oscar.oscar_kv4_gather(c, s["after"], s["first"], s["back_starts"],
                           max(PAGE, s["case"]["hi"]), s["k_back"], s["v_back"])
    return s["k_back"], s["v_back"]


def _own_back(s):
    _library().oscar_kv4_gather(_cache(s, s["case"]["hkv"]), s["after"], s["first"], s["back_starts"],
                                s["case"]["hi"], s["k_back"], s["v_back"])
    return s["k_back"], s["v_back"]


def _own_attend(s):
    case = s["case"]
    oscar, c, rows = _library(), _cache(s, case["hq"]), case["rows"]
    if "ws" not in s:
        s["ws"] = torch.empty(oscar.oscar_kv4_workspace_size(c, case["batch"], rows, case["hi"]),
                              dtype=torch.uint8, device=DEV)
    oscar.oscar_kv4_attention(c, s["q"], s["lens"], case["hi"],
                              s["out"] if rows > 1 else s["out"][:, 0], s["ws"],
                              q_pos=s["pos"] if rows > 1 else None)
    return s["out"]


def _own_uncode(s):
    oscar, case = _library(), s["case"]
    if "cache" not in s:
        s["cache"] = oscar.Cache(case["hkv"], case["hkv"], case["d"], SINK, WINDOW, s["pool"], s["bf16"],
                                 s["coded"], s["plain"], s["r_k"], s["r_v"], s["clip"], s["clip"],
                                 s["status"], case["bits"])
    oscar.oscar_gather(s["cache"], s["after"], s["first"], s["back_starts"], case["hi"], s["k_back"],
                       s["v_back"])
    return s["k_back"], s["v_back"]


def _plain_place(s):
    case = s["case"]
    d = case["d"]
    before, after, starts, table = (s[k].long() for k in ("before", "after", "starts", "table"))
    row = torch.arange(s["k"].shape[0], device=DEV)
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
    s["pool"][table[b, top // PAGE]] = _fill_pages(torch.where(old, tail_k[b], s["k"][src]),
                                                   torch.where(old, tail_v[b], s["v"][src]))
    # the tokens behind the last whole page
    rest = row[pos // PAGE >= full]
    tail_k = tail_k.clone()
    tail_v = tail_v.clone()
    tail_k[seq[rest], pos[rest] % PAGE] = s["k"][rest]
    tail_v[seq[rest], pos[rest] % PAGE] = s["v"][rest]
    s["tail"][:, :, 0] = _key_order(tail_k.permute(0, 2, 1, 3))
    s["tail"][:, :, 1] = _value_order(tail_v.permute(0, 2, 1, 3))
    return _plain_back(s)


def _rows_back(s):
    """Of the rows read back: which, their sequences and positions."""
    back = torch.arange(s["k_back"].shape[0], device=DEV)
    seq = torch.searchsorted(s["back_starts"][1:].long(), back, right=True)
    back, seq = back[seq < s["case"]["batch"]], seq[seq < s["case"]["batch"]]
    return back, seq, s["first"].long()[seq] + back - s["back_starts"].long()[seq]


def _plain_back(s):
    d = s["case"]["d"]
    back, seq, pos = _rows_back(s)
    paged = pos // PAGE < (s["after"].long() // PAGE)[seq]
    tail = [_key_tokens(s["tail"][:, :, 0], d), _value_tokens(s["tail"][:, :, 1], d)]
    for out, x in zip((s["k_back"], s["v_back"]), tail):
        out[back[~paged]] = x[seq[~paged], :, pos[~paged] % PAGE]
    back, seq, pos = back[paged], seq[paged], pos[paged]
    for at in range(0, len(back), 1 << 16):
        r, q, t = (x[at:at + (1 << 16)] for x in (back, seq, pos))
        ids, number = torch.unique(s["table"].long()[q, t // PAGE], return_inverse=True)
        for out, x in zip((s["k_back"], s["v_back"]), _page_values(s["pool"][ids])):
            out[r] = x[number, :, t % PAGE].bfloat16()
    return s["k_back"], s["v_back"]


def _plain_attend(s):
    case = s["case"]
    m, hq, hkv, d = (case[k] for k in ("rows", "hq", "hkv", "d"))
    slot = torch.arange(PAGE, device=DEV)
    # a few sequences at a time: pages of the table that are not theirs are masked
    step = max(1, 400000 // (case["hi"] + PAGE))
    for at in range(0, case["batch"], step):
        lens, table, tail = s["lens"][at:at + step].long(), s["table"][at:at + step].long(), s["tail"][at:at + step]
        b, pages = table.shape
        k, v = (x.view(b, pages, hkv, PAGE, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, pages * PAGE, d)
                for x in _page_values(s["pool"][table.clamp(min=0).view(-1)]))
        k = torch.cat([k, _key_tokens(tail[:, :, 0].contiguous(), d).float()], 2)
        v = torch.cat([v, _value_tokens(tail[:, :, 1].contiguous(), d).float()], 2)
        t = torch.arange(pages * PAGE, device=DEV)
        whole = (lens // PAGE * PAGE)[:, None]
        pos = torch.cat([torch.where(t[None] < whole, t[None], 1 << 30),
                         torch.where(whole + slot[None] < lens[:, None], whole + slot[None], 1 << 30)], 1)
        limit = s["pos"][at:at + step].long() if m > 1 else lens[:, None] - 1
        seen = pos[:, None, :] <= limit[:, :, None]                     # [b, m, tokens]
        q = s["q"][at:at + step].float().view(b, m, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
        logits = q @ k.transpose(-1, -2) / math.sqrt(d)
        del k
        logits = logits.view(b, hkv, m, hq // hkv, -1).masked_fill(~seen[:, None, :, None, :], -math.inf)
        top = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - torch.where(torch.isfinite(top), top, 0.0))
        total = p.sum(-1, keepdim=True)
        o = (p.view(b, hkv, m * (hq // hkv), -1) @ v).view(b, hkv, m, hq // hkv, d)
        o = torch.where(total > 0, o / total, 0.0)
        s["out"][at:at + step] = o.permute(0, 2, 1, 3, 4).reshape(b, m, hq, d)
    return s["out"]


def _uncoded(block, d, bits, kv, dtype):
    """Rotated values [n, hkv, 16, d] of code blocks: code * s + z."""
    n, h, _ = block.shape
    planes, ng = bits // 2, d // 32
    start = 0 if kv == 0 else 4 * d * planes + 2 * d
    fields = _code_fields(d, kv == 1)
    code = torch.zeros(n, h, PAGE * d, dtype=torch.uint8, device=DEV)
    for plane in range(planes):
        area = block[:, :, start + 4 * d * plane:start + 4 * d * (plane + 1)]
        f = (area[..., None] >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=DEV)) & 3
        one = torch.empty_like(code)
        one[:, :, fields.flatten()] = f.reshape(n, h, -1)
        code = code * 4 + one
    at = start + 4 * d * planes
    sz = block[:, :, at:at + 2 * d].contiguous().view(torch.float16).to(dtype)
    if kv == 0:
        sz = sz.view(n, h, PAGE, ng, 2)
        step, zero = sz[..., 0], sz[..., 1]
    else:
        step, zero = (x[:, :, _value_groups(d)] for x in sz.view(n, h, 2, PAGE * ng).unbind(2))
    code = code.view(n, h, PAGE, ng, 32).to(dtype)
    return (code * step[..., None] + zero[..., None]).view(n, h, PAGE, d)


def _plain_uncode(s):
    case = s["case"]
    d, hkv, bits = case["d"], case["hkv"], case["bits"]
    back, seq, pos = _rows_back(s)
    lens = s["after"].long()[seq]
    is_plain = (pos < SINK) | (pos >= lens - WINDOW)
    outs, rot = (s["k_back"], s["v_back"]), (s["r_k"], s["r_v"])
    r, q, t = back[is_plain], seq[is_plain], pos[is_plain]
    ids = s["plain"].long()[q, t // PAGE]
    for kv in range(2):
        x = s["bf16"][:, :, kv][ids]                                   # [rows, hkv, 16 d]
        at = _bf16_elements(d, kv == 1)[t % PAGE][:, None].expand(-1, hkv, -1)
        outs[kv][r] = x.gather(2, at)
    back, seq, pos = back[~is_plain], seq[~is_plain], pos[~is_plain]
    for at in range(0, len(back), 1 << 15):
        r, q, t = (x[at:at + (1 << 15)] for x in (back, seq, pos))
        ids, number = torch.unique(s["coded"].long()[q, t // PAGE], return_inverse=True)
        block = s["pool"][ids]
        for kv in range(2):
            x = _uncoded(block, d, bits, kv, torch.float32) @ rot[kv].transpose(-1, -2)
            outs[kv][r] = x[number, :, t % PAGE].bfloat16()
    return outs


# ----------------------------------------------------------------------- floors

def work(case):
    op = case["op"]
    tokens = case["batch"] * (case["lo"] + case["hi"]) / 2
    if op == "attend":
        rows = case["batch"] * case["rows"] * case["hq"]
        return {"bytes": tokens * case["hkv"] * (18 * case["d"] + 8) / PAGE + rows * case["d"] * 4,
                "flops": 4.0 * tokens * case["rows"] * case["hq"] * case["d"]}
    width, code = case["hkv"] * case["d"] * 2, 9.0 / 16
    if op == "place":
        # an append's page is read back whole: half of one, on average
        back = tokens if case["hi"] > 1 else case["batch"] * (PAGE + 1) / 2
        # bf16 in, codes out; codes in, bf16 out
        return {"bytes": width * (tokens * (2 + code) + back * (code + 2)),
                "flops": width * (tokens * 3 + back)}
    lens = _lens(case, _host_rng(0))
    back = float((lens - _spans(case, lens)[0]).sum())
    if op == "back":
        return {"bytes": back * width * (2 + code), "flops": back * width * 2}
    return {"bytes": back * width * (2 + case["bits"] / 8 + 1.0 / 8) + 8 * case["hkv"] * case["d"] ** 2,
            "flops": back * width * (2 * case["d"] + 2)}


# ------------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    return {"place": _exact_place, "back": _exact_back, "attend": _exact_attend,
            "uncode": _exact_uncode}[case["op"]](s)


def _element(d, value):
    """Index of (token, channel) in a tail's keys or values, [16, d]."""
    t = torch.arange(PAGE, device=DEV)[:, None]
    c = torch.arange(d, device=DEV)[None, :]
    if value:
        return (c // 32 * 32 + 4 * (c // 4 % 8) + t // 4) * 16 + 4 * (c % 4) + t % 4
    return ((c // 64 * 2 + t % 2) * 32 + 4 * (t // 2) + c // 16 % 4) * 16 + c % 16


def _minifloat(y, mantissa, least, top):
    """y >= 0 to the nearest number of `mantissa` bits behind the point, exponents from `least`,
    ties to even, at most `top`."""
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** least))) - mantissa)
    return (torch.round(y / step) * step).clamp(max=top)


def _as_coded(x, value):
    """Pages [n, 16, hkv, d] of float64 values as the cache holds them: maxima, the scales and
    their reciprocals in 32 bits as the format defines them, the rest in 64."""
    n, _, h, d = x.shape
    a = x.abs().amax((1, 3), keepdim=True)
    live = a >= 2.0 ** -97
    a = torch.where(live, a, 1.0)
    f32 = lambda y: y.float().double()  # noqa: E731
    mids, tops = torch.full_like(a, 448.0), torch.full_like(a, 2688.0)
    m = x.view(n, 16, h, d // 16, 16).abs().amax(-1).repeat_interleave(16, -1) if value else \
        x.abs().amax(1, keepdim=True).expand_as(x)
    s = _minifloat(f32(m * f32(mids / a)), 3, -6, 448.0)
    r = torch.where(s > 0, f32(f32(tops / a) / torch.where(s > 0, s, 1.0)), 0.0)
    y = f32(x * r)
    return torch.where(live, torch.sign(y) * _minifloat(y.abs(), 1, 0, 6.0) * s * f32(a / tops), 0.0)


def _exact_place(s):
    case = s["case"]
    d = case["d"]
    starts, back_starts, before = (s[k].tolist() for k in ("starts", "back_starts", "before"))
    out = []
    for which, rows in ((0, s["k"]), (1, s["v"])):
        back = torch.zeros(s["k_back"].shape, dtype=torch.float64, device=DEV)
        el = _element(d, which == 1)
        for b in range(case["batch"]):
            n_old = before[b] % PAGE
            old = s["tail"][b, :, which][:, el[:n_old]].permute(1, 0, 2).double()
            y = torch.cat([old, rows[starts[b]:starts[b + 1]].double()])
            whole = len(y) // PAGE * PAGE
            y[:whole] = _as_coded(y[:whole].view(-1, PAGE, case["hkv"], d), which == 1).view(whole, case["hkv"], d)
            back[back_starts[b]:back_starts[b + 1]] = y
        out.append(back)
    return tuple(out)


def _stored_tokens(s, i, n):
    """Keys and values [n][hkv][d] of sequence i in 64 bits, byte by byte of its blocks."""
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    blocks = s["pool"][s["table"][i, :n // PAGE].long()].cpu()
    t, c = torch.arange(PAGE)[:, None], torch.arange(d)[None, :]
    mag = torch.tensor(_MAGNITUDES, dtype=torch.float64)
    page = blocks[:, :, 18 * d:18 * d + 8].contiguous().view(torch.float32).double()
    out = []
    for which in (0, 1):
        if which == 0:
            byte = ((c // 64) * 32 + 4 * (t // 2) + c // 16 % 4) * 16 + 8 * (t % 2) + c % 16 // 2
            high, scale = (c % 2).expand(PAGE, d), (16 * d + c).expand(PAGE, d)
        else:
            byte = 8 * d + (c // 64 * 32 + 4 * (c // 4 % 8) + t // 4) * 16 + 8 * (c // 32 % 2) + 2 * (c % 4) + t % 4 // 2
            high, b = (t % 2).expand(PAGE, d), c // 16
            scale = 17 * d + b // 4 * 64 + (b % 2 * 4 + t // 4) * 8 + b // 2 % 2 * 4 + t % 4
        x = torch.where(high == 1, blocks[:, :, byte] >> 4, blocks[:, :, byte] & 15)
        x = mag[(x & 7).long()] * torch.where(x >= 8, -1.0, 1.0)
        x = x * blocks[:, :, scale].view(torch.float8_e4m3fn).double() * page[:, :, which, None, None]
        x = x.permute(0, 2, 1, 3).reshape(n // PAGE * PAGE, hkv, d).to(DEV)
        tail = s["tail"][i, :, which][:, _element(d, which == 1)[:n % PAGE]].permute(1, 0, 2).double()
        out.append(torch.cat([x, tail]))
    return out


def _exact_back(s):
    case = s["case"]
    starts, first = s["back_starts"].tolist(), s["first"].tolist()
    out = [torch.zeros(s["k_back"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
    for b, n in enumerate(s["after"].tolist()):
        for o, x in zip(out, _stored_tokens(s, b, n)):
            o[starts[b]:starts[b + 1]] = x[first[b]:]
    return tuple(out)


def _exact_attend(s):
    case = s["case"]
    b, m, hq, hkv, d = (case[k] for k in ("batch", "rows", "hq", "hkv", "d"))
    if m * case["hi"] * hq * b > 2 ** 30:
        return None
    q = s["q"].double().view(b, m, hkv, hq // hkv, d)
    out = torch.zeros(b, m, hkv, hq // hkv, d, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens"].tolist()):
        k, v = _stored_tokens(s, i, n)
        limit = s["pos"][i].long() if m > 1 else torch.tensor([n - 1], device=DEV)
        hidden = torch.arange(n, device=DEV)[None] > limit[:, None]
        for h in range(hkv):
            w = torch.einsum("mgd,td->gmt", q[i, :, h], k[:, h]) * d ** -0.5
            w = torch.softmax(w.masked_fill(hidden[None], -math.inf), -1).nan_to_num(0.0)
            out[i, :, h] = torch.einsum("gmt,td->mgd", w, v[:, h])
    return out.view(b, m, hq, d)


def _exact_uncode(s):
    """Each sequence's pages on their own, each code found by its bit's place."""
    case = s["case"]
    d, hkv, bits = case["d"], case["hkv"], case["bits"]
    ng, planes = d // 32, bits // 2
    starts, first = s["back_starts"].tolist(), s["first"].tolist()
    out = [torch.zeros(s["k_back"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
    t, j = torch.arange(PAGE, device=DEV)[:, None], torch.arange(d, device=DEV)[None, :]
    for b, n in enumerate(s["after"].tolist()):
        pos = torch.arange(n, device=DEV)
        near = (pos < SINK) | (pos >= n - WINDOW)
        blocks = s["pool"][s["coded"][b].long().clamp(min=0)].int()
        pages = s["bf16"][s["plain"][b].long().clamp(min=0)]
        for which in (0, 1):
            base = 0 if which == 0 else 4 * d * planes + 2 * d
            if which == 0:
                lane, s_bit, e = 4 * (t % 8) + j // 2 % 4, 2 * (t // 8) + j // 8 % 2, j % 2
                place = base + 4 * d * planes + 4 * (t * ng + j // 32)
                step_at, zero_at = place, place + 2
                el = 2 * ((j // 16 * 32 + lane) * 4 + t // 8 + 2 * (j // 8 % 2)) + j % 2
            else:
                lane, s_bit, e = 4 * (j % 8) + t // 2 % 4, j // 8 % 2 + 2 * (t // 8), t % 2
                place = 2 * (((t // 2 % 4 * 2 + t // 8) * ng + j // 32) * 2 + t % 2)
                step_at = base + 4 * d * planes + place
                zero_at = step_at + d
                el = 2 * ((j // 16 * 32 + lane) * 4 + j // 8 % 2 + 2 * (t // 8)) + t % 2
            bit = 32 * (lane * ng + j // 32) + 16 * e + 4 * s_bit + 2 * (j // 16 % 2)
            code = torch.zeros((), device=DEV)
            for plane in range(planes):
                code = 4 * code + (blocks[:, :, base + 4 * d * plane + bit // 8] >> (bit % 8)) % 4
            half = lambda at: (blocks[:, :, at] + 256 * blocks[:, :, at + 1]).to(torch.uint16).view(torch.float16).double()  # noqa: E731
            y = code.double() * half(step_at) + half(zero_at)
            x = torch.einsum("phtc,hjc->pthj", y, (s["r_k"], s["r_v"])[which].double())
            x = x.reshape(-1, hkv, d)[:n]
            raw = pages[:, :, which][:, :, el].permute(0, 2, 1, 3).reshape(-1, hkv, d)[:n].double()
            out[which][starts[b]:starts[b + 1]] = torch.where(near[:, None, None], raw, x)[first[b]:]
    return tuple(out)

"""Workloads of the latent-attention operators: a paged cache of one latent vector (512) and one
rotary key (64) a token, shared by every query head.

Four operators: the append that lays new tokens out in the pages (bf16, or E4M3 codes with one
power-of-two scale for 32 dims), the read-back of a token range, attention of new tokens over the
pages in the absorbed form (queries of 512 + 64, values = the latents), and causal attention in
the expanded form (keys of 128 a head + the 64 shared, values of 128 a head).

A block holds 64 tokens of one layer.  16-byte units of a 128-byte row are stored at unit
index u ^ (token % 8):
  bf16:   9 chunks [64 tokens][128 B]: latent dims 64c .. 64c + 63, then the rotary key.
  mxfp8:  8 chunks [64 tokens][64 B] of E4M3 codes (not permuted), the rotary chunk
          [64][128 B] in bf16, then scale bytes [64 tokens][16] (2^(byte - 127)).
"""
import math

import torch

own = False

LAT, ROPE, PAGE = 512, 64, 64
NOPE, VDIM = 128, 128
BLOCK = {"bf16": 9 * 8192, "mxfp8": 8 * 4096 + 8192 + 1024}
ROW = {"bf16": 1152, "mxfp8": 656}
LAYERS, LAYER = 2, 1
DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch: the call that every layer makes for every new token
        {"name": "append step", "op": "append", "fmt": "mxfp8", "lanes": 32, "most": 1, "least": 1, "past": 4000},
        # ragged chunks of several prompts
        {"name": "append chunks", "op": "append", "fmt": "bf16", "lanes": 8, "most": 5003, "least": 1, "past": 300},
        # a long prompt, as long as this repository's prefill prefix
        {"name": "append prompt", "op": "append", "fmt": "mxfp8", "lanes": 1, "most": 65536, "least": 65536, "past": 0},
        # a short prefix read back for the expanded form
        {"name": "read prefix", "op": "read", "fmt": "bf16", "lanes": 1, "most": 1025, "least": 1025, "past": 70},
        # whole histories, this repository's decode sizes
        {"name": "read histories", "op": "read", "fmt": "mxfp8", "lanes": 8, "most": 40960, "least": 33000, "past": 0},
        # one short conversation: latency
        {"name": "decode short", "op": "absorbed", "fmt": "bf16", "lanes": 1, "heads": 16, "most": 257, "least": 257, "nq": 1},
        # this repository's decode workload: 8 lanes of 40,960 tokens
        {"name": "decode 8 x 40960", "op": "absorbed", "fmt": "bf16", "lanes": 8, "heads": 128, "most": 40960, "least": 40960, "nq": 1},
        # one long lane beside short ones (this repository's mixed pool), few heads
        {"name": "decode mixed", "op": "absorbed", "fmt": "mxfp8", "lanes": 9, "heads": 16, "most": 131072, "least": 4096, "nq": 1, "one_long": True},
        # four drafted tokens a lane, ragged lanes
        {"name": "decode drafted", "op": "absorbed", "fmt": "mxfp8", "lanes": 16, "heads": 128, "most": 16001, "least": 500, "nq": 4},
        # short new turns of several users
        {"name": "prefill short", "op": "expanded", "lanes": 6, "heads": 16, "most": 300, "least": 1, "prefix": 0},
        # a whole prompt
        {"name": "prefill prompt", "op": "expanded", "lanes": 1, "heads": 128, "most": 4096, "least": 4096, "prefix": 0},
        # a chunk after a long prefix
        {"name": "prefill chunk", "op": "expanded", "lanes": 1, "heads": 32, "most": 1024, "least": 1024, "prefix": 15000},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "absorbed", "absorbed", "expanded", "expanded"])
    if op in ("append", "read"):
        lanes = _log(rng, 1, 64)
        most = _log(rng, 1, 200000 // lanes)
        return {"op": op, "fmt": rng.choice(["bf16", "mxfp8"]), "lanes": lanes, "most": most,
                "least": rng.randint(1, most), "past": rng.randint(0, 500)}
    if op == "absorbed":
        heads, nq = rng.choice([8, 16, 24, 32, 64, 128]), rng.choice([1, 1, 1, 2, 3, 4, 7])
        lanes = _log(rng, 1, 64)
        most = _log(rng, 1, max(1, min(131072, 42000000 // (heads * nq * lanes), 320000 // lanes)))
        most = max(most, nq)
        return {"op": op, "fmt": rng.choice(["bf16", "mxfp8"]), "lanes": lanes, "heads": heads, "most": most,
                "least": rng.randint(nq, most), "nq": nq}
    heads = rng.choice([8, 16, 32, 64, 128])
    most = _log(rng, 1, 4096)
    cells = 2100000000 // (heads * most)
    prefix = rng.choice([0, 0, _log(rng, 1, 16000)])
    prefix = max(0, min(prefix, cells - most))
    lanes = max(1, min(8, cells // (most + prefix)))
    lanes = rng.randint(1, lanes)
    return {"op": op, "lanes": lanes, "heads": heads, "most": most, "least": rng.randint(1, most), "prefix": prefix}


def _lengths(case):
    """Lengths of the lanes: the first has the most; the others fall to the least, each by the
    same ratio, or all have the least ("one_long")."""
    n, a, b = case["lanes"], case["most"], case["least"]
    if n == 1 or case.get("one_long"):
        return [a] + [b] * (n - 1)
    return [a] + [min(a, max(b, int(round(a * (b / a) ** (i / (n - 1)))))) for i in range(1, n)]


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _latents(n, gen):
    """Normed latents: N(0, 1) with a gain a dim, some of them large; bf16 [n, 512]."""
    gain = torch.exp(0.35 * torch.randn(LAT, generator=gen, device=DEV))
    out = torch.empty(n, LAT, dtype=torch.bfloat16, device=DEV)
    for i in range(0, n, 65536):
        m = min(65536, n - i)
        out[i:i + m] = (torch.randn(m, LAT, generator=gen, device=DEV) * gain).to(torch.bfloat16)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _swizzle():
    t, u = torch.arange(PAGE, device=DEV), torch.arange(8, device=DEV)
    return u[None, :] ^ (t[:, None] & 7)


def _table(lens, gen):
    """A permuted page table wide enough for every lane, and the pages of the pool."""
    need = [-(-n // PAGE) for n in lens]
    width, total = max(need), sum(need)
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _fill(pool, fmt, table, lens, lat, rope):
    """Writes the lanes' tokens (rows of lat / rope in lane order) into their pages, as the format says."""
    pages = pool.view(-1, LAYERS, BLOCK[fmt])[:, LAYER]
    sw, at = _swizzle(), 0
    for b, n in enumerate(lens):
        k = -(-n // PAGE)
        x = torch.zeros(k * PAGE, LAT + ROPE, dtype=torch.bfloat16, device=DEV)
        x[:n, :LAT], x[:n, LAT:] = lat[at:at + n], rope[at:at + n]
        at += n
        u = x.view(k, PAGE, 9, 8, 8).permute(0, 2, 1, 3, 4)
        u = torch.gather(u, 3, sw[None, None, :, :, None].expand(k, 9, PAGE, 8, 8)).contiguous()
        if fmt == "bf16":
            blk = u.view(k, -1).view(torch.uint8)
        else:
            codes, scale = _encode(x[:, :LAT])
            c = codes.view(torch.uint8).view(k, PAGE, 8, 64).permute(0, 2, 1, 3).reshape(k, -1)
            blk = torch.cat([c, u[:, 8].reshape(k, -1).view(torch.uint8), scale.view(k, -1)], 1)
        pages[table[b, :k].long()] = blk


def _encode(x):
    """E4M3 codes and scale bytes of rows [n, 512]: 2^e with e the least that keeps the group's
    largest value within 448, in [-120, 7]."""
    g = x.float().view(-1, 16, 32)
    m, p = torch.frexp(g.abs().amax(-1))
    e = torch.where(m <= 0.875, p - 9, p - 8)
    e = torch.where(m == 0, torch.full_like(e, -120), e).clamp(-120, 7)
    codes = torch.ldexp(g, -e[..., None]).view(-1, LAT).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = _gen(seed)
    if case["op"] == "expanded":
        new = _lengths(case)
        keys = [n + case["prefix"] for n in new]
        rows, krows, h = sum(new), sum(keys), case["heads"]
        rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
        # the query and the expanded keys and values as a model's projections leave them: one
        # row of q holds 128 + 64 dims a head, one row of the expansion 128 of k and 128 of v
        q, kv = rnd(rows, h, NOPE + ROPE), rnd(krows, h, NOPE + VDIM)
        return {"case": case, "q_nope": q[..., :NOPE], "q_rope": q[..., NOPE:], "k_nope": kv[..., :NOPE],
                "v": kv[..., NOPE:], "k_rope": rnd(krows, ROPE), "new": new, "keys": keys,
                "q_pos0": _i32([case["prefix"]] * len(new)), "n_q": _i32(new), "q_off": _i32(_offsets(new)[:-1]),
                "n_k": _i32(keys), "k_off": _i32(_offsets(keys)[:-1]), "scale": 1.0 / math.sqrt(NOPE + ROPE),
                "status": torch.zeros(1, dtype=torch.int32, device=DEV),
                "out": torch.empty(rows, h, VDIM, dtype=torch.bfloat16, device=DEV)}
    fmt, lens = case["fmt"], _lengths(case)
    if case["op"] in ("append", "read"):
        past = case["past"]
        table, pages = _table([past + n for n in lens], gen)
    else:
        table, pages = _table(lens, gen)
    pool = torch.zeros(pages * LAYERS * BLOCK[fmt], dtype=torch.uint8, device=DEV)
    lat = _latents(sum(lens), gen)
    rope = torch.randn(sum(lens), ROPE, generator=gen, device=DEV).to(torch.bfloat16)
    s = {"case": case, "fmt": fmt, "pool": pool, "table": table, "lens": lens,
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if case["op"] in ("append", "read"):
        s |= {"start": _i32([past] * len(lens)), "n": _i32(lens), "off": _i32(_offsets(lens)[:-1]), "past": past}
        if case["op"] == "append":
            return s | {"lat": lat, "rope": rope}
        held = [past + n for n in lens]
        lat, rope = _latents(sum(held), gen), torch.randn(sum(held), ROPE, generator=gen, device=DEV).to(torch.bfloat16)
        _fill(pool, fmt, table, held, lat, rope)
        return s | {"lat": torch.empty(sum(lens), LAT, dtype=torch.bfloat16, device=DEV),
                    "rope": torch.empty(sum(lens), ROPE, dtype=torch.bfloat16, device=DEV)}
    _fill(pool, fmt, table, lens, lat, rope)
    nq, h = case["nq"], case["heads"]
    rows = nq * len(lens)
    # the absorbed product leaves its result head first: [heads][rows][512]
    q_lat = torch.randn(h, rows, LAT, generator=gen, device=DEV).to(torch.bfloat16).transpose(0, 1)
    q_rope = torch.randn(rows, h, ROPE, generator=gen, device=DEV).to(torch.bfloat16)
    return s | {"q_lat": q_lat, "q_rope": q_rope, "scale": 1.0 / math.sqrt(NOPE + ROPE),
                "q_pos0": _i32([n - nq for n in lens]), "n_q": _i32([nq] * len(lens)),
                "q_off": _i32([nq * b for b in range(len(lens))]), "seq_len": _i32(lens),
                "out": torch.empty(rows, h, LAT, dtype=torch.bfloat16, device=DEV)}


# ------------------------------------------------------------------------------------- plain forms
def _positions(s):
    """Lane and position of every row of an append or a read, and its page and slot."""
    lane = torch.repeat_interleave(torch.arange(len(s["lens"]), device=DEV), s["n"].long())
    pos = torch.arange(lane.numel(), device=DEV) - s["off"].long()[lane] + s["start"].long()[lane]
    return s["table"].long()[lane, pos // PAGE], pos % PAGE


def _held(s):
    """What the layer's part of the pool holds: views of its blocks."""
    blocks = s["pool"].view(-1, LAYERS, BLOCK[s["fmt"]])[:, LAYER]
    n = blocks.shape[0]
    if s["fmt"] == "bf16":
        return (blocks.view(torch.bfloat16).view(n, 9, PAGE, 8, 8),)
    codes = blocks[:, :32768].view(torch.float8_e4m3fn).view(n, 8, PAGE, 64)
    rope = blocks[:, 32768:40960].view(torch.bfloat16).view(n, PAGE, 8, 8)
    return codes, rope, blocks[:, 40960:].view(n, PAGE, 16)


def _plain_append(s):
    page, slot = _positions(s)
    at = torch.arange(8, device=DEV)[None, :] ^ (slot[:, None] & 7)
    if s["fmt"] == "bf16":
        x = torch.cat([s["lat"], s["rope"]], 1).view(-1, 9, 8, 8)
        units, = _held(s)
        units[page[:, None, None], torch.arange(9, device=DEV)[None, :, None], slot[:, None, None], at[:, None, :]] = x
        return (units,)
    codes, rope, scale = _held(s)
    c, e = _encode(s["lat"])
    codes.view(torch.uint8)[page, :, slot] = c.view(torch.uint8).view(-1, 8, 64)
    rope[page[:, None], slot[:, None], at] = s["rope"].view(-1, 8, 8)
    scale[page, slot] = e
    return codes, rope, scale


def _rows(s, page, slot):
    """The tokens at (page, slot): latents and rotary keys in 32 bits."""
    at = torch.arange(8, device=DEV) ^ (slot[..., None] & 7)
    if s["fmt"] == "bf16":
        units, = _held(s)
        chunk = torch.arange(9, device=DEV)[:, None]
        x = units[page[..., None, None], chunk, slot[..., None, None], at[..., None, :]].float().flatten(-3)
        return x[..., :LAT], x[..., LAT:]
    codes, rope, scale = _held(s)
    c = codes.view(torch.uint8)[page[..., None], torch.arange(8, device=DEV), slot[..., None]]
    c = c.view(torch.float8_e4m3fn).float().flatten(-2).unflatten(-1, (16, 32))
    x = torch.ldexp(c, (scale[page, slot].int() - 127)[..., None]).flatten(-2)
    return x, rope[page[..., None], slot[..., None], at].float().flatten(-2)


def _plain_read(s):
    lat, rope = _rows(s, *_positions(s))
    return lat.to(torch.bfloat16), rope.to(torch.bfloat16)


def _softmax_rows(x, ok):
    """Softmax over the last axis where `ok` (in 32 bits); rows without a key are zeros."""
    x = x.masked_fill(~ok, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-1e30))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_absorbed(s):
    nq, most = s["case"]["nq"], s["case"]["most"]
    pos = torch.arange(most, device=DEV)
    page = s["table"].long()[:, pos // PAGE].clamp_min(0)
    lat, rope = _rows(s, page, (pos % PAGE).expand(page.shape))
    b, h = page.shape[0], s["case"]["heads"]
    ql = s["q_lat"].float().reshape(b, nq * h, LAT)
    qr = s["q_rope"].float().reshape(b, nq * h, ROPE)
    sc = (ql @ lat.transpose(1, 2) + qr @ rope.transpose(1, 2)) * s["scale"]
    last = s["q_pos0"][:, None] + torch.arange(nq, device=DEV)
    ok = pos <= last.repeat_interleave(h, 1)[..., None]
    return (_softmax_rows(sc, ok) @ lat).view(b * nq, h, LAT).to(torch.bfloat16)


def _plain_expanded(s):
    h, lanes = s["case"]["heads"], len(s["new"])
    mq, mk = max(s["new"]), max(s["keys"])
    qi, ki = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    qrow = (s["q_off"].long()[:, None] + qi).clamp_max(s["out"].shape[0] - 1)
    krow = (s["k_off"].long()[:, None] + ki).clamp_max(s["k_rope"].shape[0] - 1)
    grab = lambda x, r: x[r].float().transpose(1, 2)  # noqa: E731
    sc = grab(s["q_nope"], qrow) @ grab(s["k_nope"], krow).transpose(2, 3)
    sc = sc + grab(s["q_rope"], qrow) @ s["k_rope"][krow].float().transpose(1, 2)[:, None]
    ok = (ki <= (s["q_pos0"][:, None] + qi)[..., None]) & (ki < s["n_k"][:, None])[:, None]
    out = (_softmax_rows(sc * s["scale"], ok[:, None]) @ grab(s["v"], krow)).transpose(1, 2)
    return out[qi < s["n_q"][:, None]].view(-1, h, VDIM).to(torch.bfloat16)


# ------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "absorbed": _plain_absorbed,
                "expanded": _plain_expanded}[case["op"]](s)
    from compressed_paged_kv_quant_gb300 import kvq
    if case["op"] == "expanded":
        if "ws" not in s:
            s["ws"] = torch.empty(kvq.latent_prefill_workspace_bytes(len(s["new"]), case["heads"], s["out"].shape[0],
                                                                     max(s["new"]), max(s["keys"])),
                                  dtype=torch.uint8, device=DEV)
        kvq.latent_prefill_attn(s["q_pos0"], s["n_q"], s["q_off"], max(s["new"]), s["n_k"], s["k_off"], max(s["keys"]),
                                s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"], s["scale"], s["ws"],
                                s["out"], s["status"])
        return s["out"]
    if "geom" not in s:
        fmt = kvq.LATENT_BF16 if s["fmt"] == "bf16" else kvq.LATENT_MXFP8
        s["geom"] = kvq.latent_geom(fmt, LAYERS, case.get("heads", 1))
    g = s["geom"]
    if case["op"] == "append":
        kvq.latent_append(g, LAYER, s["pool"], s["table"], s["start"], s["n"], s["off"], max(s["lens"]), s["lat"],
                          s["rope"], s["status"])
        return _held(s)
    if case["op"] == "read":
        kvq.latent_read(g, LAYER, s["pool"], s["table"], s["start"], s["n"], s["off"], max(s["lens"]), s["lat"],
                        s["rope"], s["status"])
        return s["lat"], s["rope"]
    if "ws" not in s:
        s["ws"] = torch.empty(kvq.latent_workspace_bytes(g, len(s["lens"]), case["nq"], case["most"]),
                              dtype=torch.uint8, device=DEV)
    kvq.paged_latent_attn(g, LAYER, s["pool"], s["table"], s["q_pos0"], s["n_q"], s["q_off"], case["nq"],
                          s["seq_len"], case["most"], s["q_lat"], s["q_rope"], s["scale"], s["ws"], s["out"],
                          s["status"])
    return s["out"]


def work(case):
    lens = _lengths(case)
    n = sum(lens)
    if case["op"] in ("append", "read"):
        return {"bytes": n * (1152 + ROW[case["fmt"]]), "flops": 0}
    if case["op"] == "absorbed":
        h, nq = case["heads"], case["nq"]
        pairs = sum(nq * k - nq * (nq - 1) // 2 for k in lens)
        return {"bytes": n * ROW[case["fmt"]] + len(lens) * nq * h * (1152 + 1024), "flops": 2 * pairs * h * (LAT + ROPE + LAT)}
    h, p = case["heads"], case["prefix"]
    pairs = sum(k * p + k * (k + 1) // 2 for k in lens)
    keys = n + p * len(lens)
    return {"bytes": n * h * 2 * (NOPE + ROPE + VDIM) + keys * (h * 2 * (NOPE + VDIM) + 2 * ROPE),
            "flops": 2 * pairs * h * (NOPE + ROPE + VDIM)}


# ------------------------------------------------------------------------------------- in 64 bits
def _e4m3(x):
    """The nearest E4M3 value of a double within +-448, ties to the even mantissa."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _groups64(x):
    """Codes (as values) and exponents of rows [n, 512] from the definition."""
    g = x.double().view(-1, 16, 32)
    a = g.abs().amax(-1)
    ladder = torch.exp2(torch.arange(-120, 8, device=DEV, dtype=torch.float64)) * 448.0
    e = torch.searchsorted(ladder, a).clamp_max(127) - 120
    return _e4m3(g / torch.exp2(e.double())[..., None]).view(-1, 8, 64), e


def _token64(block, fmt, slot):
    """One slot of blocks [n, bytes] in doubles: latents [n, 512] and rotary keys [n, 64]."""
    swap = [u ^ (slot % 8) for u in range(8)]
    if fmt == "bf16":
        x = block.view(torch.bfloat16).view(-1, 9, PAGE, 8, 8)[:, :, slot][:, :, swap].double().reshape(-1, LAT + ROPE)
        return x[:, :LAT], x[:, LAT:]
    byte = block[:, :32768].reshape(-1, 8, PAGE, 64)[:, :, slot].reshape(-1, 16, 32).long()
    mant, expo = byte % 8, byte // 8 % 16
    mag = torch.where(expo == 0, mant.double() * 2.0 ** -9, (8 + mant).double() * torch.exp2(expo.double() - 10))
    val = torch.where(byte >= 128, -mag, mag)
    sc = torch.exp2(block[:, 40960:].reshape(-1, PAGE, 16)[:, slot].double() - 127)
    rope = block[:, 32768:40960].reshape(-1, 8192).view(torch.bfloat16).view(-1, PAGE, 8, 8)[:, slot][:, swap]
    return (val * sc[..., None]).reshape(-1, LAT), rope.double().reshape(-1, ROPE)


def _lane64(s, b, n):
    """The first n tokens of lane b in doubles."""
    k = -(-n // PAGE)
    blk = s["pool"].view(-1, LAYERS, BLOCK[s["fmt"]])[s["table"][b, :k].long(), LAYER]
    got = [_token64(blk, s["fmt"], t) for t in range(PAGE)]
    return tuple(torch.stack([x[i] for x in got], 1).flatten(0, 1)[:n] for i in (0, 1))


def _attend64(q, k, v, scale, first):
    """Rows of q [h, n, d] at positions first + i against k [h or 1, m, d], v [h or 1, m, e]."""
    n, m = q.shape[1], k.shape[1]
    out = torch.empty(q.shape[0], n, v.shape[2], dtype=torch.float64, device=DEV)
    for i in range(0, n, 512):
        j = min(n, i + 512)
        x = (q[:, i:j] @ k.transpose(1, 2)) * scale
        mask = torch.arange(m, device=DEV)[None] > first + torch.arange(i, j, device=DEV)[:, None]
        p = torch.softmax(x.masked_fill_(mask, -math.inf), -1)
        out[:, i:j] = p @ v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        held = [x.clone() for x in _held(s)]
        vals = [torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in held[:2]]
        codes, e = _groups64(s["lat"])
        expo = torch.zeros(held[0].shape[0], PAGE, 16, dtype=torch.uint8, device=DEV)
        at = 0
        for b, n in enumerate(s["lens"]):
            pos = torch.arange(s["past"], s["past"] + n, device=DEV)
            page, slot = s["table"][b].long()[pos // PAGE], pos % PAGE
            r = slice(at, at + n)
            at += n
            for u in range(8):
                place = u ^ (slot % 8)
                if case["fmt"] == "bf16":
                    x = torch.cat([s["lat"][r], s["rope"][r]], 1).double().view(n, 9, 8, 8)
                    for c in range(9):
                        vals[0][page, c, slot, place] = x[:, c, u]
                else:
                    vals[1][page, slot, place] = s["rope"][r].double().view(n, 8, 8)[:, u]
            if case["fmt"] == "mxfp8":
                for c in range(8):
                    vals[0][page, c, slot] = codes[r, c]
                expo[page, slot] = (e[r] + 127).to(torch.uint8)
        return (vals[0],) if case["fmt"] == "bf16" else (vals[0], vals[1], expo)
    if case["op"] == "read":
        got = [_lane64(s, b, s["past"] + n) for b, n in enumerate(s["lens"])]
        return tuple(torch.cat([x[i][s["past"]:] for x in got]) for i in (0, 1))
    if case["op"] == "absorbed":
        out = []
        for b, n in enumerate(s["lens"]):
            lat, rope = _lane64(s, b, n)
            r = slice(b * case["nq"], (b + 1) * case["nq"])
            q = torch.cat([s["q_lat"][r], s["q_rope"][r]], -1).double().transpose(0, 1)
            out.append(_attend64(q, torch.cat([lat, rope], 1)[None], lat[None], s["scale"], n - case["nq"]).transpose(0, 1))
        return torch.cat(out)
    out, qa, ka = [], 0, 0
    for n, m in zip(s["new"], s["keys"]):
        heads = []
        for h in range(0, case["heads"], 8):
            q = torch.cat([s["q_nope"][qa:qa + n, h:h + 8], s["q_rope"][qa:qa + n, h:h + 8]], -1).double().transpose(0, 1)
            kr = s["k_rope"][ka:ka + m, None].expand(m, q.shape[0], ROPE)
            k = torch.cat([s["k_nope"][ka:ka + m, h:h + 8], kr], -1).double().transpose(0, 1)
            v = s["v"][ka:ka + m, h:h + 8].double().transpose(0, 1)
            heads.append(_attend64(q, k, v, s["scale"], m - n))
        out.append(torch.cat(heads).transpose(0, 1))
        qa, ka = qa + n, ka + m
    return torch.cat(out)

"""Cases, plain forms and 64-bit definitions of the prompt and eviction operators.

The operators, in the order a serving program meets them:
  prompt   causal attention over whole prompts packed behind one another, with
           the log-sum-exp of every row and, where asked for, the attention
           weight that every tile of T tokens receives (its mass)
  decode   one decode step over the packed 2/3/4/8-bit pages that adds the
           step's attention weight to the masses
  evict    drops the tiles with the least mass from a cache: block tables,
           lengths and masses are compacted in place
``run`` computes them with elementary torch operations, or through the
library's calls where ``own`` is true.  ``exact`` gives the same outputs from
the definitions in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

PAGE = 16            # tokens per page
PLAIN_ELEMS = 1 << 28  # scores held at once by the plain forms


# ------------------------------------------------------------------ cases
def _prompt(name, lens, hkv, g, d=128, t=64, mass=False, window=0):
    return {"name": name, "op": "prompt", "lens": ",".join(str(x) for x in lens), "hkv": hkv, "g": g, "d": d, "t": t,
            "mass": mass, "window": window}


def _decode(name, lens, hkv, g, d=128, t=64, bits_k=4, bits_v=4):
    return {"name": name, "op": "decode", "lens": ",".join(str(x) for x in lens), "hkv": hkv, "g": g, "d": d, "t": t,
            "bits_k": bits_k, "bits_v": bits_v}


def _evict(name, lens, keep, sink=1, recent=1, t=64):
    return {"name": name, "op": "evict", "lens": ",".join(str(x) for x in lens), "keep": keep, "sink": sink,
            "recent": recent, "t": t}


def _log_lens(seed, count, lo, hi):
    r = random.Random(seed)
    return [int(math.exp(r.uniform(math.log(lo), math.log(hi + 1)))) for _ in range(count)]


def listed():
    return [
        # one short chat turn arriving alone: what counts is latency
        _prompt("prompt_turn_37", [37], 8, 4),
        # a scheduler's batch of prompts of all lengths packed together, one of
        # them empty and one a single token (Qwen3-32B-shaped heads)
        _prompt("prompt_ragged_16", [0, 1] + _log_lens(7, 14, 33, 2048), 8, 8, t=128),
        # the 16K-token prompts of the Qwen3-32B-shaped burst
        _prompt("prompt_16384", [16384], 8, 8, t=128),
        # the other head sizes of the library
        _prompt("prompt_d64", [2047, 1300, 4096], 8, 8, d=64),
        _prompt("prompt_d256", [2500, 701], 4, 2, d=256),
        # prompts of a cache that will evict: every query counts
        _prompt("prompt_mass_4x4096", [4096] * 4, 8, 4, mass=True),
        # a long document whose last 64 tokens say which tiles matter
        _prompt("prompt_window_32768", [32768], 8, 4, mass=True, window=64),
        # one short sequence, one KV head: latency
        _decode("decode_tiny", [1024], 1, 8),
        # the Qwen3-4B-shaped batch at 128K context (one token into its tail)
        _decode("decode_qwen3_4b", [131073] * 6, 8, 4),
        # the Qwen3-32B-shaped burst
        _decode("decode_burst", [16385] * 64, 8, 8, t=128, bits_k=4, bits_v=2),
        # a batch of mixed lengths brought down to 256 tiles a sequence
        _evict("evict_mixed_256", _log_lens(1005, 256, 1024, 131072), 256),
        # long contexts at twice their budget
        _evict("evict_6x131072", [131072] * 6, 1024, sink=4, recent=16),
    ]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "evict"])
    t = rng.choice([32, 64, 128])

    def log(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))

    if op == "prompt":
        count = log(1, 24)
        top = log(2, min(16384, 49152 // count))
        lens = [rng.randint(0, 2) if rng.random() < 0.1 else log(max(1, top // 16), top) for _ in range(count)]
        if not any(lens):
            lens[0] = top
        mass = rng.random() < 0.5
        window = rng.choice([0, log(1, 512)]) if mass else 0
        c = _prompt("", lens, rng.choice([1, 2, 4, 8]), rng.randint(1, 8), rng.choice([64, 128, 128, 128, 256]), t,
                    mass, window)
    elif op == "decode":
        count = log(1, 64)
        top = log(16, min(131072, 786432 // count))
        lens = [rng.randint(0, 2) if rng.random() < 0.1 else log(max(1, top // 16), top) for _ in range(count)]
        if not any(lens):
            lens[0] = top
        bits = rng.choice([(4, 4), (4, 4), (4, 2), (2, 2), (2, 4), (3, 3), (8, 8)])
        d = rng.choice([64, 128, 128, 128, 128, 256])
        if d != 128:  # the library's plain path: smaller caches
            lens = [x // 16 + 1 for x in lens]
        c = _decode("", lens, rng.choice([1, 2, 4, 8]), rng.randint(1, 8), d, t, *bits)
    else:
        count = log(1, 256)
        top = log(64, 131072)
        lens = [rng.randint(0, t) if rng.random() < 0.1 else log(max(1, top // 16), top) for _ in range(count)]
        sink, recent = rng.randint(0, 4), rng.randint(0, 16)
        c = _evict("", lens, max(sink + recent, log(1, max(2, top // t))), sink, recent, t)
    del c["name"]
    return c


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ page format
def _code_slots(d, bits, is_v):
    """Slot (bit offset / bits) of the code of (channel, token) in a page, [d][PAGE]."""
    c, p = np.meshgrid(np.arange(d), np.arange(PAGE), indexing="ij")
    if not is_v or bits == 3:
        return p * d + c
    n, g, t, u, s = c // 8, c % 8, (p % 8) // 2, p // 8, p % 2
    h = 16 // bits
    k, e, lane = 2 * (n // h) + u, n % h, 4 * g + t
    r = min(4, d * bits // 64)
    byte = ((k // r) * 32 + lane) * 4 * r + (k % r) * 4
    return (8 * byte + bits * (e + h * s)) // bits


def _geometry(d, t, bits):
    codes = PAGE * d * bits // 8
    cs = 2 * d * PAGE // t
    return codes, cs, (codes + 64 + cs + 15) // 16 * 16


def _pages(gen, tiles, hkv, d, t, bits, is_v):
    """Packed pages [tiles * t / PAGE][hkv][page_bytes] of rows as they stand after
    the rotation and the normalization: N(0, 1) with channel and token factors."""
    codes_bytes, cs, page_bytes = _geometry(d, t, bits)
    ppt = t // PAGE
    pool = torch.zeros((tiles, ppt, hkv, page_bytes), dtype=torch.uint8, device="cuda")
    slots = torch.from_numpy(_code_slots(d, bits, is_v)).cuda().t().reshape(-1)  # [PAGE * d], token-major
    at_slot = torch.argsort(slots)
    step = max(1, (1 << 26) // (hkv * t * d))
    for a in range(0, tiles, step):
        n = min(step, tiles - a)
        y = torch.randn((n, hkv, t, d), generator=gen, device="cuda")
        lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
        s = (hi - lo) / (2 ** bits - 1)
        code = torch.round((y - lo) / s).clamp_(0, 2 ** bits - 1).to(torch.uint8)
        r = torch.exp(0.2 * torch.randn((n, hkv, t, 1), generator=gen, device="cuda"))
        meta = torch.cat([s * r, lo * r], dim=-1).half()                              # [n][hkv][t][2]
        chan = torch.exp((0.0 if is_v else 0.5) * torch.randn((n, hkv, d), generator=gen, device="cuda"))
        chan = (chan * (1.0 if is_v else 1.2)).half()
        flat = code.view(n, hkv, ppt, PAGE * d).index_select(-1, at_slot)
        if bits == 3:
            w = flat.view(n, hkv, ppt, -1, 8).int()
            v = sum(w[..., i] << (3 * i) for i in range(8))
            packed = torch.stack([v & 255, (v >> 8) & 255, v >> 16], dim=-1).to(torch.uint8).flatten(-2)
        else:
            w = flat.view(n, hkv, ppt, -1, 8 // bits)
            packed = w[..., 0].clone()
            for i in range(1, 8 // bits):
                packed |= w[..., i] << (bits * i)
        dst = pool[a:a + n].permute(0, 2, 1, 3)                                        # [n][hkv][ppt][bytes]
        dst[..., :codes_bytes] = packed
        dst[..., codes_bytes:codes_bytes + 64] = meta.view(n, hkv, ppt, PAGE * 2).view(torch.uint8)
        dst[..., codes_bytes + 64:codes_bytes + 64 + cs] = chan.view(n, hkv, ppt, -1).view(torch.uint8)
    return pool.view(tiles * ppt, hkv, page_bytes)


# ------------------------------------------------------------------ states
def prepare(case, seed):
    return {"prompt": _prepare_prompt, "decode": _prepare_decode, "evict": _prepare_evict}[case["op"]](case, seed)


def _config(case):
    from quantized_paged_kv_tile_b200 import kvq
    return kvq.Config(num_kv_heads=case.get("hkv", 8), group_size=case.get("g", 4), tile_tokens=case["t"],
                      bits_k=case.get("bits_k", 4), bits_v=case.get("bits_v", 4), iters=4,
                      head_dim=case.get("d", 128))


def _channel_std(gen, hkv, d):
    """K channel stds: lognormal(0, 1) per (head, channel), 2% of them ten times that."""
    std = torch.exp(torch.randn((hkv, d), generator=gen, device="cuda"))
    top = torch.rand((hkv, d), generator=gen, device="cuda").argsort(-1)[:, :math.ceil(0.02 * d)]
    return std.scatter(1, top, std.gather(1, top) * 10.0)


def _prepare_prompt(case, seed):
    lens, hkv, g, d, t = _lens(case), case["hkv"], case["g"], case["d"], case["t"]
    n = sum(lens)
    gen = _gen(seed, 1)
    # the projection's output as a model has it: q, k and v side by side in one row
    qkv = torch.randn((n, hkv * g + 2 * hkv, d), generator=gen, device="cuda")
    qkv[:, hkv * g:hkv * (g + 1)] *= _channel_std(gen, hkv, d)
    qkv = qkv.half()
    tiles = max(1, -(-max(lens) // t))
    st = {"case": case, "lens": lens, "qkv": qkv, "q": qkv[:, :hkv * g], "k": qkv[:, hkv * g:hkv * (g + 1)],
          "v": qkv[:, hkv * (g + 1):], "cu": _ints([0] + list(np.cumsum(lens))), "tiles": tiles}
    if own:
        from quantized_paged_kv_tile_b200 import kvq
        st["cfg"] = _config(case)
        st["status"] = _ints([0])
        if case["mass"]:
            need = kvq.prompt_workspace_bytes(st["cfg"], len(lens), n, max(lens), case["window"])
            st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return st


def _prepare_decode(case, seed):
    lens, hkv, g, d, t = _lens(case), case["hkv"], case["g"], case["d"], case["t"]
    b, ppt = len(lens), case["t"] // PAGE
    gen = _gen(seed, 2)
    max_tiles = max(lens) // t + 1
    total = sum(x // t for x in lens)
    # every page somewhere else in the pool
    where = torch.randperm(total * ppt + 1, generator=gen, device="cuda")[:total * ppt].int()
    table = torch.zeros((b, max_tiles * ppt), dtype=torch.int32, device="cuda")
    k_pool = torch.zeros((total * ppt + 1, hkv, _geometry(d, t, case["bits_k"])[2]), dtype=torch.uint8, device="cuda")
    v_pool = torch.zeros((total * ppt + 1, hkv, _geometry(d, t, case["bits_v"])[2]), dtype=torch.uint8, device="cuda")
    if total:
        k_pool[where.long()] = _pages(gen, total, hkv, d, t, case["bits_k"], False)
        v_pool[where.long()] = _pages(gen, total, hkv, d, t, case["bits_v"], True)
    at = 0
    for i, x in enumerate(lens):
        n = x // t * ppt
        table[i, :n] = where[at:at + n]
        at += n
    tail = torch.randn((2, b, hkv, t, d), generator=gen, device="cuda")
    tail[0] *= _channel_std(gen, hkv, d)[None, :, None]
    tail = tail.half()
    st = {"case": case, "lens": lens, "k_pool": k_pool, "v_pool": v_pool, "table": table, "k_tail": tail[0],
          "v_tail": tail[1], "seq_lens": _ints(lens),
          "q": torch.randn((b, hkv * g, d), generator=gen, device="cuda").half(),
          "mass": torch.rand((b, max_tiles), generator=gen, device="cuda") * 8.0}
    if own:
        from quantized_paged_kv_tile_b200 import kvq
        st["cfg"] = _config(case)
        st["status"] = _ints([0])
        st["ws"] = torch.empty(kvq.decode_mass_workspace_bytes(st["cfg"], b, table.shape[1]), dtype=torch.uint8,
                               device="cuda")
    return st


def _prepare_evict(case, seed):
    lens, t = _lens(case), case["t"]
    b, ppt = len(lens), case["t"] // PAGE
    gen = _gen(seed, 3)
    max_tiles = max(lens) // t + 2
    # masses fall off with a long tail; fresh tiles have none yet, some are equal
    mass = torch.exp(2.0 * torch.randn((b, max_tiles), generator=gen, device="cuda"))
    coarse = torch.rand((b, max_tiles), generator=gen, device="cuda")
    mass = torch.where(coarse < 0.05, torch.zeros_like(mass), torch.where(coarse < 0.15, mass.round(), mass))
    held = _ints([-(-x // t) for x in lens])[:, None]
    mass = torch.where(torch.arange(max_tiles, device="cuda")[None] < held, mass, torch.zeros_like(mass))
    table = torch.randperm(b * max_tiles * ppt, generator=gen, device="cuda").int().view(b, max_tiles * ppt)
    # the three arrays that the call changes sit in one buffer, so that a pass restores them in one copy
    # (each starts on a 16-byte boundary)
    parts = [table.flatten(), mass.view(torch.int32).flatten(), _ints(lens)]
    flat = torch.cat([torch.nn.functional.pad(x, (0, -x.numel() % 4)) for x in parts])
    st = {"case": case, "flat": flat, "b": b, "tiles": max_tiles, "ppt": ppt}
    if own:
        from quantized_paged_kv_tile_b200 import kvq
        st["cfg"] = _config(case)
        st["status"] = _ints([0])
        st["ws"] = torch.empty(kvq.evict_workspace_bytes(st["cfg"], b, max_tiles * ppt), dtype=torch.uint8,
                               device="cuda")
    return st


def _evict_views(st, flat):
    b, tiles, ppt = st["b"], st["tiles"], st["ppt"]
    n_table, n_mass = b * tiles * ppt, b * tiles
    at_mass = (n_table + 3) // 4 * 4
    at_lens = at_mass + (n_mass + 3) // 4 * 4
    return (flat[:n_table].view(b, tiles * ppt), flat[at_mass:at_mass + n_mass].view(torch.float32).view(b, tiles),
            flat[at_lens:at_lens + b])


# ------------------------------------------------------------------ passes
def run(state):
    return {"prompt": _run_prompt, "decode": _run_decode, "evict": _run_evict}[state["case"]["op"]](state)


def _run_prompt(st):
    case = st["case"]
    q, k, v = st["q"], st["k"], st["v"]
    b = len(st["lens"])
    if own:
        from quantized_paged_kv_tile_b200 import kvq
        out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        mass = torch.zeros((b, st["tiles"]), dtype=torch.float32, device="cuda") if case["mass"] else None
        kvq.prompt_attention(st["cfg"], q, k, v, out, st["cu"], max(st["lens"]), lse=lse, mass=mass,
                             mass_window=case["window"], workspace=st.get("ws"), dev_status=st["status"])
        return {"out": out, "lse": lse, "mass": mass} if case["mass"] else {"out": out, "lse": lse}
    g, d, t, hkv = case["g"], case["d"], case["t"], case["hkv"]
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    mass = torch.zeros((b, st["tiles"]), dtype=torch.float32, device="cuda")
    scale = d ** -0.5
    at = 0
    for s, n in enumerate(st["lens"]):
        first = n - case["window"] if case["window"] else 0  # queries from here on count towards the mass
        kk = k[at:at + n].float()
        vv = v[at:at + n].float()
        for h in range(hkv):
            qq = q[at:at + n, h * g:(h + 1) * g].float()
            step = max(1, PLAIN_ELEMS // max(1, g * n))
            for r0 in range(0, n, step):
                r1 = min(n, r0 + step)
                x = qq[r0:r1].reshape(-1, d) @ kk[:r1, h].t() * scale  # [(r1 - r0) * g][r1]
                row = torch.arange(r0, r1, device="cuda").repeat_interleave(g)[:, None]
                x.masked_fill_(torch.arange(r1, device="cuda")[None] > row, -math.inf)
                m = x.amax(-1, keepdim=True)
                e = torch.exp(x.sub_(m))
                z = e.sum(-1, keepdim=True)
                p = e.div_(z)
                out[at + r0:at + r1, h * g:(h + 1) * g] = (p @ vv[:r1, h]).view(r1 - r0, g, d).half()
                lse[at + r0:at + r1, h * g:(h + 1) * g] = (m + torch.log(z)).view(r1 - r0, g)
                if case["mass"] and r1 > first:
                    w = p[max(0, first - r0) * g:].sum(0)
                    w = torch.nn.functional.pad(w, (0, -(-r1 // t) * t - r1)).view(-1, t).sum(-1)
                    mass[s, :w.numel()] += w
        at += n
    return {"out": out, "lse": lse, "mass": mass} if case["mass"] else {"out": out, "lse": lse}


def _hadamard(d, dtype):
    h = torch.ones((1, 1), dtype=dtype, device="cuda")
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(d)


def _unpack(pool, blocks, d, t, bits, is_v, heads, dtype):
    """(codes, s, z, c) of the tiles of ``blocks`` [tiles * t / PAGE]: codes
    [tiles][heads][t][d], s and z [tiles][heads][t], c [tiles][heads][d]."""
    codes_bytes, cs, _ = _geometry(d, t, bits)
    ppt = t // PAGE
    page = pool[blocks.long()][:, heads]                                       # [pages][heads][bytes]
    nh = page.shape[1]
    bit = torch.from_numpy(_code_slots(d, bits, is_v).T.reshape(-1) * bits).cuda()  # [PAGE * d]
    raw = page.index_select(-1, bit // 8)
    if bits == 3:  # a code may straddle two bytes
        raw = raw.int() | (page.index_select(-1, bit // 8 + 1).int() << 8)
    code = ((raw >> (bit % 8).to(raw.dtype)) & (2 ** bits - 1)).to(dtype)
    code = code.view(-1, ppt, nh, PAGE, d).transpose(1, 2).reshape(-1, nh, t, d)
    meta = page[..., codes_bytes:codes_bytes + 64].contiguous().view(torch.float16).to(dtype)
    meta = meta.view(-1, ppt, nh, PAGE, 2).transpose(1, 2).reshape(-1, nh, t, 2)
    c = page[..., codes_bytes + 64:codes_bytes + 64 + cs].contiguous().view(torch.float16).to(dtype)
    return code, meta[..., 0], meta[..., 1], c.view(-1, ppt, nh, d // ppt).transpose(1, 2).reshape(-1, nh, d)


def _run_decode(st):
    case = st["case"]
    q = st["q"]
    mass = st["mass"].clone()
    if own:
        from quantized_paged_kv_tile_b200 import kvq
        out = torch.empty_like(q)
        kvq.paged_decode_attention_mass(st["cfg"], q, out, mass, st["seq_lens"], st["table"], st["k_pool"],
                                        st["v_pool"], st["k_tail"], st["v_tail"], st["ws"], dev_status=st["status"])
        return {"out": out, "mass": mass}
    g, d, t, hkv = case["g"], case["d"], case["t"], case["hkv"]
    out = torch.zeros_like(q)
    had = _hadamard(d, torch.float32)
    ppt = t // PAGE
    every = slice(0, hkv)
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        full, tau = n // t, n % t
        qq = q[b].float().view(hkv, g, d) * d ** -0.5
        qr = qq @ had
        x = torch.empty((hkv, g, n), device="cuda")
        step = max(1, (1 << 27) // (hkv * t * d))
        for a in range(0, full, step):
            e = min(full, a + step)
            code, s, z, c = _unpack(st["k_pool"], st["table"][b, a * ppt:e * ppt], d, t, case["bits_k"], False, every,
                                    torch.float32)
            kk = (code * s[..., None] + z[..., None]) * c[:, :, None]               # [tiles][hkv][t][d]
            kk = kk.transpose(0, 1).reshape(hkv, -1, d)
            x[:, :, a * t:e * t] = qr @ kk.transpose(1, 2)
        if tau:
            x[:, :, full * t:] = qq @ st["k_tail"][b, :, :tau].float().transpose(1, 2)
        x = torch.exp(x - x.amax(-1, keepdim=True))
        p = x / x.sum(-1, keepdim=True)
        acc = torch.zeros((hkv, g, d), device="cuda")
        for a in range(0, full, step):
            e = min(full, a + step)
            code, s, z, c = _unpack(st["v_pool"], st["table"][b, a * ppt:e * ppt], d, t, case["bits_v"], True, every,
                                    torch.float32)
            vv = (code * s[..., None] + z[..., None]) * c[:, :, None]
            acc += p[:, :, a * t:e * t] @ vv.transpose(0, 1).reshape(hkv, -1, d)
        acc = acc @ had
        if tau:
            acc += p[:, :, full * t:] @ st["v_tail"][b, :, :tau].float()
        out[b] = acc.view(hkv * g, d).half()
        w = p.sum((0, 1))
        tiles = -(-n // t)
        mass[b, :tiles] += torch.nn.functional.pad(w, (0, tiles * t - n)).view(tiles, t).sum(-1)
    return {"out": out, "mass": mass}


def _run_evict(st):
    case = st["case"]
    table, mass, lens = _evict_views(st, st["flat"].clone())
    if own:
        from quantized_paged_kv_tile_b200 import kvq
        kept = torch.empty((st["b"], st["tiles"]), dtype=torch.int32, device="cuda")
        kvq.evict_tiles(st["cfg"], mass, lens, table, case["keep"], sink_tiles=case["sink"],
                        recent_tiles=case["recent"], kept=kept, workspace=st["ws"], dev_status=st["status"])
        return {"table": table, "mass": mass, "lens": lens, "kept": kept}
    t, b, tiles, ppt = case["t"], st["b"], st["tiles"], st["ppt"]
    full = (lens // t)[:, None]
    gone = (full - case["keep"]).clamp_min(0)                               # tiles to evict
    idx = torch.arange(tiles, device="cuda")[None].expand(b, tiles)
    free = (idx >= case["sink"]) & (idx < full - case["recent"])
    # free tiles by ascending mass, equal ones by index, then all others
    order = torch.argsort(mass, dim=1, stable=True)
    order = order.gather(1, torch.argsort((~free).gather(1, order).int(), dim=1, stable=True))
    rank = torch.empty_like(order).scatter_(1, order, idx)
    evicted = free & (rank < gone)
    # kept tiles in order, the evicted ones behind them, the rest where it was
    group = torch.where(evicted, 1, torch.where(idx < full, 0, 2))
    src = torch.argsort(group, dim=1, stable=True)
    table = table.view(b, tiles, ppt).gather(1, src[..., None].expand(b, tiles, ppt)).view(b, tiles * ppt)
    left = full - gone
    moved = mass.gather(1, src)
    tail = mass.gather(1, full.long().clamp_max(tiles - 1))                # the unfinished tile's mass
    mass = torch.where(gone > 0, torch.where(idx < left, moved, torch.where(idx == left, tail, 0.0)), mass)
    kept = torch.where(idx < left, src, -1).int()
    lens = lens - (gone * t)[:, 0]
    return {"table": table, "mass": mass, "lens": lens.int(), "kept": kept}


# ------------------------------------------------------------------ costs
def work(case):
    lens, t = _lens(case), case["t"]
    if case["op"] == "evict":
        b = len(lens)
        tiles = max(lens) // t + 2
        # table, masses and lengths in and out, the kept list out
        return {"bytes": b * (8 * tiles * t // PAGE + 8 * tiles + 8 + 4 * tiles), "flops": b * tiles}
    hq, d = case["hkv"] * case["g"], case["d"]
    if case["op"] == "prompt":
        n = sum(lens)
        size = 2 * n * d * (2 * hq + 2 * case["hkv"]) + 4 * n * hq
        if case["mass"]:
            size += 4 * sum(-(-x // t) for x in lens)
        return {"bytes": size, "flops": 4 * d * hq * sum(x * (x + 1) // 2 for x in lens)}
    per_page = sum(_geometry(d, t, case[k])[2] for k in ("bits_k", "bits_v")) * case["hkv"] + 4
    full = sum(x // t for x in lens)
    size = full * (t // PAGE) * per_page + sum(x % t for x in lens) * case["hkv"] * d * 4
    size += 4 * len(lens) * hq * d + 8 * sum(-(-x // t) for x in lens)
    return {"bytes": size, "flops": 4 * d * hq * sum(lens)}


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(st)
    lens, hkv, g, d, t = _lens(case), case["hkv"], case["g"], case["d"], case["t"]
    if case["op"] == "prompt":
        n_all = sum(lens)
        out = torch.zeros((n_all, hkv * g, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((n_all, hkv * g), dtype=torch.float64, device="cuda")
        mass = torch.zeros((len(lens), st["tiles"]), dtype=torch.float64, device="cuda")
        lo = 0
        for s, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            tile_of = pos // t
            for hq in range(hkv * g):
                keys = st["k"][lo:lo + n, hq // g].double()
                vals = st["v"][lo:lo + n, hq // g].double()
                for i in range(0, n, 4096):
                    j = min(n, i + 4096)
                    score = st["q"][lo + i:lo + j, hq].double() @ keys[:j].T / math.sqrt(d)
                    score = torch.where(pos[None, :j] <= pos[i:j, None], score, -math.inf)
                    norm = torch.logsumexp(score, dim=1)
                    weight = torch.exp(score - norm[:, None])
                    out[lo + i:lo + j, hq] = weight @ vals[:j]
                    lse[lo + i:lo + j, hq] = norm
                    if case["mass"]:
                        counts = pos[i:j] >= (n - case["window"] if case["window"] else 0)
                        mass[s].index_add_(0, tile_of[:j], (weight * counts[:, None]).sum(0))
            lo += n
        res = {"out": out, "lse": lse}
        if case["mass"]:
            res["mass"] = mass
        return res
    out = torch.zeros((len(lens), hkv * g, d), dtype=torch.float64, device="cuda")
    mass = st["mass"].double()
    had = _hadamard(d, torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        full, tau = n // t, n % t
        blocks = st["table"][b, :full * t // PAGE]
        for h in range(hkv):
            keys, vals = [], []
            for rows, pool, tail, bits, is_v in ((keys, "k_pool", "k_tail", case["bits_k"], False),
                                                 (vals, "v_pool", "v_tail", case["bits_v"], True)):
                if full:
                    code, sc, zero, chan = _unpack(st[pool], blocks, d, t, bits, is_v, slice(h, h + 1), torch.float64)
                    x = (code * sc.unsqueeze(-1) + zero.unsqueeze(-1)) * chan.unsqueeze(2)
                    rows.append(x.reshape(full * t, d) @ had)                      # back in the original domain
                rows.append(st[tail][b, h, :tau].double())
            keys, vals = torch.cat(keys), torch.cat(vals)
            weight = torch.softmax(st["q"][b, h * g:(h + 1) * g].double() @ keys.T / math.sqrt(d), dim=1)
            out[b, h * g:(h + 1) * g] = weight @ vals
            mass[b].index_add_(0, torch.arange(n, device="cuda") // t, weight.sum(0))
    return {"out": out, "mass": mass}


def _exact_evict(st):
    """By the definition, one sequence at a time on the host."""
    case = st["case"]
    table, mass, lens = (x.cpu().numpy().copy() for x in _evict_views(st, st["flat"]))
    t, ppt = case["t"], st["ppt"]
    kept = np.full((st["b"], st["tiles"]), -1, dtype=np.int32)
    for b in range(st["b"]):
        full = int(lens[b]) // t
        gone = max(0, full - case["keep"])
        free = range(case["sink"], full - case["recent"])
        out = set(sorted(free, key=lambda i: (mass[b, i], i))[:gone])
        stay = [i for i in range(full) if i not in out]
        kept[b, :len(stay)] = stay
        if gone:
            new = stay + sorted(out)
            table[b, :full * ppt] = table[b].reshape(-1, ppt)[new].reshape(-1)
            row = np.zeros_like(mass[b])
            row[:len(stay)] = mass[b, stay]
            row[len(stay)] = mass[b, full]
            mass[b] = row
            lens[b] -= gone * t
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    return {"table": dev(table), "mass": dev(mass).double(), "lens": dev(lens), "kept": dev(kept)}

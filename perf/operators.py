"""Measured cases of the paged 4-bit cache and of the prompt attention.

Four operators, as a serving loop runs them on one layer:

* append: rotate the new tokens' queries and keys by position, write keys and
  values into 4-bit pages (and read the written tokens back, which is how the
  cached values are seen);
* gather: pages back to contiguous keys and values (the history of a chunk);
* decode: one query token per sequence over the 4-bit pages;
* prompt: causal attention of packed sequences with grouped heads.

``run`` computes them in elementary torch operations where ``own`` is false,
and by the library's calls where it is true.  ``exact`` computes them in 64
bits from the definitions.

Pages.  A cell holds 16 tokens of one KV head in 20 d bytes, G = d / 32 groups:
key codes [8 d], value codes [8 d], key scales [32 G], key zeros [32 G], value
scales [32 G], value zeros [32 G]; a page holds h_kv x (page / 16) cells.  With
P = min(G, 4), token n = 8 s + 2 t + e and channel c = 32 j + r:
  key nibble    byte (j/P) 256 P + n 16 P + (r/8) 4 P + (j%P) 4 + (r%8)/2, high half for odd r
  value nibble  byte (j/P) 256 P + s 128 P + ((r/4) 4 + t) 4 P + (j%P) 4 + 2 e + (r%4)/2, high half for odd r
  key zero      half n G + j
  other scales and zeros  half t 4 G + j 4 + s 2 + e
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
THETA = 500000.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _append(name, dtype, d, h_q, h_kv, page, batch, new, past, rotary, interleaved=False):
    return {"name": name, "op": "append", "dtype": dtype, "d": d, "h_q": h_q, "h_kv": h_kv, "page": page, "batch": batch,
            "new_lo": new[0], "new_hi": new[1], "past_lo": past[0], "past_hi": past[1], "rotary": rotary,
            "interleaved": interleaved, "shape": 1}


def _cached(name, op, dtype, d, h_q, h_kv, page, batch, lo, hi):
    return {"name": name, "op": op, "dtype": dtype, "d": d, "h_q": h_q, "h_kv": h_kv, "page": page, "batch": batch, "lo": lo,
            "hi": hi, "shape": 1}


def _prompt(name, dtype, d, h_q, h_kv, batch, lo, hi, past_hi=0):
    return {"name": name, "op": "prompt", "dtype": dtype, "d": d, "h_q": h_q, "h_kv": h_kv, "batch": batch, "lo": lo, "hi": hi,
            "past_hi": past_hi, "shape": 1}


def listed():
    return [
        # one decode step's append: the batched workload's 32 sequences, one token each
        _append("append_step_b32", "bf16", 128, 32, 8, 64, 32, (1, 1), (16384, 32767), 128),
        # one chunk of the long-context workload: 4 sequences x 8192 tokens behind 32K cached ones
        _append("append_chunk_4x8192", "bf16", 128, 32, 8, 128, 4, (8192, 8192), (32768, 32768), 128),
        # ragged prompts of a small model, half-precision, rotation of adjacent pairs over half the channels
        _append("append_ragged_f16", "f16", 64, 12, 2, 16, 23, (1, 700), (0, 900), 32, True),
        # the history of a chunked prompt: the qwen-shaped layer's longest context
        _cached("gather_1x16384", "gather", "bf16", 128, 12, 2, 64, 1, 16384, 16384),
        # the histories of a ragged batch, small pages
        _cached("gather_ragged_b16", "gather", "f16", 64, 8, 8, 16, 16, 1, 9000),
        # single-stream decode (llama-shaped layer): latency
        _cached("decode_1x4096", "decode", "bf16", 128, 32, 8, 64, 1, 4096, 4096),
        # the batched workload: ragged 16K-32K contexts
        _cached("decode_b32_32k", "decode", "bf16", 128, 32, 8, 64, 32, 16384, 32768),
        # long contexts, few sequences
        _cached("decode_4x131072", "decode", "bf16", 128, 32, 8, 128, 4, 131072, 131072),
        # many short ragged sequences, wide heads, six query heads a KV head, half precision
        _cached("decode_b61_short_f16", "decode", "f16", 256, 12, 2, 16, 61, 0, 1500),
        # one short prompt of the qwen-shaped layer: latency
        _prompt("prompt_1x512", "bf16", 128, 12, 2, 1, 512, 512),
        # one long prompt of the llama-shaped layer
        _prompt("prompt_1x8192", "bf16", 128, 32, 8, 1, 8192, 8192),
        # packed ragged prompts, some behind a cached history, half precision
        _prompt("prompt_ragged_f16", "f16", 64, 16, 8, 9, 1, 3000, 1700),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prompt", "prompt"])
    d = rng.choice([64, 128, 128, 256])
    h_kv = rng.choice([1, 2, 3, 4, 8])
    h_q = h_kv * rng.choice([1, 2, 4, 5, 6, 8])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    page = rng.choice([16, 32, 64, 128])
    c = {"op": op, "dtype": dtype, "d": d, "h_q": h_q, "h_kv": h_kv}
    if op == "append":
        batch = _log(rng, 1, 64)
        most = 32768 * 8 * 128 // (batch * d * h_kv) // (1 + h_q // h_kv)
        hi = _log(rng, 1, max(1, min(8192, most)))
        rotary = rng.choice([0, d // 2, d, d])
        c.update({"page": page, "batch": batch, "new_lo": rng.choice([hi, (hi + 1) // 2, 0]), "new_hi": hi, "past_lo": 0,
                  "past_hi": _log(rng, 1, 20000), "rotary": rotary, "interleaved": rng.random() < 0.4})
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    elif op in ("gather", "decode"):
        batch = _log(rng, 1, 64)
        most = 32 * 24576 * 8 * 128 // (batch * d * h_kv) // (2 if op == "decode" else 8)
        hi = _log(rng, 1, max(1, min(131072, most)))
        c.update({"page": page, "batch": batch, "lo": rng.choice([hi, (hi + 1) // 2, 0]), "hi": hi})
        if op == "gather":
            c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    else:
        batch = _log(rng, 1, 16)
        most = int(math.sqrt(8192 * 8192 * 32 * 128 / (batch * h_q * max(d, 128)) / 2))
        hi = _log(rng, 1, max(1, min(8192, most)))
        c.update({"batch": batch, "lo": rng.choice([hi, (hi + 1) // 2, 0]), "hi": hi, "past_hi": rng.choice([0, 0, hi // 2])})
    c["shape"] = rng.randrange(1 << 20)
    return c


def _lengths(c):
    """(tokens of each sequence in the call, tokens cached before them); the same for every seed."""
    rng = random.Random(c["shape"])
    if c["op"] == "append":
        new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
        new[0] = c["new_hi"]
        return new, [rng.randint(c["past_lo"], c["past_hi"]) for _ in new]
    n = [rng.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]
    n[0] = c["hi"]
    if c["op"] == "prompt":
        return n, [rng.randint(0, c["past_hi"]) for _ in n]
    return n, [0] * len(n)


def work(c):
    n, past = _lengths(c)
    d, h_q, h_kv = c["d"], c["h_q"], c["h_kv"]
    size = 4 if c["dtype"] == "f32" else 2
    T = sum(n)
    record = 1.25 * d
    if c["op"] == "append":
        io = T * d * size * (h_q + 2 * h_kv) + T * d * size * (h_q + h_kv) + T * c["rotary"] * 4
        back = T * h_kv * 2 * d * size
        return {"bytes": io + 2 * T * h_kv * record + back, "flops": T * (3 * c["rotary"] * (h_q + h_kv) + 8 * 2 * h_kv * d)}
    if c["op"] == "gather":
        return {"bytes": T * h_kv * (record + 2 * d * size), "flops": T * h_kv * 2 * d * 2}
    if c["op"] == "decode":
        return {"bytes": T * h_kv * record + 2 * c["batch"] * h_q * d * size, "flops": 4 * d * h_q * T}
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, past))
    rows = T + sum(past)
    return {"bytes": size * d * (2 * T * h_q + 2 * rows * h_kv), "flops": 4 * d * h_q * pairs}


# --------------------------------------------------------------------------
# the pages' layout and the 4-bit codec
# --------------------------------------------------------------------------
_MAPS = {}


def _maps(d, dev):
    """Byte and shift of every key and value nibble [16, d], half index of every key zero and of the other scales [16, G],
    and for packing the (token, channel) of each low and high nibble."""
    if (d, dev) in _MAPS:
        return _MAPS[d, dev]
    G = d // 32
    P = min(G, 4)
    n = torch.arange(16).view(16, 1)
    c = torch.arange(d).view(1, d)
    j, r = c // 32, c % 32
    s, t, e = n // 8, (n % 8) // 2, n % 2
    kb = j // P * 256 * P + n * 16 * P + r // 8 * 4 * P + j % P * 4 + r % 8 // 2
    vb = j // P * 256 * P + s * 128 * P + (r // 4 * 4 + t) * 4 * P + j % P * 4 + 2 * e + r % 4 // 2
    sh = (r % 2 * 4).expand(16, d)
    g = torch.arange(G).view(1, G)
    zk = n * G + g
    sc = t * 4 * G + g * 4 + s * 2 + e
    flat = n * d + c

    def inverse(b):
        at = torch.empty(2, 8 * d, dtype=torch.long)
        at[sh.reshape(-1) // 4, b.reshape(-1)] = flat.reshape(-1)
        return at.to(dev)

    def places(i):
        at = torch.empty(16 * G, dtype=torch.long)
        at[i.reshape(-1)] = torch.arange(16 * G)
        return at.to(dev)

    m = {"kb": kb.to(dev), "vb": vb.to(dev), "sh": sh.to(dev).to(torch.uint8), "zk": zk.to(dev), "sc": sc.to(dev), "ki": inverse(kb),
         "vi": inverse(vb), "zki": places(zk), "sci": places(sc)}
    _MAPS[d, dev] = m
    return m


def _half(x):
    """fp16 of 64-bit values, rounded once (through a 32-bit value rounded to odd)."""
    f = x.float()
    f = torch.where(f.double().abs() > x.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    odd = (f.double() != x).to(torch.int32)
    return (f.contiguous().view(torch.int32) | odd).view(torch.float32).half()


def _encode(x):
    """[..., d] 32-bit values -> codes uint8 [..., d], scale and zero fp16 [..., G]."""
    g = x.unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1), g.amax(-1)
    zero = lo.half()
    scale = _half((hi.double() - lo.double()) / 15)
    code = torch.round((g.double() - zero.double().unsqueeze(-1)) / scale.double().unsqueeze(-1)).clamp(0, 15)
    code = torch.where(scale.unsqueeze(-1) == 0, torch.zeros_like(code), code)
    return code.to(torch.uint8).flatten(-2), scale, zero


def _decode(code, scale, zero):
    """codes, scale, zero -> 32-bit values [..., d]."""
    g = code.unflatten(-1, (-1, 32)).float()
    return (g * scale.float().unsqueeze(-1) + zero.float().unsqueeze(-1)).flatten(-2)


def _pack(k, v):
    """Encoded cells: keys and values [cells, 16, d] (32 bits) -> bytes [cells, 20 d]."""
    m = _maps(k.shape[-1], k.device)
    n = k.shape[0]
    out = []
    for x, inv in ((k, "ki"), (v, "vi")):
        code, scale, zero = _encode(x)
        code = code.reshape(n, -1)
        out.append((code[:, m[inv][0]] | (code[:, m[inv][1]] << 4), scale, zero))
    halves = [out[0][1].reshape(n, -1)[:, m["sci"]], out[0][2].reshape(n, -1)[:, m["zki"]], out[1][1].reshape(n, -1)[:, m["sci"]],
              out[1][2].reshape(n, -1)[:, m["sci"]]]
    return torch.cat([out[0][0], out[1][0]] + [h.contiguous().view(torch.uint8) for h in halves], 1)


def _unpack(cells):
    """Bytes [..., 20 d] -> keys, values [..., 16, d] in 32 bits."""
    d = cells.shape[-1] // 20
    G = d // 32
    m = _maps(d, cells.device)
    half = cells[..., 16 * d:].contiguous().view(torch.float16)
    ks, kz, vs, vz = half.unflatten(-1, (4, 16 * G)).unbind(-2)
    k = _decode((cells[..., : 8 * d][..., m["kb"]] >> m["sh"]) & 15, ks[..., m["sc"]], kz[..., m["zk"]])
    v = _decode((cells[..., 8 * d : 16 * d][..., m["vb"]] >> m["sh"]) & 15, vs[..., m["sc"]], vz[..., m["sc"]])
    return k, v


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _cu(n, dev):
    at = [0]
    for x in n:
        at.append(at[-1] + x)
    return _i32(at, dev)


def _scales(g, shape, dev):
    """Per-channel scales: log-normal, two outlier channels of ten times the size in each head."""
    s = torch.exp(0.5 * torch.randn(shape, generator=g, device=dev))
    s[..., 3::64] *= 10
    return s


def _table(positions, rotary, dev):
    """Cosines and sines [positions, rotary] of the rotation's angles, as a model keeps them."""
    inv = THETA ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=dev) / rotary)
    a = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _block_table(g, c, total, dev):
    """Pages of every sequence, in random order over the pool: [batch, most pages] and the pool's size."""
    page = c["page"]
    need = [-(-n // page) for n in total]
    most, pool = max(1, max(need)), sum(need) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(need), most, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at : at + n]
        at += n
    return table, pool


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n, past = _lengths(c)
    d, h_q, h_kv, dt = c["d"], c["h_q"], c["h_kv"], DTYPES[c["dtype"]]
    T = sum(n)
    st = {"case": {k: v for k, v in c.items() if k != "name"}, "n": n, "past": past}
    if c["op"] == "append":
        # one projection's output holds q, k and v of a token next to each other
        qkv = torch.randn(T, h_q + 2 * h_kv, d, generator=g, device=dev)
        qkv[:, h_q:] *= _scales(g, (2 * h_kv, d), dev)
        qkv = qkv.to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :h_q], qkv[:, h_q : h_q + h_kv], qkv[:, h_q + h_kv :]
        total = [a + b for a, b in zip(n, past)]
        st["len"], st["first"], st["cu"] = _i32(total, dev), _i32(past, dev), _cu(n, dev)
        st["table"], pool = _block_table(g, c, total, dev)
        st["pages"] = torch.zeros(pool, h_kv * (c["page"] // 16) * 20 * d, dtype=torch.uint8, device=dev)
        st["rope"] = _table(max(total) + 1, c["rotary"], dev) if c["rotary"] else None
        st["pos"] = torch.cat([torch.arange(b, a + b, device=dev) for a, b in zip(n, past)])
        for name, h in (("q_out", h_q), ("k_out", h_kv), ("kc", h_kv), ("vc", h_kv)):
            st[name] = torch.zeros(T, h, d, dtype=dt, device=dev)
    elif c["op"] in ("gather", "decode"):
        ks, vs = _scales(g, (h_kv, 1, d), dev), _scales(g, (h_kv, 1, d), dev)
        st["table"], pool = _block_table(g, c, n, dev)
        cells = c["page"] // 16
        pages = torch.empty(pool, h_kv * cells * 20 * d, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (h_kv * c["page"] * d))
        for a in range(0, pool, step):
            m = min(step, pool - a)
            shape = (m, h_kv, cells * 16, d)
            k = (torch.randn(shape, generator=g, device=dev) * ks).view(-1, 16, d)
            v = (torch.randn(shape, generator=g, device=dev) * vs).view(-1, 16, d)
            pages[a : a + m] = _pack(k, v).view(m, -1)
        st["pages"], st["len"], st["most"] = pages, _i32(n, dev), max(n)
        if c["op"] == "gather":
            st["cu"] = _cu(n, dev)
            st["seq"] = torch.repeat_interleave(torch.arange(len(n), device=dev), st["len"].long())
            st["pos"] = torch.arange(T, device=dev) - st["cu"].long()[st["seq"]]
            st["kc"], st["vc"] = (torch.zeros(T, h_kv, d, dtype=dt, device=dev) for _ in range(2))
        else:
            q = torch.randn(c["batch"], h_kv, h_q // h_kv, d, generator=g, device=dev) / ks.view(h_kv, 1, d)
            st["q"] = (1.5 * q).view(c["batch"], h_q, d).to(dt)
            st["out"] = torch.zeros_like(st["q"])
    else:
        rows = T + sum(past)
        st["q"] = (1.5 * torch.randn(T, h_q, d, generator=g, device=dev)).to(dt)
        # rotated keys lie by themselves, values next to the projection's other outputs
        st["k"] = torch.randn(rows, h_kv, d, generator=g, device=dev).to(dt)
        st["v"] = torch.randn(rows, 2 * h_kv, d, generator=g, device=dev).to(dt)[:, h_kv:]
        st["cu_q"], st["cu_k"] = _cu(n, dev), _cu([a + b for a, b in zip(n, past)], dev)
        st["out"] = torch.zeros(T, h_q, d, dtype=dt, device=dev)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    c = st["case"]
    if own:
        return {"append": _own_append, "gather": _own_gather, "decode": _own_decode, "prompt": _own_prompt}[c["op"]](st, c)
    return {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode, "prompt": _plain_prompt}[c["op"]](st, c)


def _rotate(x, table, pos, interleaved):
    """[T, h, d] rotated by position: products and sum in 64 bits, rounded to 32."""
    if table is None:
        return x.float()
    rot = table.shape[1]
    cos, sin = table[pos].double().unsqueeze(1).chunk(2, -1)
    y = x[..., :rot].double()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else y.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y.float(), x[..., rot:].float()], -1)


def _plain_append(st, c):
    dt = DTYPES[c["dtype"]]
    q = _rotate(st["q"], st["rope"], st["pos"], c["interleaved"])
    k = _rotate(st["k"], st["rope"], st["pos"], c["interleaved"])
    return {"q": q.to(dt), "k": k.to(dt), "k_cached": _decode(*_encode(k)).to(dt), "v_cached": _decode(*_encode(st["v"].float())).to(dt)}


def _plain_gather(st, c):
    dt, page, h_kv = DTYPES[c["dtype"]], c["page"], c["h_kv"]
    of = st["table"][st["seq"], st["pos"] // page].long()
    cells = st["pages"].view(-1, h_kv, page // 16, 20 * c["d"])
    # each token's own bytes of its cell
    k, v = _unpack_tokens(cells[of, :, st["pos"] % page // 16], st["pos"] % 16, c["d"])
    return {"k": k.to(dt), "v": v.to(dt)}


def _unpack_tokens(cells, slot, d):
    """One token of each cell: bytes [T, h, 20 d], slots [T] -> keys, values [T, h, d] in 32 bits."""
    G = d // 32
    m = _maps(d, cells.device)
    half = cells[..., 16 * d:].contiguous().view(torch.float16)
    h = cells.shape[1]

    def take(x, at):
        return torch.gather(x, 2, at[slot].unsqueeze(1).expand(-1, h, -1))

    sh = m["sh"][slot].unsqueeze(1)
    ks, kz = take(half[..., : 16 * G], m["sc"]), take(half[..., 16 * G : 32 * G], m["zk"])
    vs, vz = take(half[..., 32 * G : 48 * G], m["sc"]), take(half[..., 48 * G :], m["sc"])
    k = _decode((take(cells[..., : 8 * d], m["kb"]) >> sh) & 15, ks, kz)
    v = _decode((take(cells[..., 8 * d : 16 * d], m["vb"]) >> sh) & 15, vs, vz)
    return k, v


def _plain_decode(st, c):
    d, h_kv, page = c["d"], c["h_kv"], c["page"]
    B, L = c["batch"], st["table"].shape[1] * page
    cells = st["pages"].view(-1, h_kv, page // 16, 20 * d)[st["table"].long()]  # [B, pages, h_kv, cells, bytes]
    k, v = _unpack(cells.transpose(1, 2).reshape(B, h_kv, L // 16, 20 * d))
    k, v = k.reshape(B, h_kv, L, d), v.reshape(B, h_kv, L, d)
    q = st["q"].float().view(B, h_kv, -1, d)
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    seen = torch.arange(L, device=s.device) < st["len"][:, None]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e30))
    o = torch.matmul(p, v.masked_fill(~seen[:, None, :, None], 0.0)) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return {"out": o.view(B, -1, d).to(st["q"].dtype)}


def _plain_prompt(st, c):
    d, h_kv, h_q, B = c["d"], c["h_kv"], c["h_q"], c["batch"]
    dev = st["q"].device
    n, m = max(st["n"]), max(a + b for a, b in zip(st["n"], st["past"]))
    nq, nk = st["cu_q"].diff().long(), st["cu_k"].diff().long()
    i, j = torch.arange(n, device=dev), torch.arange(m, device=dev)
    in_q, in_k = i < nq[:, None], j < nk[:, None]

    def pad(x, inside):
        y = torch.zeros(inside.shape + x.shape[1:], device=dev)
        y[inside] = x.float()
        return y.transpose(1, 2)

    q = pad(st["q"], in_q).reshape(B, h_kv, h_q // h_kv * n, d)
    k, v = pad(st["k"], in_k), pad(st["v"], in_k)
    s = torch.matmul(q, k.transpose(-1, -2)).view(B, h_kv, -1, n, m).div_(math.sqrt(d))
    hidden = ~((j <= (i[:, None] + (nk - nq)[:, None, None])) & in_k[:, None])
    s.masked_fill_(hidden[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    o = torch.matmul(s.view(B, h_kv, -1, m), v).view(B, h_q, n, d) / s.sum(-1).view(B, h_q, n, 1).clamp_min(1e-30)
    return {"out": o.transpose(1, 2)[in_q].to(st["q"].dtype)}


def _handles(st, c):
    """The cache, batch, rotation and workspace handles that a serving loop keeps."""
    from kv_cache_quantization_turboquantprod_b200 import tq

    if "tq" not in st:
        st["tq"] = tq
        if c["op"] != "prompt":
            st["cache"] = tq.PagedCache(c["d"], c["h_kv"], c["page"], st["pages"].shape[0], buffer=st["pages"])
            st["batch"] = tq.PagedBatch(st["len"], st["table"])
        if c["op"] == "append":
            st["rotation"] = tq.Rope(st["rope"], interleaved=c["interleaved"]) if st["rope"] is not None else None
        if c["op"] == "decode":
            st["ws"] = tq.paged_workspace_for(st["cache"], st["batch"], c["h_q"])
    return tq


def _own_append(st, c):
    tq = _handles(st, c)
    tq.tq_paged_append(st["cache"], st["batch"], st["cu"], st["k"], st["v"], q=st["q"], rope=st["rotation"], q_out=st["q_out"],
                       k_out=st["k_out"])
    tq.tq_paged_gather(st["cache"], st["batch"], st["cu"], st["kc"], st["vc"], first=st["first"])
    return {"q": st["q_out"], "k": st["k_out"], "k_cached": st["kc"], "v_cached": st["vc"]}


def _own_gather(st, c):
    tq = _handles(st, c)
    tq.tq_paged_gather(st["cache"], st["batch"], st["cu"], st["kc"], st["vc"])
    return {"k": st["kc"], "v": st["vc"]}


def _own_decode(st, c):
    tq = _handles(st, c)
    tq.tq_paged_decode_attention(st["cache"], st["batch"], st["q"], st["out"], st["ws"])
    return {"out": st["out"]}


def _own_prompt(st, c):
    tq = _handles(st, c)
    tq.tq_prompt_attention(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["out"])
    return {"out": st["out"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(c, seed):
    st = prepare(c, seed)
    return {"append": _exact_append, "gather": _exact_gather, "decode": _exact_decode, "prompt": _exact_prompt}[c["op"]](st, c)


def _nearest_level(x):
    """[..., d] (32-bit values held in 64 bits) -> their 4-bit values: the nearest of the group's sixteen levels."""
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    zero = lo.float().half().double()
    width = (hi - lo) / 15
    # fp16 of the exact width: the nearer of the two halves around its 32-bit value
    near = width.float().half()
    bits = near.view(torch.int16)
    cand = torch.stack([(bits - 1).clamp_min(0), bits, bits + 1]).view(torch.float16).double()
    off = (cand - width).abs() + (torch.stack([bits - 1, bits, bits + 1]) & 1) * 1e-300
    scale = torch.gather(cand, 0, off.argmin(0, keepdim=True))[0]
    level = ((g - zero) / torch.where(scale > 0, scale, torch.ones_like(scale))).round().clamp(0, 15)
    return (zero + torch.where(scale > 0, level * scale, torch.zeros_like(level))).reshape(x.shape)


def _exact_append(st, c):
    out = []
    for name in ("q", "k"):
        x = st[name].double()
        rot = c["rotary"]
        y = x.clone()
        if rot:
            half = rot // 2
            first = torch.arange(half, device=x.device) * (2 if c["interleaved"] else 1)
            second = first + (1 if c["interleaved"] else half)
            angle = st["rope"].double()[st["pos"]][:, None]
            z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle[..., :half], angle[..., half:])
            y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    k32 = out[1].float().double()
    return {"q": out[0], "k": out[1], "k_cached": _nearest_level(k32), "v_cached": _nearest_level(st["v"].double())}


def _sequence(st, c, b):
    """Keys and values [h_kv, len, d] of sequence b in 64 bits, read nibble by nibble from its pages."""
    d, h_kv, page = c["d"], c["h_kv"], c["page"]
    G, n = d // 32, st["n"][b]
    P = min(G, 4)
    raw = st["pages"][st["table"][b, : -(-n // page)].long()].view(-1, h_kv, page // 16, 20 * d).transpose(0, 1).reshape(h_kv, -1, 20 * d)
    half = raw[..., 16 * d :].contiguous().view(torch.float16).view(h_kv, -1, 4, 16 * G).double()

    def words(x):  # [h, cells, 8 d bytes] -> nibbles, low half first, in words of eight
        return torch.stack([x & 15, x >> 4], -1).reshape(h_kv, x.shape[1], G // P, -1, P, 8)

    k = words(raw[..., : 8 * d])  # [h, cells, j/P, (n, r/8), j%P, r%8]
    k = k.reshape(h_kv, -1, G // P, 16, 4, P, 8).permute(0, 1, 3, 2, 5, 4, 6).reshape(h_kv, -1, 16, G, 32)
    v = words(raw[..., 8 * d : 16 * d])  # [h, cells, j/P, (s, r/4, t), j%P, (e, r%4)]
    v = v.reshape(h_kv, -1, G // P, 2, 8, 4, P, 2, 4).permute(0, 1, 3, 5, 7, 2, 6, 4, 8).reshape(h_kv, -1, 16, G, 32)

    def spread(x):  # [h, cells, (t, j, s, e)] -> [h, cells, n, j]
        return x.reshape(h_kv, -1, 4, G, 2, 2).permute(0, 1, 4, 2, 5, 3).reshape(h_kv, -1, 16, G)

    k = k * spread(half[:, :, 0]).unsqueeze(-1) + half[:, :, 1].reshape(h_kv, -1, 16, G, 1)
    v = v * spread(half[:, :, 2]).unsqueeze(-1) + spread(half[:, :, 3]).unsqueeze(-1)
    return k.reshape(h_kv, -1, d)[:, :n], v.reshape(h_kv, -1, d)[:, :n]


def _exact_gather(st, c):
    got = [_sequence(st, c, b) for b in range(c["batch"])]
    return {name: torch.cat([x[i].transpose(0, 1) for x in got]) for i, name in enumerate(("k", "v"))}


def _exact_decode(st, c):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    for b in range(c["batch"]):
        if st["n"][b]:
            k, v = _sequence(st, c, b)
            q = st["q"][b].double().view(c["h_kv"], -1, c["d"])
            w = torch.softmax(q @ k.transpose(1, 2) * c["d"] ** -0.5, -1)
            out[b] = (w @ v).view(-1, c["d"])
    return {"out": out}


def _exact_prompt(st, c):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    G, at, ak = c["h_q"] // c["h_kv"], 0, 0
    for nq, past in zip(st["n"], st["past"]):
        nk = nq + past
        for h in range(c["h_q"]):
            q = st["q"][at : at + nq, h].double()
            k, v = (st[x][ak : ak + nk, h // G].double() for x in ("k", "v"))
            for a in range(0, nq, 4096):
                s = q[a : a + 4096] @ k.T / math.sqrt(c["d"])
                rows = torch.arange(a, a + s.shape[0], device=s.device)[:, None]
                s[torch.arange(nk, device=s.device)[None] > rows + past] = -math.inf
                out[at + a : at + a + s.shape[0], h] = torch.softmax(s, -1) @ v
        at, ak = at + nq, ak + nk
    return {"out": out}

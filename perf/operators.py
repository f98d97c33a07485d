"""What is measured of the block-scaled 8-bit cache: appending to it, reading it back, attending over it.

The cache holds OCP E4M3 codes in 64-token blocks, [num_blocks][H_kv][64][d], with one fp32 scale
for each block and head, [num_blocks][H_kv], a power of two (0 for a block of zeros):

* append: the new K and V rows of every sequence (one token of a decode step, or a ragged run of a
  prompt) are quantised into their blocks.  A block whose first row is written starts afresh; a
  block that was begun earlier keeps its scale, or grows it and rounds its rows to the new one.
* read: a run of cached positions of every sequence, dequantised into dense rows.
* decode: attention of the last q_len positions of every sequence over its cached keys, query
  heads sharing K/V heads in contiguous groups, with an optional window and kept first positions.

Every case is a dict of plain values; the lengths of its sequences follow from it alone.
"""
import math

import torch

own = False

BLOCK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _append(name, B, H, d, start, new, dtype="bf16"):
    return {"name": name, "op": "append", "B": B, "H_kv": H, "d": d, "start_lo": start[0],
            "start_hi": start[1], "new_lo": new[0], "new_hi": new[1], "dtype": dtype}


def _read(name, B, H, d, start, new, dtype="bf16"):
    return {**_append(name, B, H, d, start, new, dtype), "op": "read"}


def _decode(name, B, H_q, H_kv, d, T, q_len=1, window=0, sink=0):
    return {"name": name, "op": "decode", "B": B, "H_q": H_q, "H_kv": H_kv, "d": d, "T_lo": T[0],
            "T_hi": T[1], "q_len": q_len, "window": window, "sink": sink}


def listed():
    return [
        # one decode step of a batch: a token a sequence, most blocks begun earlier
        _append("append step 16x8x128", 16, 8, 128, (4000, 4200), (1, 1)),
        # a chunk of several prompts at once, of odd lengths, after cached prefixes
        _append("append ragged chunks", 7, 8, 128, (0, 1000), (1, 3001)),
        # whole prompts of a model with as many K/V heads as query heads, K and V in fp32
        _append("append prompts f32", 8, 32, 64, (0, 0), (4096, 4096), "f32"),
        # cached prefixes of a few sequences, read back for a kernel that takes dense rows
        _read("read prefixes d256", 3, 4, 256, (0, 70), (100, 1500)),
        # a batch of long caches, read back whole
        _read("read long", 8, 8, 128, (0, 0), (8192, 8192)),
        # the smallest call: one sequence shortly after its start
        _decode("decode one short", 1, 4, 2, 64, (77, 77)),
        # an ordinary step: 32 query heads over 8 K/V heads
        _decode("decode 32/8/128 B16", 16, 32, 8, 128, (4096, 4096)),
        # every query head its own K/V head, long caches: the most bytes
        _decode("decode 32/32/128 B8", 8, 32, 32, 128, (32768, 32768)),
        # all query heads over one K/V head, long caches: the most arithmetic for a byte
        _decode("decode 32/1/128 B8", 8, 32, 1, 128, (32768, 32768)),
        # a window layer with kept first tokens, wide heads, ragged lengths
        _decode("decode 24/4/256 window", 16, 24, 4, 256, (1024, 32768), 1, 4096, 64),
        # one long sequence alone: the key axis has to be split
        _decode("decode 32/8/128 long", 1, 32, 8, 128, (131071, 131071)),
        # drafted tokens being verified: five query positions a sequence
        _decode("decode five drafted", 12, 32, 8, 128, (300, 9000), 5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode"])
    d = rng.choice([64, 128, 256])
    B = _log_int(rng, 1, 48)
    if op != "decode":
        H = rng.choice([1, 2, 4, 8, 12, 32])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = max(1, min(9000, 8 * 4096 * 32 * 64 // (B * H * d)))     # tokens a sequence
        single = op == "append" and rng.random() < 0.3
        hi = 1 if single else _log_int(rng, 1, most)
        lo = max(1, int(hi * rng.uniform(0.1, 1)))
        start = rng.choice([0, 1, 63, 64, _log_int(rng, 1, 4000)])
        return _append("", B, H, d, (start // 2, start), (lo, hi), dtype) | {"op": op, "name": ""}
    H_q, H_kv = rng.choice([(4, 2), (8, 8), (32, 8), (24, 4), (32, 1), (32, 32), (12, 1), (40, 8)])
    q_len = rng.choice([1, 1, 1, 2, 3, 6])
    most = max(2, min(131072, 2 ** 30 // (B * H_kv * d)))               # tokens a sequence
    hi = _log_int(rng, 2, most)
    lo = max(1, int(hi * rng.uniform(0.05, 1)))
    window, sink = rng.choice([(0, 0), (0, 0), (_log_int(rng, 1, 5000), 0),
                               (_log_int(rng, 1, 5000), rng.randint(1, 200))])
    return _decode("", B, H_q, H_kv, d, (lo, hi), q_len, window, sink)


def _spread(lo, hi, B, shift):
    """B whole numbers over [lo, hi], both ends among them where B > 1, in no order."""
    if B == 1 or lo == hi:
        return [hi] * B
    return [lo + round((hi - lo) * (((i * 0.6180339887498949 + shift) % 1.0) if 1 < i else float(i)))
            for i in range(B)]


def _lengths(case):
    """Host lists of a case: (starts, counts) of its token runs, or its cached lengths."""
    if case["op"] == "decode":
        return _spread(case["T_lo"], case["T_hi"], case["B"], 0.37)
    return (_spread(case["start_lo"], case["start_hi"], case["B"], 0.11),
            _spread(case["new_lo"], case["new_hi"], case["B"], 0.53))


# ------------------------------------------------------------------ inputs

def _cache(gen, num_blocks, H, d):
    """Codes and block scales as left by rows of unit variance.  The largest of 64 d normal values
    is near 4, so a block's scale is 2^-7 or 2^-6 (448 times it has to reach the largest)."""
    scale = torch.exp2(torch.randint(-7, -5, (num_blocks, H), generator=gen, device="cuda").float())
    codes = torch.empty((num_blocks, H, BLOCK, d), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (H * BLOCK * d))
    for i in range(0, num_blocks, step):
        s = scale[i:i + step, :, None, None]
        x = torch.randn((s.shape[0], H, BLOCK, d), generator=gen, device="cuda") / s
        codes[i:i + step] = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def _table(gen, blocks):
    """Block table of sequences that hold `blocks` blocks each: a permutation of the pool, -1 behind."""
    total, width = sum(blocks), max(blocks)
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(blocks), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, d = case["B"], case["H_kv"], case["d"]

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")
    s = {"case": dict(case)}
    if case["op"] == "decode":
        lens = _lengths(case)
        table, total = _table(gen, [-(-t // BLOCK) for t in lens])
        s["seq_lens"] = ints(lens)
        shape = (B, case["q_len"], case["H_q"], d)
        s["q"] = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    else:
        starts, counts = _lengths(case)
        table, total = _table(gen, [-(-(p + n) // BLOCK) for p, n in zip(starts, counts)])
        offsets = [0]
        for n in counts:
            offsets.append(offsets[-1] + n)
        s["positions"], s["counts"], s["offsets"] = ints(starts), ints(counts), ints(offsets)
        s["tokens"] = offsets[-1]
        dtype = DTYPES[case["dtype"]]
        shape = (offsets[-1], H, d)
        if case["op"] == "append":
            s["k_new"] = torch.randn(shape, generator=gen, device="cuda").to(dtype)
            s["v_new"] = torch.randn(shape, generator=gen, device="cuda").to(dtype)
    s["table"] = table
    s["k"], s["k_scale"] = _cache(gen, total, H, d)
    s["v"], s["v_scale"] = _cache(gen, total, H, d)
    if case["op"] == "append":
        # the codes as the values they are (the same memory)
        s["k_values"], s["v_values"] = (s[n].view(torch.float8_e4m3fn) for n in ("k", "v"))
    return s


# ------------------------------------------------------------------ plain forms

def _positions(s):
    """Sequence, physical block and row of every token of a ragged run."""
    n = s["tokens"]
    seq = torch.repeat_interleave(torch.arange(s["table"].shape[0], device="cuda"),
                                  s["counts"].long(), output_size=n)
    pos = (s["positions"].long()[seq] + torch.arange(n, device="cuda") - s["offsets"].long()[seq])
    return s["table"].long()[seq, pos // BLOCK], pos % BLOCK


def _power_of_two_scale(amax):
    """The smallest power of two s, at least 2^-126, with amax <= 448 s; 0 for amax = 0."""
    m, e = torch.frexp(amax)                               # amax = m 2^e, m in [0.5, 1)
    e = e - 9 + (m > 448.0 / 512.0).to(e.dtype)            # 448 = (7/8) 2^9
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e.clamp(min=-126)), 0.0)


def _to_codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _append_one(s, new, codes, scale, phys, row):
    x = new.float()
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=2)                  # [tokens][H]
    need = torch.zeros_like(scale).index_reduce_(0, phys, amax, "amax")
    new_block = torch.zeros_like(scale[:, :1]).index_reduce_(
        0, phys, (row == 0).float()[:, None], "amax") > 0
    old = torch.where(new_block, 0.0, scale)
    grown = torch.maximum(old, _power_of_two_scale(need))
    # rows cached earlier in the block that each sequence's run begins in
    first = s["positions"].long()
    block = s["table"].long().gather(1, (first // BLOCK)[:, None])[:, 0]
    kept = codes[block]
    ratio = torch.where(grown > 0, scale / grown, 1.0)[block][:, :, None, None]
    again = _to_codes(kept.view(torch.float8_e4m3fn).float() * ratio)
    earlier = torch.arange(BLOCK, device="cuda")[None, :] < (first % BLOCK)[:, None]
    codes[block] = torch.where(earlier[:, None, :, None], again, kept)
    scale.copy_(grown)
    by = grown[phys][:, :, None]
    codes[phys, :, row] = _to_codes(torch.where(by > 0, x / by, 0.0))


def _plain_append(s):
    phys, row = _positions(s)
    _append_one(s, s["k_new"], s["k"], s["k_scale"], phys, row)
    _append_one(s, s["v_new"], s["v"], s["v_scale"], phys, row)


def _plain_read(s):
    phys, row = _positions(s)
    dtype = DTYPES[s["case"]["dtype"]]

    def one(codes, scale):
        x = codes[phys, :, row].view(torch.float8_e4m3fn).float()
        return (x * scale[phys][:, :, None]).to(dtype)
    return {"k": one(s["k"], s["k_scale"]), "v": one(s["v"], s["v_scale"])}


def _plain_decode(s):
    c = s["case"]
    B, L, H_q, H, d = c["B"], c["q_len"], c["H_q"], c["H_kv"], c["d"]
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * BLOCK

    def dense(codes, scale):
        x = codes[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, n, d)
    k, v = dense(s["k"], s["k_scale"]), dense(s["v"], s["v_scale"])
    q = s["q"].float().reshape(B, L, H, H_q // H, d).permute(0, 2, 1, 3, 4).reshape(B, H, -1, d)
    score = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    at = s["seq_lens"].long()[:, None] - L + torch.arange(L, device="cuda")          # [B][L]
    j = torch.arange(n, device="cuda")
    seen = j <= at[:, :, None]
    if c["window"] > 0:
        seen &= (j > at[:, :, None] - c["window"]) | (j < c["sink"])
    seen = seen[:, None, :, None, :].expand(B, H, L, H_q // H, n).reshape(B, H, -1, n)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(dim=3, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(dim=3, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    out = out.reshape(B, H, L, H_q // H, d).permute(0, 2, 1, 3, 4).reshape(B, L, H_q, d)
    return out.to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import decode_attention_kv_paged_b200 as attn
        c = s["case"]
        if op == "append":
            attn.kv_append_fp8_block(s["k_new"], s["v_new"], s["k"], s["v"], s["k_scale"],
                                     s["v_scale"], s["positions"], s["table"],
                                     offsets=s["offsets"])
        elif op == "read":
            k, v = attn.kv_read_fp8_block(s["k"], s["v"], s["k_scale"], s["v_scale"],
                                          s["positions"], s["table"], s["tokens"],
                                          offsets=s["offsets"], dtype=DTYPES[c["dtype"]])
            return {"k": k, "v": v}
        else:
            if "workspace" not in s:       # kept by the program from its first step on
                s["workspace"] = attn.fp8_block_workspace(s["q"], s["k"])
            return {"out": attn.decode_gqa_fp8_block(
                s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["seq_lens"], s["table"],
                1.0 / math.sqrt(c["d"]), window=c["window"], sink_tokens=c["sink"],
                workspace=s["workspace"])}
    elif op == "append":
        _plain_append(s)
    elif op == "read":
        return _plain_read(s)
    else:
        return {"out": _plain_decode(s)}
    return {"k": s["k_values"], "v": s["v_values"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


# ------------------------------------------------------------------ work

def _visible(case, T, i):
    """Keys that query i of q_len sees in a sequence of T cached tokens."""
    at = T - case["q_len"] + i
    if at < 0:
        return 0
    if case["window"] <= 0 or at + 1 <= case["window"]:
        return at + 1
    return case["window"] + min(case["sink"], at + 1 - case["window"])


def work(case):
    H, d = case["H_kv"], case["d"]
    if case["op"] == "decode":
        keys = read = 0
        for T in _lengths(case):
            keys += sum(_visible(case, T, i) for i in range(case["q_len"]))
            # rows that any of the sequence's queries sees
            reach = dict(case, window=case["window"] + case["q_len"] - 1 if case["window"] else 0)
            read += _visible(reach, T, case["q_len"] - 1)
        rows = case["B"] * case["q_len"] * case["H_q"] * d
        return {"bytes": 2 * read * H * d + 2 * -(-read // BLOCK) * H * 4 + 2 * 2 * rows,
                "flops": 4 * keys * case["H_q"] * d}
    starts, counts = _lengths(case)
    size = 2 if case["dtype"] == "bf16" else 4
    blocks = sum((p + n - 1) // BLOCK - p // BLOCK + 1 for p, n in zip(starts, counts))
    n = 2 * sum(counts) * H * d
    return {"bytes": n * (1 + size) + 2 * blocks * H * 4 + 4 * blocks, "flops": 2 * n}


# ------------------------------------------------------------------ the definition, in 64 bits

def _value(codes):
    """The number that each E4M3 code is, from the format: sign, 4 bits of exponent with bias 7,
    3 bits of fraction; exponent 0 holds the subnormals; S.1111.111 is NaN."""
    c = torch.arange(256, device=codes.device)
    e, f = (c >> 3) & 15, (c & 7).double()
    size = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2((e - 7).double()))
    size = torch.where((c & 127) == 127, math.nan, size)
    return torch.where(c >= 128, -size, size)[codes.long()]


def _nearest(x):
    """The E4M3 number nearest to x, ties to the even one, at most 448 either way."""
    e = torch.frexp(x.abs())[1].clamp(min=-5) - 1          # x in [2^e, 2^(e+1)), or subnormal
    step = torch.exp2((e - 3).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    got = {}
    starts, counts = _lengths(s["case"])
    H, d = s["case"]["H_kv"], s["case"]["d"]
    for name in ("k", "v"):
        value, scale = _value(s[name]), s[name + "_scale"].double()
        at = 0
        for b, (p, n) in enumerate(zip(starts, counts)):
            lead, blocks = p % BLOCK, (p % BLOCK + n - 1) // BLOCK + 1
            ids = s["table"][b, p // BLOCK:p // BLOCK + blocks].long()
            x = torch.zeros((blocks * BLOCK, H, d), dtype=torch.float64, device="cuda")
            x[lead:lead + n] = s[name + "_new"][at:at + n].double()
            x = x.view(blocks, BLOCK, H, d).transpose(1, 2)            # [blocks][H][64][d]
            at += n
            amax = x.abs().amax(dim=(2, 3))
            need = torch.exp2(torch.ceil(torch.log2(amax / 448))).clamp(min=2.0 ** -126)
            need = torch.where(amax > 0, need, 0.0)
            held = scale[ids]
            held[1:] = 0
            if lead == 0:
                held[0] = 0
            s_new = torch.maximum(held, need)
            safe = torch.where(s_new > 0, s_new, 1.0)[:, :, None, None]
            coded = _nearest(x / safe)
            old = value[ids]
            rescaled = _nearest(old[0] * scale[ids][0][:, None, None] / safe[0])
            t = torch.arange(blocks * BLOCK, device="cuda").view(blocks, 1, BLOCK, 1)
            put = torch.where((t >= lead) & (t < lead + n), coded, old)
            put[0] = torch.where(t[0] < lead, rescaled, put[0])
            value[ids], scale[ids] = put, s_new
        got[name], got[name + "_scale"] = value, scale
    return got


def _exact_read(s):
    got = {"k": [], "v": []}
    for b, (p, n) in enumerate(zip(*_lengths(s["case"]))):
        ids = s["table"][b, p // BLOCK:(p + n - 1) // BLOCK + 1].long()
        for name in got:
            x = _value(s[name][ids]) * s[name + "_scale"][ids].double()[:, :, None, None]
            x = x.transpose(1, 2).reshape(-1, *x.shape[1:2], x.shape[3])
            got[name].append(x[p % BLOCK:p % BLOCK + n])
    return {name: torch.cat(rows) for name, rows in got.items()}


def _exact_decode(s):
    c = s["case"]
    L, G = c["q_len"], c["H_q"] // c["H_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, T in enumerate(_lengths(c)):
        ids = s["table"][b, :-(-T // BLOCK)].long()
        for h in range(c["H_kv"]):
            k, v = (_value(s[n][ids, h]) * s[n + "_scale"][ids, h].double()[:, None, None]
                    for n in ("k", "v"))
            k, v = (x.reshape(-1, c["d"])[:T] for x in (k, v))
            heads = slice(h * G, (h + 1) * G)
            for i in range(max(0, L - T), L):
                at = T - L + i
                keys = torch.arange(at + 1, device="cuda")
                if c["window"] > 0:
                    keys = keys[(keys > at - c["window"]) | (keys < c["sink"])]
                w = torch.softmax(s["q"][b, i, heads].double() @ k[keys].T / math.sqrt(c["d"]), -1)
                out[b, i, heads] = w @ v[keys]
    return {"out": out}


def exact(case, seed):
    # one state is made and read; a case of several hundred (sequence, head) pairs of long caches
    # takes a few seconds
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "decode": _exact_decode}[case["op"]](s)

"""Cases, plain forms and 64-bit forms of the operators on the 8-bit key/value cache.

The cache holds keys and values of decoded tokens as 8-bit integers, in blocks of `block` tokens that a block
table strings together per sequence, with one fp32 scale for each block and head (keys and values apart).
Three operators work on it:

  write      new tokens' keys and values are quantised into the cache: with a the largest magnitude that the
             new tokens of a block have in a head, the head's scale in that block becomes fl(a / 127), or, where
             the block already holds earlier tokens, the larger of that and the scale it has; then a value x has
             the code clamp(rint(fl(x / scale)), -127, 127), and earlier codes q of a block whose scale grew
             become rint(fl(fl(q * old) / new)), all in fp32 with one rounding an operation
  read       a range of positions of each sequence comes back as numbers, fl(code * scale)
  attention  softmax(scale * q . k) . v over the cached tokens that a query may see: those up to its own
             position (the last query of a sequence stands at the sequence's last token), and with a window only
             the last `window` of these; query heads share a key/value head in groups; a query that sees
             nothing gives zeros

Case fields: kind; batch sequences; past tokens in the cache before the call and new ones of the call (both the
longest sequence's: sequence b has a share of them between 1 - ragged and 1); idle sequences without any cached
token; kv_heads, group (query heads for each), head_dim, block; dtype of k, v and q; out, the type of what comes
back; window (0: none).
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def _case(name, kind, **kw):
    c = dict(name=name, kind=kind, batch=1, past=0, new=1, ragged=0.0, idle=0, kv_heads=8, group=1, head_dim=128,
             block=64, dtype="bf16", out="bf16", window=0)
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token: 8 heads of 128 (a 1024-wide k and v projection); latency is all that counts
        _case("append-one", "write", past=530, out="f32"),
        # a decode step of a serving batch, k and v straight from the fp32 products of the projections
        _case("append-batch", "write", batch=64, past=4095, ragged=0.9, idle=3, dtype="f32"),
        # a prompt that continues a short one: the first block is partly filled already
        _case("prompt", "write", past=37, new=2011),
        # many long prompts of different lengths: as fast as memory allows
        _case("prompts-many", "write", batch=16, past=100, new=8192, ragged=0.5),
        # a short cache read back in full precision, heads of 64 in blocks of 32
        _case("read-one", "read", past=777, head_dim=64, block=32, out="f32"),
        # caches of a batch brought back, to be moved or to be used by another program
        _case("read-many", "read", batch=16, past=8192, ragged=0.5),
        # one user's next token, 32 query heads on 8
        _case("decode-one", "attention", past=776, group=4),
        # a decode step of a serving batch, 64 query heads on 8, q straight from the fp32 product, two idle slots
        _case("decode-batch", "attention", batch=32, past=4096, ragged=0.6, idle=2, group=8, dtype="f32"),
        # a decode step over long documents
        _case("decode-long", "attention", batch=4, past=131071, group=8),
        # five proposed tokens a sequence checked at once, heads of 64 and a sliding window
        _case("check-draft", "attention", batch=8, past=3000, new=5, ragged=0.4, group=4, head_dim=64, block=32,
              window=1024),
        # prompts from their start, the query rows of a 2048-token prefill
        _case("prefill", "attention", batch=2, new=2048, ragged=0.3, group=4),
        # the last piece of a long prompt that is taken in pieces
        _case("prefill-piece", "attention", past=30001, new=2048, group=8, block=128),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    kind = rng.choice(["write", "write", "read", "attention", "attention", "attention"])
    c = _case("", kind, kv_heads=rng.choice([1, 2, 3, 4, 5, 8, 8, 16]), head_dim=rng.choice([64, 128, 128, 256]),
              block=rng.choice([32, 64, 64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
              ragged=round(rng.uniform(0.0, 0.9), 2))
    del c["name"]
    width = c["kv_heads"] * c["head_dim"]
    if kind != "attention":
        c["out"] = rng.choice(["bf16", "f32"])
        most = 64_000_000 // width  # tokens: under what the largest listed ones of these kinds have
        if kind == "read":
            c["past"] = _log(rng, 1, min(most, 30000))
            c["new"] = 0
            c["batch"] = _log(rng, 1, max(1, min(64, most // c["past"])))
        elif rng.random() < 0.5:
            c["past"], c["new"] = _log(rng, 1, 10000), rng.choice([1, 1, 2, 5])
            c["batch"] = _log(rng, 1, 128)
        else:
            c["past"], c["new"] = rng.choice([0, rng.randrange(1, 500)]), _log(rng, 2, min(most, 10000))
            c["batch"] = _log(rng, 1, max(1, min(64, most // c["new"])))
        c["idle"] = rng.randrange(0, c["batch"]) // 4
        return c
    c["window"] = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    if rng.random() < 0.6:  # a few query tokens over a long cache
        c["new"] = rng.choice([1, 1, 1, 2, 3, 5])
        c["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        c["past"] = _log(rng, 1, min(130000, 400_000_000 // width))
        c["batch"] = _log(rng, 1, max(1, min(64, 400_000_000 // (width * c["past"]))))
        c["idle"] = rng.randrange(0, c["batch"]) // 4
        return c
    c["group"] = rng.choice([1, 2, 3, 4, 8])
    c["new"] = _log(rng, 16, 4096)
    c["past"] = rng.choice([0, _log(rng, 1, 16000)])
    pairs = 400_000_000_000 // (width * c["group"] * c["new"] * (c["new"] + c["past"]))
    while pairs < 1:  # too much work for one sequence: fewer query heads, then a shorter piece
        if c["group"] > 1:
            c["group"] = 1
        else:
            c["new"] = c["new"] // 2 + 1
        pairs = 400_000_000_000 // (width * c["group"] * c["new"] * (c["new"] + c["past"]))
    c["batch"] = _log(rng, 1, min(16, pairs))
    return c


def _lengths(case):
    """(past, new) of each sequence."""
    share = [1.0 - case["ragged"] * ((0.6180339887498949 * b) % 1.0) for b in range(case["batch"])]
    past = [int(round(case["past"] * s)) for s in share]
    new = [max(1, int(round(case["new"] * s))) if case["new"] else 0 for s in share]
    for b in range(case["batch"] - case["idle"], case["batch"]):
        past[b] = 0
        if case["kind"] == "attention":
            new[b] = -new[b]  # query rows of a slot without tokens
        else:
            new[b] = 0
    return past, new


def work(case):
    past, new = _lengths(case)
    h, d, blk = case["kv_heads"], case["head_dim"], case["block"]
    size = 4 if case["dtype"] == "f32" else 2
    back = 4 if case["out"] == "f32" else 2
    blocks = lambda a, b: 2 * 4 * h * max(0, -(-b // blk) - a // blk)  # scales of a range of positions
    if case["kind"] == "read":
        n = sum(past)
        return {"bytes": 2 * n * h * d * (1 + back) + sum(blocks(0, p) for p in past), "flops": 2 * n * h * d}
    if case["kind"] == "write":
        n = sum(new)
        seen = sum(p + m - p // blk * blk for p, m in zip(past, new) if m)
        return {"bytes": 2 * n * h * d * (size + 1) + 2 * seen * h * d * (1 + back)
                + 2 * sum(blocks(p, p + m) for p, m in zip(past, new)), "flops": 2 * (3 * n + seen) * h * d}
    rows, kv, scales, pairs = 0, 0, 0, 0
    for p, m in zip(past, new):
        rows += abs(m)
        if m <= 0:
            continue
        w = case["window"] or p + m
        lo = max(0, p + 1 - w)
        kv += p + m - lo
        scales += blocks(lo, p + m)
        pairs += sum(min(w, p + i + 1) for i in range(m))
    return {"bytes": rows * h * case["group"] * d * (size + back) + 2 * kv * h * d + scales,
            "flops": 4 * pairs * h * case["group"] * d}


# ---------------------------------------------------------------- inputs

def _inputs(case, seed):
    """Random keys, values and queries of every token, and a block table, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    past, new = _lengths(case)
    h, d, blk, B = case["kv_heads"], case["head_dim"], case["block"], case["batch"]
    real = [max(0, m) for m in new]
    total = [p + m for p, m in zip(past, real)]
    typ = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def normal(n, heads, spread):
        x = torch.randn(n, heads, d, generator=g, device="cuda")
        return (x * spread).to(typ)

    # a few strong channels in each head's keys, tokens of different weight in the values
    strong = 1.0 + 4.0 * (torch.rand(1, h, d, generator=g, device="cuda") < 0.03)
    # tokens of the call come apart from those that the cache has already
    def tokens(n):
        return normal(n, h, strong), normal(n, h, torch.exp(0.4 * torch.randn(n, 1, 1, generator=g, device="cuda")))

    width = max(1, max(-(-t // blk) for t in total))
    blocks = B * width
    table = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).view(B, width)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    offsets = lambda v: i32([sum(v[:b]) for b in range(B + 1)])
    x = dict(past=past, new=new, real=real, total=total, table=table, blocks=blocks, i32=i32, offsets=offsets)
    if case["kind"] == "attention":
        x["k"], x["v"] = tokens(sum(total))
        x["q"] = normal(sum(abs(m) for m in new), h * case["group"], 1.0)
    else:
        # of the tokens before the call, a write meets those in the block that it goes on with
        x["before"] = [p % blk if m else 0 for p, m in zip(past, real)] if case["kind"] == "write" else past
        x["at"] = [p - n for p, n in zip(past, x["before"])]
        x["k_before"], x["v_before"] = tokens(sum(x["before"]))
        x["k"], x["v"] = tokens(sum(real))
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    i32, offsets, h, d, blk = x["i32"], x["offsets"], case["kv_heads"], case["head_dim"], case["block"]
    # a program keeps its cache in the framework's layout: it is made and filled by the framework's own calls there
    if own:
        import block_wise_mixed_amd as msq
        cache = msq.allocate_kv_cache(x["blocks"], h, d, blk)
    else:
        cache = _plain_cache(x["blocks"], h, d, blk)

    def write(k, v, at, count):
        if sum(count) == 0:
            return
        args = (cache, k, v, x["table"], i32(at), offsets(count))
        if own:
            msq.kv_write(*args, max_count=max(count))
        else:
            _plain_write(*args, max(count))

    s = dict(case=case, cache=cache, table=x["table"], out=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    if case["kind"] == "attention":
        write(x["k"], x["v"], [0] * len(x["total"]), x["total"])
        rows = [abs(m) for m in x["new"]]
        s.update(q=x["q"], kv_len=i32(x["total"]), max_kv_len=max(x["total"]), offset=offsets(rows), max_count=max(rows))
        if own:
            need = msq.kv_attention_workspace_bytes(cache, sum(rows), h * case["group"], len(rows), max(rows),
                                                    max(x["total"]), window=case["window"])
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        return s
    write(x["k_before"], x["v_before"], x["at"], x["before"])
    if case["kind"] == "write":
        s.update(k=x["k"], v=x["v"], first=i32(x["past"]), offset=offsets(x["real"]), max_count=max(x["real"]))
        back = [p + m - p // blk * blk if m else 0 for p, m in zip(x["past"], x["real"])]
        s["back_first"] = i32([p // blk * blk for p in x["past"]])
    else:
        back = x["past"]
        s["back_first"] = i32([0] * len(back))
    s.update(back_offset=offsets(back), back_total=sum(back), back_max=max(back))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        import block_wise_mixed_amd as msq
        if c["kind"] == "attention":
            return msq.kv_attention(s["q"], s["cache"], s["table"], s["kv_len"], s["offset"], max_count=s["max_count"],
                                    max_kv_len=s["max_kv_len"], window=c["window"], out_dtype=s["out"],
                                    workspace=s["workspace"])
        if c["kind"] == "write":
            msq.kv_write(s["cache"], s["k"], s["v"], s["table"], s["first"], s["offset"], max_count=s["max_count"])
        k, v = msq.kv_read(s["cache"], s["table"], s["back_first"], s["back_offset"], total=s["back_total"],
                           max_count=s["back_max"], dtype=s["out"])
    else:
        if c["kind"] == "attention":
            return _plain_attention(s)
        if c["kind"] == "write":
            _plain_write(s["cache"], s["k"], s["v"], s["table"], s["first"], s["offset"], s["max_count"])
        k, v = _plain_read(s["cache"], s["table"], s["back_first"], s["back_offset"], s["back_total"], s["out"])
    if c["kind"] == "read":
        return {"k": k, "v": v}
    if own:
        return {"k": k, "v": v, "k_scale": s["cache"].k_scale, "v_scale": s["cache"].v_scale}
    # the plain cache ends with one block that takes what belongs nowhere
    return {"k": k, "v": v, "k_scale": s["cache"]["k_scale"][:-1], "v_scale": s["cache"]["v_scale"][:-1]}


# ---------------------------------------------------------------- plain forms

def _plain_cache(blocks, h, d, blk):
    codes = lambda: torch.zeros(blocks + 1, h, blk, d, dtype=torch.int8, device="cuda")
    scale = lambda: torch.zeros(blocks + 1, h, device="cuda")
    return dict(k=codes(), v=codes(), k_scale=scale(), v_scale=scale(), block=blk)


def _plain_write(cache, k, v, table, first, offset, max_count):
    """Every block that a sequence's new tokens can reach, all at once: [batch, reach, block slot, head, dim]."""
    blk = cache["block"]
    nowhere = cache["k"].shape[0] - 1
    reach = (max_count + blk - 2) // blk + 1
    count = offset[1:] - offset[:-1]
    at = torch.div(first, blk, rounding_mode="floor")[:, None] + torch.arange(reach, device="cuda")
    place = at[..., None] * blk + torch.arange(blk, device="cuda")
    is_new = (place >= first[:, None, None]) & (place < (first + count)[:, None, None])
    is_old = (place < first[:, None, None]) & (count > 0)[:, None, None]
    row = (offset[:-1] - first)[:, None, None] + place
    row = torch.where(is_new, row, 0).long()
    ids = torch.gather(table, 1, at.clamp(max=table.shape[1] - 1).long())
    ids = torch.where(is_new.any(-1), ids, nowhere).long()
    is_new, is_old = is_new[..., None, None], is_old[..., None, None]
    begun = is_old.any(2)[..., 0]  # the block holds earlier tokens
    _plain_quantise(cache["k"], cache["k_scale"], k, row, ids, is_new, is_old, begun)
    _plain_quantise(cache["v"], cache["v_scale"], v, row, ids, is_new, is_old, begun)


def _plain_quantise(codes, scales, values, row, ids, is_new, is_old, begun):
    x = torch.where(is_new, values[row].float(), 0.0)
    top = x.abs().amax(dim=(2, 4))
    scale = top / torch.full_like(top, 127.0)
    had = torch.where(begun, scales[ids], 0.0)
    scale = torch.maximum(scale, had)
    by = torch.where(scale > 0, scale, 1.0)[:, :, None, :, None]
    x = torch.clamp(torch.round(x / by), -127, 127)
    q = codes[ids].transpose(2, 3)
    grown = torch.round(q.float() * had[:, :, None, :, None] / by)
    q = torch.where((scale > had)[:, :, None, :, None], grown, q.float())
    q = torch.where(is_new, x, torch.where(is_old, q, 0.0))
    codes[ids] = q.to(torch.int8).transpose(2, 3)
    scales[ids] = scale


def _plain_rows(offset, total):
    """(sequence, index within it) of each of the rows that the sequences' ranges take in turn."""
    seq = torch.repeat_interleave(torch.arange(offset.numel() - 1, device="cuda"), (offset[1:] - offset[:-1]).long(),
                                  output_size=total)
    return seq, torch.arange(total, device="cuda") - offset[seq]


def _plain_read(cache, table, first, offset, total, out):
    blk = cache["block"]
    seq, i = _plain_rows(offset, total)
    place = first[seq] + i
    ids = table[seq, torch.div(place, blk, rounding_mode="floor")].long()
    slot = place % blk
    k = cache["k"][ids, :, slot].float() * cache["k_scale"][ids][..., None]
    v = cache["v"][ids, :, slot].float() * cache["v_scale"][ids][..., None]
    return k.to(out), v.to(out)


def _plain_attention(s):
    """All sequences padded to the longest: scores [batch, kv head, query token * group, cached token]."""
    c, cache = s["case"], s["cache"]
    B, h, g, d, blk = c["batch"], c["kv_heads"], c["group"], c["head_dim"], c["block"]
    n, length = s["max_count"], s["max_kv_len"]
    offset, q = s["offset"], s["q"]
    count = offset[1:] - offset[:-1]
    i = torch.arange(n, device="cuda")
    row = torch.where(i < count[:, None], offset[:-1, None] + i, 0).long()
    q = q[row].float().view(B, n, h, g, d).permute(0, 2, 1, 3, 4).reshape(B, h, n * g, d)
    width = max(1, -(-length // blk))
    ids = s["table"][:, :width].long()

    def cached(codes, scale):
        x = codes[ids].float() * scale[ids][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, h, width * blk, d)

    scores = torch.matmul(q, cached(cache["k"], cache["k_scale"]).transpose(2, 3))
    scores *= 1.0 / math.sqrt(d)
    place = torch.arange(width * blk, device="cuda")
    stands = (s["kv_len"] - count)[:, None] + i
    sees = place <= stands[..., None]
    if c["window"]:
        sees &= place > stands[..., None] - c["window"]
    sees = sees[:, None, :, None, :]
    scores.view(B, h, n, g, -1).masked_fill_(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores -= torch.where(top == -math.inf, 0.0, top)
    scores.exp_()
    total = scores.sum(-1, keepdim=True)
    o = torch.matmul(scores, cached(cache["v"], cache["v_scale"]))
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(B, h, n, g, d).permute(0, 2, 1, 3, 4).reshape(B, n, h * g, d)
    seq, at = _plain_rows(offset, s["q"].shape[0])
    return o[seq, at].to(s["out"])


# ---------------------------------------------------------------- 64 bits

def _exact_block(x, code, old, begun):
    """Codes and scale of one block: x [tokens, head, dim] new values, code the earlier tokens' codes. The roundings to
    32 bits are part of the definition; a 64-bit quotient of 32-bit numbers, rounded to 32, is the 32-bit quotient."""
    f32 = lambda t: t.to(torch.float32).double()
    scale = f32(x.abs().amax(dim=(0, 2)) / 127.0)
    if begun:
        scale = torch.maximum(scale, old)
    by = torch.where(scale > 0, scale, 1.0)[None, :, None]
    new = torch.round(f32(x / by)).clamp(-127, 127)
    if begun:
        moved = torch.round(f32(f32(code * old[None, :, None]) / by))
        code = torch.where((scale > old)[None, :, None], moved, code)
        new = torch.cat([code, new])
    return new, scale


def _exact_fill(x, blk, code=None, scale=None):
    """Codes [tokens, head, dim] and scales [blocks, head] of a run of tokens; code, scale: its first block's so far."""
    codes, scales, at = [], [], 0
    have = 0 if code is None else code.shape[0]
    while at < x.shape[0]:
        n = min(blk - have, x.shape[0] - at)
        q, s = _exact_block(x[at:at + n], code, scale, have > 0)
        codes.append(q)
        scales.append(s)
        at, have = at + n, 0
    return torch.cat(codes), torch.stack(scales)


def exact(case, seed):
    x = _inputs(case, seed)
    h, d, blk, g = case["kv_heads"], case["head_dim"], case["block"], case["group"]
    if case["kind"] == "attention":
        outs, at, rows = [], 0, 0
        for m, p, n in zip(x["new"], x["past"], x["total"]):
            q = x["q"][rows:rows + abs(m)].double().view(abs(m), h, g, d)
            o = torch.zeros_like(q)
            rows += abs(m)
            if n:
                both = []
                for t in (x["k"], x["v"]):
                    code, scale = _exact_fill(t[at:at + n].double(), blk)
                    both.append(code * scale.repeat_interleave(blk, 0)[:n, :, None])
                k, v = both
                j = torch.arange(n, device="cuda")
                stands = p + torch.arange(m, device="cuda")
                sees = j[None, :] <= stands[:, None]
                if case["window"]:
                    sees &= j[None, :] > stands[:, None] - case["window"]
                for e in range(h * g):
                    w = q[:, e // g, e % g] @ k[:, e // g].T / math.sqrt(d)
                    o[:, e // g, e % g] = torch.softmax(w.masked_fill(~sees, -math.inf), -1) @ v[:, e // g]
            at += n
            outs.append(o.reshape(abs(m), h * g, d))
        return torch.cat(outs)
    result = {}
    for name in ("k", "v"):
        back = []
        scales = torch.zeros(x["blocks"], h, dtype=torch.float64, device="cuda")
        before = new = 0
        for b in range(case["batch"]):
            p, m, had = x["past"][b], x["real"][b], x["before"][b]
            code = scale = None
            if had:
                code, scale = _exact_fill(x[name + "_before"][before:before + had].double(), blk)
            if case["kind"] == "write" and m:
                part = (code, scale[0]) if had else (None, None)
                code, scale = _exact_fill(x[name][new:new + m].double(), blk, *part)
                ids = x["table"][b, p // blk:p // blk + scale.shape[0]].long()
                scales[ids] = scale
            elif case["kind"] == "write":
                code = None
            if code is not None:
                back.append(code * scale.repeat_interleave(blk, 0)[:code.shape[0], :, None])
            before, new = before + had, new + m
        result[name] = torch.cat(back)
        if case["kind"] == "write":
            result[name + "_scale"] = scales
    return result if case["kind"] == "read" else {n: result[n] for n in ("k", "v", "k_scale", "v_scale")}

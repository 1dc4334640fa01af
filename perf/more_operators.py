"""Cases, plain forms and 64-bit forms of the operators with which drafted tokens are served from the 8-bit cache.

A small model drafts some tokens of a sequence, as a chain or as a tree; the large one looks at all of them in one
pass, and as many are kept as its own probabilities allow.  Rows of a call are nodes: row 0 of a sequence is the
last token that is certain, the others are drafted, each below a parent with a smaller row number.

  rotate   positions into queries or keys: of the first `part` dims of a head the values a, b of pair i become
           a cos - b sin, b cos + a sin with the angle position * frequency i; pairs are the dims i and part / 2 + i
           (half) or 2 i and 2 i + 1 (pairs).  cos and sin of fl64(position * frequency), times the amplitude, are
           rounded to 32 bits, and the rest is in 32 bits with one rounding an operation
  append   keys rotated to their positions and quantised into the cache with their values (the quantiser of
           perf/operators.py), queries rotated on the way
  tree     from the parents, for each row the set of its call's rows that it sees (itself and its ancestors, as bits
           of 32-bit words) and its position, the sequence's first one and its depth
  attend   softmax(scale * q . k) . v over the cached tokens before the call's rows and, of these, the ones that a
           row's set has; with a window the last `window` of them all
  verify   goes down the tree: a drafted child x of the row reached is taken if u q(x) m < r(x), where r begins as
           the target's probabilities there (m = 1) and after each child that is not taken becomes max(r / m - q, 0),
           m its sum (without draft probabilities q(x) = 1 and r(x) becomes 0, m falls by it); where none is taken
           the next token is the first whose running sum of r passes u times its sum (r as at the start if that is
           0).  Without numbers u: a child is taken if it is the target's largest entry, which is the next token else

Case fields: kind; batch sequences; past tokens in the cache before the call and new rows of the call (both the
longest sequence's: sequence b has a share of them between 1 - ragged and 1); idle sequences without any cached
token (attend) or any row (append); first, the position that the sequence's tokens begin at (rotate); kv_heads,
group (query heads for each), head_dim, block; dtype of what comes in; out, of what comes back; layout, part, base,
factor, original of the rotation; window (0: none); chain (no tree); vocab; draft (draft probabilities are there);
greedy (no numbers u).
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def _case(name, kind, **kw):
    c = dict(name=name, kind=kind, batch=1, past=0, new=1, ragged=0.0)
    if kind in ("rotate", "append"):
        c.update(kv_heads=8, group=1, head_dim=128, dtype="bf16", out="bf16", layout="half", part=128, base=10000.0,
                 factor=1.0, original=0, first=0)
    if kind in ("append", "attend"):
        c.update(kv_heads=8, group=4, head_dim=128, block=64, dtype="bf16", out="bf16", idle=0)
    if kind == "attend":
        c.update(window=0)
    if kind == "verify":
        c.update(vocab=32000, dtype="f32", draft=False, greedy=False, chain=False)
    c.update(kw)
    return c


def listed():
    return [
        # queries of a decode step far into long documents, 64 heads straight from the fp32 product of the projection
        _case("rotate-step", "rotate", batch=64, new=1, kv_heads=64, first=100000, dtype="f32", out="f32",
              base=500000.0, factor=8.0, original=8192),
        # queries of a batch of prompts, neighbouring dims paired, half of each head
        _case("rotate-prompts", "rotate", batch=8, new=4096, ragged=0.3, kv_heads=32, layout="pairs", part=64),
        # a decode step of a serving batch: q, k and v straight from the fp32 products, some slots without a token
        _case("append-step", "append", batch=64, past=4095, ragged=0.9, idle=3, group=8, dtype="f32", out="f32",
              base=500000.0, factor=8.0, original=8192),
        # long prompts of different lengths: as fast as memory allows
        _case("append-prompts", "append", batch=16, past=100, new=8192, ragged=0.5),
        # one user's tree of drafted tokens
        _case("tree-one", "tree", new=26),
        # those of a large serving batch
        _case("tree-batch", "tree", batch=256, new=64, ragged=0.5),
        # one user's tree on a short text
        _case("attend-one", "attend", past=751, new=26),
        # trees of a serving batch, 64 query heads on 8, q in fp32, two idle slots
        _case("attend-batch", "attend", batch=32, past=4063, new=33, ragged=0.6, idle=2, group=8, dtype="f32"),
        # trees over long documents
        _case("attend-long", "attend", batch=4, past=131000, new=64, group=8, block=128),
        # chains of four drafted tokens against a large vocabulary, drafted from known probabilities
        _case("verify-chains", "verify", batch=64, new=5, vocab=128000, draft=True, chain=True),
        # one user's tree by its largest entries, the fp32 products of a last projection as they come
        _case("verify-one", "verify", new=26, greedy=True),
        # trees of a serving batch
        _case("verify-trees", "verify", batch=16, new=32, ragged=0.4, vocab=128000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotate", "append", "append", "tree", "attend", "attend", "verify", "verify"])
    c = _case("", kind, ragged=round(rng.uniform(0.0, 0.9), 2))
    del c["name"]
    if kind in ("rotate", "append"):
        c["head_dim"] = rng.choice([64, 128, 128, 256])
        c["part"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2, 16, 48])
        c["layout"] = rng.choice(["half", "half", "pairs"])
        c["base"] = rng.choice([10000.0, 500000.0])
        c["factor"], c["original"] = rng.choice([(1.0, 0), (4.0, 0), (8.0, 8192), (32.0, 4096)])
        c["dtype"], c["out"] = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"])
    if kind == "rotate":
        c["kv_heads"] = rng.choice([1, 2, 5, 8, 16, 32, 64, 71])
        c["first"] = rng.choice([0, _log(rng, 1, 1000000)])
        most = 100_000_000 // (c["kv_heads"] * c["head_dim"])
        c["new"] = _log(rng, 1, min(most, 16000))
        c["batch"] = _log(rng, 1, max(1, min(64, most // c["new"])))
    if kind in ("append", "attend"):
        c["kv_heads"] = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        c["block"] = rng.choice([32, 64, 64, 128])
    if kind == "append":
        c["group"] = rng.choice([1, 2, 3, 4, 8])
        most = 48_000_000 // (c["kv_heads"] * c["head_dim"] * c["group"])
        if rng.random() < 0.5:
            c["past"], c["new"] = _log(rng, 1, 10000), rng.choice([1, 1, 5, 26, 64])
            c["batch"] = _log(rng, 1, max(1, min(128, most // c["new"])))
        else:
            c["past"], c["new"] = rng.choice([0, rng.randrange(1, 500)]), _log(rng, 2, min(most, 10000))
            c["batch"] = _log(rng, 1, max(1, min(64, most // c["new"])))
        c["idle"] = rng.randrange(0, c["batch"]) // 4
    if kind == "tree":
        c["new"] = _log(rng, 1, 256)
        c["batch"] = _log(rng, 1, 16384 // c["new"] if c["new"] > 64 else 256)
        c["past"] = _log(rng, 1, 100000)
    if kind == "attend":
        c["head_dim"] = rng.choice([64, 128, 128, 256])
        c["dtype"], c["out"] = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"])
        c["group"] = rng.choice([1, 2, 3, 4, 5, 8, 16])
        c["window"] = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
        c["new"] = _log(rng, 1, 130)
        width = c["kv_heads"] * c["head_dim"]
        c["past"] = _log(rng, 1, min(100000, 400_000_000 // width))
        pairs = 100_000_000_000 // (width * c["group"] * c["new"] * c["past"])
        c["batch"] = _log(rng, 1, max(1, min(48, 400_000_000 // (width * c["past"]), pairs)))
        c["idle"] = rng.randrange(0, c["batch"]) // 4
    if kind == "verify":
        c["vocab"] = _log(rng, 500, 130000)
        c["new"] = rng.choice([1, 2, 5, 8, _log(rng, 1, 64)])
        c["batch"] = _log(rng, 1, max(1, min(128, 60_000_000 // (c["vocab"] * c["new"]))))
        c["dtype"] = rng.choice(["f32", "f32", "bf16"])
        c["draft"], c["greedy"] = rng.choice([(True, False), (False, False), (False, True)])
        c["chain"] = rng.random() < 0.4
    return c


def _lengths(case):
    """(past, new) of each sequence."""
    share = [1.0 - case["ragged"] * ((0.6180339887498949 * b) % 1.0) for b in range(case["batch"])]
    past = [int(round(case["past"] * s)) for s in share]
    new = [max(1, int(round(case["new"] * s))) for s in share]
    for b in range(case["batch"] - case.get("idle", 0), case["batch"]):
        past[b] = 0
        new[b] = 0 if case["kind"] == "append" else -new[b]  # query rows of a slot without tokens
    return past, new


def _size(name):
    return 4 if name == "f32" else 2


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def work(case):
    past, new = _lengths(case)
    rows = sum(abs(m) for m in new)
    if case["kind"] == "tree":
        words = -(-max(new) // 32)
        return {"bytes": 4 * (rows * (2 + words) + 2 * case["batch"]), "flops": rows}
    if case["kind"] == "verify":
        # the row where each sequence stops, with draft probabilities the drafter's too; by largest entries the rows
        # of the nodes that are taken, one of them at the least beside the first
        read = 2 if case["draft"] or case["greedy"] and case["new"] > 1 else 1
        n = case["batch"] * case["vocab"] * read
        return {"bytes": n * _size(case["dtype"]) + rows * 16, "flops": 3 * n}
    h, d, size, back = case["kv_heads"], case["head_dim"], _size(case["dtype"]), _size(case["out"])
    if case["kind"] == "rotate":
        return {"bytes": rows * (h * d * (size + back) + 4) + 4 * case["part"],
                "flops": rows * h * case["part"] * 3 + rows * case["part"] * 20}
    blk = case["block"]
    blocks = lambda a, b: 2 * 4 * h * max(0, -(-b // blk) - a // blk)  # scales of a range of positions
    if case["kind"] == "append":
        seen = sum(p + m - p // blk * blk for p, m in zip(past, new) if m)
        return {"bytes": 2 * rows * h * d * (size + 1) + rows * h * case["group"] * d * (size + back)
                + 2 * seen * h * d * (1 + back) + 2 * sum(blocks(p, p + m) for p, m in zip(past, new)),
                "flops": rows * h * (1 + case["group"]) * case["part"] * 3 + 2 * (3 * rows + seen) * h * d}
    kv, scales, pairs = 0, 0, 0
    for p, m in zip(past, new):
        if m <= 0:
            continue
        lo = max(0, p - case["window"] + 1) if case["window"] else 0
        kv += p + m - lo
        scales += blocks(lo, p + m)
        pairs += m * (p - lo + 1)  # and a few of the call's own rows
    return {"bytes": rows * h * case["group"] * d * (size + back) + 2 * kv * h * d + scales,
            "flops": 4 * pairs * h * case["group"] * d}


# ---------------------------------------------------------------- inputs

def _parents(g, new, chain=False):
    """int32 [rows]: the parent of each row, counted in its sequence, -1 for the first; most trees are wide near the
    root."""
    i = torch.cat([torch.arange(abs(m), device="cuda") for m in new])
    if chain:
        return (i - 1).to(torch.int32)
    u = torch.rand(i.numel(), generator=g, device="cuda", dtype=torch.float64)
    p = (u ** 1.5 * i).long().clamp(max=(i - 1))
    return torch.where(i > 0, p, -1).to(torch.int32)


def _frequencies(case):
    """float64 [part / 2] and the amplitude: base^(-2 i / part), divided by factor, or with an original length only
    where it holds fewer than 1 to 32 turns (in between, by the share of 32)."""
    i = torch.arange(0, case["part"], 2, dtype=torch.float64)
    f = torch.exp(-math.log(case["base"]) * i / case["part"])
    if not case["original"]:
        return (f / case["factor"]).cuda(), 1.0
    keep = ((case["original"] * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return (f * (keep + (1 - keep) / case["factor"])).cuda(), 0.1 * math.log(case["factor"]) + 1.0


def _inputs(case, seed):
    """Everything that a case starts from, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    past, new = _lengths(case)
    B = case["batch"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    offsets = lambda v: i32([0] + torch.tensor(v).cumsum(0).tolist())
    rows = [abs(m) for m in new]
    x = dict(past=past, new=new, rows=rows, i32=i32, offsets=offsets)
    if case["kind"] == "tree":
        x["parents"] = _parents(g, new)
        return x
    if case["kind"] == "verify":
        n, V = sum(rows), case["vocab"]
        x["parents"] = _parents(g, new, case["chain"])
        start = torch.tensor([0] + rows[:-1], device="cuda").cumsum(0)
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(rows, device="cuda"))
        above = (start[seq] + x["parents"]).clamp(min=0)  # row of the parent
        logits = 2.5 * torch.randn(n, V, generator=g, device="cuda")
        near = logits + 0.7 * torch.randn(n, V, generator=g, device="cuda")  # what the drafter thinks
        if case["draft"]:
            u = torch.rand(n, V, generator=g, device="cuda").clamp(min=1e-12)
            tokens = (near[above] - torch.log(-torch.log(u))).argmax(-1)  # drawn from its probabilities
            x["draft"] = torch.softmax(near, -1).to(_type(case["dtype"]))
        else:  # its likeliest tokens, in turn for the children of a row
            same = (above[:, None] == above[None, :]) & (x["parents"] >= 0)[None, :]
            rank = same.tril(-1).sum(-1)
            best = near.topk(min(V, 64), -1).indices
            tokens = best[above, rank.clamp(max=best.shape[1] - 1)]
        x["tokens"] = tokens.to(torch.int32)
        x["target"] = logits.to(_type(case["dtype"])) if case["greedy"] else torch.softmax(logits, -1).to(_type(case["dtype"]))
        x["uniform"] = torch.rand(n, generator=g, device="cuda")
        return x
    h, d = case["kv_heads"], case["head_dim"]
    typ = _type(case["dtype"])

    def normal(n, heads, spread):
        t = torch.randn(n, heads, d, generator=g, device="cuda")
        t *= spread
        return t.to(typ)

    if case["kind"] == "rotate":
        x["x"] = normal(sum(rows), h, 1.0)
        x["positions"] = torch.cat([torch.arange(m, device="cuda") + (case["first"] + 37 * b)
                                    for b, m in enumerate(rows)]).to(torch.int32)
        return x
    real = [max(0, m) for m in new]
    total = [p + m for p, m in zip(past, real)]
    # a few strong channels in each head's keys, tokens of different weight in the values
    strong = 1.0 + 4.0 * (torch.rand(1, h, d, generator=g, device="cuda") < 0.03)

    def tokens(n):
        return normal(n, h, strong), normal(n, h, torch.exp(0.4 * torch.randn(n, 1, 1, generator=g, device="cuda")))

    width = max(1, max(-(-t // case["block"]) for t in total))
    x["table"] = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    x.update(real=real, total=total, blocks=B * width)
    if case["kind"] == "attend":
        x["k"], x["v"] = tokens(sum(total))
        x["parents"] = _parents(g, new)
    else:
        # of the tokens before the call, an append meets those in the block that it goes on with
        x["before"] = [p % case["block"] if m else 0 for p, m in zip(past, real)]
        x["at"] = [p - n for p, n in zip(past, x["before"])]
        x["k_before"], x["v_before"] = tokens(sum(x["before"]))
        x["k"], x["v"] = tokens(sum(real))
    x["q"] = normal(sum(rows), h * case["group"], 1.0)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    i32, offsets, kind = x["i32"], x["offsets"], case["kind"]
    if own:
        import block_wise_mixed_amd as msq
    s = dict(case=case, offset=offsets(x["rows"]), max_count=max(x["rows"]))
    if kind == "tree":
        s.update(parents=x["parents"], first=i32(x["past"]))
        return s
    if kind == "verify":
        s.update(tokens=x["tokens"], parents=None if case["chain"] else x["parents"], target=x["target"],
                 draft=x.get("draft"), uniform=None if case["greedy"] else x["uniform"])
        if own:
            need = msq.verify_draft_workspace_bytes(sum(x["rows"]), case["batch"], case["vocab"], s["max_count"],
                                                    greedy=case["greedy"])
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        return s
    h, d, blk = case["kv_heads"], case["head_dim"], case.get("block")
    s["out"] = _type(case["out"])
    if kind in ("rotate", "append"):
        f, amplitude = _frequencies(case)
        pairs = case["layout"] == "pairs"
        s["rot"] = msq.Rotary(f, interleaved=pairs, amplitude=amplitude) if own else (f, pairs, amplitude)
    if kind == "rotate":
        s.update(x=x["x"], positions=x["positions"])
        return s
    # a program keeps its cache in the framework's layout: it is made and filled by the framework's own calls there
    cache = s["cache"] = msq.allocate_kv_cache(x["blocks"], h, d, blk) if own else _plain_cache(x["blocks"], h, d, blk)
    s["table"] = x["table"]

    def write(k, v, at, count):
        if sum(count) == 0:
            return
        args = (cache, k, v, x["table"], i32(at), offsets(count))
        if own:
            msq.kv_write(*args, max_count=max(count))
        else:
            _plain_write(*args, max(count))

    s["q"] = x["q"]
    if kind == "attend":
        write(x["k"], x["v"], [0] * len(x["total"]), x["total"])
        s.update(kv_len=i32(x["total"]), max_kv_len=max(x["total"]))
        # the sets of a step serve all layers of a model
        if own:
            s["tree"], _ = msq.draft_tree(x["parents"], s["offset"], max_count=s["max_count"])
            need = msq.kv_attention_workspace_bytes(cache, sum(x["rows"]), h * case["group"], len(x["rows"]),
                                                    s["max_count"], max(x["total"]), window=case["window"])
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        else:
            s["tree"], _ = _plain_sets(x["parents"], s["offset"], s["max_count"])
        return s
    write(x["k_before"], x["v_before"], x["at"], x["before"])
    back = [p + m - p // blk * blk if m else 0 for p, m in zip(x["past"], x["real"])]
    s.update(k=x["k"], v=x["v"], first=i32(x["past"]), back_first=i32([p // blk * blk for p in x["past"]]),
             back_offset=offsets(back), back_total=sum(back), back_max=max(back))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    kind = c["kind"]
    if not own:
        return {"rotate": _plain_rotate_pass, "append": _plain_append, "tree": _plain_tree, "attend": _plain_attend,
                "verify": _plain_verify}[kind](s)
    import block_wise_mixed_amd as msq
    if kind == "rotate":
        return msq.rotary(s["x"], s["positions"], s["rot"], out_dtype=s["out"])
    if kind == "tree":
        sets, positions = msq.draft_tree(s["parents"], s["offset"], s["first"], max_count=s["max_count"])
        return {"sets": sets, "positions": positions}
    if kind == "attend":
        return msq.kv_attention(s["q"], s["cache"], s["table"], s["kv_len"], s["offset"], max_count=s["max_count"],
                                max_kv_len=s["max_kv_len"], window=c["window"], out_dtype=s["out"],
                                workspace=s["workspace"], tree=s["tree"])
    if kind == "verify":
        token, taken, path = msq.verify_draft(s["tokens"], s["target"], s["offset"], parents=s["parents"],
                                              draft=s["draft"], uniform=s["uniform"], max_count=s["max_count"],
                                              workspace=s["workspace"])
        return {"token": token, "taken": taken, "path": path}
    q = msq.kv_append(s["cache"], s["k"], s["v"], s["table"], s["first"], s["rot"], q=s["q"], offset=s["offset"],
                      max_count=s["max_count"], q_dtype=s["out"])
    k, v = msq.kv_read(s["cache"], s["table"], s["back_first"], s["back_offset"], total=s["back_total"],
                       max_count=s["back_max"], dtype=s["out"])
    return {"q": q, "k": k, "v": v, "k_scale": s["cache"].k_scale, "v_scale": s["cache"].v_scale}


# ---------------------------------------------------------------- plain forms

def _plain_rotate(x, positions, rot):
    """x [rows, heads, dim] in 32 bits, rotated."""
    f, pairs, amplitude = rot
    angle = positions.double()[:, None] * f
    cos, sin = ((amplitude * t).float()[:, None, :] for t in (torch.cos(angle), torch.sin(angle)))
    n = 2 * f.numel()
    x = x.float()
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if pairs else (x[..., :n // 2], x[..., n // 2:n])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., n:]], -1)


def _plain_rotate_pass(s):
    return _plain_rotate(s["x"], s["positions"], s["rot"]).to(s["out"])


def _plain_append(s):
    offset, cache = s["offset"], s["cache"]
    seq, i = _plain_rows(offset, s["k"].shape[0])
    at = s["first"][seq] + i
    _plain_write(cache, _plain_rotate(s["k"], at, s["rot"]), s["v"], s["table"], s["first"], offset, s["max_count"])
    k, v = _plain_read(cache, s["table"], s["back_first"], s["back_offset"], s["back_total"], s["out"])
    # the plain cache ends with one block that takes what belongs nowhere
    return {"q": _plain_rotate(s["q"], at, s["rot"]).to(s["out"]), "k": k, "v": v,
            "k_scale": cache["k_scale"][:-1], "v_scale": cache["v_scale"][:-1]}


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
    row = torch.where(is_new, (offset[:-1] - first)[:, None, None] + place, 0).long()
    ids = torch.gather(table, 1, at.clamp(max=table.shape[1] - 1).long())
    ids = torch.where(is_new.any(-1), ids, nowhere).long()
    is_new, is_old = is_new[..., None, None], is_old[..., None, None]
    begun = is_old.any(2)[..., 0]  # the block holds earlier tokens
    for codes, scales, values in ((cache["k"], cache["k_scale"], k), (cache["v"], cache["v_scale"], v)):
        x = torch.where(is_new, values[row].float(), 0.0)
        top = x.abs().amax(dim=(2, 4))
        had = torch.where(begun, scales[ids], 0.0)
        scale = torch.maximum(top / torch.full_like(top, 127.0), had)
        by = torch.where(scale > 0, scale, 1.0)[:, :, None, :, None]
        x = torch.clamp(torch.round(x / by), -127, 127)
        q = codes[ids].transpose(2, 3).float()
        q = torch.where((scale > had)[:, :, None, :, None], torch.round(q * had[:, :, None, :, None] / by), q)
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


def _plain_sets(parents, offset, max_count):
    """(bool [rows, max_count]: itself and its ancestors; depth) of each row: powers of the step to the parent."""
    seq, i = _plain_rows(offset, parents.numel())
    B, n = offset.numel() - 1, max_count
    sees = torch.zeros(B, n, n, device="cuda")
    sees[seq, i, torch.where(parents >= 0, parents, i).long()] = 1.0
    sees[seq, i, i] = 1.0
    for _ in range(max(1, math.ceil(math.log2(max(2, n))))):
        sees = torch.matmul(sees, sees).clamp(max=1.0)
    sees = sees[seq, i]
    return sees > 0, (sees.sum(-1) - 1).to(torch.int32)


def _plain_tree(s):
    sees, depth = _plain_sets(s["parents"], s["offset"], s["max_count"])
    words = -(-s["max_count"] // 32)
    bits = torch.nn.functional.pad(sees.long(), (0, 32 * words - sees.shape[1])).view(-1, words, 32)
    sets = (bits << torch.arange(32, device="cuda")).sum(-1)
    sets = torch.where(sets >= 2 ** 31, sets - 2 ** 32, sets).to(torch.int32)
    seq, _ = _plain_rows(s["offset"], depth.numel())
    return {"sets": sets, "positions": s["first"][seq] + depth}


def _plain_attend(s):
    """All sequences padded to the longest: scores [batch, kv head, query row * group, cached token]."""
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

    scores = torch.matmul(q, cached(cache["k"], cache["k_scale"]).transpose(2, 3).contiguous())
    scores *= 1.0 / math.sqrt(d)
    place = torch.arange(width * blk, device="cuda")
    own_row = place - (s["kv_len"] - count)[:, None]  # which of the call's rows a place is
    tree = s["tree"][row]
    sees = torch.gather(tree, 2, own_row.clamp(0, n - 1)[:, None].expand(B, n, -1).long())
    sees = torch.where(own_row[:, None] < 0, True, sees & (own_row < count[:, None])[:, None])
    sees &= (place < s["kv_len"][:, None])[:, None]
    if c["window"]:
        after = sees.flip(-1).cumsum(-1).flip(-1)  # how many it sees from here on
        sees &= after <= c["window"]
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


def _plain_verify(s):
    """Rows in their order: a child comes after its parent, so one sweep goes down every sequence's tree."""
    offset, tokens, target, draft, u = s["offset"], s["tokens"].long(), s["target"], s["draft"], s["uniform"]
    B, V, total = offset.numel() - 1, target.shape[1], tokens.numel()
    start, count = offset[:-1].long(), (offset[1:] - offset[:-1]).long()
    parents = s["parents"]
    if parents is None:
        parents = (_plain_rows(offset, total)[1] - 1).to(torch.int32)
    at = torch.zeros(B, dtype=torch.long, device="cuda")
    taken = (count > 0).to(torch.int32)
    path = torch.full((total + 1,), -1, dtype=torch.int32, device="cuda")  # the last one takes what belongs nowhere
    path[torch.where(count > 0, start, total)] = start.to(torch.int32)
    if u is None:
        largest = target.float().argmax(-1)
    else:
        r, m = target[start].double(), torch.ones(B, dtype=torch.float64, device="cuda")
    for j in range(1, s["max_count"]):
        row = torch.where(j < count, start + j, 0)
        below = (j < count) & (parents[row] == at)
        x = tokens[row]
        if u is None:
            take = below & (x == largest[start + at])
        else:
            rx = torch.gather(r, 1, x[:, None])[:, 0]
            q = draft[start + at].double() if draft is not None else None
            qx = torch.gather(q, 1, x[:, None])[:, 0] if draft is not None else 1.0
            take = below & (u[row].double() * qx * m < rx)
            not_taken = below & ~take
            if draft is not None:
                left = torch.clamp(r / torch.where(m > 0, m, 1.0)[:, None] - q, min=0.0)
                r = torch.where(not_taken[:, None], left, r)
                m = torch.where(not_taken, r.sum(-1), m)
            else:
                m = torch.where(not_taken, m - rx, m)
                r = r.scatter(1, x[:, None], torch.where(not_taken, 0.0, rx)[:, None])
        at = torch.where(take, j, at)
        path[torch.where(take, start + taken, total)] = (start + j).to(torch.int32)
        taken = taken + take.to(torch.int32)
        if u is not None:
            r = torch.where(take[:, None], target[start + at].double(), r)
            m = torch.where(take, 1.0, m)
    if u is None:
        token = largest[start + at]
    else:
        r = torch.where(r.sum(-1, keepdim=True) > 0, r, target[start + at].double())
        run = r.cumsum(-1)
        token = torch.searchsorted(run, (u[start].double() * run[:, -1])[:, None], right=True)[:, 0]
        last = V - 1 - (r > 0).flip(-1).int().argmax(-1)
        token = torch.minimum(token, last)
    return {"token": torch.where(count > 0, token, -1).to(torch.int32), "taken": taken, "path": path[:-1]}


# ---------------------------------------------------------------- 64 bits

def _f32(t):
    return t.to(torch.float32).double()


def _exact_turn(x, positions, case, rounded):
    """x rotated, by complex numbers; `rounded`: with the roundings to 32 bits that the definition has for keys."""
    f, amplitude = _frequencies(case)
    n = case["part"]
    x = x.double()
    if case["layout"] == "pairs":
        a, b = x[..., :n].unflatten(-1, (n // 2, 2)).unbind(-1)
    else:
        a, b = x[..., :n].unflatten(-1, (2, n // 2)).unbind(-2)
    if rounded:
        w = torch.outer(positions.double(), f)
        c, s = _f32(w.cos() * amplitude)[:, None], _f32(w.sin() * amplitude)[:, None]
        re, im = _f32(_f32(a * c) - _f32(b * s)), _f32(_f32(b * c) + _f32(a * s))
    else:
        w = torch.polar(torch.full((), amplitude, dtype=torch.float64, device="cuda").expand(len(positions), n // 2).contiguous(),
                        torch.outer(positions.double(), f))
        z = torch.complex(a, b) * w[:, None]
        re, im = z.real, z.imag
    y = x.clone()
    if case["layout"] == "pairs":
        y[..., 0:n:2], y[..., 1:n:2] = re, im
    else:
        y[..., :n // 2], y[..., n // 2:n] = re, im
    return y


def _exact_block(x, code, old, begun):
    """Codes and scale of one block: x [tokens, head, dim] new values, code the earlier tokens' codes. The roundings to
    32 bits are part of the definition; a 64-bit quotient of 32-bit numbers, rounded to 32, is the 32-bit quotient."""
    scale = _f32(x.abs().amax(dim=(0, 2)) / 127.0)
    if begun:
        scale = torch.maximum(scale, old)
    by = torch.where(scale > 0, scale, 1.0)[None, :, None]
    new = torch.round(_f32(x / by)).clamp(-127, 127)
    if begun:
        moved = torch.round(_f32(_f32(code * old[None, :, None]) / by))
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


def _exact_sets(parents):
    """bool [n][n]: itself and its ancestors, by walking up."""
    p = parents.tolist()
    sees = torch.zeros(len(p), len(p), dtype=torch.bool)
    for i in range(len(p)):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = p[j]
    return sees.cuda()


def exact(case, seed):
    if case["kind"] in ("tree", "verify"):  # whole numbers
        return None
    x = _inputs(case, seed)
    if case["kind"] == "rotate":
        return _exact_turn(x["x"], x["positions"], case, False)
    h, d, blk, g = case["kv_heads"], case["head_dim"], case["block"], case["group"]
    if case["kind"] == "attend":
        outs, at, rows = [], 0, 0
        for m, p, n in zip(x["new"], x["past"], x["total"]):
            q = x["q"][rows:rows + abs(m)].double().view(abs(m), h, g, d)
            o = torch.zeros_like(q)
            if n:
                both = []
                for t in (x["k"], x["v"]):
                    code, scale = _exact_fill(t[at:at + n].double(), blk)
                    both.append(code * scale.repeat_interleave(blk, 0)[:n, :, None])
                k, v = both
                own_rows = _exact_sets(x["parents"][rows:rows + m])
                sees = torch.cat([torch.ones(m, p, dtype=torch.bool, device="cuda"), own_rows], 1)
                if case["window"]:
                    sees &= sees.sum(1, keepdim=True) - sees.cumsum(1) < case["window"]
                for e in range(h * g):
                    w = q[:, e // g, e % g] @ k[:, e // g].T / math.sqrt(d)
                    o[:, e // g, e % g] = torch.softmax(w.masked_fill(~sees, -math.inf), -1) @ v[:, e // g]
            at += n
            rows += abs(m)
            outs.append(o.reshape(abs(m), h * g, d))
        return torch.cat(outs)
    at = torch.cat([torch.arange(m, device="cuda") + p for p, m in zip(x["past"], x["real"])])
    result = {"q": _exact_turn(x["q"], at, case, False)}
    for name in ("k", "v"):
        back = []
        scales = torch.zeros(x["blocks"], h, dtype=torch.float64, device="cuda")
        before = new = 0
        values = _exact_turn(x["k"], at, case, True) if name == "k" else x["v"].double()
        for b in range(case["batch"]):
            p, m, had = x["past"][b], x["real"][b], x["before"][b]
            if m:
                part = (None, None)
                if had:
                    code, scale = _exact_fill(x[name + "_before"][before:before + had].double(), blk)
                    part = (code, scale[0])
                code, scale = _exact_fill(values[new:new + m], blk, *part)
                scales[x["table"][b, p // blk:p // blk + scale.shape[0]].long()] = scale
                back.append(code * scale.repeat_interleave(blk, 0)[:code.shape[0], :, None])
            before, new = before + had, new + m
        result[name] = torch.cat(back)
        result[name + "_scale"] = scales
    return {n: result[n] for n in ("q", "k", "v", "k_scale", "v_scale")}

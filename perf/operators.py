"""Measured cases of the operators that decode over part of a paged cache.

Five operators, in the order a serving step uses them:

* ``bounds``   ``pa_update_key_bounds``: elementwise minimum and maximum of the keys of
  each block that a step has appended to;
* ``select``   ``pa_select_blocks``: an upper bound of q.k for every block of a sequence
  from those minima and maxima, and the ``count`` best blocks for each K/V head;
* ``selected`` ``pa_decode_selected_blocks``: decode attention over the listed blocks;
* ``weights``  ``pa_decode_accumulate_weights``: decode attention that also adds each
  position's attention weight to a running sum;
* ``evict``    ``pa_evict_tokens``: keep the positions of largest weight and move them to
  the front of the cache.

``own = False`` runs them as elementary torch operations, ``own = True`` through the
library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, dtype, batch, ctx_min, ctx_max, heads, kv_heads, head_dim, block, **more):
    return dict(name=name, op=op, dtype=dtype, batch=batch, ctx_min=ctx_min, ctx_max=ctx_max,
                heads=heads, kv_heads=kv_heads, head_dim=head_dim, block=block, **more)


def listed():
    return [
        # the decode step of a batch of chats: one appended token per sequence, so one block
        # per sequence gets new minima and maxima (smallest call: latency)
        _case("bounds_step", "bounds", "bf16", 128, 16, 4096, 64, 8, 128, 16, new=1),
        # four long prompts have just been appended: every block is summarised once
        _case("bounds_prompt", "bounds", "bf16", 4, 32768, 131072, 32, 8, 128, 64, new=131072),
        # one user, a document of 8K tokens: latency
        _case("select_one", "select", "bf16", 1, 8191, 8191, 32, 8, 128, 16, count=64, first=1,
              last=2),
        # a batch of chats with ragged lengths, many of them shorter than the selection
        _case("select_batch", "select", "bf16", 128, 16, 4096, 64, 8, 128, 16, count=64, first=1,
              last=2),
        # sixteen long documents: 64K to 128K tokens in 16-token blocks
        _case("select_long", "select", "bf16", 16, 65536, 131072, 32, 8, 128, 16, count=256,
              first=4, last=8),
        # one user over 64 of a long document's blocks: latency
        _case("selected_one", "selected", "bf16", 1, 32768, 32768, 32, 8, 128, 16, count=64,
              first=1, last=2),
        # a batch of chats, each K/V head over its own 64 blocks
        _case("selected_batch", "selected", "bf16", 128, 256, 4096, 64, 8, 128, 16, count=64,
              first=1, last=2),
        # the smallest float32 decode: four short sequences
        _case("weights_tiny", "weights", "fp32", 4, 5, 40, 4, 4, 64, 16),
        # a Llama-2-7B-shaped batch that keeps track of its attention weights
        _case("weights_llama", "weights", "bf16", 64, 128, 2048, 32, 32, 128, 16),
        # long documents: the weights of up to 128K positions
        _case("weights_long", "weights", "bf16", 4, 32768, 131072, 32, 8, 128, 64),
        # a batch of chats that has outgrown its memory, cut back to 1024 tokens each
        _case("evict_batch", "evict", "bf16", 64, 1500, 4096, 64, 8, 128, 16, count=1024, first=4,
              last=256),
        # long documents cut back to 16K tokens each
        _case("evict_long", "evict", "bf16", 4, 32768, 131072, 32, 8, 128, 64, count=16384,
              first=4, last=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bounds", "select", "selected", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    head_dim = rng.choice([64, 128])
    block = rng.choice([16, 32, 64])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
    group = rng.choice([1, 2, 3, 4, 8, 8, 16]) if kv_heads < 32 else 1
    ctx_max = _log_int(rng, 5, 131072)
    # K/V bytes of the whole batch stay well below the largest listed case
    room = 5e8 / (kv_heads * head_dim * (2 if dtype == "bf16" else 4)) / ctx_max / 2
    batch = _log_int(rng, 1, max(1, min(128, int(room))))
    ctx_min = max(1, int(ctx_max * rng.uniform(0.1, 1.0)))
    if batch * ctx_max * kv_heads * head_dim > 1.5e8:  # one very long, wide sequence
        ctx_min = ctx_max = int(1.5e8 / (batch * kv_heads * head_dim))
    case = _case("", op, dtype, batch, ctx_min, ctx_max, kv_heads * group, kv_heads, head_dim,
                 block)
    del case["name"]
    blocks = -(-ctx_max // block)
    if op == "bounds":
        case["new"] = rng.choice([1, _log_int(rng, 1, ctx_max), ctx_max])
    elif op in ("select", "selected"):
        case["count"] = min(_log_int(rng, 1, 512), max(1, blocks))
        case["first"] = min(rng.choice([0, 1, 4]), case["count"] // 2)
        case["last"] = min(rng.choice([0, 1, 2, 8]), case["count"] // 2)
    elif op == "evict":
        case["count"] = max(1, int(ctx_max * rng.uniform(0.05, 0.6)))
        case["first"] = min(rng.choice([0, 4, 17]), case["count"] // 4)
        case["last"] = int(case["count"] * rng.choice([0.0, 0.1, 0.5]))
    return case


def _lens(case):
    """Context lengths: spread evenly over the case's range, in a fixed mixed order."""
    n, lo, hi = case["batch"], case["ctx_min"], case["ctx_max"]
    if n == 1:
        return [hi]
    lens = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    step = next(s for s in (37, 41, 43, 47) if math.gcd(s, n) == 1)
    return [lens[i * step % n] for i in range(n)]


def _new_lens(case):
    return [min(n, case["new"]) for n in _lens(case)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(gen, num_blocks, case, dtype):
    """[num_blocks, kv_heads, block, head_dim], filled in pieces."""
    shape = (num_blocks, case["kv_heads"], case["block"], case["head_dim"])
    pool = torch.empty(shape, dtype=dtype, device="cuda")
    piece = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, num_blocks, piece):
        part = pool[i:i + piece]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.float32))
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, op = DTYPES[case["dtype"]], case["op"]
    B, H, D, bs = case["batch"], case["kv_heads"], case["head_dim"], case["block"]
    lens = _lens(case)
    max_ctx = max(lens)
    width = -(-max_ctx // bs)
    dst_width = -(-case["count"] // bs) if op == "evict" else 0
    num_blocks = B * (width + dst_width) + 1
    order = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    s = {"case": dict(case), "max_ctx": max_ctx, "scale": 1.0 / math.sqrt(D),
         "block_tables": order[:B * width].reshape(B, width).contiguous(),
         "context_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if op in ("select", "selected", "weights"):
        s["q"] = _normal(gen, (B, case["heads"], D), dtype)
    if op == "bounds":
        s["k_cache"] = _pool(gen, num_blocks, case, dtype)
        s["new_lens"] = torch.tensor(_new_lens(case), dtype=torch.int32, device="cuda")
        s["max_new"] = max(_new_lens(case))
        s["key_bounds"] = torch.zeros(num_blocks, H, 2, D, dtype=dtype, device="cuda")
    elif op == "select":
        # minimum and maximum of `block` keys: a normal key's expected extremes, with a spread
        # of their own for each block
        reach = math.sqrt(2.0 * math.log(bs))
        s["key_bounds"] = torch.empty(num_blocks, H, 2, D, dtype=dtype, device="cuda")
        piece = max(1, (1 << 26) // (H * 2 * D))
        for i in range(0, num_blocks, piece):
            part = s["key_bounds"][i:i + piece]
            r = torch.randn(part.shape, generator=gen, device="cuda") * 0.5
            r[:, :, 0] -= reach * 0.8
            r[:, :, 1] += reach * 0.8
            part[:, :, 0] = torch.minimum(r[:, :, 0], r[:, :, 1]).to(dtype)
            part[:, :, 1] = torch.maximum(r[:, :, 0], r[:, :, 1]).to(dtype)
        s["selected"] = torch.empty(B, H, case["count"], dtype=torch.int32, device="cuda")
    elif op == "selected":
        s["k_cache"] = _pool(gen, num_blocks, case, dtype)
        s["v_cache"] = _pool(gen, num_blocks, case, dtype)
        # the first and last blocks of each sequence and a random choice between them
        n = (s["context_lens"].long() + bs - 1) // bs
        at = torch.arange(width, device="cuda")
        key = torch.rand(B, H, width, generator=gen, device="cuda")
        forced = (at < case["first"]) | (at >= n[:, None, None] - case["last"])
        key = torch.where(forced, key + 2, key)
        key = torch.where(at < n[:, None, None], key, key.new_tensor(-1.0))
        best, which = key.topk(min(case["count"], width), dim=-1)
        which = torch.where(best >= 0, which, width).sort(dim=-1).values
        sel = torch.full((B, H, case["count"]), -1, dtype=torch.int32, device="cuda")
        sel[:, :, :which.shape[-1]] = torch.where(which < width, which, -1).to(torch.int32)
        s["selected"] = sel
        s["out"] = torch.empty_like(s["q"])
    elif op == "weights":
        s["k_cache"] = _pool(gen, num_blocks, case, dtype)
        s["v_cache"] = _pool(gen, num_blocks, case, dtype)
        s["weights_in"] = _old_weights(gen, B, H, max_ctx)
        s["weights_out"] = torch.zeros_like(s["weights_in"])
        s["out"] = torch.empty_like(s["q"])
    elif op == "evict":
        s["k_cache"] = _pool(gen, num_blocks, case, dtype)
        s["v_cache"] = _pool(gen, num_blocks, case, dtype)
        s["dst_tables"] = order[B * width:B * (width + dst_width)].reshape(
            B, dst_width).contiguous()
        s["weights_in"] = _old_weights(gen, B, H, max_ctx)
        s["weights_out"] = torch.zeros_like(s["weights_in"])
        s["kept"] = torch.empty(B, H, case["count"], dtype=torch.int32, device="cuda")
        s["new_context_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    if own:
        s["call"] = _own_call(s)  # the marshalled call that a decode loop keeps
    return s


def _old_weights(gen, B, H, n):
    """Attention mass collected so far: heavy-tailed, a tenth of the positions never attended
    (equal weights), the first positions the heaviest."""
    w = torch.exp(1.5 * torch.randn(B, H, n, generator=gen, device="cuda") - 2.0)
    w = torch.where(torch.rand(B, H, n, generator=gen, device="cuda") < 0.1, w.new_zeros(()), w)
    w[:, :, :4] += 20.0
    return w


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own_call(s):
    """The library's calls, their arguments marshalled once (pa.prepare_*)."""
    from pagedattention_paged_kv_02_b200 import pa

    c = s["case"]
    op = c["op"]
    if op == "bounds":
        return pa.prepare_update_key_bounds(s["key_bounds"], s["k_cache"], s["block_tables"],
                                            s["context_lens"], s["new_lens"], s["max_new"])
    if op == "select":
        return pa.prepare_select_blocks(s["selected"], s["q"], s["key_bounds"],
                                        s["block_tables"], s["context_lens"], s["max_ctx"],
                                        c["block"], c["first"], c["last"])
    if op == "selected":
        n = pa.pa_decode_selected_blocks_workspace_size(c["batch"], c["heads"], c["kv_heads"],
                                                        c["head_dim"], c["block"], c["count"])
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        return pa.prepare_decode_selected_blocks(
            s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
            s["selected"], s["scale"], workspace=ws)
    if op == "weights":
        n = pa.pa_decode_accumulate_weights_workspace_size(c["batch"], c["heads"], c["head_dim"],
                                                           s["max_ctx"])
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        return pa.prepare_decode_accumulate_weights(
            s["out"], s["weights_out"], s["weights_in"], s["q"], s["k_cache"], s["v_cache"],
            s["block_tables"], s["context_lens"], s["max_ctx"], s["scale"], workspace=ws)
    return pa.prepare_evict_tokens(
        s["k_cache"], s["v_cache"], s["weights_out"], s["weights_in"], s["kept"],
        s["new_context_lens"], s["block_tables"], s["dst_tables"], s["context_lens"],
        s["max_ctx"], c["count"], c["first"], c["last"])


def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
    elif op == "bounds":
        _plain_bounds(s)
    elif op == "select":
        _plain_select(s)
    elif op == "selected":
        _plain_selected(s)
    elif op == "weights":
        _plain_weights(s)
    else:
        _plain_evict(s)
    return _outputs(s)


def _outputs(s):
    op = s["case"]["op"]
    if op == "bounds":
        return {"key_bounds": s["key_bounds"]}
    if op == "select":
        return {"selected": s["selected"]}
    if op == "selected":
        return {"out": s["out"]}
    if op == "weights":
        return {"out": s["out"], "weights": s["weights_out"]}
    return {"kept": s["kept"], "lens": s["new_context_lens"], "weights": s["weights_out"],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_bounds(s):
    bs = s["case"]["block"]
    ctx, new = s["context_lens"].long(), s["new_lens"].long()
    first = (ctx - new) // bs
    many = (s["max_new"] + bs - 2) // bs + 1
    blk = first[:, None] + torch.arange(many, device="cuda")
    live = blk * bs < ctx[:, None]
    phys = s["block_tables"].long().gather(1, blk.clamp(max=s["block_tables"].shape[1] - 1))
    phys = phys[live]
    pos = blk[live][:, None] * bs + torch.arange(bs, device="cuda")
    valid = pos < ctx[:, None].expand_as(blk)[live][:, None]
    k = s["k_cache"][phys].float()
    hole = ~valid[:, None, :, None]
    lo = k.masked_fill(hole, math.inf).amin(2)
    hi = k.masked_fill(hole, -math.inf).amax(2)
    s["key_bounds"][phys] = torch.stack((lo, hi), 2).to(s["key_bounds"].dtype)


def _plain_select(s):
    c = s["case"]
    B, H, bs, K = c["batch"], c["kv_heads"], c["block"], c["count"]
    # in 64 bits: a block is in or out by its place in the order of the scores
    q = s["q"].double().view(B, H, -1, c["head_dim"])
    bounds = s["key_bounds"][s["block_tables"].long()].double()  # [B, N, H, 2, D]
    score = torch.einsum("bhgd,bnhd->bhgn", q.clamp(min=0), bounds[:, :, :, 1])
    score = score + torch.einsum("bhgd,bnhd->bhgn", q.clamp(max=0), bounds[:, :, :, 0])
    score = score.amax(2)
    N = score.shape[-1]
    n = ((s["context_lens"].long() + bs - 1) // bs)[:, None, None]
    at = torch.arange(N, device="cuda")
    score = score.masked_fill((at < c["first"]) | (at >= n - c["last"]), math.inf)
    score = score.masked_fill(at >= n, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[:, :, :K]
    taken = torch.arange(order.shape[-1], device="cuda") < n
    order = torch.where(taken, order, N).sort(dim=-1).values
    s["selected"].fill_(-1)
    s["selected"][:, :, :order.shape[-1]] = torch.where(order < N, order, -1).to(torch.int32)


def _plain_selected(s):
    c = s["case"]
    B, H, bs, D = c["batch"], c["kv_heads"], c["block"], c["head_dim"]
    sel = s["selected"].long()
    phys = s["block_tables"].long()[:, None].expand(B, H, -1).gather(2, sel.clamp(min=0))
    head = torch.arange(H, device="cuda")[None, :, None]
    pos = sel[..., None] * bs + torch.arange(bs, device="cuda")
    valid = (sel[..., None] >= 0) & (pos < s["context_lens"].long()[:, None, None, None])
    valid = valid.view(B, H, 1, -1)
    k = s["k_cache"][phys, head].float().view(B, H, -1, D)
    q = s["q"].float().view(B, H, -1, D) * s["scale"]
    logits = (q @ k.transpose(2, 3)).masked_fill(~valid, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(logits - top)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    v = s["v_cache"][phys, head].float().view(B, H, -1, D)
    s["out"].copy_((p @ v).view(s["out"].shape))


def _plain_weights(s):
    c = s["case"]
    B, H, bs, D = c["batch"], c["kv_heads"], c["block"], c["head_dim"]
    T = s["max_ctx"]
    table = s["block_tables"].long()
    k = s["k_cache"][table].transpose(1, 2).reshape(B, H, -1, D)[:, :, :T].float()
    q = s["q"].float().view(B, H, -1, D) * s["scale"]
    valid = torch.arange(T, device="cuda") < s["context_lens"].long()[:, None, None, None]
    logits = (q @ k.transpose(2, 3)).masked_fill(~valid, -math.inf)
    del k
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = s["v_cache"][table].transpose(1, 2).reshape(B, H, -1, D)[:, :, :T].float()
    s["out"].copy_((p @ v).view(s["out"].shape))
    new = s["weights_in"] + p.sum(2)
    s["weights_out"].copy_(torch.where(valid[:, :, 0], new, s["weights_out"]))


def _plain_evict(s):
    c = s["case"]
    B, H, bs, K = c["batch"], c["kv_heads"], c["block"], c["count"]
    T = s["max_ctx"]
    ctx = s["context_lens"].long()[:, None, None]
    at = torch.arange(T, device="cuda")
    key = s["weights_in"].masked_fill((at < c["first"]) | (at >= ctx - c["last"]), math.inf)
    key = key.masked_fill(at >= ctx, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices[:, :, :K]
    taken = torch.arange(order.shape[-1], device="cuda") < ctx
    order = torch.where(taken, order, T).sort(dim=-1).values
    live = order < T  # [B, H, kept]
    src = order.clamp(max=T - 1)
    s["kept"].fill_(-1)
    s["kept"][:, :, :order.shape[-1]] = torch.where(live, order, -1).to(torch.int32)
    s["new_context_lens"].copy_(s["context_lens"].clamp(max=K))
    new = torch.zeros_like(s["weights_in"])
    new[:, :, :order.shape[-1]] = s["weights_in"].gather(2, src) * live
    s["weights_out"].copy_(torch.where(at < ctx, new, s["weights_out"]))
    b, h, i = live.nonzero(as_tuple=True)
    j = src[b, h, i]
    from_block = s["block_tables"].long()[b, j // bs]
    to_block = s["dst_tables"].long()[b, i // bs]
    s["k_cache"][to_block, h, i % bs] = s["k_cache"][from_block, h, j % bs]
    s["v_cache"][to_block, h, i % bs] = s["v_cache"][from_block, h, j % bs]


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def _listed_tokens(case):
    """Tokens of each row's listed blocks (the last one may be partly filled)."""
    bs, total = case["block"], 0
    for n in _lens(case):
        blocks = -(-n // bs)
        if blocks <= case["count"]:
            total += n
        else:  # the short last block is listed when last blocks always are
            total += case["count"] * bs - (blocks * bs - n if case["last"] else 0)
    return total


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, H, Hq, D, bs = (case[k] for k in ("batch", "kv_heads", "heads", "head_dim", "block"))
    lens, op = _lens(case), case["op"]
    table = sum(4 * -(-n // bs) for n in lens) + 4 * B
    q_out = B * Hq * D * e
    if op == "bounds":
        tokens = blocks = 0
        for n, new in zip(lens, _new_lens(case)):
            first = (n - new) // bs
            tokens += n - first * bs
            blocks += -(-n // bs) - first
        return {"bytes": (tokens + 2 * blocks) * H * D * e + 4 * blocks + 8 * B,
                "flops": 2 * tokens * H * D}
    if op == "select":
        blocks = sum(-(-n // bs) for n in lens)
        return {"bytes": blocks * H * 2 * D * e + q_out + table + 4 * B * H * case["count"],
                "flops": 4 * blocks * Hq * D}
    if op == "selected":
        tokens = _listed_tokens(case)
        return {"bytes": 2 * tokens * H * D * e + 2 * q_out + 8 * B * H * case["count"] + 4 * B,
                "flops": 4 * tokens * Hq * D}
    if op == "weights":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * H * D * e + 8 * tokens * H + 2 * q_out + table,
                "flops": 4 * tokens * Hq * D}
    kept = sum(min(n, case["count"]) for n in lens)
    return {"bytes": 8 * sum(lens) * H + 4 * kept * H * D * e + 4 * B * H * case["count"] + table,
            "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, row by row
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "select":
        return None  # whole numbers only
    bs, H = c["block"], c["kv_heads"]
    group = c["heads"] // H
    lens, tables = _lens(c), s["block_tables"].long()

    def rows(cache, b, n):  # [n, H, D] tokens of row b, in order
        blocks = cache[tables[b, :-(-n // bs)]]
        return blocks.permute(0, 2, 1, 3).flatten(0, 1)[:n]

    if op == "bounds":
        want = s["key_bounds"].double()
        for b, (n, new) in enumerate(zip(lens, _new_lens(c))):
            k = rows(s["k_cache"], b, n).double()
            start = (n - new) // bs
            full = n // bs
            if full > start:
                part = k[start * bs:full * bs].unflatten(0, (full - start, bs))
                ids = tables[b, start:full]
                want[ids, :, 0] = torch.min(part, dim=1).values
                want[ids, :, 1] = torch.max(part, dim=1).values
            if n % bs:
                tail = k[full * bs:]
                want[tables[b, full], :, 0] = torch.min(tail, dim=0).values
                want[tables[b, full], :, 1] = torch.max(tail, dim=0).values
        return {"key_bounds": want}

    if op == "evict":
        K = c["count"]
        weights = s["weights_out"].double()
        pools = {"k_cache": s["k_cache"].clone(), "v_cache": s["v_cache"].clone()}
        for b, n in enumerate(lens):
            keep = min(n, K)
            dst = s["dst_tables"][b].long().repeat_interleave(bs)[:keep]
            off = torch.arange(keep, device="cuda") % bs
            for h in range(H):
                w = s["weights_in"][b, h, :n].double()
                chosen = torch.zeros(n, dtype=torch.bool, device="cuda")
                if keep == n:
                    chosen[:] = True
                else:
                    stop = n - c["last"]
                    chosen[:c["first"]] = True
                    chosen[stop:] = True
                    room = keep - c["first"] - c["last"]
                    mid = w[c["first"]:stop]
                    if room > 0:
                        cut = torch.topk(mid, room).values[-1]
                        above = mid > cut
                        level = mid == cut
                        level &= level.cumsum(0) <= room - above.sum()
                        chosen[c["first"]:stop] |= above | level
                at = chosen.nonzero()[:, 0]
                weights[b, h, :n] = 0
                weights[b, h, :keep] = w[at]
                blk = tables[b, at // bs]
                for name in pools:
                    pools[name][dst, h, off] = s[name][blk, h, at % bs]
        return {"kept": None, "lens": None, "weights": weights,
                "k_cache": pools["k_cache"].double(), "v_cache": pools["v_cache"].double()}

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights_out"].double() if op == "weights" else None
    for b, n in enumerate(lens):
        k, v = rows(s["k_cache"], b, n), rows(s["v_cache"], b, n)
        for h in range(H):
            at = None
            if op == "selected":
                sel = s["selected"][b, h].long()
                at = (sel[sel >= 0][:, None] * bs + torch.arange(bs, device="cuda")).flatten()
                at = at[at < n]
            kh = (k[:, h] if at is None else k[at, h]).double()
            vh = (v[:, h] if at is None else v[at, h]).double()
            qh = s["q"][b, h * group:(h + 1) * group].double()
            p = torch.softmax(qh.mul(s["scale"]).matmul(kh.mT), dim=-1)
            out[b, h * group:(h + 1) * group] = p.matmul(vh)
            if weights is not None:
                weights[b, h, :n] = s["weights_in"][b, h, :n].double() + p.sum(0)
    return {"out": out} if weights is None else {"out": out, "weights": weights}

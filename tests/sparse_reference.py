"""Plain 64-bit forms of the operators that decode over part of a paged cache,
row by row on the CPU, written from their formulas: what the GPU tests compare
the library with."""
import torch


def tokens(cache, table, n, h):
    """Positions 0..n-1 of one row and K/V head, [n, D] in float64."""
    bs = cache.shape[2]
    ids = table[:-(-n // bs)].long()
    return cache[ids, h].reshape(-1, cache.shape[3])[:n].double()


def update_key_bounds(key_bounds, k_cache, tables, lens, new_lens):
    """``key_bounds`` (changed in place) as pa_update_key_bounds leaves it."""
    bs = k_cache.shape[2]
    for b, (n, new) in enumerate(zip(lens.tolist(), new_lens.tolist())):
        if new == 0:
            continue
        for j in range((n - new) // bs, -(-n // bs)):
            p = int(tables[b, j])
            part = k_cache[p, :, :min(bs, n - j * bs)]
            key_bounds[p, :, 0] = part.amin(1)
            key_bounds[p, :, 1] = part.amax(1)
    return key_bounds


def block_scores(q, key_bounds, table, n, h, group):
    """Scores of a row's first n blocks for K/V head h, float64 [n]."""
    kb = key_bounds[table[:n].long(), h].double()
    qh = q[h * group:(h + 1) * group].double()
    # a zero weight times an infinite bound is NaN, as in the formula
    s = (qh.clamp(min=0)[:, None] * kb[None, :, 1] + qh.clamp(max=0)[:, None] * kb[None, :, 0])
    return s.sum(-1).amax(0)


def _best(values, need):
    """Indices of the ``need`` largest: NaN above everything, ties to the lowest
    index, ascending."""
    key = [(0 if v != v else 1, 0.0 if v != v else -v, i) for i, v in enumerate(values.tolist())]
    return sorted(i for _, _, i in sorted(key)[:need])


def select_blocks(q, key_bounds, tables, lens, bs, count, first, last):
    B, H_q, _ = q.shape
    H = key_bounds.shape[1]
    out = torch.full((B, H, count), -1, dtype=torch.int32)
    for b, ctx in enumerate(lens.tolist()):
        n = -(-ctx // bs)
        for h in range(H):
            if n <= count:
                idx = list(range(n))
            else:
                s = block_scores(q[b], key_bounds, tables[b], n, h, H_q // H)
                mid = s[first:n - last]
                idx = (list(range(first)) + [first + i for i in _best(mid, count - first - last)] +
                       list(range(n - last, n)))
            out[b, h, :len(idx)] = torch.tensor(idx, dtype=torch.int32)
    return out


def attend(q, k, v, scale):
    """softmax(scale q K^T) V and the weights, float64; no tokens gives zeros."""
    if k.shape[0] == 0:
        return torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64), q.new_zeros(
            (q.shape[0], 0)).double()
    p = torch.softmax(scale * (q.double() @ k.T), dim=-1)
    return p @ v, p


def decode_selected(q, k_cache, v_cache, tables, lens, selected, scale):
    B, H_q, D = q.shape
    H, bs = k_cache.shape[1], k_cache.shape[2]
    G = H_q // H
    out = torch.zeros(B, H_q, D, dtype=torch.float64)
    for b, ctx in enumerate(lens.tolist()):
        n = -(-ctx // bs)
        for h in range(H):
            at = []
            for j in selected[b, h].tolist():
                if 0 <= j < n:
                    at += range(j * bs, min(ctx, (j + 1) * bs))
            at = torch.tensor(at, dtype=torch.long)
            k = tokens(k_cache, tables[b], ctx, h)[at]
            v = tokens(v_cache, tables[b], ctx, h)[at]
            out[b, h * G:(h + 1) * G] = attend(q[b, h * G:(h + 1) * G], k, v, scale)[0]
    return out


def decode_weights(q, k_cache, v_cache, tables, lens, scale, weights_in, stride):
    """Outputs, and the new weights (None at positions past each row's length)."""
    B, H_q, D = q.shape
    H = k_cache.shape[1]
    G = H_q // H
    out = torch.zeros(B, H_q, D, dtype=torch.float64)
    weights = torch.full((B, H, stride), float("nan"), dtype=torch.float64)
    for b, ctx in enumerate(lens.tolist()):
        for h in range(H):
            k, v = tokens(k_cache, tables[b], ctx, h), tokens(v_cache, tables[b], ctx, h)
            o, p = attend(q[b, h * G:(h + 1) * G], k, v, scale)
            out[b, h * G:(h + 1) * G] = o
            weights[b, h, :ctx] = p.sum(0)
            if weights_in is not None:
                weights[b, h, :ctx] += weights_in[b, h, :ctx].double()
    return out, weights


def evict(weights, lens, budget, first, last):
    """Kept positions of each row and head, as lists."""
    kept = []
    for b, n in enumerate(lens.tolist()):
        row = []
        for h in range(weights.shape[1]):
            if n <= budget:
                row.append(list(range(n)))
            else:
                mid = weights[b, h, first:n - last].double()
                row.append(list(range(first)) +
                           [first + i for i in _best(mid, budget - first - last)] +
                           list(range(n - last, n)))
        kept.append(row)
    return kept

"""The operators over a paged KV cache that perf/ measures, with their plain forms.

Three operators that a sliding-window layer of a served model runs next to the
library's attention calls:

  window   grouped-query attention in which a row sees the first ``sinks``
           positions and the last ``window`` ones, over pages (decode, verify
           windows, prompt chunks);
  rope     the row write with rotary positions of several axes: query and key
           rows are turned by their (time, height, width) positions, keys and
           values land in their pages;
  pages    the cache's pages, shared by reference count: ``beam`` is one
           reordering of beams (fork by parent, free the old beams, grow by
           one position with a copy of each shared page that is written to),
           ``evict`` frees the pages behind every stream's window and
           compacts the pool.

``own = False`` computes them with elementary torch operations; ``own = True``
makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

# A workspace and a list of page moves as a serving program keeps them: sized
# once from the largest shape it runs.
WORKSPACE_BYTES = 48 << 20


def listed():
    return [
        # one short chat, one KV head: a call's latency
        dict(name="window_decode_1x1037", op="window", streams=1, kv_heads=1, group=4, dim=128, page=512,
             rows=1, len_lo=1037, len_hi=1037, window=256, sinks=4),
        # a serving batch far into its contexts
        dict(name="window_decode_12x40k", op="window", streams=12, kv_heads=8, group=4, dim=128, page=512,
             rows=1, len_lo=40960, len_hi=40960, window=4096, sinks=4),
        # a large batch of mixed lengths over small pages, eight query heads a KV head
        dict(name="window_decode_64_ragged_p64", op="window", streams=64, kv_heads=4, group=8, dim=128, page=64,
             rows=1, len_lo=900, len_hi=32768, window=8192, sinks=64),
        # draft-verify windows at head dim 512
        dict(name="window_verify_hd512", op="window", streams=16, kv_heads=2, group=8, dim=512, page=512,
             rows=4, len_lo=2048, len_hi=9216, window=1024, sinks=4),
        # an odd chunk over odd pages, shorter than its window in part
        dict(name="window_prompt_100_p37", op="window", streams=3, kv_heads=2, group=4, dim=128, page=37,
             rows=100, len_lo=100, len_hi=1536, window=333, sinks=5),
        # the largest prompt chunk
        dict(name="window_prompt_4096", op="window", streams=2, kv_heads=8, group=4, dim=128, page=512,
             rows=4096, len_lo=9216, len_hi=12000, window=4096, sinks=4),
        # a decode step's row per stream, three axes
        dict(name="rope_decode_64", op="rope", streams=64, kv_heads=8, group=4, dim=128, page=512, rows=1,
             len_lo=1, len_hi=40960, axes=3, rotary=128, adjacent=False, far=131072),
        # long image and video prompts
        dict(name="rope_prompt_4x4096", op="rope", streams=4, kv_heads=8, group=4, dim=128, page=512, rows=4096,
             len_lo=4096, len_hi=9216, axes=3, rotary=128, adjacent=False, far=131072),
        # one request with four beams
        dict(name="beam_1x4", op="beam", prompts=1, beams=4, kv_heads=8, dim=128, page=512, len_lo=700,
             len_hi=1000, spare=0.5),
        # a batch of beam searches over small pages
        dict(name="beam_32x8", op="beam", prompts=32, beams=8, kv_heads=8, dim=128, page=128, len_lo=300,
             len_hi=2000, spare=0.5),
        # a few streams, a small pool
        dict(name="evict_4_p64", op="evict", streams=4, kv_heads=2, dim=128, page=64, len_lo=500, len_hi=4000,
             window=512, sinks=4, spare=0.2),
        # a serving batch whose window layers hold their whole contexts until now
        dict(name="evict_12_p512", op="evict", streams=12, kv_heads=8, dim=128, page=512, len_lo=9000,
             len_hi=40960, window=16384, sinks=4, spare=0.2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# a drawn case costs no more than the largest listed ones
MOST_BYTES, MOST_FLOPS = 7e8, 5e11


def draw(rng):
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


def _draw(rng):
    op = rng.choice(["window", "window", "window", "rope", "beam", "evict"])
    dim = rng.choice([128, 128, 256, 512])
    page = rng.choice([16, 37, 64, 128, 200, 512, 512])
    if op == "window":
        rows = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 2048)])
        streams = _log_int(rng, 1, 64 if rows == 1 else 16 if rows <= 8 else 2)
        len_hi = max(rows, _log_int(rng, 16, 40960 if rows <= 8 else 12000))
        return dict(op=op, streams=streams, kv_heads=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 3, 4, 8]), dim=dim,
                    page=page, rows=rows, len_lo=max(rows, len_hi // rng.choice([1, 2, 7])), len_hi=len_hi,
                    window=_log_int(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 4, 64, 130]))
    if op == "rope":
        rows = rng.choice([1, rng.randint(2, 8), _log_int(rng, 9, 4096)])
        len_hi = max(rows, _log_int(rng, 16, 40960))
        return dict(op=op, streams=_log_int(rng, 1, 64 if rows <= 8 else 2), kv_heads=rng.choice([1, 2, 8]),
                    group=rng.choice([1, 3, 4, 8]), dim=dim, page=page, rows=rows,
                    len_lo=max(rows, len_hi // rng.choice([1, 3])), len_hi=len_hi, axes=rng.choice([1, 2, 3, 3, 4]),
                    rotary=rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)]), adjacent=rng.choice([True, False]),
                    far=_log_int(rng, 1, 1 << 20))
    if op == "beam":
        len_hi = _log_int(rng, 4, 2000)
        return dict(op=op, prompts=_log_int(rng, 1, 32), beams=rng.randint(1, 8), kv_heads=rng.choice([1, 2, 8]), dim=128,
                    page=page, len_lo=max(1, len_hi // 3), len_hi=len_hi, spare=rng.uniform(0.1, 1.0))
    len_hi = _log_int(rng, 64, 20000)
    return dict(op=op, streams=_log_int(rng, 1, 12), kv_heads=rng.choice([1, 2, 8]), dim=128, page=page,
                len_lo=max(1, len_hi // 4), len_hi=len_hi, window=_log_int(rng, 1, 16384), sinks=rng.choice([0, 4, 64]),
                spare=rng.uniform(0.05, 1.0))


# ---- inputs -----------------------------------------------------------------

def _dev():
    return torch.device("cuda")


def _lens(case, r, n):
    return r.integers(case["len_lo"], case["len_hi"] + 1, n).astype(np.int64)


def _normal(g, shape):
    return torch.randn(shape, generator=g, device=_dev(), dtype=torch.float32).to(torch.bfloat16)


def _pools(case, g, n_pages):
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    return _normal(g, shape), _normal(g, shape)


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(_dev())


def _prepare_window(case, r, g):
    S, P, W = case["streams"], case["page"], case["rows"]
    lens = _lens(case, r, S)
    # the pages a sliding-window layer still holds: those with a visible
    # position; the others went back to the pool (-1)
    stride = -(-case["len_hi"] // P)
    j = np.arange(stride)[None, :]
    start = np.maximum(lens - W - case["window"] + 1, 0)[:, None]
    held = (j * P < lens[:, None]) & ((j * P < case["sinks"]) | ((j + 1) * P > start))
    need = int(held.sum())
    n_pages = need + max(1, need // 8)
    table = np.full((S, stride), -1, np.int32)
    table[held] = r.permutation(n_pages)[:need]
    k_pool, v_pool = _pools(case, g, n_pages)
    q = _normal(g, (S, W, case["kv_heads"] * case["group"], case["dim"]))
    return dict(k_pool=k_pool, v_pool=v_pool, table=_up(table), lens=_up(lens.astype(np.int32)), q=q,
                out=torch.empty(q.shape, dtype=torch.float32, device=_dev()), max_len=int(lens.max()),
                scale=1.0 / math.sqrt(case["dim"]),
                workspace=torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=_dev()))


def _pair_axis(case):
    """The axis of each rotated pair: sections of nearly equal size in order, as in the (time, height, width) split."""
    n = case["rotary"] // 2
    return [min(case["axes"] - 1, i * case["axes"] // n) for i in range(n)]


def _prepare_rope(case, r, g):
    S, P, W, D = case["streams"], case["page"], case["rows"], case["dim"]
    Hkv, Hq = case["kv_heads"], case["kv_heads"] * case["group"]
    lens = _lens(case, r, S)
    stride = -(-case["len_hi"] // P)
    first = (lens - W) // P  # only the pages that are written need to exist here
    j = np.arange(stride)[None, :]
    held = (j * P < lens[:, None]) & (j >= first[:, None])
    need = int(held.sum())
    n_pages = S * ((W + P - 2) // P + 1) + 1
    table = np.full((S, stride), -1, np.int32)
    table[held] = r.permutation(n_pages)[:need]
    k_pool, v_pool = _pools(case, g, n_pages)
    qkv = _normal(g, (S, W, Hq + 2 * Hkv, D))  # one projection's output: the rows are slices of it
    # text rows move every axis together; an image's rows share a time and walk its height and width
    base = r.integers(0, case["far"] + 1, (S, 1, 1))
    row = np.arange(W)[None, :, None]
    step = np.stack([row // 64, row // 8 % 8, row % 8, row % 5], -1)[..., : case["axes"]].reshape(1, W, case["axes"])
    image = r.random((S, 1, 1)) < 0.5
    positions = np.where(image, base + step, base + row).astype(np.int32)
    inv_freq = 10000.0 ** (-np.arange(case["rotary"] // 2) * 2.0 / case["rotary"])
    return dict(k_pool=k_pool, v_pool=v_pool, table=_up(table), lens=_up(lens.astype(np.int32)), max_len=int(lens.max()),
                q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:], positions=_up(positions),
                inv_freq=_up(inv_freq.astype(np.float32)), pair_axis=_pair_axis(case),
                axis_index=_up(np.array(_pair_axis(case), np.int64)),
                q_out=torch.empty((S, W, Hq, D), dtype=torch.bfloat16, device=_dev()))


def _views(flat, shapes):
    out, at = [], 0
    for s in shapes:
        n = int(np.prod(s))
        out.append(flat[at:at + n].view(s))
        at += n
    return out


def _meta(arrays):
    """The page bookkeeping in one buffer, and a copy of it to begin each pass with: a pass changes it in place."""
    flat = _up(np.concatenate([np.asarray(a, np.int32).reshape(-1) for a in arrays]))
    now = flat.clone()
    return flat, now, _views(now, [np.shape(a) for a in arrays])


def _move_list(n):
    return torch.zeros((1 + n, 4), dtype=torch.int32, device=_dev())


def _prepare_beam(case, r, g):
    B, N, P = case["prompts"], case["beams"], case["page"]
    n_rows = B * N
    lens = np.repeat(_lens(case, r, B), N)
    stride = -(-(case["len_hi"] + 1) // P)
    shared = (lens * 2 // 3) // P  # the whole pages of the prompt are shared by its beams
    pages = -(-lens // P)
    # the pool holds the largest prompts, a page more for each beam, and some to spare
    any_len = np.arange(case["len_lo"], case["len_hi"] + 1)
    any_shared = any_len * 2 // 3 // P
    most = B * int((any_shared + N * (-(-any_len // P) - any_shared)).max())
    n_pages = most + n_rows + 1 + int(case["spare"] * most)
    ids = r.permutation(n_pages)
    table = np.full((n_rows, stride), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    at = 0
    for p in range(B):
        s, own_pages = int(shared[p * N]), int((pages - shared)[p * N])
        for b in range(N):
            table[p * N + b, :s] = ids[at:at + s]
        for b in range(N):
            o = at + s + b * own_pages
            table[p * N + b, s:s + own_pages] = ids[o:o + own_pages]
        at += s + N * own_pages
    np.add.at(refs, table[table >= 0], 1)
    parents = (np.arange(n_rows) // N) * N + r.integers(0, N, n_rows)
    start, now, (refs, table, lens, new_table, new_lens) = _meta([refs, table, lens, np.full_like(table, -1), np.zeros_like(lens)])
    k_pool, v_pool = _pools(case, g, n_pages)
    return dict(k_pool=k_pool, v_pool=v_pool, start=start, now=now, refs=refs, table=table, lens=lens, new_table=new_table,
                new_lens=new_lens, parents=_up(parents.astype(np.int32)), moves=_move_list(2 * n_rows), page=P)


def _prepare_evict(case, r, g):
    S, P = case["streams"], case["page"]
    lens = _lens(case, r, S)
    stride = -(-case["len_hi"] // P)
    held = np.arange(stride)[None, :] * P < lens[:, None]
    used = int(held.sum())
    n_pages = S * stride + 1 + int(case["spare"] * S * stride)
    table = np.full((S, stride), -1, np.int32)
    table[held] = r.permutation(n_pages)[:used]
    refs = np.zeros(n_pages, np.int32)
    refs[table[held]] = 1
    start, now, (refs, table, lens) = _meta([refs, table, lens])
    k_pool, v_pool = _pools(case, g, n_pages)
    return dict(k_pool=k_pool, v_pool=v_pool, start=start, now=now, refs=refs, table=table, lens=lens,
                moves=_move_list(n_pages // 2), page=P)


def prepare(case, seed):
    r = np.random.default_rng([seed, 17])
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    make = {"window": _prepare_window, "rope": _prepare_rope, "beam": _prepare_beam, "evict": _prepare_evict}[case["op"]]
    state = make(case, r, g)
    state["case"] = dict(case)
    return state


# ---- sliding-window attention --------------------------------------------------

def _plain_window(s):
    c = s["case"]
    P, W, window, sinks, Hkv, G = c["page"], c["rows"], c["window"], c["sinks"], c["kv_heads"], c["group"]
    q, lens = s["q"].float(), s["lens"].long()[:, None]
    S, _, Hq, D = q.shape
    # the positions some row of the stream sees: the first ones, then the window of the first row on
    n = min(s["max_len"], sinks + window + W - 1)
    i = torch.arange(n, device=q.device)[None, :]
    start = (lens - W - window + 1).clamp(min=sinks)
    pos = torch.where(i < sinks, i, i - sinks + start)
    there = pos < lens
    at = torch.where(there, pos, 0)
    page = s["table"].long().gather(1, at // P)
    there_d = there[:, :, None, None]
    k = torch.where(there_d, s["k_pool"][page, :, at % P].float(), 0.0)
    v = torch.where(there_d, s["v_pool"][page, :, at % P].float(), 0.0)
    row = lens + torch.arange(W, device=q.device) - W  # [S][W]: the rows' positions
    row, p = row[:, :, None], pos[:, None, :]
    sees = (p <= row) & ((p > row - window) | (p < sinks))
    sees = sees[:, None, :, None, :].expand(S, Hkv, W, G, n).reshape(S, Hkv, W * G, n)
    qh = q.view(S, W, Hkv, G, D).transpose(1, 2).reshape(S, Hkv, W * G, D)
    scores = (qh @ k.permute(0, 2, 3, 1)) * s["scale"]
    scores = scores.masked_fill(~sees, float("-inf"))
    w = torch.exp(scores - scores.amax(-1, keepdim=True))
    out = (w @ v.transpose(1, 2)) / w.sum(-1, keepdim=True)
    return out.view(S, Hkv, W, G, D).transpose(1, 2).reshape(S, W, Hq, D)


def _own_window(s):
    import verify_paged_gqa_b200 as tf
    c = s["case"]
    call = (tf.tf_paged_attn_decode_window if c["rows"] == 1 else
            tf.tf_paged_attn_verify_window if c["rows"] <= 8 else tf.tf_paged_attn_prompt_window)
    return call(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["q"], c["window"], c["sinks"], s["scale"], s["out"],
                s["workspace"], s["max_len"])


# ---- rotary positions of several axes, and the row write ----------------------------

def _turn(x, cos, sin, rotary, adjacent):
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if adjacent else (x[..., :rotary // 2], x[..., rotary // 2:rotary])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    if adjacent:
        y[..., 0:rotary:2], y[..., 1:rotary:2] = lo, hi
    else:
        y[..., :rotary // 2], y[..., rotary // 2:rotary] = lo, hi
    return y.to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    P, W = c["page"], c["rows"]
    angle = s["positions"].double()[..., s["axis_index"]] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    q = _turn(s["q"], cos, sin, c["rotary"], c["adjacent"])
    k = _turn(s["k"], cos, sin, c["rotary"], c["adjacent"])
    pos = s["lens"].long()[:, None] + torch.arange(W, device=q.device) - W
    page = s["table"].long().gather(1, pos // P)
    s["k_pool"][page, :, pos % P] = k
    s["v_pool"][page, :, pos % P] = s["v"]
    return q, s["k_pool"], s["v_pool"]


def _own_rope(s):
    import verify_paged_gqa_b200 as tf
    c = s["case"]
    rope = s.get("rope")
    if rope is None:  # the plan a program keeps: it depends on the layer's settings alone
        rope = s["rope"] = tf.Rope(s["inv_freq"], s["pair_axis"], c["axes"], adjacent=c["adjacent"])
    q = tf.tf_kv_put_rows_rope(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["q"], s["k"], s["v"], s["positions"], rope,
                               s["max_len"], q_out=s["q_out"])
    return q, s["k_pool"], s["v_pool"]


# ---- pages ------------------------------------------------------------------------

def _plain_release(refs, table, gone):
    """Drops the entries of `table` that `gone` names."""
    gone = gone & (table >= 0)
    refs.scatter_add_(0, table.clamp(min=0).long().view(-1), -gone.to(refs.dtype).view(-1))
    table.masked_fill_(gone, -1)


def _plain_beam(s):
    P, refs, table, new = s["page"], s["refs"], s["table"], s["new_table"]
    stride = table.shape[1]
    j = torch.arange(stride, device=table.device)[None, :]
    # fork: a child holds its parent's pages
    parents = s["parents"].long()
    lens = s["lens"][parents]
    new.copy_(torch.where(j * P < lens[:, None], table[parents], -1))
    refs.scatter_add_(0, new.clamp(min=0).long().view(-1), (new >= 0).to(refs.dtype).view(-1))
    # free the old beams
    _plain_release(refs, table, torch.ones_like(table, dtype=torch.bool))
    # grow by one position: a page of its own under each row's new position
    at = (lens // P).long()[:, None]
    s["new_lens"].copy_(lens + 1)
    page = new.gather(1, at)[:, 0].long()
    shared = (page >= 0) & (refs[page.clamp(min=0)] > 1)
    need = (page < 0) | shared
    rank = need.to(torch.int64).cumsum(0) - 1
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)  # free pages first, lowest id first
    got = torch.where(need, free[rank.clamp(min=0)], page)
    new.scatter_(1, at, got.to(new.dtype)[:, None])
    refs.scatter_add_(0, page.clamp(min=0), -shared.to(refs.dtype))
    refs.scatter_add_(0, got, need.to(refs.dtype))
    # the positions before the new one move along
    src = torch.where(shared, page, got)
    keep = (torch.arange(P, device=table.device)[None, :] < (lens % P)[:, None])[:, None, :, None] & shared[:, None, None, None]
    s["k_pool"][got] = torch.where(keep, s["k_pool"][src], s["k_pool"][got])
    s["v_pool"][got] = torch.where(keep, s["v_pool"][src], s["v_pool"][got])


def _own_beam(s):
    import verify_paged_gqa_b200 as tf
    refs, P = s["refs"], s["page"]
    tf.tf_kv_pages_fork(refs, P, s["table"], s["lens"], s["parents"], s["new_table"], s["new_lens"])
    tf.tf_kv_pages_free(refs, P, s["table"])
    s["new_lens"].add_(1)
    tf.tf_kv_pages_grow(refs, P, s["new_table"], s["new_lens"], 1, s["moves"])
    tf.tf_kv_pages_move(s["k_pool"], s["v_pool"], s["moves"])


def _beam(s):
    s["now"].copy_(s["start"])
    _own_beam(s) if own else _plain_beam(s)
    return s["new_table"], s["new_lens"], s["table"], s["refs"], s["k_pool"], s["v_pool"]


def _plain_evict(s):
    c = s["case"]
    P, refs, table = s["page"], s["refs"], s["table"]
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    # a later row sits at position lens or beyond: it sees the sinks and positions past lens - window
    _plain_release(refs, table, (j * P >= c["sinks"]) & ((j + 1) * P - 1 <= s["lens"][:, None] - c["window"]))
    # compact: the live pages past the number of live pages move into the holes below it
    ids = torch.arange(refs.shape[0], device=refs.device)
    live = refs > 0
    n_live = live.sum()
    src, dst = ids[live & (ids >= n_live)], ids[~live & (ids < n_live)]
    to = ids.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(table.dtype), -1))
    refs[dst] = refs[src]
    refs[src] = 0
    s["k_pool"][dst] = s["k_pool"][src]
    s["v_pool"][dst] = s["v_pool"][src]


def _own_evict(s):
    import verify_paged_gqa_b200 as tf
    c = s["case"]
    refs, P = s["refs"], s["page"]
    tf.tf_kv_pages_free_window(refs, P, s["table"], s["lens"], c["window"], c["sinks"])
    tf.tf_kv_pages_compact(refs, P, s["table"], s["moves"])
    tf.tf_kv_pages_move(s["k_pool"], s["v_pool"], s["moves"])


def _evict(s):
    s["now"].copy_(s["start"])
    _own_evict(s) if own else _plain_evict(s)
    return s["table"], s["refs"], s["k_pool"], s["v_pool"]


def run(state):
    op = state["case"]["op"]
    if op == "window":
        return _own_window(state) if own else _plain_window(state)
    if op == "rope":
        return _own_rope(state) if own else _plain_rope(state)
    return _beam(state) if op == "beam" else _evict(state)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    kv_row = 2 * case["kv_heads"] * case["dim"] * 2  # a position's K and V, bytes
    mid = (case["len_lo"] + case["len_hi"]) / 2
    if op == "window":
        W, window, sinks = case["rows"], case["window"], case["sinks"]
        Hq = case["kv_heads"] * case["group"]
        n = min(mid, sinks + window + W - 1)
        seen = min(mid, sinks + window)  # by a row, about
        if mid < sinks + window:
            seen = mid - (W - 1) / 2
        rows = case["streams"] * W * Hq
        return dict(bytes=case["streams"] * n * kv_row + rows * case["dim"] * 6, flops=4 * rows * seen * case["dim"])
    if op == "rope":
        rows = case["streams"] * case["rows"]
        Hq = case["kv_heads"] * case["group"]
        return dict(bytes=rows * (2 * kv_row + 4 * Hq * case["dim"] + 4 * case["axes"]),
                    flops=rows * (Hq + case["kv_heads"]) * case["rotary"] * 3)
    if op == "beam":
        rows = case["prompts"] * case["beams"]
        pages = -(-mid // case["page"])
        # most children share their parent's last page: about half a page is copied
        n = case["beams"]
        copies = rows * max(0.0, 1 - (1 - 1 / n) ** (n - 1)) if n > 1 else 0.0
        return dict(bytes=rows * pages * 4 * 4 + 2 * copies * kv_row * min(mid, case["page"] / 2), flops=0)
    pages = case["streams"] * mid / case["page"]
    kept = case["streams"] * (min(mid, case["window"] + case["sinks"]) / case["page"] + 1)
    total = case["streams"] * case["len_hi"] / case["page"] * (1 + case["spare"])
    moved = min(kept, pages) * max(0.0, 1 - kept / total)
    return dict(bytes=8 * total + 8 * pages + 2 * moved * case["page"] * kv_row, flops=0)


# ---- the definitions in 64 bits ---------------------------------------------------------

def _exact_window(case, s):
    P, W, Hkv, G = case["page"], case["rows"], case["kv_heads"], case["group"]
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=_dev())
    for b, n in enumerate(lens):
        n = int(n)
        first = max(0, n - W - case["window"] + 1)
        pos = [p for p in range(n) if p < case["sinks"] or p >= first]
        page = _up(table[b][np.array(pos) // P].astype(np.int64))
        slot = _up(np.array(pos) % P)
        pos = _up(np.array(pos))
        for h in range(Hkv):
            k, v = s["k_pool"][page, h, slot].double(), s["v_pool"][page, h, slot].double()
            for r0 in range(0, W, 1024):
                r1 = min(W, r0 + 1024)
                at = torch.arange(n - W + r0, n - W + r1, device=_dev())[:, None, None]
                hidden = (pos > at) | ((pos >= case["sinks"]) & (at - pos >= case["window"]))
                x = s["q"][b, r0:r1, h * G:(h + 1) * G].double() * s["scale"]
                a = torch.einsum("rgd,nd->rgn", x, k).masked_fill(hidden, -math.inf)
                out[b, r0:r1, h * G:(h + 1) * G] = torch.einsum("rgn,nd->rgd", torch.softmax(a, -1), v)
    return out


def _exact_rope(case, s):
    P, W, half = case["page"], case["rows"], case["rotary"] // 2
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    turned = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        for i in range(half):
            a = s["positions"][..., s["pair_axis"][i]].double()[:, :, None] * float(s["inv_freq"][i])
            d0, d1 = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + half)
            y[..., d0] = x[..., d0] * torch.cos(a) - x[..., d1] * torch.sin(a)
            y[..., d1] = x[..., d0] * torch.sin(a) + x[..., d1] * torch.cos(a)
        turned[name] = y
    for b, n in enumerate(lens):
        pos = np.arange(n - W, n)
        page, slot = _up(table[b][pos // P].astype(np.int64)), _up(pos % P)
        k_pool[page, :, slot] = turned["k"][b]
        v_pool[page, :, slot] = s["v"][b].double()
    return turned["q"], k_pool, v_pool


def exact(case, seed):
    if case["op"] not in ("window", "rope"):
        return None  # whole numbers and copied bits: compared as they are
    s = prepare(case, seed)
    return _exact_window(case, s) if case["op"] == "window" else _exact_rope(case, s)

"""Measured cases of the rotary, cache-append and window-with-sinks attention operators.

Each case names one call of the library and its sizes.  ``run`` computes it either
through the library (``own`` true) or in its plain form: elementary torch operations in
32 bits (angles in 64), rounded once at the end.  ``exact`` gives the same outputs in 64
bits from the definitions.

  rope / rope_bwd   rotary positions of Q and K inside a training step, and their gradient
  append            new keys and values, rotated, into a paged cache (bf16 or E4M3)
  window            causal attention with a sliding window and visible first tokens
  paged_window      the same for query tokens appended to a paged cache
  window_bwd        its gradients
  decode_window     single-token attention over a paged cache, window and first tokens
"""
import math

import torch

own = False

DEVICE = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # Q and K of a training step's long sequence, as views of the fused projection
        {"name": "rope_8k", "op": "rope", "batch": 1, "heads": 32, "kv_heads": 8, "seq": 8192,
         "dim": 128, "rotary": 128, "interleaved": False, "scaling": "none", "start": 0},
        # its gradient for shorter rows, half of the head rotated, interleaved pairs, positions
        # far into a document whose frequencies were stretched for it
        {"name": "rope_bwd_2k_far", "op": "rope_bwd", "batch": 4, "heads": 16, "kv_heads": 16,
         "seq": 2048, "dim": 128, "rotary": 64, "interleaved": True, "scaling": "ramp",
         "start": 200000},
        # one decode step of a serving batch: every sequence's new token into its last page
        {"name": "append_step_64", "op": "append", "seqs": 64, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "new_min": 1, "new_max": 1, "len_min": 512, "len_max": 8191,
         "rotary": 128, "interleaved": False, "cache": "bf16"},
        # a mix of prompts and chunks of prompts
        {"name": "append_chunks_8", "op": "append", "seqs": 8, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "new_min": 131, "new_max": 4097, "len_min": 1, "len_max": 4000,
         "rotary": 128, "interleaved": False, "cache": "bf16"},
        # a decode step of a small batch over an 8-bit cache, part of the head rotated
        {"name": "append_step_5_e4m3", "op": "append", "seqs": 5, "heads": 16, "kv_heads": 4,
         "dim": 64, "page": 64, "new_min": 1, "new_max": 1, "len_min": 3, "len_max": 2000,
         "rotary": 32, "interleaved": True, "cache": "e4m3"},
        # a padded batch of short rows, lengths that end inside a tile
        {"name": "window_1k_padded", "op": "window", "batch": 3, "heads": 8, "kv_heads": 2,
         "seq_q": 1000, "seq_k": 1000, "dim": 64, "window": 200, "sinks": 4, "padded": True},
        # the long rows of a model whose layers see a window
        {"name": "window_8k", "op": "window", "batch": 2, "heads": 32, "kv_heads": 8,
         "seq_q": 8192, "seq_k": 8192, "dim": 128, "window": 1024, "sinks": 4, "padded": False},
        # prompts processed in chunks against what the cache already holds
        {"name": "paged_window_8", "op": "paged_window", "seqs": 8, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "new_min": 5, "new_max": 1024, "len_min": 1, "len_max": 7168,
         "window": 1024, "sinks": 4},
        # gradients of a short odd-sized batch
        {"name": "window_bwd_700", "op": "window_bwd", "batch": 2, "heads": 4, "kv_heads": 2,
         "seq_q": 700, "seq_k": 700, "dim": 64, "window": 100, "sinks": 3, "padded": True},
        # gradients of the long rows
        {"name": "window_bwd_8k", "op": "window_bwd", "batch": 1, "heads": 32, "kv_heads": 8,
         "seq_q": 8192, "seq_k": 8192, "dim": 128, "window": 1024, "sinks": 4, "padded": False},
        # a decode step of a serving batch
        {"name": "decode_window_64", "op": "decode_window", "seqs": 64, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "len_min": 512, "len_max": 8192,
         "window": 1024, "sinks": 4, "cache": "bf16"},
        # a decode step of a single conversation over an 8-bit cache: latency
        {"name": "decode_window_1_e4m3", "op": "decode_window", "seqs": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "len_min": 5000, "len_max": 5000,
         "window": 2000, "sinks": 4, "cache": "e4m3"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 4]), kv


def _sinks(rng):
    return rng.choice([0, 1, 4, 16, rng.randint(1, 200)])


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "append", "window", "paged_window",
                     "window_bwd", "decode_window", "decode_window"])
    heads, kv = _heads(rng)
    dim = rng.choice([64, 128])
    case = {"op": op, "heads": heads, "kv_heads": kv, "dim": dim}
    if op in ("rope", "rope_bwd"):
        case["seq"] = _log_int(rng, 1, 8192)
        case["batch"] = rng.randint(1, max(1, min(8, 8192 // case["seq"])))
        case["rotary"] = 16 * rng.randint(1, dim // 16)
        case["interleaved"] = rng.random() < 0.5
        case["scaling"] = rng.choice(["none", "linear", "ramp"])
        case["start"] = rng.choice([0, _log_int(rng, 1, 1000000)])
    elif op == "append":
        case["page"] = rng.choice([16, 32, 64, 128])
        case["cache"] = rng.choice(["bf16", "e4m3"])
        case["rotary"] = 16 * rng.randint(1, dim // 16)
        case["interleaved"] = rng.random() < 0.5
        case["seqs"] = _log_int(rng, 1, 64)
        top = 1 if rng.random() < 0.5 else _log_int(rng, 2, max(2, 16384 // case["seqs"]))
        case["new_max"] = top
        case["new_min"] = rng.randint(1, top)
        case["len_max"] = _log_int(rng, 1, 8000)
        case["len_min"] = rng.randint(1, case["len_max"])
    elif op in ("window", "window_bwd"):
        case["seq_q"] = _log_int(rng, 1, 8192)
        case["seq_k"] = case["seq_q"] if rng.random() < 0.6 else \
            min(8192, case["seq_q"] + _log_int(rng, 1, 2000))
        case["batch"] = rng.randint(1, max(1, min(4, 8192 // case["seq_q"])))
        case["window"] = _log_int(rng, 16, 4096)
        case["sinks"] = _sinks(rng)
        case["padded"] = rng.random() < 0.4
        if op == "window_bwd":
            case["batch"] = min(case["batch"], 2)
    elif op == "paged_window":
        case["page"] = rng.choice([16, 32, 64, 128])
        case["seqs"] = _log_int(rng, 1, 8)
        case["new_max"] = _log_int(rng, 1, 1024)
        case["new_min"] = rng.randint(1, case["new_max"])
        case["len_max"] = _log_int(rng, 1, 7000)
        case["len_min"] = rng.randint(1, case["len_max"])
        case["window"] = _log_int(rng, 16, 4096)
        case["sinks"] = _sinks(rng)
    else:
        case["page"] = rng.choice([16, 32, 64, 128])
        case["cache"] = rng.choice(["bf16", "e4m3"])
        case["seqs"] = _log_int(rng, 1, 64)
        case["len_max"] = _log_int(rng, 1, 8192)
        case["len_min"] = rng.randint(1, case["len_max"])
        case["window"] = _log_int(rng, 16, 1500)
        case["sinks"] = _sinks(rng)
    return case


# ------------------------------------------------------------------- sizes of a case

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spaced over their logarithm (the same for every seed)."""
    if n == 1:
        return [hi]
    return [min(hi, max(lo, round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * i / (n - 1)))))
            for i in range(n)]


def _lengths(case):
    """(new tokens, cached + new tokens) of each sequence of a paged case."""
    n = case["seqs"]
    cached = _spread(case["len_min"], case["len_max"], n)
    if "new_max" not in case:
        return [1] * n, cached
    new = _spread(case["new_min"], case["new_max"], n)[::-1]
    return new, [c + w for c, w in zip(cached, new)]


def _seen(p, window, sinks):
    """Keys that the row at key position p sees."""
    if p < 0:
        return 0
    own_window = min(p + 1, window)
    return own_window + min(sinks, p + 1 - own_window)


def _padded_lengths(case):
    """Key length of each row of a batch: whole, or shorter by up to a quarter."""
    n, sk = case["batch"], case["seq_k"]
    if not case["padded"]:
        return [sk] * n
    return [sk - (sk // 4) * (i + 1) // n for i in range(n)]


def work(case):
    op, hq, hkv, d = case["op"], case["heads"], case["kv_heads"], case["dim"]
    if op in ("rope", "rope_bwd"):
        rows = case["batch"] * case["seq"] * (hq + hkv)
        return {"bytes": 4 * rows * d, "flops": 3 * rows * case["rotary"]}
    if op == "append":
        new, _ = _lengths(case)
        out = 2 if case["cache"] == "bf16" else 1
        total = sum(new)
        return {"bytes": total * d * (4 * hq + 2 * (2 + out) * hkv),
                "flops": 3 * total * (hq + hkv) * case["rotary"]}
    if op in ("window", "window_bwd"):
        sq, sk = case["seq_q"], case["seq_k"]
        pairs = sum(_seen(i + n - sq, case["window"], case["sinks"])
                    for n in _padded_lengths(case) for i in range(sq)) * hq
        rows_q, rows_k = case["batch"] * sq * hq, case["batch"] * sk * hkv
        if op == "window":
            return {"bytes": 2 * d * (2 * rows_q + 2 * rows_k) + 4 * rows_q,
                    "flops": 4 * d * pairs}
        return {"bytes": 2 * d * (4 * rows_q + 4 * rows_k) + 4 * rows_q, "flops": 10 * d * pairs}
    new, total = _lengths(case)
    w, s = case["window"], case["sinks"]
    if op == "paged_window":
        pairs = sum(_seen(t - n + i, w, s) for n, t in zip(new, total) for i in range(n)) * hq
        keys = sum(min(t, w + n - 1 + s) for n, t in zip(new, total))
        rows = sum(new) * hq
        return {"bytes": 4 * d * rows + 4 * rows + 4 * d * keys * hkv, "flops": 4 * d * pairs}
    keys = sum(_seen(t - 1, w, s) for t in total)
    size = 2 if case["cache"] == "bf16" else 1
    return {"bytes": 2 * size * d * keys * hkv + 4 * d * case["seqs"] * hq,
            "flops": 4 * d * keys * hq}


# ----------------------------------------------------------------------------- inputs

def _frequencies(case):
    """Radians per token of each rotated pair, float64, and the factor on cos and sin."""
    half = case["rotary"] // 2
    i = torch.arange(half, dtype=torch.float64)
    freq = 10000.0 ** (-i / half)
    kind = case.get("scaling", "none")
    if kind == "linear":
        return freq / 4.0, 1.0
    if kind == "ramp":  # low frequencies stretched, high ones kept, a linear ramp between
        factor, original = 32.0, 8192.0
        turns = original * freq / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return freq * keep + freq / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return freq, 1.0


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.bfloat16)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _codes(g, *shape):
    """E4M3 codes of normal values over about a tenth of the format's range."""
    x = torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
    return (x.mul_(40.0).clamp_(-E4M3_MAX, E4M3_MAX)).to(torch.float8_e4m3fn).view(torch.uint8)


def _paged(case, seed):
    """A page pool, its block table and the sequences' lengths."""
    g = _generator(seed)
    hkv, d, page = case["kv_heads"], case["dim"], case["page"]
    new, total = _lengths(case)
    order = torch.randperm(case["seqs"], generator=torch.Generator().manual_seed(seed)).tolist()
    new, total = [new[i] for i in order], [total[i] for i in order]
    per = [-(-t // page) for t in total]
    pages, most = sum(per) + 3, max(per)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 1)).tolist()
    table, at = [], 0
    for n in per:
        table.append(perm[at:at + n] + [-1] * (most - n))
        at += n
    state = {"case": case, "block_table": _int32(table), "seq_lens": _int32(total),
             "new": new, "total": total}
    if case.get("cache") == "e4m3":
        state["k_cache"] = _codes(g, pages, page, hkv, d)
        state["v_cache"] = _codes(g, pages, page, hkv, d)
        for name in ("k_scale", "v_scale"):
            state[name] = (torch.rand(pages, hkv, generator=g, device=DEVICE) + 0.5) / 40.0
    else:
        state["k_cache"] = _normal(g, pages, page, hkv, d)
        state["v_cache"] = _normal(g, pages, page, hkv, d)
    return state, g


def prepare(case, seed):
    op, hq, hkv, d = case["op"], case["heads"], case["kv_heads"], case["dim"]
    if op in ("rope", "rope_bwd"):
        g = _generator(seed)
        freq, factor = _frequencies(case)
        b, s = case["batch"], case["seq"]
        state = {"case": case, "inv_freq": freq.to(DEVICE), "factor": factor,
                 "positions": _int32([case["start"] + i for i in range(s)])}
        if op == "rope":
            # the fused projection's output: Q, K and V heads of a token next to each other
            state["qkv"] = _normal(g, b, s, hq + 2 * hkv, d)
        else:
            # what the attention's backward pass hands on, and the buffer that the
            # projection's gradient is collected in
            state["dq"], state["dk"] = _normal(g, b, hq, s, d), _normal(g, b, hkv, s, d)
            state["dqkv"] = torch.zeros(b, s, hq + 2 * hkv, d, device=DEVICE, dtype=torch.bfloat16)
        return state
    if op == "append":
        state, g = _paged(case, seed)
        freq, factor = _frequencies(case)
        total = sum(state["new"])
        cu = [0]
        for n in state["new"]:
            cu.append(cu[-1] + n)
        return state | {"qkv": _normal(g, total, hq + 2 * hkv, d), "inv_freq": freq.to(DEVICE),
                        "factor": factor, "cu": None if case["new_max"] == 1 else _int32(cu)}
    if op in ("window", "window_bwd"):
        g = _generator(seed)
        b, sq, sk = case["batch"], case["seq_q"], case["seq_k"]
        state = {"case": case, "q": _normal(g, b, hq, sq, d), "k": _normal(g, b, hkv, sk, d),
                 "v": _normal(g, b, hkv, sk, d),
                 "k_lens": _int32(_padded_lengths(case)) if case["padded"] else None}
        if op == "window_bwd":  # what the forward pass saved
            state["o"], state["lse"] = _window_plain(state)
            state["d_o"] = _normal(g, b, hq, sq, d)
        return state
    state, g = _paged(case, seed)
    if op == "paged_window":
        cu = [0]
        for n in state["new"]:
            cu.append(cu[-1] + n)
        return state | {"q": _normal(g, cu[-1], hq, d), "cu": _int32(cu),
                        "max_new": max(state["new"])}
    return state | {"q": _normal(g, case["seqs"], hq, d)}


# ------------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, rotary, interleaved):
    """Rotates the first `rotary` elements of the last axis pair by pair (float32)."""
    x = x.float()
    head, tail = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = head[..., :rotary // 2], head[..., rotary // 2:]
        head = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((head, tail), dim=-1)


def _cos_sin(positions, inv_freq, factor):
    angle = positions.double()[:, None] * inv_freq
    return (angle.cos() * factor).float(), (angle.sin() * factor).float()


def _rope_plain(state):
    case = state["case"]
    cos, sin = _cos_sin(state["positions"], state["inv_freq"], state["factor"])
    how = (case["rotary"], case["interleaved"])
    hq, hkv = case["heads"], case["kv_heads"]
    if case["op"] == "rope":
        q, k = state["qkv"][:, :, :hq], state["qkv"][:, :, hq:hq + hkv]
        cos, sin = cos[:, None], sin[:, None]
        return [_rotate(x, cos, sin, *how).to(torch.bfloat16).transpose(1, 2).contiguous()
                for x in (q, k)]
    to = state["dqkv"]
    to[:, :, :hq] = _rotate(state["dq"], cos, -sin, *how).transpose(1, 2)
    to[:, :, hq:hq + hkv] = _rotate(state["dk"], cos, -sin, *how).transpose(1, 2)
    return to


def _append_plain(state):
    case = state["case"]
    hq, hkv, page = case["heads"], case["kv_heads"], case["page"]
    qkv, lens = state["qkv"], state["seq_lens"].long()
    n = qkv.shape[0]
    token = torch.arange(n, device=DEVICE)
    if state["cu"] is None:
        seq, position = token, lens - 1
    else:
        cu = state["cu"].long()
        seq = (token[:, None] >= cu[None, 1:]).sum(1)
        position = lens[seq] - cu[seq + 1] + token
    cos, sin = _cos_sin(position, state["inv_freq"], state["factor"])
    how = (cos[:, None], sin[:, None], case["rotary"], case["interleaved"])
    q = _rotate(qkv[:, :hq], *how).to(torch.bfloat16)
    k = _rotate(qkv[:, hq:hq + hkv], *how)
    v = qkv[:, hq + hkv:]
    where = state["block_table"].long()[seq, position // page]
    row = position % page
    if case["cache"] == "bf16":
        state["k_cache"][where, row] = k.to(torch.bfloat16)
        state["v_cache"][where, row] = v
        return q, state["k_cache"], state["v_cache"]
    for x, cache, scale in ((k, "k_cache", "k_scale"), (v.float(), "v_cache", "v_scale")):
        y = x / state[scale][where][:, :, None]
        y = y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        state[cache][where, row] = y.view(torch.uint8)
    return (q, state["k_cache"].view(torch.float8_e4m3fn),
            state["v_cache"].view(torch.float8_e4m3fn))


def _visible(rows, keys, key_len, offset, case):
    """Whether query row i sees key j, from the row's own place p = i + offset among the keys."""
    p = rows + offset
    near = keys > p - case["window"]
    first = keys < case["sinks"]
    return (keys <= p) & (keys < key_len) & (near | first)


def _softmax_plain(s, visible):
    """(weights, log-sum-exp) of the last axis of s where visible; empty rows: zeros, -inf."""
    s = s.masked_fill_(~visible, -math.inf)
    m = s.amax(-1, keepdim=True)
    base = m.masked_fill(m == -math.inf, 0.0)
    e = s.sub_(base).exp_()
    total = e.sum(-1, keepdim=True)
    return e.div_(total.masked_fill(total == 0.0, 1.0)), (base + total.log()).squeeze(-1)


def _batch_mask(state):
    case = state["case"]
    sq, sk = case["seq_q"], case["seq_k"]
    lens = state["k_lens"]
    lens = torch.full((case["batch"],), sk, device=DEVICE) if lens is None else lens.long()
    lens = lens[:, None, None]
    rows = torch.arange(sq, device=DEVICE)[None, :, None]
    keys = torch.arange(sk, device=DEVICE)[None, None, :]
    return _visible(rows, keys, lens, lens - sq, case)[:, None, None]


def _grouped(state):
    """Q, K, V in 32 bits with the query heads of a KV head as an axis of their own."""
    case = state["case"]
    b, hq, hkv, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    q = state["q"].float().reshape(b, hkv, hq // hkv * case["seq_q"], d)
    return q, state["k"].float(), state["v"].float()


def _window_plain(state):
    case = state["case"]
    b, hq, hkv, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    sq, sk = case["seq_q"], case["seq_k"]
    q, k, v = _grouped(state)
    s = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).view(b, hkv, hq // hkv, sq, sk)
    p, lse = _softmax_plain(s, _batch_mask(state))
    o = p.view(b, hkv, -1, sk) @ v
    return o.view(b, hq, sq, d).to(torch.bfloat16), lse.reshape(b, hq, sq)


def _window_bwd_plain(state):
    case = state["case"]
    b, hq, hkv, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    sq, sk = case["seq_q"], case["seq_k"]
    scale = d ** -0.5
    q, k, v = _grouped(state)
    d_o = state["d_o"].float()
    delta = (d_o * state["o"].float()).sum(-1).view(b, hkv, -1, 1)
    d_o = d_o.reshape(q.shape)
    lse = state["lse"].view(b, hkv, hq // hkv, sq, 1)
    p = (q @ k.transpose(-1, -2)).mul_(scale).view(b, hkv, hq // hkv, sq, sk)
    p = p.sub_(lse.masked_fill(lse == -math.inf, 0.0)).exp_()
    p = p.masked_fill_(~_batch_mask(state), 0.0).view(b, hkv, -1, sk)
    dv = p.transpose(-1, -2) @ d_o
    ds = (d_o @ v.transpose(-1, -2)).sub_(delta).mul_(p)
    dq = (ds @ k).mul_(scale).view(b, hq, sq, d)
    dk = (ds.transpose(-1, -2) @ q).mul_(scale)
    return [x.to(torch.bfloat16) for x in (dq, dk, dv)]


def _paged_window_plain(state):
    case = state["case"]
    hq, hkv, d, n = case["heads"], case["kv_heads"], case["dim"], case["seqs"]
    cu, lens, most = state["cu"].long(), state["seq_lens"].long(), state["max_new"]
    sk = state["block_table"].shape[1] * case["page"]
    new = cu[1:] - cu[:-1]
    row = torch.arange(most, device=DEVICE)
    token = (cu[:-1, None] + row).clamp(max=state["q"].shape[0] - 1)
    q = state["q"][token].float().transpose(1, 2).reshape(n, hkv, hq // hkv * most, d)
    pages = state["block_table"].long().clamp(min=0)
    k = state["k_cache"][pages].float().view(n, sk, hkv, d).permute(0, 2, 3, 1)
    v = state["v_cache"][pages].float().view(n, sk, hkv, d).transpose(1, 2)
    keys = torch.arange(sk, device=DEVICE)[None, None, :]
    seen = _visible(row[None, :, None], keys, lens[:, None, None], (lens - new)[:, None, None],
                    case)
    s = (q @ k).mul_(d ** -0.5).view(n, hkv, hq // hkv, most, sk)
    p, lse = _softmax_plain(s, seen[:, None, None])
    o = (p.view(n, hkv, -1, sk) @ v).view(n, hq, most, d).transpose(1, 2)
    lse = lse.reshape(n, hq, most).transpose(1, 2)
    at = torch.arange(state["q"].shape[0], device=DEVICE)
    seq = (at[:, None] >= cu[None, 1:]).sum(1)
    at = at - cu[seq]
    return o[seq, at].to(torch.bfloat16), lse[seq, at].t().contiguous()


def _decode_window_plain(state):
    case = state["case"]
    hq, hkv, d, n = case["heads"], case["kv_heads"], case["dim"], case["seqs"]
    lens, page = state["seq_lens"].long()[:, None], case["page"]
    near = lens - case["window"] + torch.arange(case["window"], device=DEVICE)
    first = torch.arange(case["sinks"], device=DEVICE).expand(n, -1)
    token = torch.cat((first, near), 1)
    valid = torch.cat((first < lens - case["window"], near >= 0), 1)
    token = token.clamp(min=0).minimum(lens - 1)
    where = state["block_table"].long().gather(1, token // page)
    k, v = state["k_cache"][where, token % page], state["v_cache"][where, token % page]
    if case["cache"] == "e4m3":
        k = k.view(torch.float8_e4m3fn).float() * state["k_scale"][where][..., None]
        v = v.view(torch.float8_e4m3fn).float() * state["v_scale"][where][..., None]
    q = state["q"].float().view(n, hkv, hq // hkv, d)
    s = (q @ k.float().permute(0, 2, 3, 1)).mul_(d ** -0.5)
    p, lse = _softmax_plain(s, valid[:, None, None])
    o = p @ v.float().transpose(1, 2)
    return o.reshape(n, hq, d).to(torch.bfloat16), lse.reshape(n, hq)


# ------------------------------------------------------------------- the library's calls

def _rope_own(state):
    from exact_softmax_attention_fwd_b200 import attn_rope, attn_rope_bwd
    case = state["case"]
    hq, hkv = case["heads"], case["kv_heads"]
    if case["op"] == "rope":
        qkv = state["qkv"]
        q, k = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hkv].transpose(1, 2)
        return attn_rope(q, k, state["inv_freq"], state["positions"],
                         interleaved=case["interleaved"], mscale=state["factor"])
    to = state["dqkv"]
    attn_rope_bwd(state["dq"], state["dk"], state["inv_freq"], state["positions"],
                  interleaved=case["interleaved"], mscale=state["factor"],
                  q_out=to[:, :, :hq].transpose(1, 2), k_out=to[:, :, hq:hq + hkv].transpose(1, 2))
    return to


def _append_own(state):
    from exact_softmax_attention_fwd_b200 import attn_append_paged, attn_append_paged_fp8
    case, qkv = state["case"], state["qkv"]
    hq, hkv = case["heads"], case["kv_heads"]
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    kc, vc = state["k_cache"], state["v_cache"]
    how = {"cu_seqlens": state["cu"], "q": q, "inv_freq": state["inv_freq"],
           "interleaved": case["interleaved"], "mscale": state["factor"]}
    if case["cache"] == "bf16":
        return attn_append_paged(k, v, kc, vc, state["block_table"], state["seq_lens"], **how), kc, vc
    q = attn_append_paged_fp8(k, v, kc, vc, state["k_scale"], state["v_scale"],
                              state["block_table"], state["seq_lens"], **how)
    return q, kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)


def _window_own(state):
    from exact_softmax_attention_fwd_b200 import attn_fwd_window_sinks
    case = state["case"]
    return attn_fwd_window_sinks(state["q"], state["k"], state["v"], case["dim"] ** -0.5,
                                 case["window"], case["sinks"], k_lens=state["k_lens"])


def _window_bwd_own(state):
    from exact_softmax_attention_fwd_b200 import attn_bwd_window_sinks
    case = state["case"]
    return attn_bwd_window_sinks(state["q"], state["k"], state["v"], state["o"], state["lse"],
                                 state["d_o"], case["dim"] ** -0.5, case["window"], case["sinks"],
                                 k_lens=state["k_lens"])


def _paged_window_own(state):
    from exact_softmax_attention_fwd_b200 import attn_fwd_paged_window
    case = state["case"]
    return attn_fwd_paged_window(state["q"], state["k_cache"], state["v_cache"],
                                 state["block_table"], state["cu"], state["seq_lens"],
                                 state["max_new"], case["dim"] ** -0.5, case["window"],
                                 case["sinks"])


def _decode_window_own(state):
    from exact_softmax_attention_fwd_b200 import (attn_decode_paged_window,
                                                  attn_decode_paged_window_fp8)
    case = state["case"]
    rest = (state["block_table"], state["seq_lens"], case["dim"] ** -0.5, case["window"],
            case["sinks"])
    if case["cache"] == "bf16":
        return attn_decode_paged_window(state["q"], state["k_cache"], state["v_cache"], *rest)
    return attn_decode_paged_window_fp8(state["q"], state["k_cache"], state["v_cache"],
                                        state["k_scale"], state["v_scale"], *rest)


_PLAIN = {"rope": _rope_plain, "rope_bwd": _rope_plain, "append": _append_plain,
          "window": _window_plain, "window_bwd": _window_bwd_plain,
          "paged_window": _paged_window_plain, "decode_window": _decode_window_plain}
_OWN = {"rope": _rope_own, "rope_bwd": _rope_own, "append": _append_own, "window": _window_own,
        "window_bwd": _window_bwd_own, "paged_window": _paged_window_own,
        "decode_window": _decode_window_own}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# -------------------------------------------------------------------------- definitions

def _turned(x, angle, factor, rotary, interleaved):
    """x (float64) times exp(i angle) on each pair, as complex numbers."""
    pairs = x[..., :rotary]
    pairs = pairs.unflatten(-1, (-1, 2)) if interleaved else \
        pairs.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, factor), angle)
    z = torch.view_as_real(z)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, x[..., rotary:]), -1)


def _to_e4m3(x):
    """Nearest value of the 8-bit format (ties to the even one), in 64 bits."""
    _, exponent = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), exponent.sub(4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_row(q, k, v, p, window, sinks):
    """softmax attention of queries q [h, n, d] at places p [n] over keys k, v [m, d] (float64)."""
    j = torch.arange(k.shape[0], device=k.device)
    hidden = (j > p[:, None]) | ((j <= p[:, None] - window) & (j >= sinks))
    s = (q @ k.t()) / math.sqrt(q.shape[-1])
    lse = torch.logsumexp(s.masked_fill(hidden, -math.inf), -1)
    a = torch.exp(s - lse.masked_fill(lse == -math.inf, math.inf)[..., None])
    return a.masked_fill(hidden, 0.0) @ v, lse


def _gathered(state, b, name):
    """Keys or values of sequence b in order, float64."""
    pages = state["block_table"][b].long()
    pages = pages[pages >= 0]
    x = state[name + "_cache"][pages]
    if x.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn).double() * state[name + "_scale"][pages].double()[:, None, :, None]
    return x.double().flatten(0, 1)[:state["total"][b]]


def exact(case, seed):
    state = prepare(case, seed)
    op, hq, hkv = case["op"], case["heads"], case["kv_heads"]
    group = hq // hkv
    if op in ("rope", "rope_bwd"):
        sign = 1.0 if op == "rope" else -1.0
        angle = sign * state["positions"].double()[:, None] * state["inv_freq"]
        how = (angle, state["factor"], case["rotary"], case["interleaved"])
        if op == "rope":
            x = state["qkv"].double().transpose(1, 2)
            return [_turned(x[:, :hq], *how), _turned(x[:, hq:hq + hkv], *how)]
        dx = [_turned(state[n].double(), *how).transpose(1, 2) for n in ("dq", "dk")]
        return torch.cat(dx + [torch.zeros_like(dx[1])], 2)
    if op == "append":
        fp8 = case["cache"] == "e4m3"
        caches = [state[n].view(torch.float8_e4m3fn).double() if fp8 else state[n].double()
                  for n in ("k_cache", "v_cache")]
        x, done, at = state["qkv"].double(), [], 0
        for b, (n, total) in enumerate(zip(state["new"], state["total"])):
            t = torch.arange(total - n, total, device=DEVICE)
            angle = (t.double()[:, None] * state["inv_freq"])[:, None]
            qk = _turned(x[at:at + n, :hq + hkv], angle, state["factor"], case["rotary"],
                         case["interleaved"])
            done.append(qk[:, :hq])
            page = state["block_table"][b].long()[t // case["page"]]
            for cache, new, scale in ((caches[0], qk[:, hq:], "k_scale"),
                                      (caches[1], x[at:at + n, hq + hkv:], "v_scale")):
                if fp8:
                    new = _to_e4m3(new / state[scale][page].double()[..., None])
                cache[page, t % case["page"]] = new
            at += n
        return [torch.cat(done)] + caches
    if op in ("window", "window_bwd"):
        q, k, v = (state[n].double() for n in ("q", "k", "v"))
        out = [torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, device=DEVICE,
                                               dtype=torch.float64)]
        grads = [torch.zeros_like(x) for x in (q, k, v)]
        sq = case["seq_q"]
        for b, n in enumerate(_padded_lengths(case)):
            p = torch.arange(sq, device=DEVICE) + n - sq
            for h in range(hkv):
                hs = slice(h * group, (h + 1) * group)
                if op == "window":
                    out[0][b, hs], out[1][b, hs] = _exact_row(q[b, hs], k[b, h, :n], v[b, h, :n],
                                                              p, case["window"], case["sinks"])
                    continue
                with torch.enable_grad():
                    x = [t.clone().requires_grad_() for t in (q[b, hs], k[b, h, :n], v[b, h, :n])]
                    o, _ = _exact_row(*x, p, case["window"], case["sinks"])
                    g = torch.autograd.grad(o, x, state["d_o"][b, hs].double())
                grads[0][b, hs], grads[1][b, h, :n], grads[2][b, h, :n] = g
        return out if op == "window" else grads
    q = state["q"].double()
    if op == "decode_window":
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEVICE, dtype=torch.float64)
        starts, lse_rows = list(range(case["seqs"])), lse
    else:
        o = torch.empty_like(q)
        lse = torch.empty(hq, q.shape[0], device=DEVICE, dtype=torch.float64)
        starts, lse_rows = [sum(state["new"][:b]) for b in range(case["seqs"])], lse.t()
    for b, (n, total) in enumerate(zip(state["new"], state["total"])):
        k, v = _gathered(state, b, "k"), _gathered(state, b, "v")
        rows = slice(starts[b], starts[b] + n)
        p = torch.arange(total - n, total, device=DEVICE)
        for h in range(hkv):
            hs = slice(h * group, (h + 1) * group)
            got = _exact_row(q[rows, hs].transpose(0, 1), k[:, h], v[:, h], p, case["window"],
                             case["sinks"])
            o[rows, hs], lse_rows[rows, hs] = got[0].transpose(0, 1), got[1].t()
    return [o, lse]

"""Cases of the cache-side operators: appending tokens to a paged latent cache,
decoding a batch that shares a long prefix, keeping one int8 key per page, and
decoding over the pages that those keys select.

Each operator has a plain form (elementary torch operations) and the call that a
user makes of the library; ``own`` says which of the two ``run`` takes.
"""
import math

import torch

own = False

PAGE = 64
D_QK, D_V, D_ROPE = 576, 512, 64
ROPE_BASE = 1e4
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # appending: one token for each of a batch's sequences, bf16 rows (a decode step)
        {"name": "append_step_bf16", "op": "append", "fmt": "bf16", "n": 64, "blocks": 1024,
         "pad": 3, "norm": True, "strided": True},
        # a prompt chunk of ordinary length, FP8 rows, and the rows for its own attention
        {"name": "append_prompt_fp8", "op": "append", "fmt": "656", "n": 4096, "blocks": 1024,
         "pad": 0, "norm": True, "strided": True},
        # an odd number of tokens, 528-byte rows of an already normalised latent
        {"name": "append_odd_528", "op": "append", "fmt": "528", "n": 1023, "blocks": 512,
         "pad": 17, "norm": False, "strided": False},
        # several long prompts in one call, FP4 rows
        {"name": "append_bulk_fp4", "op": "append", "fmt": "288", "n": 32768, "blocks": 1024,
         "pad": 100, "norm": True, "strided": True},
        # a small batch behind a short system prompt: latency counts
        {"name": "prefix_small", "op": "prefix", "batch": 8, "s_q": 1, "h_q": 16, "prefix": 1000,
         "own_max": 100},
        # many short answers to one long document, 16 heads
        {"name": "prefix_h16", "op": "prefix", "batch": 128, "s_q": 1, "h_q": 16,
         "prefix": 32768, "own_max": 1024},
        # speculative pairs of tokens, 64 heads, odd lengths
        {"name": "prefix_pairs_h64", "op": "prefix", "batch": 23, "s_q": 2, "h_q": 64,
         "prefix": 8190, "own_max": 2001},
        # all 128 heads of a full batch
        {"name": "prefix_h128", "op": "prefix", "batch": 64, "s_q": 1, "h_q": 128,
         "prefix": 16384, "own_max": 512},
        # the pages that a decode step has just written to
        {"name": "page_keys_step", "op": "page_keys", "batch": 64, "len_max": 8192, "tail": 1},
        # every page of a batch of prompts
        {"name": "page_keys_prompt", "op": "page_keys", "batch": 16, "len_max": 32768,
         "tail": 512},
        # one request with a short context
        {"name": "page_sparse_small", "op": "page_sparse", "batch": 1, "s_q": 1, "h_q": 16,
         "len_max": 4096, "topk": 16},
        # a batch of long contexts, 128 heads
        {"name": "page_sparse_h128", "op": "page_sparse", "batch": 32, "s_q": 1, "h_q": 128,
         "len_max": 65536, "topk": 32},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "prefix", "prefix", "page_keys", "page_sparse"])
    if op == "append":
        n = _log_int(rng, 1, 32768)
        return {"op": op, "fmt": rng.choice(["bf16", "656", "528", "288"]), "n": n,
                "blocks": n // PAGE + rng.randint(2, 400), "pad": rng.randint(0, n // 8),
                "norm": rng.random() < 0.7, "strided": rng.random() < 0.7}
    if op == "prefix":
        h_q = rng.choice([1, 8, 16, 20, 32, 64, 96, 128])
        s_q = rng.choice([1, 1, 1, 2, 3])
        batch = max(1, min(_log_int(rng, 1, 200), 8000 // (h_q * s_q)))
        return {"op": op, "batch": batch, "s_q": s_q, "h_q": h_q,
                "prefix": _log_int(rng, 64, 16384), "own_max": _log_int(rng, 1, 1024)}
    if op == "page_keys":
        length = _log_int(rng, 64, 32768)
        return {"op": op, "batch": _log_int(rng, 1, 16), "len_max": length,
                "tail": _log_int(rng, 1, 512)}
    return {"op": op, "batch": _log_int(rng, 1, 32), "s_q": rng.choice([1, 1, 2]),
            "h_q": rng.choice([8, 16, 32, 64, 128]), "len_max": _log_int(rng, 200, 32768),
            "topk": _log_int(rng, 1, 32)}


# ------------------------------------------------------------------ inputs

def _row_bytes(fmt):
    return 2 * D_QK if fmt == "bf16" else int(fmt)


def _width(fmt):
    return D_QK if fmt in ("bf16", "656") else D_V


def _table(lengths, total, gen, device):
    """`total` blocks dealt out to the sequences at random; -1 behind a sequence's last page."""
    pages = [-(-n // PAGE) for n in lengths]
    perm = torch.randperm(total, generator=gen, device=device).to(torch.int32)
    width = max(1, max(pages))
    count = torch.tensor(pages, device=device)
    at = torch.arange(width, device=device)[None, :]
    first = (torch.cumsum(count, 0) - count)[:, None]
    table = torch.where(at < count[:, None], perm[(first + at).clamp(max=total - 1)],
                        torch.full((), -1, dtype=torch.int32, device=device))
    return table.contiguous()


def _lengths(n, low, high, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(low, high + 1, (n,), generator=g).tolist()
    x[seed % n] = high
    return x


def _bf16(shape, gen, device):
    return torch.randn(shape, generator=gen, device=device, dtype=torch.float32).to(torch.bfloat16)


def _cache(blocks, gen, device):
    out = torch.empty((blocks, PAGE, 1, D_QK), dtype=torch.bfloat16, device=device)
    for i in range(0, blocks, 4096):
        out[i:i + 4096] = torch.randn(out[i:i + 4096].shape, generator=gen, device=device,
                                      dtype=torch.float32)
    return out


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    return {"append": _prepare_append, "prefix": _prepare_prefix, "page_keys": _prepare_page_keys,
            "page_sparse": _prepare_page_sparse}[case["op"]](case, seed, gen, device)


def _prepare_append(case, seed, gen, device):
    n, d = case["n"], _width(case["fmt"])
    # the latent is a column range of the down projection's output, or a tensor of its own
    wide = torch.randn((n, d + 512 if case["strided"] else d), generator=gen, device=device)
    wide = (wide * torch.exp(0.5 * torch.randn(wide.shape[1], generator=gen, device=device))).to(
        torch.bfloat16)
    kv = wide[:, 512:] if case["strided"] else wide
    gain = 1 + 0.1 * torch.randn(D_V, generator=gen, device=device) if case["norm"] else None
    # tokens in order over shuffled blocks, from the middle of one; the last block stays free
    order = torch.randperm(case["blocks"] - 1, generator=gen, device=device)
    t = torch.arange(n, device=device) + seed % PAGE
    slots = (order[(t // PAGE) % order.numel()] * PAGE + t % PAGE).to(torch.int32)
    if case["pad"]:
        slots[n - case["pad"]:] = -1
    positions = (t + (seed * 977) % 100000).to(torch.int32)
    if case["fmt"] == "bf16":
        cache = _cache(case["blocks"], gen, device)
    else:  # valid codes and scales everywhere
        cache = torch.randint(40, 72, (case["blocks"], PAGE, _row_bytes(case["fmt"])),
                              generator=gen, device=device, dtype=torch.uint8)
        if case["fmt"] == "656":
            some = torch.rand((case["blocks"], PAGE, 4), generator=gen, device=device)
            cache[..., D_V:D_V + 16] = (0.005 + 0.01 * some).view(torch.uint8)
            cache[..., D_V + 16:] = _bf16((case["blocks"], PAGE, D_ROPE), gen, device).view(
                torch.uint8)
    rows = None
    if case["fmt"] != "bf16":
        rows = torch.zeros((n, d), dtype=torch.bfloat16, device=device)
    return {"case": case, "kv": kv, "gain": gain, "slots": slots, "positions": positions,
            "cache": cache, "rows": rows}


def _prepare_prefix(case, seed, gen, device):
    b, rows = case["batch"], case["s_q"] * case["h_q"]
    lengths = _lengths(b, min(case["s_q"], case["own_max"]), case["own_max"], seed)
    blocks = -(-case["prefix"] // PAGE) + b * -(-case["own_max"] // PAGE) + 3
    table = _table([case["prefix"]] + lengths, blocks, gen, device)
    n_prefix, n_own = -(-case["prefix"] // PAGE), max(1, -(-max(lengths) // PAGE))
    state = {"case": case, "q": _bf16((b, case["s_q"], case["h_q"], D_QK), gen, device),
             "cache": _cache(blocks, gen, device), "prefix_table": table[0, :n_prefix].contiguous(),
             "table": table[1:, :n_own].contiguous(),
             "lengths": torch.tensor(lengths, dtype=torch.int32, device=device)}
    if own:  # the plan of a decode step, shared by its layers
        from mla_paged_kv_03_b200 import binding as B
        state["plan"] = B.mla_shared_prefix_get_metadata(state["lengths"], case["prefix"], rows)
    return state


def _prepare_page_keys(case, seed, gen, device):
    lengths = _lengths(case["batch"], max(1, case["len_max"] // 2), case["len_max"], seed)
    blocks = case["batch"] * -(-case["len_max"] // PAGE) + 3
    table = _table(lengths, blocks, gen, device)
    used = torch.zeros(blocks, dtype=torch.int32, device=device)
    used[table.clamp(min=0).long().reshape(-1)] = 1
    return {"case": case, "cache": _cache(blocks, gen, device), "table": table,
            "lengths": torch.tensor(lengths, dtype=torch.int32, device=device),
            "spare": torch.argmin(used),  # a block that no sequence owns
            "keys": torch.zeros((blocks, D_QK), dtype=torch.int8, device=device),
            "scales": torch.ones((blocks,), device=device)}


def _prepare_page_sparse(case, seed, gen, device):
    state = _prepare_page_keys(case, seed, gen, device)
    # keys drawn like the mean of a page's rows, without the pass over the whole cache
    blocks = state["keys"].shape[0]
    mean = torch.randn((blocks, D_QK), generator=gen, device=device) / 8
    amax = mean.abs().amax(1)
    state["scales"] = amax / 127
    state["keys"] = torch.round(mean / state["scales"][:, None]).to(torch.int8)
    state["q"] = _bf16((case["batch"], case["s_q"], case["h_q"], D_QK), gen, device)
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    return {"append": _append, "prefix": _prefix, "page_keys": _page_keys,
            "page_sparse": _page_sparse}[state["case"]["op"]](state)


def _append_outputs(state):
    fmt, cache = state["case"]["fmt"], state["cache"]
    if fmt == "bf16":
        return {"cache": cache}
    if fmt == "288":  # codes are compared as the rows that they stand for
        return {"rows": state["rows"], "scales": cache[..., 256:].view(torch.float8_e4m3fn)}
    out = {"rows": state["rows"], "codes": cache[..., :512].view(torch.float8_e4m3fn)}
    if fmt == "528":
        return out | {"scales": cache[..., 512:].view(torch.float8_e8m0fnu)}
    return out | {"scales": cache[..., 512:528].view(torch.float32),
                  "rope": cache[..., 528:].view(torch.bfloat16)}


def _append(state):
    if own:
        from mla_paged_kv_03_b200 import binding as B
        B.mla_cache_append(state["kv"], state["slots"], state["cache"],
                           positions=state["positions"], norm_gain=state["gain"], eps=EPS,
                           rope_base=ROPE_BASE, rows=state["rows"])
        return _append_outputs(state)
    fmt = state["case"]["fmt"]
    x = state["kv"].float()
    n, d = x.shape
    if state["gain"] is not None:
        z = x[:, :D_V]
        z = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * state["gain"]
        x = torch.cat([z, x[:, D_V:]], 1)
    # angles of far positions in 64 bits
    freq = ROPE_BASE ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64, device=x.device) / D_ROPE)
    angle = state["positions"].double()[:, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = x[:, d - D_ROPE::2], x[:, d - D_ROPE + 1::2]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], 2).reshape(n, D_ROPE)
    x = torch.cat([x[:, :d - D_ROPE], turned], 1)
    live = state["slots"] >= 0
    cache = state["cache"]
    flat = cache.view(-1, cache.shape[-1])
    if fmt == "bf16":
        row, stands = x.to(torch.bfloat16), None
    elif fmt == "656":
        g = x[:, :D_V].reshape(n, 4, 128)
        amax = g.abs().amax(2, keepdim=True)
        scale = torch.where(amax > 0, amax / 448, 1.0)
        code = (g / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        rope = x[:, D_V:].to(torch.bfloat16)
        row = torch.cat([code.view(torch.uint8).reshape(n, D_V),
                         scale.reshape(n, 4).view(torch.uint8), rope.view(torch.uint8)], 1)
        stands = torch.cat([(code.float() * scale).reshape(n, D_V).to(torch.bfloat16), rope], 1)
    elif fmt == "528":
        g = x.reshape(n, 16, 32)
        amax = g.abs().amax(2, keepdim=True)
        m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 2^9
        e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), 0).clamp(-127, 127)
        scale = torch.ldexp(torch.ones_like(amax), e)
        code = (g / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        row = torch.cat([code.view(torch.uint8).reshape(n, D_V),
                         (e + 127).to(torch.uint8).reshape(n, 16)], 1)
        stands = (code.float() * scale).reshape(n, D_V).to(torch.bfloat16)
    else:
        g = x.reshape(n, 32, 16)
        amax = g.abs().amax(2, keepdim=True)
        scale8 = torch.where(amax > 0, amax / 6, 1.0).clamp(max=448).to(torch.float8_e4m3fn)
        scale8 = torch.where(scale8.float() > 0, scale8.float(), 1.0).to(torch.float8_e4m3fn)
        scale = scale8.float()
        v = g / scale
        # nearest magnitude: between 0, .5, .. 6 the midpoints, ties to the even code
        mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
        up = torch.tensor([False, True, False, True, False, True, False], device=x.device)
        w = v.abs().unsqueeze(-1)
        code = ((w > mid) | ((w == mid) & up)).sum(-1)
        value = torch.tensor(E2M1, device=x.device)[code] * torch.where(v < 0, -1.0, 1.0)
        code = (code + 8 * (v < 0)).to(torch.uint8).reshape(n, 256, 2)
        row = torch.cat([code[..., 0] | (code[..., 1] << 4),
                         scale8.view(torch.uint8).reshape(n, 32)], 1)
        stands = (value * scale).reshape(n, D_V).to(torch.bfloat16)
    # a token without a slot rewrites the last, unused row with what it holds
    last = flat.shape[0] - 1
    at = torch.where(live, state["slots"], last).long()
    flat[at] = torch.where(live[:, None], row, flat[last])
    if stands is not None:
        state["rows"].copy_(torch.where(live[:, None], stands, state["rows"]))
    return _append_outputs(state)


def _rows_of(cache, table, tokens):
    """Cache rows of the first `tokens` tokens behind each table row: [..., tokens, 576]."""
    t = torch.arange(tokens, device=cache.device)
    slot = table.clamp(min=0).long()[..., t // PAGE] * PAGE + t % PAGE
    return cache.view(-1, D_QK)[slot]


def _prefix(state):
    case = state["case"]
    if own:
        from mla_paged_kv_03_b200 import binding as B
        metadata, splits, parts = state["plan"]
        out, lse = B.mla_shared_prefix_decode_fwd(
            state["q"], state["cache"], state["prefix_table"], case["prefix"], state["table"],
            state["lengths"], metadata, splits, parts)
        return {"out": out, "lse": lse}
    b, s, h, p = case["batch"], case["s_q"], case["h_q"], case["prefix"]
    q = state["q"].float().view(b, s * h, D_QK) / math.sqrt(D_QK)
    kp = _rows_of(state["cache"], state["prefix_table"], p).float()
    ko = _rows_of(state["cache"], state["table"], state["table"].shape[1] * PAGE).float()
    x = torch.cat([(q.reshape(-1, D_QK) @ kp.T).view(b, s * h, p), q @ ko.transpose(1, 2)], 2)
    # query i of s sees prefix + length - s + 1 + i tokens
    i = torch.arange(s, device=q.device).repeat_interleave(h)
    sees = state["lengths"][:, None] - s + 1 + i
    t = torch.arange(-p, ko.shape[1], device=q.device)
    x.masked_fill_(t >= sees[:, :, None], -math.inf)
    top = x.amax(2, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(2, keepdim=True)
    e /= total
    o = (e[..., :p].reshape(-1, p) @ kp[:, :D_V]).view(b, s * h, D_V) + e[..., p:] @ ko[..., :D_V]
    return {"out": o.to(torch.bfloat16).view(b, s, h, D_V),
            "lse": (top + torch.log(total)).view(b, s, h)}


def _page_keys(state):
    case = state["case"]
    if own:
        from mla_paged_kv_03_b200 import binding as B
        B.mla_page_keys_update(state["cache"], state["table"], state["lengths"], state["keys"],
                               state["scales"], tail_pages=case["tail"])
        return {"keys": state["keys"], "scales": state["scales"]}
    table, lengths = state["table"], state["lengths"].long()
    n = (lengths + PAGE - 1) // PAGE
    k = min(case["tail"], table.shape[1])
    page = n[:, None] - k + torch.arange(k, device=table.device)
    live = (page >= 0).reshape(-1)
    page = page.clamp(min=0)
    block = torch.gather(table, 1, page.clamp(max=table.shape[1] - 1)).long().reshape(-1)
    block = block.clamp(min=0)
    count = (lengths[:, None] - page * PAGE).clamp(1, PAGE).reshape(-1)
    x = state["cache"][block, :, 0]
    mask = torch.arange(PAGE, device=table.device)[None, :] < count[:, None]
    # sums in 64 bits: a mean next to a rounding border decides a code
    total = torch.where(mask[..., None], x.double(), 0.0).sum(1)
    mean = (total / count[:, None]).float()
    amax = mean.abs().amax(1)
    scale = torch.where(amax > 0, amax / 127, 1.0)
    code = torch.round(mean / scale[:, None]).to(torch.int8)
    # a place without a page rewrites the block that no sequence owns
    spare = state["spare"]
    at = torch.where(live, block, spare)
    state["keys"][at] = torch.where(live[:, None], code, state["keys"][spare])
    state["scales"][at] = torch.where(live, scale, state["scales"][spare])
    return {"keys": state["keys"], "scales": state["scales"]}


def _page_sparse(state):
    case = state["case"]
    if own:
        from mla_paged_kv_03_b200 import binding as B
        out, lse, pages = B.mla_page_sparse_decode(state["q"], state["cache"], state["keys"],
                                                   state["scales"], state["table"],
                                                   state["lengths"], case["topk"])
        return {"out": out, "lse": lse, "pages": pages}
    b, s, h, k = case["batch"], case["s_q"], case["h_q"], case["topk"]
    table, device = state["table"], state["table"].device
    width = table.shape[1]
    q = state["q"].float()
    amax = q.abs().amax(3, keepdim=True)
    q_scale = torch.where(amax > 0, amax / 127, 1.0)
    code = torch.round(q / q_scale)
    block = table.clamp(min=0).long()
    # whole numbers below 2^24: these products and sums are exact in 32 bits
    dot = code.view(b, s * h, D_QK) @ state["keys"][block].float().transpose(1, 2)
    score = (dot.view(b, s, h, width) * q_scale).amax(2) * state["scales"][block][:, None, :]
    sees = (state["lengths"][:, None] - s + 1 + torch.arange(s, device=device)).clamp(min=0)
    last = (sees + PAGE - 1) // PAGE - 1  # the page that ends a query's tokens is always taken
    page = torch.arange(width, device=device)
    score = torch.where(page < last[..., None], score, -math.inf)
    score = torch.where(page == last[..., None], math.inf, score)
    order = torch.sort(score, dim=2, descending=True, stable=True)[1][..., :k]
    if order.shape[2] < k:
        order = torch.nn.functional.pad(order, (0, k - order.shape[2]), value=width)
    pages = torch.sort(torch.where(order <= last[..., None], order, width), dim=2)[0]
    pages = torch.where(pages < width, pages, -1)
    # tokens of the pages, and which of them a query sees
    at = torch.gather(block[:, None].expand(b, s, width), 2, pages.clamp(min=0))
    t = torch.arange(PAGE, device=device)
    kv = state["cache"].view(-1, D_QK)[(at[..., None] * PAGE + t).reshape(b * s, k * PAGE)].float()
    seen = (pages[..., None] >= 0) & (pages[..., None] * PAGE + t < sees[..., None, None])
    x = (q.view(b * s, h, D_QK) / math.sqrt(D_QK)) @ kv.transpose(1, 2)
    x.masked_fill_(~seen.reshape(b * s, 1, k * PAGE), -math.inf)
    top = x.amax(2, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(2, keepdim=True)
    o = (e / torch.where(total > 0, total, 1.0)) @ kv[..., :D_V]
    return {"out": o.to(torch.bfloat16).view(b, s, h, D_V),
            "lse": (top + torch.log(total)).view(b, s, h), "pages": pages.to(torch.int32)}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "append":
        n, d = case["n"], _width(case["fmt"])
        live = n - case["pad"]
        rows = 0 if case["fmt"] == "bf16" else 2 * d
        return {"bytes": live * (2 * d + 4 + _row_bytes(case["fmt"]) + rows) + 4 * n
                + (4 * D_V if case["norm"] else 0), "flops": live * d * 6}
    if case["op"] == "prefix":
        rows = case["batch"] * case["s_q"] * case["h_q"]
        mean = (min(case["s_q"], case["own_max"]) + case["own_max"]) / 2
        tokens = case["prefix"] + case["batch"] * mean
        return {"bytes": tokens * 2 * D_QK + rows * (2 * D_QK + 2 * D_V + 4),
                "flops": 2 * rows * (case["prefix"] + mean) * (D_QK + D_V)}
    low = max(1, case["len_max"] // 2)
    pages = -(-(low + case["len_max"]) // (2 * PAGE))
    if case["op"] == "page_keys":
        pages = case["batch"] * min(case["tail"], pages)
        return {"bytes": pages * (PAGE * 2 * D_QK + D_QK + 4), "flops": pages * PAGE * D_QK}
    pairs = case["batch"] * case["s_q"]
    taken = min(case["topk"], pages)
    return {"bytes": case["batch"] * pages * (D_QK + 8) + pairs * taken * PAGE * 2 * D_QK
            + pairs * case["h_q"] * (2 * D_QK + 2 * D_V + 4) + pairs * 4 * case["topk"],
            "flops": 2 * pairs * case["h_q"] * (pages * D_QK + taken * PAGE * (D_QK + D_V))}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"append": _exact_append, "prefix": _exact_prefix, "page_keys": _exact_page_keys,
            "page_sparse": _exact_page_sparse}[case["op"]](state)


def _nearest_e4m3(v):
    """v rounded to the nearest E4M3 value (3 fraction bits, least exponent -6, at most 448)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_append(state):
    fmt, slots = state["case"]["fmt"], state["slots"].long()
    y = state["kv"].double()
    n, d = y.shape
    if state["gain"] is not None:
        rms = torch.sqrt(y[:, :D_V].pow(2).sum(1) / D_V + EPS)
        y[:, :D_V] = y[:, :D_V] / rms[:, None] * state["gain"].double()
    pair = torch.view_as_complex(y[:, d - D_ROPE:].reshape(n, D_ROPE // 2, 2).contiguous())
    k = torch.arange(D_ROPE // 2, device=y.device, dtype=torch.float64)
    angle = state["positions"].double()[:, None] * torch.pow(ROPE_BASE, -2 * k / D_ROPE)
    pair = pair * torch.polar(torch.ones_like(angle), angle)
    y[:, d - D_ROPE:] = torch.view_as_real(pair).reshape(n, D_ROPE)
    keep = torch.nonzero(slots >= 0)[:, 0]
    slots, y = slots[keep], y[keep]
    m = keep.numel()
    old = {k: v.double() for k, v in _append_outputs(state).items()}
    new = {}
    if fmt == "bf16":
        new["cache"] = y
    elif fmt in ("656", "528"):
        size = 128 if fmt == "656" else 32
        g = y[:, :D_V].reshape(m, D_V // size, size)
        amax = g.abs().amax(2, keepdim=True)
        scale = amax / 448
        if fmt == "528":
            e = torch.ceil(torch.log2(scale))  # the least e with amax <= 448 2^e, mended below
            e = torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e)
            scale = torch.exp2(torch.where(amax > 448 * torch.exp2(e), e + 1, e))
        code = _nearest_e4m3(g / scale)
        new = {"codes": code.reshape(m, D_V), "scales": scale.reshape(m, -1),
               "rows": (code * scale).reshape(m, D_V)}
        if fmt == "656":
            new["rope"] = y[:, D_V:]
            new["rows"] = torch.cat([new["rows"], new["rope"]], 1)
    else:
        g = y.reshape(m, 32, 16)
        scale = _nearest_e4m3(g.abs().amax(2, keepdim=True) / 6)
        # E2M1: steps of 1/2 below 2, of 1 below 4, of 2 up to 6; halves go to the even step
        v = g / scale
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
        near = (torch.round(v / step) * step).clamp(-6, 6)
        new = {"scales": scale.reshape(m, 32), "rows": (near * scale).reshape(m, D_V)}
    for name, value in new.items():
        flat = old[name].view(-1, old[name].shape[-1])
        flat[keep if name == "rows" else slots] = value
    return old


def _softmax_rows(x, v):
    """(softmax(x) v, log-sum-exp) in 64 bits, one group at a time."""
    lse = torch.logsumexp(x, -1, keepdim=True)
    return torch.exp(x - lse) @ v, lse[..., 0]


def _exact_prefix(state):
    case = state["case"]
    b, s, h, p = case["batch"], case["s_q"], case["h_q"], case["prefix"]
    kp = _rows_of(state["cache"], state["prefix_table"], p).double()
    out, lse = [], []
    for j, n in enumerate(state["lengths"].tolist()):
        k = torch.cat([kp, _rows_of(state["cache"], state["table"][j], n).double()])
        x = state["q"][j].double() @ k.T / math.sqrt(D_QK)
        for i in range(s):
            x[i, :, p + n - s + 1 + i:] = -math.inf
        o, l = _softmax_rows(x, k[:, :D_V])
        out.append(o)
        lse.append(l)
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


def _exact_page_keys(state):
    # codes are whole numbers and have no unrounded value; a page's scale has
    scales = state["scales"].double()
    lengths, tail = state["lengths"].tolist(), state["case"]["tail"]
    for j, n in enumerate(lengths):
        total = -(-n // PAGE)
        for page in range(max(0, total - tail), total):
            block = int(state["table"][j, page])
            x = state["cache"][block, :min(PAGE, n - page * PAGE), 0].double()
            scales[block] = x.mean(0).abs().amax() / 127
    return {"scales": scales}


def _exact_page_sparse(state):
    case = state["case"]
    s, k = case["s_q"], case["topk"]
    out, lse, taken = [], [], []
    for j, n in enumerate(state["lengths"].tolist()):
        for i in range(s):
            sees = n - s + 1 + i
            last = -(-sees // PAGE) - 1
            q = state["q"][j, i].double()
            # the int8 query codes are part of the definition (32-bit quotients, to the nearest)
            amax = state["q"][j, i].float().abs().amax(1, keepdim=True)
            unit = torch.where(amax > 0, amax / 127, 1.0)
            code = torch.round(state["q"][j, i].float() / unit).double()
            block = state["table"][j, :last + 1].long()
            dot = code @ state["keys"][block[:last]].double().T
            score = (dot * unit.double()).amax(0) * state["scales"][block[:last]].double()
            best = torch.sort(score, descending=True, stable=True)[1][:k - 1]
            page = torch.sort(torch.cat([best, best.new_full((1,), last)]))[0]
            t = (page[:, None] * PAGE + torch.arange(PAGE, device=q.device)).reshape(-1)
            t = t[t < sees]
            rows = state["cache"].view(-1, D_QK)[block[t // PAGE] * PAGE + t % PAGE].double()
            o, l = _softmax_rows(q @ rows.T / math.sqrt(D_QK), rows[:, :D_V])
            out.append(o)
            lse.append(l)
            taken.append(torch.nn.functional.pad(page, (0, k - page.numel()), value=-1))
    shape = state["q"].shape[:3]
    return {"out": torch.stack(out).view(*shape, D_V), "lse": torch.stack(lse).view(shape),
            "pages": torch.stack(taken).view(shape[0], s, k).to(torch.int32)}

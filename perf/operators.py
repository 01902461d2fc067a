"""The operators of a decoding step around the selections: attention over a
paged key-value cache, writing and reading that cache, and beam search.

Where `own` is false, run() computes them from elementary torch operations in
32 bits (64 where candidates of different rows are compared); where it is true
it makes the library's calls on the same state.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _attend(name, batch, heads, kv_heads, d, page, longest, cache, listed=0):
    case = dict(op="attend", batch=batch, heads=heads, kv_heads=kv_heads, d=d, page=page, longest=longest,
                cache=cache, listed=listed)
    return dict(case, name=name) if name else case


def _write(name, tokens, kv_heads, d, page, cache, prefill):
    case = dict(op="write", tokens=tokens, kv_heads=kv_heads, d=d, page=page, cache=cache, prefill=prefill)
    return dict(case, name=name) if name else case


def _read(name, batch, kv_heads, d, page, longest, cache):
    case = dict(op="read", batch=batch, kv_heads=kv_heads, d=d, page=page, longest=longest, cache=cache)
    return dict(case, name=name) if name else case


def _beam(name, batch, beams, vocab, k, dtype):
    case = dict(op="beam", batch=batch, beams=beams, vocab=vocab, k=k, dtype=dtype)
    return dict(case, name=name) if name else case


def _reorder(name, tensors, batch, beams, k, width, dtype):
    case = dict(op="reorder", tensors=tensors, batch=batch, beams=beams, k=k, width=width, dtype=dtype)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one user's chat turn: a single short sequence, where the call's latency is what counts
        _attend("attend one short", 1, 32, 8, 128, 16, 1001, "bf16"),
        # a ragged serving batch with shared key-value heads, up to the selector's 32768 keys
        _attend("attend ragged batch", 16, 32, 8, 128, 16, 32768, "bf16"),
        # long contexts on a quantised cache
        _attend("attend long e4m3", 4, 32, 8, 128, 64, 131072, "e4m3"),
        # sparse attention: 512 selected keys for each of 16 x 32 heads, as the decode selector returns them
        _attend("attend selected", 16, 32, 32, 128, 64, 8192, "bf16", 512),
        # the new tokens of one decoding step of 64 sequences, quantised into scattered slots
        _write("write step e4m3", 64, 8, 128, 16, "e4m3", False),
        # a prompt's tokens quantised into their pages, the padding of a fixed-size batch left out
        _write("write prompt e4m3", 49999, 8, 128, 16, "e4m3", True),
        # one sequence's keys laid out for the selector
        _read("read one bf16", 1, 8, 128, 16, 2047, "bf16"),
        # a ragged batch of quantised keys laid out for the selector
        _read("read batch e4m3", 16, 8, 128, 64, 32768, "e4m3"),
        # one sentence's beam step on the sampling workload's vocabulary
        _beam("beam one sentence", 1, 4, 131072, 8, "f32"),
        # a batch of sentences, bf16 logits with many equal values, a vocabulary that is no multiple of anything
        _beam("beam batch bf16", 32, 8, 128255, 16, "bf16"),
        # the small per-beam state: token histories and page tables of a few sentences
        _reorder("reorder tables", 2, 4, 4, 4, 257, "i32"),
        # per-beam key and value states of a few layers
        _reorder("reorder states", 8, 4, 4, 4, 8 * 2048 * 128, "bf16"),
    ]


_MOST_ATTEND = 1_050_000_000   # cache elements (K and V) that one drawn call reads
_MOST_COPY = 130_000_000       # elements that one drawn write or read touches
_MOST_LOGITS = 33_000_000
_MOST_STATE = 130_000_000


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "read", "beam", "beam", "reorder"])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([1, 16, 16, 32, 64, 24, 128])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "attend":
        kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
        group = rng.choice([1, 2, 4, 6, 7, 8, 16, 20])
        batch = _log_int(rng, 1, 96)
        longest = _log_int(rng, 1, 131072)
        longest = min(longest, max(1, _MOST_ATTEND // (2 * batch * kv_heads * d)))
        picked = 0
        if rng.random() < 0.3:
            picked = min(_log_int(rng, 1, 2048), longest)
        return _attend("", batch, kv_heads * group, kv_heads, d, page, longest, cache, picked)
    if op == "write":
        kv_heads = rng.choice([1, 2, 4, 7, 8, 16])
        tokens = min(_log_int(rng, 1, 50000), max(1, _MOST_COPY // (2 * kv_heads * d)))
        return _write("", tokens, kv_heads, d, page, cache, rng.random() < 0.5)
    if op == "read":
        kv_heads = rng.choice([1, 2, 4, 7, 8, 16])
        batch = _log_int(rng, 1, 64)
        longest = min(_log_int(rng, 1, 40000), max(1, _MOST_COPY // (batch * kv_heads * d)))
        return _read("", batch, kv_heads, d, page, longest, cache)
    if op == "beam":
        batch = _log_int(rng, 1, 64)
        beams = rng.choice([1, 2, 3, 4, 5, 8, 12])
        vocab = min(_log_int(rng, 30, 262144), max(30, _MOST_LOGITS // (batch * beams)))
        k = rng.choice([beams, 2 * beams])
        return _beam("", batch, beams, vocab, k, rng.choice(["f32", "bf16"]))
    batch = _log_int(rng, 1, 32)
    beams = rng.choice([1, 2, 4, 5, 8])
    k = rng.choice([beams, 2 * beams])
    tensors = rng.choice([1, 2, 3, 8, 24])
    width = min(_log_int(rng, 1, 4000000), max(1, _MOST_STATE // (tensors * batch * max(beams, k))))
    return _reorder("", tensors, batch, beams, k, width, rng.choice(["i32", "bf16"]))


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Sequence lengths of a batch: the longest first, the others spread below it."""
    return [max(1, int(case["longest"] * (1.0 - 0.9375 * ((i * 0.6180339887) % 1.0)))) for i in range(case["batch"])]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pages(case, g):
    """A block table whose sequences own scattered pages, and the number of pages (a few stay unused)."""
    width = -(-case["longest"] // case["page"])
    need = case["batch"] * width
    pages = need + 3
    order = torch.randperm(pages, generator=g, device="cuda")[:need]
    return order.to(torch.int32).view(case["batch"], width), pages


def _cache(case, pages, g):
    """A filled cache [pages, kv_heads, page, d], and its scales [pages, kv_heads, page] if it is quantised."""
    shape = (pages, case["kv_heads"], case["page"], case["d"])
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    if case["cache"] == "bf16":
        return x, None
    # rows as the writer leaves them: unit normal values, the largest of a row near 448 times its power of two
    code = x.mul_(112.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    scale = torch.exp2(torch.randint(-8, -5, shape[:3], generator=g, device="cuda").float())
    return code, scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    if op in ("attend", "read"):
        s["table"], pages = _pages(case, g)
        s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        s["k_cache"], s["k_scale"] = _cache(case, pages, g)
        if op == "read":
            return s
        s["v_cache"], s["v_scale"] = _cache(case, pages, g)
        s["q"] = torch.randn(case["batch"], case["heads"], case["d"], generator=g, device="cuda").bfloat16()
        s["positions"] = None
        if case["listed"]:
            # every head's own selection: distinct positions below the sequence's length in no order, empty
            # slots behind them where the sequence is shorter than the list
            c, n = case["listed"], case["longest"]
            u = torch.rand(case["batch"], case["heads"], n, generator=g, device="cuda")
            u[(torch.arange(n, device="cuda") >= s["lens"].view(-1, 1, 1)).expand_as(u)] = 2.0
            best = torch.topk(u, c, dim=2, largest=False, sorted=False)
            s["positions"] = torch.where(best.values < 2.0, best.indices, -1).to(torch.int32)
        return s
    if op == "write":
        t, h, d, p = case["tokens"], case["kv_heads"], case["d"], case["page"]
        # keys and values are slices of one projection's output
        kv = torch.randn(t, 2 * h * d, generator=g, device="cuda").bfloat16()
        s["k"], s["v"] = kv[:, : h * d].view(t, h, d), kv[:, h * d:].view(t, h, d)
        pages = -(-t // p) + 2
        if case["prefill"]:
            at = torch.arange(t, device="cuda")
            slots = torch.randperm(pages, generator=g, device="cuda")[at // p] * p + at % p
            slots[t - t // 32:] = -1
        else:
            slots = torch.randperm(pages * p, generator=g, device="cuda")[:t].clone()
        s["slots"] = slots
        kind = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        for n in ("k", "v"):
            s[n + "_cache"] = torch.zeros(pages, h, p, d, dtype=torch.bfloat16, device="cuda").to(kind)
            s[n + "_scale"] = None if case["cache"] == "bf16" else torch.ones(pages, h, p, device="cuda")
        return s
    if op == "beam":
        shape = (case["batch"], case["beams"], case["vocab"])
        x = torch.randn(shape, generator=g, device="cuda")
        # a few tokens stand out, as in a model's logits
        x.mul_(1.5).sub_(torch.rand(case["vocab"], generator=g, device="cuda").mul_(case["vocab"]).add_(1.0).log_())
        s["logits"] = x if case["dtype"] == "f32" else x.bfloat16()
        s["scores"] = torch.rand(shape[:2], generator=g, device="cuda").mul_(-8.0)
        if case["beams"] > 2:
            s["scores"][::3, -1] = -math.inf  # a beam that has ended
        return s
    shape = (case["batch"], case["beams"], case["width"])
    if case["dtype"] == "i32":
        s["states"] = [torch.randint(0, 1 << 30, shape, generator=g, device="cuda", dtype=torch.int32)
                       for _ in range(case["tensors"])]
    else:
        s["states"] = [torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
                       for _ in range(case["tensors"])]
    s["parents"] = torch.randint(0, case["beams"], (case["batch"], case["k"]), generator=g, device="cuda",
                                 dtype=torch.int32)
    return s


# ------------------------------------------------------------------ plain forms
def _rows(cache, scale, page_ids, heads, offsets):
    x = cache[page_ids, heads, offsets].float()
    return x if scale is None else x * scale[page_ids, heads, offsets].unsqueeze(-1)


def _plain_attend(s):
    q, table, lens, pos = s["q"], s["table"].long(), s["lens"].long(), s["positions"]
    batch, heads, d = q.shape
    kv_heads, page = s["k_cache"].shape[1:3]
    if pos is None:
        at = torch.arange(table.shape[1] * page, device=q.device).expand(batch, kv_heads, -1)
        at = at[:, :, : s["case"]["longest"]]
    else:
        at = pos.long()
    live = (at >= 0) & (at < lens.view(-1, 1, 1))
    at = torch.where(live, at, 0)
    lists = at.shape[1]
    b = torch.arange(batch, device=q.device).view(-1, 1, 1)
    h = (torch.arange(lists, device=q.device) * kv_heads // lists).view(1, -1, 1)
    ids = table[b, at // page]
    k = _rows(s["k_cache"], s["k_scale"], ids, h, at % page)
    t = torch.matmul(q.float().view(batch, lists, heads // lists, d), k.transpose(2, 3)) * d ** -0.5
    del k
    t = t.masked_fill(~live.unsqueeze(2), -math.inf)
    top = t.amax(3, keepdim=True)
    p = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    v = _rows(s["v_cache"], s["v_scale"], ids, h, at % page)
    v.mul_(live.unsqueeze(3))
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = torch.log(total) + top
    return o.view(batch, heads, d).bfloat16(), lse.view(batch, heads)


def _power_scale(x):
    """The smallest power of two 2^e, e >= -127, with amax(row) <= 448 * 2^e (1 for a row of zeros)."""
    top = x.float().abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m <= E4M3_MAX / 512.0, e - 9, e - 8).clamp(min=-127)
    return torch.ldexp(torch.ones_like(top), torch.where(top == 0, 0, e))


def _plain_write(s):
    page = s["case"]["page"]
    live = s["slots"] >= 0
    at = s["slots"][live]
    for n in ("k", "v"):
        x, cache, scale = s[n][live], s[n + "_cache"], s[n + "_scale"]
        if scale is None:
            cache[at // page, :, at % page] = x
        else:
            w = _power_scale(x)
            code = (x.float() / w.unsqueeze(-1)).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[at // page, :, at % page] = code.view(torch.uint8)
            scale[at // page, :, at % page] = w
    return s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]


def _plain_read(s):
    table, lens, n = s["table"].long(), s["lens"].long(), s["case"]["longest"]
    kv_heads, page = s["k_cache"].shape[1:3]
    at = torch.arange(n, device=table.device)
    ids = table[:, at // page].unsqueeze(1)
    h = torch.arange(kv_heads, device=table.device).view(1, -1, 1)
    x = _rows(s["k_cache"], s["k_scale"], ids, h, at % page)
    return x.mul_((at < lens.view(-1, 1)).view(-1, 1, n, 1)).bfloat16()


def _plain_beam(s):
    x, k = s["logits"].float(), s["case"]["k"]
    batch, beams, vocab = x.shape
    # within a beam the order is the logits', ties to the lower token: one whole number holds both
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF) - 1)
    key = key * (1 << 32) + ((1 << 32) - 1 - torch.arange(vocab, device=x.device))
    token = torch.topk(key, min(k, vocab), dim=2).indices.sort(2).values
    x64 = x.double()
    off = s["scores"].double() - torch.logsumexp(x64, 2)
    value = (torch.gather(x64, 2, token) + off.unsqueeze(2)).view(batch, -1)
    best = value.sort(dim=1, descending=True, stable=True)
    at = best.indices[:, :k]
    score = best.values[:, :k]
    parent = at // token.shape[2]
    token = torch.gather(token.reshape(batch, -1), 1, at)
    none = score == -math.inf
    short = k - score.shape[1]
    out = score.float(), parent.masked_fill(none, -1).int(), token.masked_fill(none, -1).int()
    if short > 0:
        pad = torch.nn.functional.pad
        out = pad(out[0], (0, short), value=-math.inf), pad(out[1], (0, short), value=-1), pad(out[2], (0, short), value=-1)
    return out


def _plain_reorder(s):
    b = torch.arange(s["parents"].shape[0], device=s["parents"].device).unsqueeze(1)
    p = s["parents"].long()
    return [x[b, p] for x in s["states"]]


def run(state):
    op = state["op"]
    if not own:
        return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read, "beam": _plain_beam,
                "reorder": _plain_reorder}[op](state)
    import approximate_top_selection_b200 as atk

    if op == "attend":
        return atk.paged_attention(state["q"], state["k_cache"], state["v_cache"], state["table"], state["lens"],
                                   k_scale=state["k_scale"], v_scale=state["v_scale"],
                                   positions=state["positions"], return_lse=True)
    if op == "write":
        atk.cache_write(state["k"], state["v"], state["k_cache"], state["v_cache"], state["slots"],
                        k_scale=state["k_scale"], v_scale=state["v_scale"])
        return state["k_cache"], state["k_scale"], state["v_cache"], state["v_scale"]
    if op == "read":
        return atk.cache_read(state["k_cache"], state["table"], state["lens"], state["case"]["longest"],
                              scale=state["k_scale"])
    if op == "beam":
        return atk.topk_beam(state["logits"], state["scores"], state["case"]["k"])
    return atk.beam_reorder(state["states"], state["parents"])


def work(case):
    op, d = case["op"], case.get("d", 0)
    esz = 1 if case.get("cache") == "e4m3" else 2
    row = d * esz + (4 if esz == 1 else 0)  # one cached row with its scale
    if op == "attend":
        rows = sum(min(n, case["listed"]) * case["heads"] if case["listed"] else n * case["kv_heads"]
                   for n in _lengths(case))
        scored = sum((min(n, case["listed"]) if case["listed"] else n) * case["heads"] for n in _lengths(case))
        small = case["batch"] * case["heads"] * (4 * d + 4)
        listed_bytes = 4 * case["batch"] * case["heads"] * case["listed"]
        table = 4 * sum(-(-n // case["page"]) for n in _lengths(case))
        return {"bytes": 2 * rows * row + small + listed_bytes + table, "flops": 4 * scored * d}
    if op == "write":
        live = case["tokens"] - (case["tokens"] // 32 if case["prefill"] else 0)
        return {"bytes": 2 * live * case["kv_heads"] * (2 * d + row) + 8 * case["tokens"], "flops": 0}
    if op == "read":
        rows = sum(_lengths(case)) * case["kv_heads"]
        return {"bytes": rows * row + 2 * case["batch"] * case["kv_heads"] * case["longest"] * d, "flops": 0}
    if op == "beam":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 12 * case["batch"] * case["k"], "flops": 3 * n}
    size = 4 if case["dtype"] == "i32" else 2
    rows = case["batch"] * (min(case["beams"], case["k"]) + case["k"])
    return {"bytes": case["tensors"] * rows * case["width"] * size, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def _sequence(s, name, b, n):
    """Rows [kv_heads, n, d] of sequence b, in 64 bits."""
    ids = s["table"][b].long()
    x = s[name + "_cache"][ids].double()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][ids].double()[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attend(s, case):
    out, lse = [], []
    heads, kv_heads = case["heads"], case["kv_heads"]
    for b, n in enumerate(_lengths(case)):
        q = s["q"][b].double()
        k, v = _sequence(s, "k", b, n), _sequence(s, "v", b, n)
        if case["listed"]:
            at = s["positions"][b].long()
            at = at[at >= 0].view(heads, -1)
            of = torch.arange(heads, device=at.device)[:, None] // (heads // kv_heads)
            k, v = k[of, at], v[of, at]
        t = q.view(k.shape[0], -1, case["d"]) @ k.transpose(1, 2) / math.sqrt(case["d"])
        lse.append(torch.logsumexp(t, 2).flatten())
        out.append((torch.softmax(t, 2) @ v).view(heads, -1))
    return torch.stack(out), torch.stack(lse)


def _exact_write(s, case):
    p = case["page"]
    live = case["tokens"] - (case["tokens"] // 32 if case["prefill"] else 0)
    at = s["slots"][:live]
    got = []
    for n in ("k", "v"):
        x = s[n][:live].double()
        pages, h, _, d = s[n + "_cache"].shape
        flat = torch.zeros(pages * p, h, d, dtype=torch.float64, device=x.device)
        scale = None
        if case["cache"] == "e4m3":
            one = torch.ones((), dtype=torch.float64, device=x.device)
            m, e = torch.frexp(x.abs().amax(2) / E4M3_MAX)
            w = torch.ldexp(one, e - (m == 0.5).int())
            y = x / w[..., None]
            step = torch.ldexp(one, (torch.frexp(y).exponent - 1).clamp(min=-6) - 3)
            x = torch.round(y / step) * step
            scale = torch.ones(pages * p, h, dtype=torch.float64, device=x.device)
            scale[at] = w
            scale = scale.view(pages, p, h).transpose(1, 2).contiguous()
        flat[at] = x
        got += [flat.view(pages, p, h, d).transpose(1, 2).contiguous(), scale]
    return tuple(got)


def _exact_read(s, case):
    out = torch.zeros(case["batch"], case["kv_heads"], case["longest"], case["d"], dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        out[b, :, :n] = _sequence(s, "k", b, n)
    return out


def _exact_beam(s, case):
    """Scores alone: which token and parent they belong to are whole numbers."""
    out = []
    for b in range(case["batch"]):
        v = torch.log_softmax(s["logits"][b].double(), 1) + s["scores"][b].double()[:, None]
        v = v.flatten().topk(min(case["k"], v.numel())).values
        out.append(torch.nn.functional.pad(v, (0, case["k"] - v.numel()), value=-math.inf))
    return torch.stack(out), None, None


def exact(case, seed):
    if case["op"] == "reorder":
        return None  # a copy: compared as it is
    s = prepare(case, seed)
    return {"attend": _exact_attend, "write": _exact_write, "read": _exact_read, "beam": _exact_beam}[case["op"]](s, case)

"""Cases and plain forms of the span attention, paged attention and paged rotation operators.

Each case names one operator, its sizes and what they stand for in real use.
``run`` is one pass through the operator: through the library's entry points
where ``own`` is true, else in elementary torch operations in 32 bits.
``exact`` gives the same outputs from the definitions in 64 bits.

Operators
  span_fwd        self-attention in which query i sees the keys of one span: from
                  key_begin[i] to key_end[i], no later than i where it is causal
                  and nearer than `window`; scores capped by a tanh, a bias that
                  grows with the distance, key/value heads shared by groups
  span_bwd        dQ, dK, dV of the same, from the O and the log-sum-exp at hand
  paged_fwd       attention of a chunk of new tokens per request (one token or
                  thousands) over a cache in pages, with the same window, cap and
                  bias
  rope_paged_fwd  per-head RMS norm and rotation of queries and keys of
                  token-major projections; keys and values go to the pages
"""

import math
import random

import torch

own = False  # where true, run() calls the library


def listed():
    return [
        # fine-tuning on short prompts that are seen both ways, answers causally
        {"name": "span_prefix", "op": "span_fwd", "B": 2, "H": 8, "Hkv": 2, "N": 333, "d": 64, "mask": "prefix",
         "window": 0, "cap": 0.0, "slopes": False},
        # pretraining on packed documents, capped scores
        {"name": "span_docs", "op": "span_fwd", "B": 1, "H": 32, "Hkv": 8, "N": 8192, "d": 128, "mask": "docs",
         "window": 0, "cap": 50.0, "slopes": False},
        # a layer of a long-context model that looks back 1024 tokens
        {"name": "span_window", "op": "span_fwd", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128, "mask": "causal",
         "window": 1024, "cap": 0.0, "slopes": False},
        # training with a distance bias in the place of positions
        {"name": "span_bias", "op": "span_fwd", "B": 4, "H": 16, "Hkv": 16, "N": 2048, "d": 64, "mask": "causal",
         "window": 0, "cap": 0.0, "slopes": True},
        # the backward passes of span_prefix, span_docs and a batch with both cap and bias
        {"name": "span_bwd_prefix", "op": "span_bwd", "B": 2, "H": 8, "Hkv": 2, "N": 333, "d": 64, "mask": "prefix",
         "window": 0, "cap": 0.0, "slopes": False},
        {"name": "span_bwd_docs", "op": "span_bwd", "B": 1, "H": 32, "Hkv": 8, "N": 8192, "d": 128, "mask": "docs",
         "window": 0, "cap": 50.0, "slopes": False},
        {"name": "span_bwd_bias", "op": "span_bwd", "B": 4, "H": 16, "Hkv": 4, "N": 1000, "d": 128, "mask": "causal",
         "window": 0, "cap": 30.0, "slopes": True},
        # a served batch, one token per request
        {"name": "paged_token", "op": "paged_fwd", "B": 16, "H": 32, "Hkv": 8, "T": 1, "len": 8100, "short": 300,
         "page": 16, "d": 128, "whole": True, "tokens_first": True, "window": 0, "cap": 50.0, "slopes": False},
        # a batch in which some requests bring a chunk of their prompt and some a few tokens
        {"name": "paged_mixed", "op": "paged_fwd", "B": 6, "H": 16, "Hkv": 4, "T": 200, "len": 3001, "short": 0,
         "page": 32, "d": 64, "whole": False, "tokens_first": False, "window": 1024, "cap": 0.0, "slopes": True},
        # a long prompt, 2048 tokens at a time
        {"name": "paged_chunk", "op": "paged_fwd", "B": 2, "H": 32, "Hkv": 8, "T": 2048, "len": 16000, "short": 2000,
         "page": 64, "d": 128, "whole": True, "tokens_first": False, "window": 0, "cap": 0.0, "slopes": False},
        # the served batch's new tokens, rotated and put into their pages
        {"name": "rope_paged_token", "op": "rope_paged_fwd", "B": 16, "H": 32, "Hkv": 8, "T": 1, "len": 8100,
         "short": 300, "page": 16, "d": 128, "whole": True, "tokens_first": True, "rot": 128, "norm": False,
         "interleaved": False},
        # the prompt's chunk, normed too
        {"name": "rope_paged_chunk", "op": "rope_paged_fwd", "B": 4, "H": 32, "Hkv": 8, "T": 2048, "len": 14000,
         "short": 0, "page": 64, "d": 128, "whole": False, "tokens_first": True, "rot": 64, "norm": True,
         "interleaved": True},
    ]


def _between(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.499))))))


def draw(rng):
    op = rng.choice(["span_fwd", "span_bwd", "paged_fwd", "paged_fwd", "rope_paged_fwd"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "H": hkv * rng.choice([1, 2, 4, 5, 8]), "Hkv": hkv, "d": d}
    if op in ("span_fwd", "span_bwd"):
        case["B"] = _between(rng, 1, 8)
        # within the products of paged_chunk, were all keys seen
        scores = 1.0e9 if op == "span_fwd" else 4.0e8
        case["N"] = _between(rng, 1, min(8192, math.isqrt(int(scores / (case["B"] * case["H"])))))
        case["mask"] = rng.choice(["causal", "docs", "docs", "prefix", "full", "docs_full"])
        case["window"] = rng.choice([0, 0, _between(rng, 1, 4096)])
        case["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        case["slopes"] = rng.random() < 0.4
        return case
    case["B"] = _between(rng, 1, 32)
    case["page"] = rng.choice([16, 32, 64, 128, 256])
    case["whole"] = rng.random() < 0.5
    case["tokens_first"] = rng.random() < 0.5
    if op == "paged_fwd":
        case["T"] = _between(rng, 1, min(2048, math.isqrt(int(1.0e9 / (case["B"] * case["H"])))))
        # within half a gigabyte of pages and the scores of paged_chunk
        most = min(3.0e8 / (2 * case["B"] * hkv * d), 1.0e9 / (case["B"] * case["H"] * case["T"]))
        case["len"] = _between(rng, 1, max(1, min(65536, int(most) - case["T"]))) - 1
        case["short"] = rng.randint(0, case["len"])
        case["window"] = rng.choice([0, 0, _between(rng, 1, 4096)])
        case["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        case["slopes"] = rng.random() < 0.4
        return case
    case["T"] = _between(rng, 1, max(1, min(8192, int(4.0e7 / (case["B"] * (case["H"] + 2 * hkv) * d)))))
    case["len"] = _between(rng, 1, max(1, min(65536, int(3.0e8 / (2 * case["B"] * hkv * d)) - case["T"]))) - 1
    case["short"] = rng.randint(0, case["len"])
    case["rot"] = rng.choice([d, d, d // 2, d // 4])
    case["norm"] = rng.random() < 0.6
    case["interleaved"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# masks, lengths and pages
# ---------------------------------------------------------------------------
def _spans(case, seed=None):
    """key_begin and key_end [B, N] (None where the mask needs none) and whether it is causal.  The sizes of
    documents and prefixes are the case's own, their order the seed's."""
    B, N, mask = case["B"], case["N"], case["mask"]
    if mask in ("causal", "full"):
        return None, None, mask == "causal"
    g = None if seed is None else random.Random(seed)
    sizes = random.Random(B * 100003 + N)
    begin, end = torch.zeros((B, N), dtype=torch.int32), torch.zeros((B, N), dtype=torch.int32)
    for b in range(B):
        if mask == "prefix":
            continue
        left = N - N // 32  # the rest is padding, which sees nothing
        docs = []
        while left > 0:
            docs.append(min(left, _between(sizes, 1, max(1, N // 2))))
            left -= docs[-1]
        if g:
            g.shuffle(docs)
        at = 0
        for n in docs:
            begin[b, at:at + n] = at
            end[b, at:at + n] = at + n
            at += n
    if mask != "prefix":
        return begin, end, mask == "docs"
    prefixes = [sizes.randint(0, N) for _ in range(B)]
    if g:
        g.shuffle(prefixes)
    return None, torch.maximum(torch.arange(1, N + 1)[None], torch.tensor(prefixes)[:, None]).to(torch.int32), False


def _lens(case, g=None):
    """Tokens that the requests' caches hold: evenly spread from case["short"] to case["len"]."""
    lens = torch.linspace(case["short"], case["len"], case["B"], dtype=torch.float64).round().to(torch.int32)
    if case["B"] == 1:
        lens[0] = case["len"]
    return lens if g is None else lens[torch.randperm(case["B"], generator=g)]


def _chunks(case):
    """New tokens of each request: all T, or from T down to few, the last of a batch none."""
    if case["whole"]:
        return torch.full((case["B"],), case["T"], dtype=torch.int32)
    chunks = torch.tensor([max(1, round(case["T"] / 2 ** b)) for b in range(case["B"])], dtype=torch.int32)
    if case["B"] > 2:
        chunks[-1] = 0
    return chunks


def _paged(case, lens, chunks, g, gd):
    """Page table and pools: the requests' pages lie anywhere in a pool of a few more; entries behind a request's
    pages are -1."""
    dev, P, Hkv, d = gd.device, case["page"], case["Hkv"], case["d"]
    pages = (lens + chunks + P - 1) // P
    width = max(1, (int(lens.max()) + case["T"] + P - 1) // P)
    table = torch.full((case["B"], width), -1, dtype=torch.int32)
    count = int(pages.sum()) + 3
    order = torch.randperm(count, generator=g).to(torch.int32)
    at = 0
    for b in range(case["B"]):
        n = int(pages[b])
        table[b, :n] = order[at:at + n]
        at += n
    shape = (count, P, Hkv, d) if case["tokens_first"] else (count, Hkv, P, d)
    pools = [torch.randn(shape, generator=gd, device=dev, dtype=torch.bfloat16) for _ in range(2)]
    if case["tokens_first"]:
        pools = [x.transpose(1, 2) for x in pools]
    return table.to(dev), *pools


def _slopes(H, dev):
    return 2.0 ** (-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)


def prepare(case, seed):
    dev = torch.device("cuda")
    gd = torch.Generator(dev).manual_seed(seed)
    g = torch.Generator().manual_seed(seed + 1)

    def normal(*shape):
        return torch.randn(shape, generator=gd, device=dev, dtype=torch.bfloat16)

    B, H, Hkv, d, op = case["B"], case["H"], case["Hkv"], case["d"], case["op"]
    # a program's scratch: an allocation that every call may use
    st = {"case": case, "scale": 1.0 / math.sqrt(d), "scratch": {}}
    if op != "rope_paged_fwd":
        st["slopes"] = _slopes(H, dev) if case["slopes"] else None
    if op in ("span_fwd", "span_bwd"):
        N = case["N"]
        st["q"], st["k"], st["v"] = normal(B, H, N, d), normal(B, Hkv, N, d), normal(B, Hkv, N, d)
        if case["cap"]:
            st["q"] *= 4  # scores that the cap bends
        begin, end, st["causal"] = _spans(case, seed)
        st["begin"] = None if begin is None else begin.to(dev)
        st["end"] = None if end is None else end.to(dev)
        if op == "span_fwd":
            st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty((B, H, N), device=dev)
        else:
            st["o"], st["lse"] = _span_fwd_plain(st)
            st["dout"] = normal(B, H, N, d)
            st["dq"], st["dk"], st["dv"] = (torch.empty_like(st[x]) for x in "qkv")
        return st
    T, lens, chunks = case["T"], _lens(case, g), _chunks(case)
    st["table"], st["k_pages"], st["v_pages"] = _paged(case, lens, chunks, g, gd)
    st["lens"], st["chunks"] = lens.to(dev), None if case["whole"] else chunks.to(dev)
    # rows behind a request's last new token are left as they were
    if op == "paged_fwd":
        st["q"] = normal(B, H, T, d)
        if case["cap"]:
            st["q"] *= 4
        st["o"], st["lse"] = torch.zeros_like(st["q"]), torch.zeros((B, H, T), device=dev)
        return st
    rows = normal(B, T, H + 2 * Hkv, d)  # the projection's output, token by token
    st["q"], st["k"], st["v"] = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
    st["qw"] = st["kw"] = None
    if case["norm"]:
        st["qw"] = 1.0 + 0.2 * torch.randn((d,), generator=gd, device=dev)
        st["kw"] = 1.0 + 0.2 * torch.randn((d,), generator=gd, device=dev)
    st["eps"] = 1e-6 if case["norm"] else None
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64)
    st["freq"] = (10000.0 ** (-i / case["rot"])).to(dev)
    st["q_out"] = torch.zeros((B, H, T, d), dtype=torch.bfloat16, device=dev)
    return st


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------
def _scratch(st, nbytes):
    ws = st["scratch"].get("ws")
    if ws is None or ws.numel() < nbytes:
        ws = st["scratch"]["ws"] = torch.empty((max(16, nbytes),), dtype=torch.uint8, device="cuda")
    return ws


def _run_own(st):
    from exact_tiled_attention_08_gb300 import fa

    case = st["case"]
    op, B, H, Hkv, d = case["op"], case["B"], case["H"], case["Hkv"], case["d"]
    if op == "span_fwd":
        ws = _scratch(st, fa.fa_span_fwd_workspace_bytes(B, H, Hkv, case["N"], d))
        fa.fa_span_fwd(st["q"], st["k"], st["v"], st["begin"], st["end"], st["o"], st["lse"], ws, st["scale"],
                       causal=st["causal"], window=case["window"], cap=case["cap"], slopes=st["slopes"])
        return st["o"], st["lse"]
    if op == "span_bwd":
        ws = _scratch(st, fa.fa_span_bwd_workspace_bytes(B, H, Hkv, case["N"], d))
        fa.fa_span_bwd(st["q"], st["k"], st["v"], st["begin"], st["end"], st["o"], st["dout"], st["lse"], st["dq"],
                       st["dk"], st["dv"], ws, st["scale"], causal=st["causal"], window=case["window"],
                       cap=case["cap"], slopes=st["slopes"])
        return st["dq"], st["dk"], st["dv"]
    if op == "paged_fwd":
        capacity = st["table"].shape[1] * case["page"]
        ws = _scratch(st, fa.fa_paged_fwd_workspace_bytes(B, H, Hkv, case["T"], capacity, d))
        fa.fa_paged_fwd(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["chunks"], st["o"],
                        st["lse"], ws, st["scale"], window=case["window"], cap=case["cap"], slopes=st["slopes"])
        return st["o"], st["lse"]
    fa.fa_rope_paged_fwd(st["q"], st["k"], st["v"], st["qw"], st["kw"], st["freq"], None, st["table"], st["lens"],
                         st["chunks"], st["q_out"], st["k_pages"], st["v_pages"], eps=st["eps"],
                         interleaved=case["interleaved"])
    return st["q_out"], st["k_pages"], st["v_pages"]


# ---------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _softmax_plain(s, seen):
    """Probabilities and log-sum-exp of the rows of s over the keys seen; an empty row has none, and -inf."""
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return p / total.masked_fill(total == 0, 1.0), (m + torch.log(total))[..., 0]


def _scores_plain(st, q, k, at, to):
    """Scores [B, H, n, m] of q [B, H, n, d] and k [B, Hkv, m, d] with cap and bias, and 1 - (score / cap)^2 of the
    capped ones; at [B or 1, n] and to [m] are the positions of queries and keys."""
    case, (B, H, n, d) = st["case"], q.shape
    q = q.float().reshape(B, k.shape[1], -1, d)
    s = torch.matmul(q, k.float().transpose(-1, -2)).reshape(B, H, n, -1) * st["scale"]
    bent = None
    if case["cap"]:
        t = torch.tanh(s / case["cap"])
        s, bent = t * case["cap"], 1.0 - t * t
    if st["slopes"] is not None:
        far = (at[:, None, :, None] - to[None, None, None]).abs().float()
        s = s - st["slopes"][None, :, None, None] * far
    return s, bent


def _span_seen(st):
    """[B or 1, 1, N, N]: which keys each query sees."""
    N = st["case"]["N"]
    i = torch.arange(N, device=st["q"].device)
    seen = torch.ones((1, 1, N, N), dtype=torch.bool, device=i.device)
    if st["begin"] is not None:
        seen = seen & (i >= st["begin"][:, None, :, None])
    if st["end"] is not None:
        seen = seen & (i < st["end"][:, None, :, None])
    if st["causal"]:
        seen = seen & (i[None] <= i[:, None])
    if st["case"]["window"]:
        seen = seen & ((i[:, None] - i[None]).abs() < st["case"]["window"])
    return seen


def _times_values(p, v):
    """[B, H, n, m] and [B, Hkv, m, d] -> [B, H, n, d]"""
    B, H, n, m = p.shape
    return torch.matmul(p.reshape(B, v.shape[1], -1, m), v.float()).reshape(B, H, n, -1)


def _span_fwd_plain(st):
    i = torch.arange(st["case"]["N"], device=st["q"].device)
    p, lse = _softmax_plain(_scores_plain(st, st["q"], st["k"], i[None], i)[0], _span_seen(st))
    return _times_values(p, st["v"]).to(st["q"].dtype), lse


def _span_bwd_plain(st):
    case = st["case"]
    B, H, Hkv, N, d = case["B"], case["H"], case["Hkv"], case["N"], case["d"]
    i = torch.arange(N, device=st["q"].device)
    s, bent = _scores_plain(st, st["q"], st["k"], i[None], i)
    # a row without keys has a log-sum-exp of -inf: its scores are masked before they meet it
    s = s.masked_fill_(~_span_seen(st), -math.inf)
    p = torch.exp(s - st["lse"].masked_fill(st["lse"] == -math.inf, 0.0)[..., None])
    del s
    do, delta = st["dout"].float(), (st["dout"].float() * st["o"].float()).sum(-1, keepdim=True)
    by_kv = (B, Hkv, H // Hkv * N, -1)
    dv = torch.matmul(p.reshape(by_kv).transpose(-1, -2), do.reshape(by_kv))
    dp = torch.matmul(do.reshape(by_kv), st["v"].float().transpose(-1, -2)).reshape(B, H, N, N)
    ds = dp.sub_(delta).mul_(p)
    if bent is not None:
        ds = ds.mul_(bent)
    dq = _times_values(ds, st["k"]) * st["scale"]
    dk = torch.matmul(ds.reshape(by_kv).transpose(-1, -2), st["q"].float().reshape(by_kv)) * st["scale"]
    return dq.bfloat16(), dk.bfloat16(), dv.bfloat16()


def _gathered(pool, table):
    """[B, Hkv, width * P, d]: the pages of each request one after another."""
    x = pool[table.long().clamp(min=0)]  # [B, width, Hkv, P, d]
    return x.transpose(1, 2).flatten(2, 3)


def _new_tokens(st, B, T):
    """[B, T]: which rows are new tokens."""
    n = torch.arange(T, device=st["q"].device)[None]
    return (n >= 0).expand(B, T) if st["chunks"] is None else n < st["chunks"][:, None]


def _paged_fwd_plain(st):
    case = st["case"]
    B, T = case["B"], case["T"]
    k, v = _gathered(st["k_pages"], st["table"]), _gathered(st["v_pages"], st["table"])
    to = torch.arange(k.shape[2], device=k.device)
    at = st["lens"][:, None] + torch.arange(T, device=k.device)[None]
    new = _new_tokens(st, B, T)
    back = at[:, :, None] - to  # how far back each key lies
    seen = back >= 0
    if case["window"]:
        seen = seen & (back < case["window"])
    s, _ = _scores_plain(st, st["q"], k, at, to)
    p, lse = _softmax_plain(s, seen[:, None])
    o = _times_values(p, v).to(st["q"].dtype)
    st["o"].copy_(torch.where(new[:, None, :, None], o, st["o"]))
    st["lse"].copy_(torch.where(new[:, None], lse, st["lse"]))
    return st["o"], st["lse"]


def _rope_paged_fwd_plain(st):
    case = st["case"]
    B, T, P, rot = case["B"], case["T"], case["page"], case["rot"]
    at = st["lens"][:, None] + torch.arange(T, device=st["q"].device)[None]
    angle = at.double()[:, :, None, None] * st["freq"]  # in 64 bits: far positions lose their angle in 32
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def one(x, w):
        x = x.float()
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        y = (a * cos - b * sin, a * sin + b * cos)
        y = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
        return torch.cat((y, x[..., rot:]), -1).bfloat16()

    new = _new_tokens(st, B, T)
    st["q_out"].copy_(torch.where(new[:, None, :, None], one(st["q"], st["qw"]).transpose(1, 2), st["q_out"]))
    b, n = torch.nonzero(new, as_tuple=True)
    row = at[b, n].long()
    page = st["table"][b, row // P].long()
    st["k_pages"][page, :, row % P] = one(st["k"], st["kw"])[b, n]
    st["v_pages"][page, :, row % P] = st["v"][b, n]
    return st["q_out"], st["k_pages"], st["v_pages"]


def run(state):
    if own:
        return _run_own(state)
    return {"span_fwd": _span_fwd_plain, "span_bwd": _span_bwd_plain, "paged_fwd": _paged_fwd_plain,
            "rope_paged_fwd": _rope_paged_fwd_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _span_pairs(case):
    """Pairs of a query and a key that it sees, over the batch."""
    B, N, w = case["B"], case["N"], case["window"]
    begin, end, causal = _spans(case)
    i = torch.arange(N)[None]
    begin = torch.zeros((B, N), dtype=torch.int64) if begin is None else begin.long()
    end = torch.full((B, N), N, dtype=torch.int64) if end is None else end.long()
    if causal:
        end = torch.minimum(end, i + 1)
    if w:
        begin, end = torch.maximum(begin, i - w + 1), torch.minimum(end, i + w)
    return int((end - begin).clamp(min=0).sum())


def work(case):
    op, B, H, Hkv, d = case["op"], case["B"], case["H"], case["Hkv"], case["d"]
    if op in ("span_fwd", "span_bwd"):
        N = case["N"]
        begin, end, _ = _spans(case)
        masks = 4 * B * N * ((begin is not None) + (end is not None))
        q, kv, lse, pairs = B * H * N * d * 2, B * Hkv * N * d * 2, B * H * N * 4, H * _span_pairs(case) * d
        if op == "span_fwd":
            return {"bytes": 2 * q + 2 * kv + lse + masks, "flops": 4 * pairs}
        return {"bytes": 4 * q + 4 * kv + lse + masks, "flops": 10 * pairs}
    lens, chunks = _lens(case).long(), _chunks(case).long()
    tokens = int(chunks.sum())
    entries = 4 * int(((lens + chunks + case["page"] - 1) // case["page"]).sum())
    if op == "rope_paged_fwd":
        return {"bytes": 2 * tokens * (H + 2 * Hkv) * d * 2,
                "flops": tokens * (H + Hkv) * (3 * case["rot"] + 4 * d * case["norm"])}
    keys, pairs = 0, 0
    for n, c in zip(lens.tolist(), chunks.tolist()):
        if c:
            w = case["window"] or n + c
            keys += n + c - max(0, n - w + 1)  # from the first token's first key on
            pairs += sum(min(n + t + 1, w) for t in range(c))
    return {"bytes": 2 * keys * Hkv * d * 2 + 2 * tokens * H * d * 2 + tokens * H * 4 + entries,
            "flops": 4 * H * d * pairs}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_head(st, q, k, h, first, lowest, highest):
    """Weights [n, m] of one head, their log-sum-exps, and d score / d (scale q k); query i of q [n, d] is at position
    first + i and sees the keys lowest[i] .. highest[i]-1 of k [m, d]."""
    raw = st["scale"] * (q.double() @ k.double().T)
    slope = torch.ones_like(raw)
    cap = st["case"]["cap"]
    if cap:
        slope = 1.0 / torch.cosh(raw / cap).square()
        raw = cap * torch.tanh(raw / cap)
    to = torch.arange(raw.shape[1], device=raw.device)
    at = first + torch.arange(raw.shape[0], device=raw.device)
    if st["slopes"] is not None:
        raw = raw - float(st["slopes"][h]) * (at[:, None] - to[None]).abs().double()
    hidden = (to[None] < lowest[:, None]) | (to[None] >= highest[:, None])
    raw = raw.masked_fill(hidden, -math.inf)
    if not raw.shape[1]:
        return raw, torch.full((raw.shape[0],), -math.inf, dtype=torch.float64, device=raw.device), slope
    lse = torch.logsumexp(raw, -1)
    return torch.exp(raw - lse.clamp(min=-1e300)[:, None]), lse, slope


def _exact_bounds(st, b):
    case = st["case"]
    N, w = case["N"], case["window"]
    i = torch.arange(N, device=st["q"].device)
    low = torch.zeros_like(i) if st["begin"] is None else st["begin"][b].long()
    high = torch.full_like(i, N) if st["end"] is None else st["end"][b].long()
    if st["causal"]:
        high = high.clamp(max=i + 1)
    if w:
        low, high = low.clamp(min=i - w + 1), high.clamp(max=i + w)
    return low, high


def _exact_span(st):
    case = st["case"]
    back = case["op"] == "span_bwd"
    G = case["H"] // case["Hkv"]
    o, lse = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device), st["lse"].double().clone()
    dq = torch.zeros_like(o)
    dk, dv = (torch.zeros(st["k"].shape, dtype=torch.float64, device=o.device) for _ in range(2))
    for b in range(case["B"]):
        low, high = _exact_bounds(st, b)
        for h in range(case["H"]):
            j = h // G
            q, k, v = st["q"][b, h], st["k"][b, j], st["v"][b, j].double()
            p, l, slope = _exact_head(st, q, k, h, 0, low, high)
            if not back:
                o[b, h], lse[b, h] = p @ v, l
                continue
            # the weights of the log-sum-exp at hand
            given = st["lse"][b, h].double()
            p = p * torch.exp(torch.where(l == -math.inf, 0.0, l - given))[:, None]
            do = st["dout"][b, h].double()
            ds = p * (do @ v.T - (do * st["o"][b, h].double()).sum(-1)[:, None]) * slope * st["scale"]
            dq[b, h] = ds @ k.double()
            dk[b, j] += ds.T @ q.double()
            dv[b, j] += p.T @ do
    return (dq, dk, dv) if back else (o, lse)


def _exact_paged(st):
    case = st["case"]
    G, P = case["H"] // case["Hkv"], case["page"]
    o, lse = st["o"].double().clone(), st["lse"].double().clone()
    for b in range(case["B"]):
        n, c = int(st["lens"][b]), case["T"] if st["chunks"] is None else int(st["chunks"][b])
        if not c:
            continue
        pages = st["table"][b, :(n + c + P - 1) // P].long()
        high = torch.arange(n + 1, n + c + 1, device=o.device)
        low = (high - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(high)
        for j in range(case["Hkv"]):
            k = torch.cat([st["k_pages"][p, j] for p in pages])[:n + c]
            v = torch.cat([st["v_pages"][p, j] for p in pages])[:n + c].double()
            for h in range(j * G, j * G + G):
                w, lse[b, h, :c], _ = _exact_head(st, st["q"][b, h, :c], k, h, n, low, high)
                o[b, h, :c] = w @ v
    return o, lse


def _exact_rope_paged(st):
    case = st["case"]
    P, r = case["page"], case["rot"]
    q_out, k_pages, v_pages = st["q_out"].double(), st["k_pages"].double(), st["v_pages"].double()

    def turned(x, w, phase):
        x = x.double()
        if case["norm"]:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + st["eps"]) * w.double()
        z = x[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, r // 2)).mT
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * phase)
        return torch.cat((z.flatten(-2) if case["interleaved"] else z.mT.flatten(-2), x[..., r:]), -1)

    for b in range(case["B"]):
        n, c = int(st["lens"][b]), case["T"] if st["chunks"] is None else int(st["chunks"][b])
        if not c:
            continue
        at = torch.arange(n, n + c, device=q_out.device)
        phase = torch.polar(torch.ones((), dtype=torch.float64, device=at.device), at.double()[:, None] * st["freq"])[:, None]
        q_out[b, :, :c] = turned(st["q"][b, :c], st["qw"], phase).transpose(0, 1)
        k = turned(st["k"][b, :c], st["kw"], phase)
        for first in range(n // P * P, n + c, P):  # page by page
            page, lo, hi = int(st["table"][b, first // P]), max(n, first), min(n + c, first + P)
            k_pages[page, :, lo - first:hi - first] = k[lo - n:hi - n].transpose(0, 1)
            v_pages[page, :, lo - first:hi - first] = st["v"][b, lo - n:hi - n].double().transpose(0, 1)
    return q_out, k_pages, v_pages


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("span_fwd", "span_bwd"):
        return _exact_span(st)
    return _exact_paged(st) if case["op"] == "paged_fwd" else _exact_rope_paged(st)

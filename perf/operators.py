"""Cases and plain forms of the cross attention, draft tree attention and rotation operators.

Each case names one operator, its sizes and what they stand for in real use.
``run`` is one pass through the operator: through the library's entry points
where ``own`` is true, else in elementary torch operations in 32 bits.
``exact`` gives the same outputs from the definitions in 64 bits.

Operators
  cross_fwd  O = softmax(scale Q K^T) V and the log-sum-exp of each row, with
             keys of another length than the queries, a key length per request
             and key/value heads shared by groups of query heads
  cross_bwd  dQ, dK, dV of the same, from the O and the log-sum-exp at hand
  tree_fwd   attention of T drafted tokens per request over a cache that holds
             the request's tokens and then the drafts; a 64-bit word per token
             says which drafts it sees
  rope_fwd   per-head RMS norm (where eps is given) and rotation of queries and
             keys of token-major projections into head-major operands, with the
             values laid out beside them (into a cache, or operands of fa_fwd)
  rope_bwd   the gradients of the same
"""

import math

import torch

own = False  # where true, run() calls the library


def listed():
    return [
        # one decoder token per request over an encoder's 1500 states
        {"name": "cross_token", "op": "cross_fwd", "B": 4, "H": 16, "Hkv": 16, "Nq": 1, "Nk": 1500, "short": 1500,
         "d": 64},
        # a padded batch of decoder prompts over encoder states of many lengths
        {"name": "cross_ragged", "op": "cross_fwd", "B": 6, "H": 16, "Hkv": 4, "Nq": 333, "Nk": 1023, "short": 130,
         "d": 128},
        # training: long decoder sequences over a document's states
        {"name": "cross_long", "op": "cross_fwd", "B": 2, "H": 32, "Hkv": 8, "Nq": 8192, "Nk": 2048, "short": 2048,
         "d": 128},
        # training on short captions: 77 states, fewer than one block of keys
        {"name": "cross_bwd_short", "op": "cross_bwd", "B": 2, "H": 8, "Hkv": 8, "Nq": 96, "Nk": 77, "short": 40,
         "d": 64},
        # training on a padded batch
        {"name": "cross_bwd_ragged", "op": "cross_bwd", "B": 4, "H": 16, "Hkv": 4, "Nq": 1000, "Nk": 1500,
         "short": 400, "d": 128},
        # the backward of cross_long
        {"name": "cross_bwd_long", "op": "cross_bwd", "B": 2, "H": 32, "Hkv": 8, "Nq": 8192, "Nk": 2048,
         "short": 2048, "d": 128},
        # one user, one token at a time
        {"name": "tree_token", "op": "tree_fwd", "B": 1, "H": 32, "Hkv": 8, "T": 1, "C": 2048, "len": 1907,
         "short": 1907, "d": 128, "tree": False},
        # a served batch verifying trees of 24 drafts
        {"name": "tree_draft", "op": "tree_fwd", "B": 8, "H": 32, "Hkv": 8, "T": 24, "C": 8192, "len": 8100,
         "short": 600, "d": 128, "tree": True},
        # long contexts, small trees
        {"name": "tree_long", "op": "tree_fwd", "B": 16, "H": 32, "Hkv": 8, "T": 8, "C": 32768, "len": 32700,
         "short": 8000, "d": 128, "tree": True},
        # a served batch of single tokens: rotation at far positions (scaled frequencies), appended to the cache
        {"name": "rope_append", "op": "rope_fwd", "B": 8, "N": 1, "H": 32, "Hkv": 8, "d": 128, "rot": 128,
         "norm": False, "interleaved": False, "C": 4096, "far": 1000000, "scaled": True},
        # a training step's queries and keys, normed and rotated
        {"name": "rope_norm_prompt", "op": "rope_fwd", "B": 2, "N": 8192, "H": 32, "Hkv": 8, "d": 128, "rot": 128,
         "norm": True, "interleaved": False, "C": 8192, "far": 0, "scaled": False},
        # its backward pass, with half of each head rotated in interleaved pairs
        {"name": "rope_norm_bwd", "op": "rope_bwd", "B": 2, "N": 4001, "H": 32, "Hkv": 8, "d": 128, "rot": 64,
         "norm": True, "interleaved": True, "far": 0},
    ]


def _between(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.499))))))


def draw(rng):
    op = rng.choice(["cross_fwd", "cross_bwd", "tree_fwd", "rope_fwd", "rope_bwd"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "H": hkv * rng.choice([1, 2, 4, 5, 8]), "Hkv": hkv, "d": d}
    if op in ("cross_fwd", "cross_bwd"):
        case["B"] = _between(rng, 1, 8)
        case["Nk"] = _between(rng, 1, 4096)
        most = 1.0e9 / (case["B"] * case["H"] * case["Nk"])  # within cross_long's work
        case["Nq"] = _between(rng, 1, max(1, min(8192, int(most))))
        case["short"] = rng.choice([case["Nk"], _between(rng, 1, case["Nk"]), 0])
    elif op == "tree_fwd":
        case["B"] = _between(rng, 1, 32)
        case["T"] = _between(rng, 1, 64)
        case["C"] = _between(rng, case["T"] + 1, max(case["T"] + 1, min(65536, int(6.0e8 / (2 * case["B"] * hkv * d)))))
        case["len"] = rng.randint(0, case["C"] - case["T"])
        case["short"] = rng.randint(0, case["len"])
        case["tree"] = rng.random() < 0.7
    else:
        case["B"] = _between(rng, 1, 8)
        case["N"] = _between(rng, 1, max(1, min(16384, int(8.0e7 / (case["B"] * (case["H"] + 2 * hkv) * d)))))
        case["rot"] = rng.choice([d, d, d // 2, d // 4])
        case["norm"] = rng.random() < 0.6
        case["interleaved"] = rng.random() < 0.5
        case["far"] = rng.choice([0, 0, _between(rng, 1, 2000000)])
        if op == "rope_fwd":
            case["C"] = case["N"] + rng.choice([0, _between(rng, 1, 1000)])
            case["scaled"] = rng.random() < 0.3
    return case


def _lens(case, top, g=None):
    """The requests' lengths: evenly spread from case["short"] to top; in an order of the seed's."""
    lens = torch.linspace(case["short"], top, case["B"], dtype=torch.float64).round().to(torch.int32)
    if case["B"] == 1:
        lens[0] = top
    return lens if g is None else lens[torch.randperm(case["B"], generator=g)]


def _drafts(case):
    """Drafted tokens of each request: the last request of a batch has about half of them."""
    drafts = torch.full((case["B"],), case["T"], dtype=torch.int32)
    if case["B"] > 1:
        drafts[-1] = (case["T"] + 1) // 2
    return drafts


def _trees(case, g):
    """Which drafts each draft sees, as bits of a word: itself and its ancestors in a random tree."""
    B, T = case["B"], case["T"]
    words = torch.zeros((B, T), dtype=torch.int64)
    for i in range(T):
        bit = 1 << i if i < 63 else -(1 << 63)
        if i == 0:
            words[:, 0] = bit
            continue
        parent = torch.randint(max(0, i - 5), i, (B, 1), generator=g)
        words[:, i] = torch.gather(words, 1, parent)[:, 0] | bit
    return words


def prepare(case, seed):
    dev = torch.device("cuda")
    gd = torch.Generator(dev).manual_seed(seed)
    g = torch.Generator().manual_seed(seed + 1)

    def normal(*shape):
        return torch.randn(shape, generator=gd, device=dev, dtype=torch.bfloat16)

    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    st = {"case": case, "scale": 1.0 / math.sqrt(d)}
    op = case["op"]
    if op in ("cross_fwd", "cross_bwd"):
        Nq, Nk = case["Nq"], case["Nk"]
        st["q"], st["k"], st["v"] = normal(B, H, Nq, d), normal(B, Hkv, Nk, d), normal(B, Hkv, Nk, d)
        # a batch without padding is called without lengths
        st["lens"] = _lens(case, Nk, g).to(dev) if case["short"] != Nk else None
        if op == "cross_fwd":
            st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty((B, H, Nq), device=dev)
        else:
            st["o"], st["lse"] = _cross_fwd_plain(st)
            st["dout"] = normal(B, H, Nq, d)
            st["dq"], st["dk"], st["dv"] = (torch.empty_like(st[x]) for x in "qkv")
    elif op == "tree_fwd":
        T, C = case["T"], case["C"]
        st["q"], st["k"], st["v"] = normal(B, H, T, d), normal(B, Hkv, C, d), normal(B, Hkv, C, d)
        st["lens"] = _lens(case, case["len"], g).to(dev)
        st["drafts"] = _drafts(case).to(dev)
        st["masks"] = _trees(case, g).to(dev) if case["tree"] else None
        # rows behind a request's last draft are left as they were
        st["o"], st["lse"] = torch.zeros_like(st["q"]), torch.zeros((B, H, T), device=dev)
    else:
        N = case["N"]
        rows = normal(B, N, H + 2 * Hkv, d)  # the projection's output, token by token
        st["q"], st["k"], st["v"] = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
        st["qw"] = st["kw"] = None
        if case["norm"]:
            st["qw"] = 1.0 + 0.2 * torch.randn((d,), generator=gd, device=dev)
            st["kw"] = 1.0 + 0.2 * torch.randn((d,), generator=gd, device=dev)
        st["eps"] = 1e-6 if case["norm"] else None
        i = torch.arange(0, case["rot"], 2, dtype=torch.float64)
        st["freq"] = (10000.0 ** (-i / case["rot"])).to(dev)
        st["factor"] = 1.0
        if case.get("scaled"):
            # contexts 8 times the trained length: low frequencies slowed by 8, high ones kept
            st["freq"] = st["freq"] * torch.where(st["freq"] * 4096 < 2 * math.pi, 1.0 / 8, 1.0)
            st["factor"] = 0.1 * math.log(8) + 1.0
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=g)
        st["pos"] = (first + torch.arange(N)[None]).to(torch.int32).to(dev)
        if op == "rope_fwd":
            C = case["C"]
            st["starts"] = torch.randint(0, C - N + 1, (B,), generator=g).to(torch.int32).to(dev)
            st["q_out"] = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev)
            st["k_out"], st["v_out"] = normal(B, Hkv, C, d), normal(B, Hkv, C, d)
        else:
            st["dq_out"], st["dk_out"], st["dv_out"] = normal(B, H, N, d), normal(B, Hkv, N, d), normal(B, Hkv, N, d)
            drows = torch.empty_like(rows)
            st["dq"], st["dk"], st["dv"] = drows[:, :, :H], drows[:, :, H:H + Hkv], drows[:, :, H + Hkv:]
            st["dqw"] = torch.empty((d,), device=dev) if case["norm"] else None
            st["dkw"] = torch.empty((d,), device=dev) if case["norm"] else None
    # a program's scratch: an allocation that every call may use
    st["scratch"] = {}
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
    if op == "cross_fwd":
        ws = _scratch(st, fa.fa_cross_fwd_workspace_bytes(B, H, Hkv, case["Nq"], case["Nk"], d))
        fa.fa_cross_fwd(st["q"], st["k"], st["v"], st["lens"], st["o"], st["lse"], ws, st["scale"])
        return st["o"], st["lse"]
    if op == "cross_bwd":
        ws = _scratch(st, fa.fa_cross_bwd_workspace_bytes(B, H, Hkv, case["Nq"], case["Nk"], d))
        fa.fa_cross_bwd(st["q"], st["k"], st["v"], st["lens"], st["o"], st["dout"], st["lse"], st["dq"], st["dk"],
                        st["dv"], ws, st["scale"])
        return st["dq"], st["dk"], st["dv"]
    if op == "tree_fwd":
        ws = _scratch(st, fa.fa_tree_fwd_workspace_bytes(B, H, Hkv, case["T"], case["C"], d))
        fa.fa_tree_fwd(st["q"], st["k"], st["v"], st["lens"], st["drafts"], st["masks"], st["o"], st["lse"], ws,
                       st["scale"])
        return st["o"], st["lse"]
    if op == "rope_fwd":
        fa.fa_rope_fwd(st["q"], st["k"], st["v"], st["qw"], st["kw"], st["freq"], st["pos"], st["starts"],
                       st["q_out"], st["k_out"], st["v_out"], eps=st["eps"], factor=st["factor"],
                       interleaved=case["interleaved"])
        return st["q_out"], st["k_out"], st["v_out"]
    ws = _scratch(st, fa.fa_rope_bwd_workspace_bytes(B, H, Hkv, case["N"], d)) if case["norm"] else None
    fa.fa_rope_bwd(st["q"], st["k"], st["qw"], st["kw"], st["freq"], st["pos"], st["dq_out"], st["dk_out"],
                   st["dv_out"], st["dq"], st["dk"], st["dv"], st["dqw"], st["dkw"], ws, eps=st["eps"],
                   factor=st["factor"], interleaved=case["interleaved"])
    return tuple(st[x] for x in ("dq", "dk", "dv", "dqw", "dkw") if st[x] is not None)


# ---------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _visible(lens, n, device):
    """[B, 1, 1, n]: which keys each request has; None where it has them all."""
    return None if lens is None else torch.arange(n, device=device)[None, None, None] < lens[:, None, None, None]


def _softmax_plain(s, seen):
    """Probabilities and log-sum-exp of the rows of s over the keys seen; an empty row has none, and -inf."""
    if seen is not None:
        s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return p / total.masked_fill(total == 0, 1.0), (m + torch.log(total))[..., 0]


def _attend_plain(q, k, v, seen, scale):
    """q [B, Hkv, rows, d] over k, v [B, Hkv, n, d]."""
    p, lse = _softmax_plain(torch.matmul(q.float(), k.float().transpose(-1, -2)) * scale, seen)
    return torch.matmul(p, v.float()), lse


def _grouped(x, Hkv):
    """[B, H, N, d] -> [B, Hkv, (H / Hkv) N, d]: the rows that share a key/value head."""
    return x.reshape(x.shape[0], Hkv, -1, x.shape[-1])


def _cross_fwd_plain(st):
    q, Hkv = st["q"], st["k"].shape[1]
    o, lse = _attend_plain(_grouped(q, Hkv), st["k"], st["v"], _visible(st["lens"], st["k"].shape[2], q.device),
                           st["scale"])
    return o.reshape(q.shape).to(q.dtype), lse.reshape(q.shape[:3])


def _cross_bwd_plain(st):
    Hkv = st["k"].shape[1]
    q, o, do = (_grouped(st[x], Hkv).float() for x in ("q", "o", "dout"))
    k, v = st["k"].float(), st["v"].float()
    lse = st["lse"].reshape(*q.shape[:3], 1)
    p = torch.exp(torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"]).sub_(lse))
    seen = _visible(st["lens"], k.shape[2], q.device)
    if seen is not None:
        p = p.masked_fill_(~seen, 0.0)
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k) * st["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q) * st["scale"]
    return dq.reshape(st["q"].shape).bfloat16(), dk.bfloat16(), dv.bfloat16()


def _tree_fwd_plain(st):
    q, Hkv, C = st["q"], st["k"].shape[1], st["k"].shape[2]
    B, H, T, d = q.shape
    # place of each key among the drafts of its request: negative for the request's own tokens
    at = torch.arange(C, device=q.device)[None, None] - st["lens"][:, None, None]
    if st["masks"] is None:
        seen = at <= torch.arange(T, device=q.device)[None, :, None]
    else:
        seen = (at < 0) | ((at < 64) & ((st["masks"][:, :, None] >> at.clamp(0, 63)) & 1).bool())
    seen = seen & (at < st["drafts"][:, None, None])
    seen = seen[:, None, None].expand(B, 1, H // Hkv, T, C).reshape(B, 1, -1, C)
    o, lse = _attend_plain(_grouped(q, Hkv), st["k"], st["v"], seen, st["scale"])
    drafted = (torch.arange(T, device=q.device)[None] < st["drafts"][:, None])[:, None]
    st["o"].copy_(torch.where(drafted[..., None], o.reshape(q.shape).to(q.dtype), st["o"]))
    st["lse"].copy_(torch.where(drafted, lse.reshape(B, H, T), st["lse"]))
    return st["o"], st["lse"]


def _angles(st):
    """cos and sin [B, N, 1, rot / 2] of position times frequency: in 64 bits, far positions lose their angle in 32."""
    a = st["pos"].double()[:, :, None, None] * st["freq"]
    return (torch.cos(a) * st["factor"]).float(), (torch.sin(a) * st["factor"]).float()


def _turned(x, cos, sin, rot, interleaved):
    """x [..., d] with its first `rot` values rotated in pairs (i, i + rot / 2), or (2 i, 2 i + 1)."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., rot:]), -1)


def _normed(x, eps):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r, r


def _rope_fwd_plain(st):
    case = st["case"]
    cos, sin = _angles(st)

    def one(x, w):
        x = x.float()
        if case["norm"]:
            x = _normed(x, st["eps"])[0] * w
        return _turned(x, cos, sin, case["rot"], case["interleaved"]).transpose(1, 2).bfloat16()

    st["q_out"].copy_(one(st["q"], st["qw"]))
    at = (st["starts"][:, None] + torch.arange(case["N"], device=cos.device))[:, None, :, None]
    k = one(st["k"], st["kw"])
    at = at.long().expand(k.shape)
    st["k_out"].scatter_(2, at, k)
    st["v_out"].scatter_(2, at, st["v"].transpose(1, 2))
    return st["q_out"], st["k_out"], st["v_out"]


def _rope_bwd_plain(st):
    case = st["case"]
    cos, sin = _angles(st)

    def one(x, w, g):
        g = _turned(g.float().transpose(1, 2), cos, -sin, case["rot"], case["interleaved"])
        if not case["norm"]:
            return g.bfloat16(), None
        y, r = _normed(x.float(), st["eps"])
        dw = (g * y).sum((0, 1, 2))
        g = g * w
        return ((g - y * (g * y).mean(-1, keepdim=True)) * r).bfloat16(), dw

    dq, dqw = one(st["q"], st["qw"], st["dq_out"])
    dk, dkw = one(st["k"], st["kw"], st["dk_out"])
    return tuple(x for x in (dq, dk, st["dv_out"].transpose(1, 2), dqw, dkw) if x is not None)


def run(state):
    if own:
        return _run_own(state)
    return {"cross_fwd": _cross_fwd_plain, "cross_bwd": _cross_bwd_plain, "tree_fwd": _tree_fwd_plain,
            "rope_fwd": _rope_fwd_plain, "rope_bwd": _rope_bwd_plain}[state["case"]["op"]](state)


def work(case):
    op, B, H, Hkv, d = case["op"], case["B"], case["H"], case["Hkv"], case["d"]
    if op in ("cross_fwd", "cross_bwd"):
        keys = int(_lens(case, case["Nk"]).sum()) if case["short"] != case["Nk"] else B * case["Nk"]
        q, kv, lse = B * H * case["Nq"] * d * 2, keys * Hkv * d * 2, B * H * case["Nq"] * 4
        pairs = H * case["Nq"] * keys * d
        if op == "cross_fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs}
        # queries, O, dO and dQ; keys and values, and their gradients over the padding too
        return {"bytes": 4 * q + 2 * kv + 2 * B * case["Nk"] * Hkv * d * 2 + lse, "flops": 10 * pairs}
    if op == "tree_fwd":
        drafts, lens = _drafts(case), _lens(case, case["len"])
        keys, rows = int((lens + drafts).sum()), int(drafts.sum())
        return {"bytes": 2 * keys * Hkv * d * 2 + 2 * rows * H * d * 2 + rows * H * 4 + (8 * rows if case["tree"] else 0),
                "flops": 4 * H * d * int(((lens + drafts).long() * drafts).sum())}
    tokens = B * case["N"]
    heads = H + 2 * Hkv
    if op == "rope_fwd":
        return {"bytes": 2 * tokens * heads * d * 2, "flops": tokens * (H + Hkv) * (3 * case["rot"] + 4 * d * case["norm"])}
    moved = 2 * heads + (H + Hkv if case["norm"] else 0)  # the norm's gradient reads its input too
    return {"bytes": tokens * moved * d * 2, "flops": tokens * (H + Hkv) * (3 * case["rot"] + 10 * d * case["norm"])}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(st, b, h):
    """For request b and query head h: scores [rows, n] over its keys and values, and those keys and values."""
    case = st["case"]
    j = h // (case["H"] // case["Hkv"])
    n = st["k"].shape[2] if st["lens"] is None else int(st["lens"][b])
    if case["op"] == "tree_fwd":
        n += int(st["drafts"][b])
    k, v = st["k"][b, j, :n].double(), st["v"][b, j, :n].double()
    return st["scale"] * (st["q"][b, h].double() @ k.T), k, v, j


def _exact_attention(st):
    case = st["case"]
    o, lse = st["o"].double().clone(), st["lse"].double().clone()
    for b in range(case["B"]):
        for h in range(case["H"]):
            s, _, v, _ = _exact_rows(st, b, h)
            rows = s.shape[0]
            if case["op"] == "tree_fwd":
                rows, first = int(st["drafts"][b]), int(st["lens"][b])
                place = torch.arange(rows, device=s.device)
                if st["masks"] is None:
                    sees = place[None] <= place[:, None]
                else:
                    sees = ((st["masks"][b, :rows, None] >> place[None]) & 1) == 1
                s = s[:rows]
                s[:, first:] = torch.where(sees, s[:, first:], -math.inf)
            lse[b, h, :rows] = torch.logsumexp(s, -1) if s.shape[1] else -math.inf
            w = torch.exp(s - lse[b, h, :rows, None])
            o[b, h, :rows] = torch.nan_to_num(w, nan=0.0) @ v
    return o, lse


def _exact_cross_bwd(st):
    case = st["case"]
    dq, dk, dv = (torch.zeros(st[x].shape, dtype=torch.float64, device=st[x].device) for x in "qkv")
    for b in range(case["B"]):
        for h in range(case["H"]):
            s, k, v, j = _exact_rows(st, b, h)
            if not s.shape[1]:
                continue
            do = st["dout"][b, h].double()
            p = torch.exp(s - st["lse"][b, h].double()[:, None])
            delta = torch.einsum("nd,nd->n", do, st["o"][b, h].double())
            ds = p * (do @ v.T - delta[:, None]) * st["scale"]
            dq[b, h] = ds @ k
            dk[b, j, :s.shape[1]] += ds.T @ st["q"][b, h].double()
            dv[b, j, :s.shape[1]] += p.T @ do
    return dq, dk, dv


def _exact_pairs(x, case):
    """The rotated part of x as complex numbers, one for each pair."""
    r = case["rot"]
    x = x[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, r // 2)).mT
    return torch.view_as_complex(x.contiguous())


def _exact_turn(x, phase, case):
    z = torch.view_as_real(_exact_pairs(x, case) * phase)
    z = z.flatten(-2) if case["interleaved"] else z.mT.flatten(-2)
    return torch.cat((z, x[..., case["rot"]:]), -1)


def _exact_rope(st):
    case = st["case"]
    phase = torch.polar(torch.full((), st["factor"], dtype=torch.float64, device=st["pos"].device),
                        st["pos"].double()[..., None] * st["freq"])[:, :, None]
    back = case["op"] == "rope_bwd"
    outs, dws = [], []
    for x, w, g in ((st["q"], st["qw"], st.get("dq_out")), (st["k"], st["kw"], st.get("dk_out"))):
        x = x.double()
        inv = 1.0 / torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + st["eps"]) if case["norm"] else 1.0
        unit = x * inv
        if not back:
            outs.append(_exact_turn(unit * w.double() if case["norm"] else unit, phase, case).transpose(1, 2))
            continue
        g = _exact_turn(g.double().transpose(1, 2), phase.conj(), case)
        if case["norm"]:
            dws.append(torch.einsum("bnhd,bnhd->d", g, unit))
            g = g * w.double()
            g = inv * (g - unit * torch.einsum("bnhd,bnhd->bnh", g, unit)[..., None] / case["d"])
        outs.append(g)
    if back:
        return (*outs, st["dv_out"].double().transpose(1, 2), *dws)
    caches = [st["k_out"].double(), st["v_out"].double()]
    for cache, new in zip(caches, (outs[1], st["v"].double().transpose(1, 2))):
        for b in range(case["B"]):
            first = int(st["starts"][b])
            cache[b, :, first:first + case["N"]] = new[b]
    return outs[0], *caches


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "cross_bwd":
        return _exact_cross_bwd(st)
    if case["op"] in ("cross_fwd", "tree_fwd"):
        return _exact_attention(st)
    return _exact_rope(st)

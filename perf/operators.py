"""The cached decoding operators measured on real sizes: their plain form, their
calls, and what each has to read, write and compute.

Four operators of one token step over the paged key-value cache:

  rope     per-head RMS norms of the queries and keys with the position rotation, the
           packed projection split into its heads, and the keys and values appended to
           the cache
  decode   attention of one new token per sequence over the cached tokens (a length per
           sequence), with the attention weights added to each token's running mass
  evict    which cached tokens leave when a budget is kept: the heaviest stay, with the
           first and the most recent ones, and kept rows behind the budget fill the holes
  compact  the moves of that plan: the rows in both pools, positions and masses

`own` picks the side: the plain form in elementary torch operations, or the framework's
calls.  Masses and pools are updated in place by both sides.
"""
import math
import random

import torch

own = False

PAGE = 64
EPS = 1e-6


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def _pages(n):
    return -(-n // PAGE)


def listed():
    return [
        # one new token of each sequence of the 16K GQA workload, appended to its cache
        {"name": "rope_token", "op": "rope", "dtype": "bf16", "batch": 2, "H": 28, "H_kv": 4, "d": 128,
         "n_tok": 1, "L_ctx": 16384, "rot": 128, "norm": True, "interleaved": False, "cache": True},
        # the decode block of 32 tokens of the 32K step (32 heads, batch 4), not cached yet
        {"name": "rope_block", "op": "rope", "dtype": "bf16", "batch": 4, "H": 32, "H_kv": 32, "d": 128,
         "n_tok": 32, "L_ctx": 32768, "rot": 128, "norm": True, "interleaved": False, "cache": False},
        # an 8K prompt filling the cache of the 8K workload
        {"name": "rope_prompt", "op": "rope", "dtype": "bf16", "batch": 1, "H": 32, "H_kv": 32, "d": 128,
         "n_tok": 8192, "L_ctx": 8192, "rot": 128, "norm": True, "interleaved": False, "cache": True},
        # the smallest cache: fp32, 4 heads of 64, three short sequences of odd lengths
        {"name": "decode_tiny", "op": "decode", "dtype": "fp32", "batch": 3, "H": 4, "H_kv": 4, "d": 64,
         "L_ctx": 1024, "ragged": True, "mass": True},
        # the 16K GQA workload, one token, masses kept for a later eviction
        {"name": "decode_gqa16k", "op": "decode", "dtype": "bf16", "batch": 2, "H": 28, "H_kv": 4, "d": 128,
         "L_ctx": 16384, "ragged": False, "mass": True},
        # a serving batch of 32 sequences of very different lengths, one slot of it idle
        {"name": "decode_ragged", "op": "decode", "dtype": "bf16", "batch": 32, "H": 32, "H_kv": 8, "d": 128,
         "L_ctx": 8192, "ragged": True, "mass": True},
        # the 32K workload, full lengths: 2.1 GB of keys and values
        {"name": "decode_32k", "op": "decode", "dtype": "bf16", "batch": 4, "H": 32, "H_kv": 32, "d": 128,
         "L_ctx": 32768, "ragged": False, "mass": False},
        # a cache at its budget of 2048 that a page of new tokens has outgrown
        {"name": "evict_step", "op": "evict", "batch": 4, "H_kv": 32, "shared": False, "L_ctx": 2112,
         "budget": 2048, "n_first": 4, "n_recent": 128, "ragged": False},
        # one decision per sequence for all heads, from the column masses of the 16K workload
        {"name": "evict_shared", "op": "evict", "batch": 2, "H_kv": 4, "shared": True, "L_ctx": 16384,
         "budget": 4096, "n_first": 4, "n_recent": 256, "ragged": True},
        # a 32K prompt cut to an eighth, every head by its own masses
        {"name": "evict_prompt", "op": "evict", "batch": 4, "H_kv": 32, "shared": False, "L_ctx": 32768,
         "budget": 4096, "n_first": 4, "n_recent": 512, "ragged": False},
        # the moves of evict_step
        {"name": "compact_step", "op": "compact", "dtype": "bf16", "batch": 4, "H_kv": 32, "shared": False,
         "d": 128, "L_ctx": 2112, "budget": 2048},
        # the moves of an 8K prompt cut to a quarter
        {"name": "compact_prompt", "op": "compact", "dtype": "bf16", "batch": 4, "H_kv": 32, "shared": False,
         "d": 128, "L_ctx": 8192, "budget": 2048},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "evict", "compact"])
    H_kv = rng.choice([1, 2, 4, 8, 32])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "rope":
        H = H_kv * rng.choice([1, 2, 4, 7])
        n_tok = _log(rng, 1, 8192)
        batch = _log(rng, 1, max(1, min(32, (1 << 25) // (n_tok * (H + 2 * H_kv) * d))))
        return {"op": op, "dtype": dtype, "batch": batch, "H": H, "H_kv": H_kv, "d": d, "n_tok": n_tok,
                "L_ctx": n_tok + rng.randrange(0, 200), "rot": rng.choice([d, d, d // 2, 24]),
                "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.3, "cache": rng.random() < 0.6}
    if op == "decode":
        L = _log(rng, 1, 65536)
        batch = _log(rng, 1, max(1, min(32, (1 << 28) // (L * H_kv * d))))
        return {"op": op, "dtype": dtype, "batch": batch, "H": H_kv * rng.choice([1, 3, 4, 7, 8, 16]),
                "H_kv": H_kv, "d": d, "L_ctx": L, "ragged": rng.random() < 0.7, "mass": rng.random() < 0.6}
    L = _log(rng, 66, 32768)
    budget = _log(rng, 32, L - 1)
    shared = rng.random() < 0.3
    if op == "evict":
        keep = rng.randrange(0, budget // 2 + 1)
        return {"op": op, "batch": _log(rng, 1, 8), "H_kv": H_kv, "shared": shared, "L_ctx": L, "budget": budget,
                "n_first": min(keep, rng.choice([0, 1, 4])), "n_recent": max(0, keep - 4), "ragged": rng.random() < 0.6}
    batch = _log(rng, 1, max(1, min(8, (1 << 27) // (L * H_kv * d))))
    return {"op": op, "dtype": dtype, "batch": batch, "H_kv": H_kv, "shared": shared, "d": d, "L_ctx": L,
            "budget": budget}


def _lens(case):
    """Cached tokens of each sequence: fixed by the case, so that its work is."""
    n, L = case["batch"], case["L_ctx"]
    if not case["ragged"]:
        return [L] * n
    r = random.Random(n * 1000003 + L)
    lens = [max(1, min(L, int(math.exp(r.uniform(math.log(max(1.0, L / 64)), math.log(L + 1)))))) for _ in range(n)]
    lens[0] = L
    if n > 4:
        lens[n // 2] = 0
    return lens


def _rand(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, scale, generator=g)


def _page_table(g, batch, pages):
    """Each sequence's pages at permuted slots of the pool."""
    return torch.randperm(max(1, batch * pages), generator=g, device="cuda")[:batch * pages].to(torch.int32).reshape(batch, pages)


def _pools(g, case, pages):
    shape = (max(1, case["batch"] * pages), case["H_kv"], PAGE, case["d"])
    return _rand(g, *shape, dtype=_dtype(case)), _rand(g, *shape, dtype=_dtype(case))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"case": case, **{"rope": _prepare_rope, "decode": _prepare_decode, "evict": _prepare_evict,
                             "compact": _prepare_compact}[case["op"]](case, g)}


def _prepare_rope(case, g):
    b, n, H, H_kv, d, L = (case[k] for k in ("batch", "n_tok", "H", "H_kv", "d", "L_ctx"))
    dt = _dtype(case)
    s = {"qkv": _rand(g, b, n, (H + 2 * H_kv) * d, dtype=dt)}
    first = torch.randint(0, L - n + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    s["pos"] = first[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    rot = case["rot"]
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
    s["q_weight"] = (1.0 + _rand(g, d, scale=0.1)).to(dt) if case["norm"] else None
    s["k_weight"] = (1.0 + _rand(g, d, scale=0.1)).to(dt) if case["norm"] else None
    s["Q"] = torch.empty(b, H, n, d, device="cuda", dtype=dt)
    if case["cache"]:
        pages = _pages(L)
        s["start"], s["end"] = first, torch.empty_like(first)
        s["page_table"] = _page_table(g, b, pages)
        s["K_pool"], s["V_pool"] = (torch.zeros(b * pages, H_kv, PAGE, d, device="cuda", dtype=dt) for _ in range(2))
        s["tok_pos"] = torch.full((b, H_kv, L), -1, device="cuda", dtype=torch.int32)
        s["tok_mass"] = torch.full((b, H_kv, L), 0.5, device="cuda")
    else:
        s["K"], s["V"] = (torch.empty(b, H_kv, n, d, device="cuda", dtype=dt) for _ in range(2))
    return s


def _prepare_decode(case, g):
    b, H, H_kv, d, L = (case[k] for k in ("batch", "H", "H_kv", "d", "L_ctx"))
    pages = _pages(L)
    s = {"Q": _rand(g, b, H, d, dtype=_dtype(case)), "page_table": _page_table(g, b, pages),
         "ctx_len": torch.tensor(_lens(case), dtype=torch.int32, device="cuda")}
    s["K_pool"], s["V_pool"] = _pools(g, case, pages)
    # the first token and two of the first page draw attention, as sinks do
    for t in (0, 1 % L, 37 % L):
        slot = s["page_table"][:, 0].long()
        q = s["Q"].float().view(b, H_kv, H // H_kv, d).mean(2)
        s["K_pool"][slot, :, t] = (s["K_pool"][slot, :, t].float() + 3.0 * q).to(_dtype(case))
    s["O"] = torch.empty_like(s["Q"])
    s["lse"] = torch.empty(b, H, device="cuda")
    s["tok_mass"] = _rand(g, b, H_kv, L).square() * 0.1 if case["mass"] else None
    return s


def _prepare_evict(case, g):
    b, L = case["batch"], case["L_ctx"]
    A = 1 if case["shared"] else case["H_kv"]
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    s = {"ctx_len": lens, "tok_mass": torch.exp(1.5 * _rand(g, b, A, L) - 4.0)}
    # positions as an earlier eviction left them: in order but for some moved rows
    at = torch.arange(L, device="cuda").expand(b, A, L)
    swap = torch.rand(b, A, L, generator=g, device="cuda") < 0.05
    s["tok_pos"] = (2 * at + swap * 101).to(torch.int32).contiguous()
    most = min(case["budget"], max(L - case["budget"], 0))
    s["hole_idx"], s["fill_idx"] = (torch.empty(b, A, most, dtype=torch.int32, device="cuda") for _ in range(2))
    s["move_cnt"] = torch.empty(b, A, dtype=torch.int32, device="cuda")
    s["new_len"] = torch.empty(b, dtype=torch.int32, device="cuda")
    return s


def _moves(case):
    """Moves of each decision when a uniform choice of `budget` of L_ctx tokens stays."""
    L, B = case["L_ctx"], case["budget"]
    return max(1, (L - B) * B // L)


def _prepare_compact(case, g):
    b, H_kv, L, B = (case[k] for k in ("batch", "H_kv", "L_ctx", "budget"))
    A, m, most = 1 if case["shared"] else H_kv, _moves(case), min(B, L - B)
    pages = _pages(L)
    s = {"page_table": _page_table(g, b, pages)}
    s["K_pool"], s["V_pool"] = _pools(g, case, pages)
    pick = lambda n: torch.rand(b, A, n, generator=g, device="cuda").argsort(-1)[..., :m].sort(-1).values  # noqa: E731
    for name, idx in (("hole_idx", pick(B)), ("fill_idx", B + pick(L - B))):
        s[name] = torch.full((b, A, most), -1, dtype=torch.int32, device="cuda")
        s[name][..., :m] = idx.to(torch.int32)
    s["move_cnt"] = torch.full((b, A), m, dtype=torch.int32, device="cuda")
    s["tok_mass"] = torch.rand(b, A, L, generator=g, device="cuda")
    s["tok_pos"] = torch.randint(0, 1 << 20, (b, A, L), generator=g, device="cuda", dtype=torch.int32)
    return s


# ---- the framework's calls ----

def _desc(s, L_q=1):
    """The descriptor (and a workspace) that a user's program makes once and keeps."""
    if "desc" not in s:
        import long_context_diffusion_b200 as dl
        c = s["case"]
        H_kv = c["H_kv"]
        slots = s["K_pool"].shape[0] if "K_pool" in s else 1
        s["desc"] = dl.make_desc(c["batch"], c.get("H", H_kv), H_kv, c.get("d", 128), c["L_ctx"], 1, PAGE,
                                 _pages(c["L_ctx"]), slots, _dtype(c) if "dtype" in c else torch.bfloat16)
        if c["op"] == "decode":
            s["ws"] = torch.empty(dl.dl_workspace_size(s["desc"]), dtype=torch.uint8, device="cuda")
        s["dl"] = dl
    return s["desc"]


def _own_rope(s):
    desc, c = _desc(s), s["case"]
    more = {k: s[k] for k in ("start", "page_table", "K_pool", "V_pool", "end", "tok_pos", "tok_mass")} if c["cache"] \
        else {"K_out": s["K"], "V_out": s["V"]}
    s["dl"].dl_qk_norm_rope(desc, s["qkv"], s["pos"], s["q_weight"], s["k_weight"], EPS, s["inv_freq"], s["Q"],
                            interleaved=c["interleaved"], **more)


def _own_decode(s):
    desc = _desc(s)
    s["dl"].dl_decode_attn(desc, s["Q"], s["K_pool"], s["V_pool"], s["page_table"], s["ctx_len"], s["O"], s["lse"],
                           s["ws"], tok_mass=s["tok_mass"], decay=0.99)


def _own_evict(s):
    desc, c = _desc(s), s["case"]
    s["dl"].dl_evict_select(desc, s["tok_mass"], s["tok_pos"], s["ctx_len"], c["budget"], c["n_first"],
                            c["n_recent"], s["hole_idx"], s["fill_idx"], s["move_cnt"], s["new_len"])


def _own_compact(s):
    desc = _desc(s)
    s["dl"].dl_cache_compact(desc, s["hole_idx"], s["fill_idx"], s["move_cnt"], s["page_table"], s["K_pool"],
                             s["V_pool"], s["tok_pos"], s["tok_mass"])


# ---- the plain forms ----

def _plain_rope(s):
    c = s["case"]
    b, n, H, H_kv, d, rot = (c[k] for k in ("batch", "n_tok", "H", "H_kv", "d", "rot"))
    x = s["qkv"].float().view(b, n, H + 2 * H_kv, d)
    turn = s["pos"].double()[..., None] * s["inv_freq"].double()
    cos, sin = torch.cos(turn).float()[:, :, None], torch.sin(turn).float()[:, :, None]

    def placed(y, w):
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        head, rest = y[..., :rot], y[..., rot:]
        if c["interleaved"]:
            u, v = head[..., 0::2], head[..., 1::2]
            head = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
        else:
            u, v = head[..., :rot // 2], head[..., rot // 2:]
            head = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
        return torch.cat((head, rest), -1).to(s["qkv"].dtype)

    q, k = placed(x[:, :, :H], s["q_weight"]), placed(x[:, :, H:H + H_kv], s["k_weight"])
    v = s["qkv"].view(b, n, H + 2 * H_kv, d)[:, :, H + H_kv:]
    s["Q"].copy_(q.transpose(1, 2))
    if not c["cache"]:
        s["K"].copy_(k.transpose(1, 2))
        s["V"].copy_(v.transpose(1, 2))
        return
    at = s["start"].long()[:, None] + torch.arange(n, device="cuda")
    slot = torch.gather(s["page_table"].long(), 1, at // PAGE)
    s["K_pool"][slot, :, at % PAGE] = k
    s["V_pool"][slot, :, at % PAGE] = v
    at = at[:, None].expand(b, H_kv, n)
    s["tok_pos"].scatter_(2, at, s["pos"][:, None].expand(b, H_kv, n))
    s["tok_mass"].scatter_(2, at, 0.0)
    torch.add(s["start"], n, out=s["end"])


def _cached(pool, page_table, L):
    """[batch][H_kv][L][d] in fp32, from the pages."""
    x = pool[page_table.long()]
    b, p, H_kv, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, H_kv, p * page, d)[:, :, :L].float()


def _plain_decode(s):
    c = s["case"]
    b, H, H_kv, d, L = (c[k] for k in ("batch", "H", "H_kv", "d", "L_ctx"))
    there = torch.arange(L, device="cuda") < s["ctx_len"][:, None]
    k = _cached(s["K_pool"], s["page_table"], L)
    logits = torch.matmul(s["Q"].float().view(b, H_kv, H // H_kv, d), k.transpose(2, 3)) / math.sqrt(d)
    del k
    logits = logits.masked_fill(~there[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(top.isinf(), 0.0, top))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    v = _cached(s["V_pool"], s["page_table"], L).masked_fill(~there[:, None, :, None], 0.0)
    s["O"].copy_(torch.matmul(p, v).reshape(b, H, d))
    s["lse"].copy_((top + torch.log(total)).reshape(b, H))
    if s["tok_mass"] is not None:
        s["tok_mass"].copy_(torch.where(there[:, None], 0.99 * s["tok_mass"] + p.sum(2), s["tok_mass"]))


def _listed_at(mask, most):
    """The indices where `mask` holds, ascending, in a list of `most`, -1 behind them."""
    b, A, L = mask.shape
    at = torch.where(mask, mask.cumsum(-1) - 1, most)
    out = torch.full((b, A, most + 1), -1, dtype=torch.int32, device="cuda")
    out.scatter_(2, at, torch.arange(L, dtype=torch.int32, device="cuda").expand(b, A, L))
    return out[..., :most]


def _plain_evict(s):
    c = s["case"]
    L, B = c["L_ctx"], c["budget"]
    n = s["ctx_len"][:, None, None]
    at = torch.arange(L, device="cuda")
    there = (at < n).expand(s["tok_mass"].shape)
    pos = s["tok_pos"].long()
    last = torch.where(there, pos, -(1 << 40)).amax(-1, keepdim=True)
    held = (pos < c["n_first"]) | (pos > last - c["n_recent"])
    key = torch.where(s["tok_mass"].isnan(), -math.inf, s["tok_mass"])
    key = torch.where(held, math.inf, key).masked_fill(~there, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, at.expand_as(order))
    keep = (rank < B) & there
    out = (n > B) & there
    most = s["hole_idx"].shape[-1]
    s["hole_idx"].copy_(_listed_at(out & ~keep & (at < B), most))
    s["fill_idx"].copy_(_listed_at(out & keep & (at >= B), most))
    s["move_cnt"].copy_((out & keep & (at >= B)).sum(-1))
    s["new_len"].copy_(s["ctx_len"].clamp(max=B))


def _plain_compact(s):
    c = s["case"]
    b, H_kv, most = c["batch"], c["H_kv"], s["hole_idx"].shape[-1]
    live = torch.arange(most, device="cuda") < s["move_cnt"][..., None]
    to, frm = s["hole_idx"].long(), s["fill_idx"].long()
    for name in ("tok_mass", "tok_pos"):
        moved = torch.gather(s[name], 2, frm.clamp(min=0))
        wide = torch.cat((s[name], s[name][..., :1]), -1)  # dead moves end in a column of their own
        wide.scatter_(2, torch.where(live, to, c["L_ctx"]), moved)
        s[name].copy_(wide[..., :c["L_ctx"]])
    seq, dec, i = live.nonzero(as_tuple=True)
    heads = torch.arange(H_kv, device="cuda")[None] if c["shared"] else dec[:, None]
    table = s["page_table"].long()
    row = lambda t: ((table[seq, t // PAGE])[:, None], heads, (t % PAGE)[:, None])  # noqa: E731
    for name in ("K_pool", "V_pool"):
        s[name][row(to[seq, dec, i])] = s[name][row(frm[seq, dec, i])]


def _outputs(s):
    c = s["case"]
    if c["op"] == "rope":
        names = ("Q", "K_pool", "V_pool", "tok_pos", "tok_mass", "end") if c["cache"] else ("Q", "K", "V")
    else:
        names = {"decode": ("O", "lse", "tok_mass"), "evict": ("hole_idx", "fill_idx", "move_cnt", "new_len"),
                 "compact": ("K_pool", "V_pool", "tok_pos", "tok_mass")}[c["op"]]
    return {k: s[k] for k in names}


def run(state):
    op = state["case"]["op"]
    if own:
        {"rope": _own_rope, "decode": _own_decode, "evict": _own_evict, "compact": _own_compact}[op](state)
    else:
        {"rope": _plain_rope, "decode": _plain_decode, "evict": _plain_evict, "compact": _plain_compact}[op](state)
    return _outputs(state)


def work(case):
    b, H_kv = case["batch"], case["H_kv"]
    if case["op"] == "rope":
        rows = b * case["n_tok"] * (case["H"] + 2 * H_kv)
        book = b * case["n_tok"] * H_kv * 8 if case["cache"] else 0
        return {"bytes": 2 * rows * case["d"] * _size(case) + b * case["n_tok"] * 4 + book, "flops": 8 * rows * case["d"]}
    if case["op"] == "decode":
        n, H, d = sum(_lens(case)), case["H"], case["d"]
        mass = 8 * n * H_kv if case["mass"] else 0
        return {"bytes": 2 * n * H_kv * d * _size(case) + 2 * b * H * d * _size(case) + 4 * b * H + mass,
                "flops": 4 * n * H * d}
    A = 1 if case["shared"] else H_kv
    if case["op"] == "evict":
        most = min(case["budget"], case["L_ctx"] - case["budget"])
        return {"bytes": A * (8 * sum(_lens(case)) + 8 * b * most), "flops": 0}
    m = _moves(case)
    return {"bytes": 2 * b * m * (H_kv * 2 * case["d"] * _size(case) + 8 * A) + 8 * b * A * m, "flops": 0}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    if case["op"] == "compact":
        return _exact_compact(case, s)
    return None  # whole numbers alone


def _exact_rope(case, s):
    b, n, H, H_kv, d, rot = (case[k] for k in ("batch", "n_tok", "H", "H_kv", "d", "rot"))
    x = s["qkv"].to(torch.float64).reshape(b * n, H + 2 * H_kv, d)
    w = torch.ones(H + 2 * H_kv, d, dtype=torch.float64, device="cuda")
    normed = torch.zeros(H + 2 * H_kv, 1, dtype=torch.bool, device="cuda")
    if case["norm"]:
        w[:H], w[H:H + H_kv], normed[:H + H_kv] = s["q_weight"].double(), s["k_weight"].double(), True
    rms = ((x * x).sum(2, keepdim=True) / d + EPS).sqrt()
    x = torch.where(normed, x / rms, x) * w
    # the rotation as a complex product
    i = torch.arange(rot // 2, device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    z = torch.complex(x[:, :H + H_kv][..., lo], x[:, :H + H_kv][..., hi])
    angle = s["pos"].reshape(-1, 1).double() * s["inv_freq"].double()
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[:, :H + H_kv, lo], x[:, :H + H_kv, hi] = z.real, z.imag
    x = x.reshape(b, n, H + 2 * H_kv, d).transpose(1, 2)
    q, k, v = x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    if not case["cache"]:
        return {"Q": q, "K": k, "V": v}
    kp, vp, mass = s["K_pool"].double(), s["V_pool"].double(), s["tok_mass"].double()
    for j in range(b):
        t0 = int(s["start"][j])
        t = torch.arange(t0, t0 + n, device="cuda")
        slots = s["page_table"][j].long()[t // PAGE]
        kp[slots, :, t % PAGE], vp[slots, :, t % PAGE] = k[j].transpose(0, 1), v[j].transpose(0, 1)
        mass[j, :, t0:t0 + n] = 0.0
    return {"Q": q, "K_pool": kp, "V_pool": vp, "tok_pos": None, "tok_mass": mass, "end": None}


def _exact_decode(case, s):
    H, H_kv, d = case["H"], case["H_kv"], case["d"]
    G = H // H_kv
    O = torch.zeros(case["batch"], H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], H), -math.inf, dtype=torch.float64, device="cuda")
    mass = None if s["tok_mass"] is None else s["tok_mass"].double()
    for j, n in enumerate(_lens(case)):
        if not n:
            continue
        slots = s["page_table"][j, :_pages(n)].long()
        for h in range(H_kv):
            k = s["K_pool"][slots, h].reshape(-1, d)[:n].double()
            v = s["V_pool"][slots, h].reshape(-1, d)[:n].double()
            a = (s["Q"][j, h * G:(h + 1) * G].double() @ k.T) * d ** -0.5
            lse[j, h * G:(h + 1) * G] = torch.logsumexp(a, 1)
            p = torch.softmax(a, 1)
            O[j, h * G:(h + 1) * G] = p @ v
            if mass is not None:
                mass[j, h, :n] = 0.99 * mass[j, h, :n] + p.sum(0)
    return {"O": O, "lse": lse, "tok_mass": mass}


def _exact_compact(case, s):
    H_kv, m = case["H_kv"], _moves(case)
    out = {k: s[k].double() for k in ("K_pool", "V_pool", "tok_mass")}
    for j in range(case["batch"]):
        for h in range(H_kv):
            a = 0 if case["shared"] else h
            to, frm = s["hole_idx"][j, a, :m].long(), s["fill_idx"][j, a, :m].long()
            ps, pd = s["page_table"][j].long()[frm // PAGE], s["page_table"][j].long()[to // PAGE]
            for k in ("K_pool", "V_pool"):
                out[k][pd, h, to % PAGE] = s[k][ps, h, frm % PAGE].double()
            out["tok_mass"][j, a, to] = s["tok_mass"][j, a, frm].double()
    return {**out, "tok_pos": None}

"""Cases and plain forms of the latent cache's operators for speculative decoding and eviction.

Four operators work on one latent cache (C_KV rows of d_c, K_R rows of d_r, shared by every head),
contiguous or paged, with a length per sequence:

  tree     attention of T drafted tokens (the nodes of a tree) over a sequence's n cached tokens and
           over the drafted tokens that each node's mask names: latent output and log-sum-exp
  mass     the attention weight that every cached token received from those queries, summed over
           heads and nodes and added to what it had received before
  select   which rows an eviction keeps: the first ones, the last ones, and the largest sums between
  compact  the kept rows moved to the front of their sequence, in place, with their sums

`run` computes them in plain torch where `own` is false, and through the framework where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    mla = {"dtype": "bf16", "d_c": 512, "d_r": 64}
    tiny = {"dtype": "f32", "d_c": 64, "d_r": 16}
    return [
        # one new token of one short conversation, 16 heads: launch latency
        {"name": "tree_one_token", "op": "tree", **mla, "B": 1, "H": 16, "T": 1, "n": 1024, "page": 0, "ragged": False, "chain": True},
        # DeepSeek-V2-Lite-shaped batch, 16 drafted tokens in random trees, conversations of unlike length in pages
        {"name": "tree_v2lite", "op": "tree", **mla, "B": 8, "H": 16, "T": 16, "n": 32768, "page": 64, "ragged": True, "chain": False},
        # DeepSeek-V2-shaped: 128 heads over the shared latent, 8 drafted tokens a sequence
        {"name": "tree_v2", "op": "tree", **mla, "B": 4, "H": 128, "T": 8, "n": 32768, "page": 64, "ragged": False, "chain": False},
        # fp32 parity shape, odd sizes, a contiguous cache
        {"name": "tree_f32", "op": "tree", **tiny, "B": 2, "H": 4, "T": 7, "n": 1001, "page": 0, "ragged": True, "chain": False},
        # each decode step's weights added up, V2-Lite-shaped
        {"name": "mass_one_token", "op": "mass", **mla, "B": 8, "H": 16, "T": 1, "n": 32768, "page": 64, "ragged": False, "chain": True},
        # the last 32 tokens of a prompt score its cache before an eviction, 128 heads
        {"name": "mass_window", "op": "mass", **mla, "B": 2, "H": 128, "T": 32, "n": 16384, "page": 0, "ragged": False, "chain": True},
        {"name": "mass_f32", "op": "mass", **tiny, "B": 2, "H": 4, "T": 7, "n": 1001, "page": 0, "ragged": True, "chain": False},
        # a batch of short conversations cut back to 512 rows
        {"name": "select_batch", "op": "select", "B": 32, "n": 2048, "keep": 512, "sink": 4, "recent": 128, "ragged": True},
        # long contexts
        {"name": "select_long", "op": "select", "B": 8, "n": 131072, "keep": 16384, "sink": 64, "recent": 4096, "ragged": True},
        # the accepted path of 16 drafted tokens closes up behind each sequence's cache
        {"name": "compact_commit", "op": "compact", **mla, "B": 32, "n": 4096, "keep": 0, "T": 16, "page": 64, "ragged": True, "sums": False},
        # an eviction's kept quarter moves to the front of its pages
        {"name": "compact_evict", "op": "compact", **mla, "B": 8, "n": 32768, "keep": 8192, "T": 0, "page": 64, "ragged": False, "sums": True},
        {"name": "compact_f32", "op": "compact", **tiny, "B": 3, "n": 1001, "keep": 300, "T": 0, "page": 0, "ragged": True, "sums": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: no drawn case costs more than the largest listed one of its operator
_MOST = {"tree": (320e6, 3.0e14), "mass": (320e6, 1.6e14), "select": (5e6, 1e9), "compact": (160e6, 1e9)}


def draw(rng: random.Random):
    op = rng.choice(["tree", "tree", "mass", "mass", "select", "compact"])
    while True:
        B = _log(rng, 1, 32)
        n = _log(rng, 1, 131072 if op == "select" else 65536)
        c = {"op": op, "B": B, "n": n, "ragged": rng.random() < 0.5}
        if op == "select":  # an eviction takes something away: n is above what is kept
            c["n"] = n = max(n, 64)
            keep = _log(rng, 16, 3 * n // 4)
            c |= {"keep": keep, "sink": min(keep // 4, rng.choice([0, 1, 4, 64])), "recent": rng.randint(0, keep // 2)}
        else:
            family = rng.choice(["mla"] * 6 + ["f32", "other"])
            c |= {"mla": {"dtype": "bf16", "d_c": 512, "d_r": 64}, "f32": {"dtype": "f32", "d_c": 64, "d_r": 16},
                  "other": {"dtype": "bf16", "d_c": rng.choice([128, 256]), "d_r": 32}}[family]
            c["page"] = rng.choice([0, 64, 64, 128, 192])
            if op == "compact":
                commit = rng.random() < 0.5
                c |= {"T": rng.randint(1, 64) if commit else 0, "keep": 0 if commit else _log(rng, 1, n), "sums": not commit}
            else:
                c |= {"H": rng.choice([8, 16, 16, 24, 32, 64, 128]) if family == "mla" else rng.choice([1, 4, 6]), "T": _log(rng, 1, 64), "chain": rng.random() < 0.4}
        w = work(c)
        slow = c.get("d_c", 512) != 512  # shapes of the CUDA-core kernels stay small
        if w["bytes"] <= _MOST[op][0] and w["flops"] <= (2e10 if slow else _MOST[op][1]):
            return c


def _lengths(c):
    """Cached tokens of each sequence: n, or from n down to about n / 4 in even steps."""
    return [c["n"] - (3 * c["n"] * b) // (4 * c["B"]) if c["ragged"] else c["n"] for b in range(c["B"])]


def _drafts(c):
    """Drafted tokens of each sequence: T, or fewer in every third sequence of a ragged batch."""
    return [max(1, c["T"] - (b % 3 == 1) * (c["T"] // 3)) if c["ragged"] else c["T"] for b in range(c["B"])]


def _accepted(c):
    """Accepted drafted tokens of each sequence of a commit."""
    return [1 + (b * 5) % min(c["T"], 6) for b in range(c["B"])]


def work(c):
    lens = _lengths(c)
    if c["op"] == "select":  # each sum read once, each kept index written once
        return {"bytes": 4 * sum(lens) + 4 * sum(min(n, c["keep"]) for n in lens) + 8 * c["B"], "flops": sum(lens)}
    e = 4 if c["dtype"] == "f32" else 2
    row = e * (c["d_c"] + c["d_r"])
    if c["op"] == "compact":  # each row that moves read once and written once
        k = _accepted(c) if c["T"] else [min(n, c["keep"]) for n in lens]
        return {"bytes": (2 * row + (8 if c["sums"] else 0) + 4) * sum(k), "flops": 0}
    d = _drafts(c)
    pairs = sum(t * n + t * (t + 1) // 2 for n, t in zip(lens, d)) * c["H"]
    rows = sum(n + t for n, t in zip(lens, d))
    q = sum(d) * c["H"]
    if c["op"] == "tree":
        return {"bytes": rows * row + q * (row + e * c["d_c"] + 4), "flops": 2 * pairs * (2 * c["d_c"] + c["d_r"])}
    return {"bytes": rows * (row + 8) + q * (row + 4), "flops": 2 * pairs * (c["d_c"] + c["d_r"])}


# ------------------------------------------------------------------ inputs

def _cache(c, rows_of, g, cap):
    """Pools, block table (None: contiguous) and page size of a cache that holds rows_of[b] rows of sequence b."""
    B, dt = c["B"], torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    if c["page"]:
        page = c["page"]
        per = -(-cap // page)
        total = sum(-(-r // page) for r in rows_of) + 2
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table, at = torch.full((B, per), -1, dtype=torch.int32, device=DEV), 0
        for b, r in enumerate(rows_of):
            k = -(-r // page)
            table[b, :k] = order[at:at + k]
            at += k
    else:
        page, total, table = cap, B, None
    c_pool = torch.randn(total * page, c["d_c"], generator=g, device=DEV).to(dt)
    k_pool = torch.randn(total * page, c["d_r"], generator=g, device=DEV).to(dt)
    return c_pool, k_pool, table, page


def _masks(c, seed):
    """[B][T] words: bit j of word i says that node i sees node j (its ancestors and itself)."""
    r = np.random.default_rng([seed, 77])
    B, T = c["B"], c["T"]
    words = np.zeros((B, T), dtype=np.uint64)
    for i in range(T):
        parent = np.full(B, i - 1) if c["chain"] else r.integers(-1, i, size=B) if i else np.full(B, -1)
        up = np.where(parent >= 0, words[np.arange(B), np.maximum(parent, 0)], np.uint64(0))
        words[:, i] = up | (np.uint64(1) << np.uint64(i))
    return torch.from_numpy(words.view(np.int64)).to(DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, lens = c["B"], _lengths(c)
    s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if c["op"] == "select":
        # sums of attention weights: many small, few large, rows that were never looked at at zero
        x = torch.exp(2.0 * torch.randn(B, c["n"], generator=g, device=DEV))
        x[torch.rand(B, c["n"], generator=g, device=DEV) < 0.05] = 0.0
        s |= {"scores": x, "kept": torch.zeros(B, c["keep"], dtype=torch.int32, device=DEV),
              "kept_lens": torch.zeros(B, dtype=torch.int32, device=DEV)}
        if own:
            s["plan"] = _plan(1, 16, 512, 64, "bf16", B, c["n"])
        return s
    if c["op"] == "compact":
        cap = c["n"] + c["T"]
        s["c"], s["k"], s["table"], s["page"] = _cache(c, [n + c["T"] for n in lens], g, cap)
        s["sums"] = torch.rand(B, cap, generator=g, device=DEV) if c["sums"] else None
        x = torch.rand(B, cap, generator=g, device=DEV)
        pos = torch.arange(cap, device=DEV)[None, :]
        n = s["lens"][:, None]
        if c["T"]:   # an accepted path: nodes of rising index
            k = torch.tensor(_accepted(c), dtype=torch.int32, device=DEV)
            x = torch.where((pos >= n) & (pos < n + c["T"]), x, torch.full_like(x, -1.0))
            s["dst0"] = s["lens"]
        else:
            k = torch.tensor([min(m, c["keep"]) for m in lens], dtype=torch.int32, device=DEV)
            x = torch.where(pos < n, x, torch.full_like(x, -1.0))
            s["dst0"] = None
        most = int(k.max())
        idx = torch.argsort(x, dim=1, descending=True)[:, :most]
        idx = torch.where(torch.arange(most, device=DEV)[None, :] < k[:, None], idx, torch.full_like(idx, 1 << 30))
        s["src"], s["n_src"] = torch.sort(idx, dim=1).values.to(torch.int32), k
        if own:
            s["plan"] = _plan(1, 16, c["d_c"], c["d_r"], c["dtype"], B, cap)
        return s
    H, T = c["H"], c["T"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    d = _drafts(c)
    cap = c["n"] + T
    s["c"], s["k"], s["table"], s["page"] = _cache(c, [n + t for n, t in zip(lens, d)], g, cap)
    scale = 2.5 / math.sqrt(c["d_c"] + c["d_r"])  # logits of standard deviation 2.5: attention with some peaks
    s["q_c"] = (torch.randn(B, T, H, c["d_c"], generator=g, device=DEV) * scale).to(dt)
    s["q_r"] = (torch.randn(B, T, H, c["d_r"], generator=g, device=DEV) * scale).to(dt)
    s["mask"] = None if c["chain"] else _masks(c, seed)
    s["words"] = _masks(c, seed)
    s["drafts"] = torch.tensor(d, dtype=torch.int32, device=DEV)
    if c["op"] == "tree":
        s["out"] = torch.zeros(B, T, H, c["d_c"], dtype=dt, device=DEV)
        s["lse"] = torch.zeros(B, T, H, device=DEV)
    else:
        s["prev"] = H * torch.rand(B, cap, generator=g, device=DEV) ** 4
        s["scores"] = torch.zeros(B, cap, device=DEV)
        s["lse"] = _logits(s)[2]
    if own:
        s["plan"] = _plan(B, H, c["d_c"], c["d_r"], c["dtype"], B, cap)
        s["work"] = s["plan"].tree_workspace(T)
    return s


def _plan(B, H, d_c, d_r, dtype, batch, max_L):
    import kv_compression_b200 as kvc
    return kvc.Plan(batch, H, d_c, d_r, dtype, max_L)


# ------------------------------------------------------------------ plain forms

def _rows(s, pos):
    """Pool rows of positions pos [B][n] (int64)."""
    B = pos.shape[0]
    page = torch.arange(B, device=DEV)[:, None] if s["table"] is None else torch.gather(s["table"].long(), 1, pos // s["page"])
    return page.clamp(min=0) * s["page"] + pos % s["page"]


def _logits(s):
    """Logits [B][T*H][n] of every (node, head) against every cached and drafted token, -inf where it sees none;
    the tokens' latents; each row's log-sum-exp [B][T][H]."""
    c = s["case"]
    B, T, H = c["B"], c["T"], c["H"]
    cap = c["n"] + T
    pos = torch.arange(cap, device=DEV)
    n, d = s["lens"].long()[:, None], s["drafts"].long()[:, None]
    rows = _rows(s, torch.where(pos[None, :] < n + d, pos[None, :], torch.zeros_like(pos)[None, :]))
    C, K = s["c"][rows].float(), s["k"][rows].float()
    x = torch.matmul(s["q_c"].reshape(B, T * H, -1).float(), C.transpose(1, 2))
    x += torch.matmul(s["q_r"].reshape(B, T * H, -1).float(), K.transpose(1, 2))
    node = pos[None, :] - n                                                    # [B][cap]
    bit = (s["words"][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1        # [B][T][cap]
    seen = (node < 0)[:, None, :] | ((node >= 0) & (node < d))[:, None, :] & (bit == 1)
    seen = seen & (torch.arange(T, device=DEV)[None, :] < d)[:, :, None]       # nodes past a sequence's own: none
    x.view(B, T, H, cap).masked_fill_(~seen[:, :, None, :], -math.inf)
    top = x.amax(2, keepdim=True).clamp(min=-3e38)
    lse = (top + torch.log(torch.exp(x - top).sum(2, keepdim=True))).view(B, T, H)
    return x, C, lse


def _plain_tree(s):
    x, C, lse = _logits(s)
    B, T, H = lse.shape
    live = (torch.arange(T, device=DEV)[None, :] < s["drafts"][:, None])[:, :, None]
    p = torch.exp(x - torch.where(live, lse, torch.zeros_like(lse)).view(B, T * H, 1))
    out = torch.matmul(p, C).view(B, T, H, -1).to(s["out"].dtype)
    s["out"] = torch.where(live[..., None], out, s["out"])
    s["lse"] = torch.where(live, lse, s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_mass(s):
    x, _, _ = _logits(s)
    B, T, H = s["lse"].shape
    cap = x.shape[2]
    live = (torch.arange(T, device=DEV)[None, :] < s["drafts"][:, None])[:, :, None]
    m = torch.exp(x - torch.where(live, s["lse"], torch.zeros_like(s["lse"])).view(B, T * H, 1)).sum(1)
    pos, n, d = torch.arange(cap, device=DEV)[None, :], s["lens"][:, None], s["drafts"][:, None]
    m = torch.where(pos < n, 0.96875 * s["prev"] + m, m)
    s["scores"] = torch.where(pos < n + d, m, s["scores"])
    return {"scores": s["scores"]}


def _plain_select(s):
    c, x = s["case"], s["scores"]
    pos, n = torch.arange(c["n"], device=DEV)[None, :], s["lens"][:, None]
    safe = (pos < c["sink"]) | (pos >= n - c["recent"])
    key = torch.where(pos < n, torch.where(safe, math.inf, x), -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    k = torch.minimum(n, torch.full_like(n, c["keep"]))
    j = torch.arange(idx.shape[1], device=DEV)[None, :]
    idx = torch.sort(torch.where(j < k, idx, torch.full_like(idx, c["n"])), dim=1).values.to(torch.int32)
    s["kept"][:, :idx.shape[1]] = torch.where(j < k, idx, s["kept"][:, :idx.shape[1]])
    s["kept_lens"] = k[:, 0].to(torch.int32)
    return {"kept": s["kept"], "kept_lens": s["kept_lens"]}


def _plain_compact(s):
    src, k = s["src"].long(), s["n_src"].long()[:, None]
    B, m = src.shape
    j = torch.arange(m, device=DEV)[None, :]
    d0 = torch.zeros_like(k) if s["dst0"] is None else s["dst0"].long()[:, None]
    ok = j < k
    a = _rows(s, torch.where(ok, src, torch.zeros_like(src)))[ok]
    b = _rows(s, torch.where(ok, d0 + j, torch.zeros_like(src)))[ok]
    s["c"][b] = s["c"][a]
    s["k"][b] = s["k"][a]
    if s["sums"] is not None:
        which = torch.arange(B, device=DEV)[:, None].expand(B, m)[ok]
        s["sums"][which, (d0 + j)[ok]] = s["sums"][which, src[ok]]
        return {"c": s["c"], "k": s["k"], "sums": s["sums"]}
    return {"c": s["c"], "k": s["k"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "mass": _plain_mass, "select": _plain_select, "compact": _plain_compact}[op](s)
    plan, c = s["plan"], s["case"]
    if op == "tree":
        plan.tree_decode(s["q_c"], s["q_r"], s["c"], s["k"], s["page"], s["table"], s["lens"], s["out"], s["lse"],
                         mask=s["mask"], draft_lens=s["drafts"], workspace=s["work"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "mass":
        plan.attn_mass(s["q_c"], s["q_r"], s["c"], s["k"], s["page"], s["table"], s["lens"], s["lse"], s["scores"],
                       prev=s["prev"], decay=0.96875, mask=s["mask"], draft_lens=s["drafts"], workspace=s["work"])
        return {"scores": s["scores"]}
    if op == "select":
        plan.evict_select(s["scores"], s["lens"], c["sink"], c["recent"], s["kept"], s["kept_lens"])
        return {"kept": s["kept"], "kept_lens": s["kept_lens"]}
    plan.cache_compact(s["c"], s["k"], s["page"], s["table"], s["src"], s["n_src"], dst0=s["dst0"], scores=s["sums"])
    return {"c": s["c"], "k": s["k"], "sums": s["sums"]} if s["sums"] is not None else {"c": s["c"], "k": s["k"]}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    c = dict(case)
    if c["op"] in ("select", "compact"):
        return None            # whole numbers, and rows that are only moved
    if work(c)["flops"] > 4e14:
        return None
    s = prepare(c, seed)
    B, T, H = c["B"], c["T"], c["H"]
    lens, drafts = _lengths(c), _drafts(c)
    words = s["words"].cpu().tolist()
    out = torch.zeros(B, T, H, c["d_c"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, T, H, dtype=torch.float64, device=DEV)
    scores = torch.zeros(B, c["n"] + T, dtype=torch.float64, device=DEV)
    for b in range(B):
        n, d = lens[b], drafts[b]
        at = [b * s["page"] + t for t in range(n + d)] if s["table"] is None else None
        if at is None:
            pages = s["table"][b].cpu().tolist()
            at = [pages[t // s["page"]] * s["page"] + t % s["page"] for t in range(n + d)]
        at = torch.tensor(at, device=DEV)
        C, K = s["c"][at].double(), s["k"][at].double()
        mass = torch.zeros(n + d, dtype=torch.float64, device=DEV)
        for i in range(d):
            use = list(range(n)) + [n + j for j in range(d) if words[b][i] >> j & 1]
            use = torch.tensor(use, device=DEV)
            u, v = C[use], K[use]
            x = s["q_c"][b, i].double() @ u.T + s["q_r"][b, i].double() @ v.T
            z = torch.logsumexp(x, 1)
            lse[b, i] = z
            if c["op"] == "tree":
                out[b, i] = torch.exp(x - z[:, None]) @ u
            else:
                mass[use] += torch.exp(x - s["lse"][b, i].double()[:, None]).sum(0)
        if c["op"] == "mass":
            mass[:n] += 0.96875 * s["prev"][b, :n].double()
            scores[b, :n + d] = mass
    return {"out": out, "lse": lse} if c["op"] == "tree" else {"scores": scores}

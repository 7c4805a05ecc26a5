"""Performance cases of the cache operators: tree attention over a cache, the commit of an
accepted path, decode attention that accumulates each key's weight, and eviction by that weight.

``run`` computes an operator in its plain form (elementary fp32 torch operations) or, where
``own`` is true, through the library's entry points.  Sizes: 128-wide heads, 4 query heads per
kv head, 8 kv heads for the whole block (fewer for a head shard); caches [B, S_max, n_kv, 128].
"""
import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
D = 128
HPG = 4  # query heads per kv head
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one chat user, a small tree behind a short prompt: latency
        dict(name="tree_b1_t8_len300", op="tree", B=1, T=8, length=300, n_kv=8, ragged=False),
        # a small server batch at mixed lengths, an odd tree size
        dict(name="tree_b8_t26_len4000", op="tree", B=8, T=26, length=4000, n_kv=8, ragged=True),
        # one long-context user with a wide tree
        dict(name="tree_b1_t60_len32000", op="tree", B=1, T=60, length=32000, n_kv=8, ragged=False),
        # a large server batch with wide trees: the most work
        dict(name="tree_b32_t64_len8128", op="tree", B=32, T=64, length=8128, n_kv=8, ragged=False),
        # a head shard (2 of the 8 kv heads) with a very wide tree
        dict(name="tree_b6_t150_len2000_kv2", op="tree", B=6, T=150, length=2000, n_kv=2, ragged=True),
        # after one user's verification, and after a server batch's
        dict(name="commit_b1_t8", op="commit", B=1, T=8, length=500, n_kv=8, ragged=False),
        dict(name="commit_b64_t64", op="commit", B=64, T=64, length=700, n_kv=8, ragged=True),
        # decode steps that keep count: one user, a ragged batch, a large batch
        dict(name="weights_b1_len700", op="weights", B=1, length=700, n_kv=8, ragged=False),
        dict(name="weights_b16_len4096", op="weights", B=16, length=4096, n_kv=8, ragged=True),
        dict(name="weights_b64_len8192", op="weights", B=64, length=8192, n_kv=8, ragged=False),
        # a prompt's cache cut down for one user, and a server batch halving its caches
        dict(name="evict_b1_len4100_to1024", op="evict", B=1, length=4100, n_kv=8, ragged=False, budget=1024, first=4,
             recent=32),
        dict(name="evict_b32_len8192_to4096", op="evict", B=32, length=8192, n_kv=8, ragged=True, budget=4096, first=4,
             recent=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "weights", "weights", "evict"])
    n_kv = rng.choice([8, 8, 8, 4, 2, 1])
    ragged = rng.random() < 0.6
    if op == "tree":
        T = _log_int(rng, 1, 256)
        length = _log_int(rng, 1, 32768)
        most = min(32 * 8192 // (length + T), 32 * 64 * 8192 // (T * (length + T)))
        return dict(op=op, B=_log_int(rng, 1, max(1, min(128, most))), T=T, length=length, n_kv=n_kv, ragged=ragged)
    if op == "commit":
        return dict(op=op, B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 64), length=_log_int(rng, 1, 700), n_kv=n_kv,
                    ragged=ragged)
    if op == "weights":
        length = _log_int(rng, 1, 65536)
        return dict(op=op, B=_log_int(rng, 1, max(1, min(128, 64 * 8192 // length))), length=length, n_kv=n_kv,
                    ragged=ragged)
    length = _log_int(rng, 40, 32768)
    budget = max(8, int(length * rng.uniform(0.1, 1.1)))
    first = rng.randint(0, min(8, budget // 2))
    recent = rng.randint(0, budget // 2)
    return dict(op=op, B=_log_int(rng, 1, max(1, min(64, 32 * 4096 // budget, 32 * 8192 // length))), length=length,
                n_kv=n_kv, ragged=ragged, budget=budget, first=first, recent=recent)


def _lengths(case):
    """Length of each sequence: the case's, or spread over 1 .. it."""
    if not case["ragged"]:
        return [case["length"]] * case["B"]
    return [max(1, int(round(case["length"] * ((0.37 + 0.6180339887 * (b + 1)) % 1.0)))) for b in range(case["B"])]


def _slots(case):
    """Cache positions per sequence: the longest sequence, its draft and some room."""
    return case["length"] + case.get("T", 0) + 5


def _drafted(case):
    """Drafted tokens of each sequence (the others of the T rows are padding)."""
    T = case["T"]
    return [T - (b * 7) % (T // 4 + 1) if case["ragged"] else T for b in range(case["B"])]


def _accepted(case):
    """Length of each sequence's accepted path."""
    return [min(n, (b * 5) % 9 if case["ragged"] else 4) for b, n in enumerate(_drafted(case))]


# -------------------------------------------------------------------------------- the inputs
def _trees(case, seed):
    """Visibility of a random draft tree per sequence: bool [B, T, T], row t = token t and its
    ancestors; padding rows see nothing and nothing sees them."""
    rng = np.random.default_rng(seed)
    B, T = case["B"], case["T"]
    vis = np.zeros((B, T, T), dtype=bool)
    drafted = np.array(_drafted(case))
    for t in range(T):
        parent = np.minimum(rng.integers(-1, max(t, 1), size=B), t - 1)
        has = parent >= 0
        vis[has, t] = vis[has, parent[has]]
        vis[:, t, t] = True
    live = np.arange(T)[None, :] < drafted[:, None]
    return vis & live[:, :, None] & live[:, None, :]


def _words(vis):
    """uint32 words [B, T, ceil(T/32)] (as int32) of the visibility bits."""
    B, T, _ = vis.shape
    W = (T + 31) // 32
    bits = np.zeros((B, T, W * 32), dtype=np.uint32)
    bits[:, :, :T] = vis
    words = (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
    return words.view(np.int32)


@functools.lru_cache(maxsize=None)
def _context(n_kv):
    """The library's handle for a block with n_kv kv heads, kept as a server keeps it."""
    from transformer_gqa_attention_gb300 import abi
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ctx = abi.attn_create_shard(z(512 * n_kv, 4096), z(128 * n_kv, 4096), z(128 * n_kv, 4096), z(4096, 512 * n_kv),
                                n_kv)
    torch.cuda.synchronize()
    return ctx


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, n_kv, S = case["B"], case["n_kv"], _slots(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    s = dict(op=case["op"], B=B, n_kv=n_kv, S=S, lens=ints(_lengths(case)), k=normal(B, S, n_kv, D),
             v=normal(B, S, n_kv, D))
    if case["op"] in ("tree", "weights"):
        T = case.get("T", 1)
        s["T"] = T
        s["q"] = normal(B, T, n_kv * HPG * D) * 1.5  # a few keys stand out in each row
        s["h"] = torch.zeros(B, T, n_kv * HPG * D, dtype=torch.bfloat16, device=DEV)
    if case["op"] == "tree":
        s["mask"] = torch.from_numpy(_words(_trees(case, seed))).to(DEV)
    if case["op"] == "commit":
        rng = np.random.default_rng(seed)
        path = np.zeros((B, case["T"]), dtype=np.int32)
        for b, (n, a) in enumerate(zip(_drafted(case), _accepted(case))):
            path[b, :a] = np.sort(rng.choice(n, size=a, replace=False))
        s |= dict(T=case["T"], path=ints(path), accepted=ints(_accepted(case)), new_lens=torch.zeros_like(s["lens"]))
    if case["op"] in ("weights", "evict"):
        # weights summed over earlier steps: heavy-tailed and positive
        s["w"] = torch.exp(2.0 * torch.randn(B, n_kv, S, generator=gen, device=DEV)) / case["length"]
    if case["op"] == "evict":
        O = case["budget"] + 64  # the cut cache keeps room for what is decoded next
        s |= dict(budget=case["budget"], first=case["first"], recent=case["recent"], O=O,
                  out_k=torch.zeros(B, O, n_kv, D, dtype=torch.bfloat16, device=DEV),
                  out_v=torch.zeros(B, O, n_kv, D, dtype=torch.bfloat16, device=DEV),
                  out_w=torch.zeros(B, n_kv, O, device=DEV),
                  kept=torch.zeros(B, n_kv, case["budget"], dtype=torch.int32, device=DEV),
                  new_lens=torch.zeros_like(s["lens"]))
    if own:
        s["ctx"] = _context(n_kv)
    return s


# ------------------------------------------------------------------------------- plain forms
def _rows(s):
    """Query rows per kv head [B, n_kv, T*4, 128] fp32 and keys, values [B, n_kv, S, 128] fp32."""
    B, T, n = s["B"], s["T"], s["n_kv"]
    q = s["q"].float().view(B, T, n, HPG, D).permute(0, 2, 1, 3, 4).reshape(B, n, T * HPG, D)
    return q, s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)


def _attend(s, visible):
    """(probabilities [B, n_kv, T*4, S], merged heads [B, T, n_kv*512]) of rows that see the keys
    of `visible` (broadcast to the probabilities' shape); a row that sees none gives zeros."""
    B, T, n = s["B"], s["T"], s["n_kv"]
    q, k, v = _rows(s)
    score = torch.matmul(q, k.transpose(2, 3)) * SCALE
    score = torch.where(visible, score, torch.full((), -math.inf, device=DEV))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    h = torch.matmul(p, v).view(B, n, T, HPG, D).permute(0, 2, 1, 3, 4).reshape(B, T, n * HPG * D)
    return p, h.to(torch.bfloat16)


def _plain_tree(s):
    B, T, S = s["B"], s["T"], s["S"]
    pos = torch.arange(S, device=DEV)
    j = pos[None, :] - s["lens"][:, None].long()  # drafted index of each position
    inside = (j >= 0) & (j < T)
    jc = j.clamp(0, T - 1)
    word = torch.gather(s["mask"], 2, (jc // 32)[:, None, :].expand(B, T, S))
    bit = (word >> (jc % 32)[:, None, :].int()) & 1
    visible = (j < 0)[:, None, :] | (inside[:, None, :] & (bit == 1))
    visible = visible[:, None, :, None, :].expand(B, 1, T, HPG, S).reshape(B, 1, T * HPG, S)
    s["h"].copy_(_attend(s, visible)[1])
    return s["h"]


def _plain_commit(s):
    B, T = s["B"], s["T"]
    i = torch.arange(T, device=DEV)[None, :]
    b = torch.arange(B, device=DEV)[:, None]
    src = torch.where(i < s["accepted"][:, None], s["path"].long(), i)  # the others stay where they are
    start = s["lens"][:, None].long()
    for c in (s["k"], s["v"]):
        c[b, start + i] = c[b, start + src]
    s["new_lens"].copy_(s["lens"] + s["accepted"])
    return s["k"], s["v"], s["new_lens"]


def _plain_weights(s):
    visible = (torch.arange(s["S"], device=DEV)[None, :] < s["lens"][:, None])[:, None, None, :]
    p, h = _attend(s, visible)
    s["w"] += p.sum(2)
    s["h"].copy_(h)
    return s["h"], s["w"]


def _plain_evict(s):
    B, n, S, m = s["B"], s["n_kv"], s["S"], s["budget"]
    pos = torch.arange(S, device=DEV)[None, None, :]
    lens = s["lens"][:, None, None]
    rank = torch.where((pos < s["first"]) | (pos >= lens - s["recent"]), torch.full((), math.inf, device=DEV), s["w"])
    rank = torch.where(pos < lens, rank, torch.full((), -math.inf, device=DEV))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :, :m]
    if order.shape[2] < m:
        order = torch.cat([order, order.new_full((B, n, m - order.shape[2]), S)], 2)
    live = torch.arange(m, device=DEV)[None, None, :] < torch.minimum(lens, torch.full_like(lens, m))
    order = torch.sort(torch.where(live, order, torch.full_like(order, S)), dim=-1).values
    pick = order.clamp(max=S - 1)
    for c, o in ((s["k"], s["out_k"]), (s["v"], s["out_v"])):
        rows = torch.gather(c.transpose(1, 2), 2, pick[..., None].expand(B, n, m, D)).transpose(1, 2)
        o[:, :m] = torch.where(live.transpose(1, 2)[..., None], rows, o[:, :m])
    s["out_w"].zero_()
    s["out_w"][:, :, :m] = torch.where(live, torch.gather(s["w"], 2, pick), torch.zeros((), device=DEV))
    s["kept"].copy_(torch.where(live, order, torch.full_like(order, -1)))
    s["new_lens"].copy_(s["lens"].clamp(max=m))
    return s["out_k"], s["out_v"], s["out_w"], s["kept"], s["new_lens"]


def _own(s):
    from transformer_gqa_attention_gb300 import abi
    if s["op"] == "tree":
        abi.attn_tree_attention(s["ctx"], s["q"], s["B"], s["T"], s["mask"], s["k"], s["v"], s["S"], s["lens"], s["h"])
        return s["h"]
    if s["op"] == "commit":
        abi.attn_cache_commit(s["ctx"], s["k"], s["v"], s["B"], s["S"], s["T"], s["lens"], s["path"], s["accepted"],
                              s["new_lens"])
        return s["k"], s["v"], s["new_lens"]
    if s["op"] == "weights":
        abi.attn_decode_attention_weights(s["ctx"], s["q"], s["k"], s["v"], s["B"], s["S"], s["lens"], s["w"], s["h"])
        return s["h"], s["w"]
    abi.attn_cache_evict(s["ctx"], s["k"], s["v"], s["w"], s["B"], s["S"], s["lens"], s["budget"], s["first"],
                         s["recent"], s["out_k"], s["out_v"], s["out_w"], s["O"], s["kept"], s["new_lens"])
    return s["out_k"], s["out_v"], s["out_w"], s["kept"], s["new_lens"]


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "commit": _plain_commit, "weights": _plain_weights, "evict": _plain_evict}[
        state["op"]](state)


# --------------------------------------------------------------------- what the path cannot avoid
def work(case):
    n, lens, B = case["n_kv"], _lengths(case), case["B"]
    kv = 2 * D * 2 * n  # bytes of one position's key and value
    head = n * HPG * D * 2
    if case["op"] == "tree":
        T = case["T"]
        keys = sum(lens) + T * B
        return dict(bytes=keys * kv + 2 * B * T * head + 4 * B * T * ((T + 31) // 32) + 4 * B,
                    flops=4.0 * D * HPG * n * T * keys)
    if case["op"] == "commit":
        moved = sum(_accepted(case))
        return dict(bytes=2 * moved * kv + 4 * moved + 12 * B, flops=0)
    if case["op"] == "weights":
        return dict(bytes=sum(lens) * (kv + 8 * n) + 2 * B * head + 4 * B, flops=4.0 * D * HPG * n * sum(lens))
    kept = sum(min(x, case["budget"]) for x in lens)
    room = B * (case["budget"] + 64)
    return dict(bytes=4 * n * sum(lens) + 2 * kept * kv + 4 * n * (room + B * case["budget"]) + 8 * B, flops=0)


# ------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    B, n, lens = case["B"], case["n_kv"], _lengths(case)
    f8 = torch.float64
    if case["op"] in ("tree", "weights"):
        T = s["T"]
        tree = torch.from_numpy(_trees(case, seed)).to(DEV) if case["op"] == "tree" else None
        h = torch.zeros(B, T, n, HPG, D, dtype=f8, device=DEV)
        w = s["w"].to(f8) if case["op"] == "weights" else None
        for b in range(B):
            L = lens[b] + (T if tree is not None else 0)
            for g in range(n):
                k, v = s["k"][b, :L, g].to(f8), s["v"][b, :L, g].to(f8)
                q = s["q"][b].to(f8).view(T, n, HPG, D)[:, g]
                e = torch.einsum("thd,sd->ths", q, k) / D ** 0.5
                if tree is not None:
                    e[:, :, lens[b]:].masked_fill_(~tree[b][:, None, :], -math.inf)
                a = torch.softmax(e, -1)
                if w is not None:
                    w[b, g, :L] += a.sum((0, 1))
                h[b, :, g] = torch.einsum("ths,sd->thd", a, v)
        h = h.view(B, T, n * HPG * D)
        return h if w is None else (h, w)
    if case["op"] == "commit":
        k, v, new = s["k"].to(f8), s["v"].to(f8), []
        for b, a in enumerate(_accepted(case)):
            at = [lens[b] + int(j) for j in s["path"][b, :a].cpu()]
            k[b, lens[b]:lens[b] + a] = k[b, at].clone()
            v[b, lens[b]:lens[b] + a] = v[b, at].clone()
            new.append(lens[b] + a)
        return k, v, torch.tensor(new, dtype=torch.int32)
    m, O = case["budget"], case["budget"] + 64
    out_k = torch.zeros(B, O, n, D, dtype=f8, device=DEV)
    out_v = torch.zeros_like(out_k)
    out_w = torch.zeros(B, n, O, dtype=f8, device=DEV)
    kept = np.full((B, n, m), -1, dtype=np.int32)
    weights = s["w"].cpu().numpy().astype(np.float64)
    for b, L in enumerate(lens):
        for g in range(n):
            take = np.arange(L)
            if L > m:
                edge = np.concatenate([take[:case["first"]], take[L - case["recent"]:]])
                middle = take[case["first"]:L - case["recent"]]
                by = np.lexsort((middle, -weights[b, g, middle]))[:m - case["first"] - case["recent"]]
                take = np.sort(np.concatenate([edge, middle[by]]))
            kept[b, g, :len(take)] = take
            at = torch.from_numpy(take).to(DEV)
            out_k[b, :len(take), g] = s["k"][b, at, g].to(f8)
            out_v[b, :len(take), g] = s["v"][b, at, g].to(f8)
            out_w[b, g, :len(take)] = s["w"][b, g, at].to(f8)
    return out_k, out_v, out_w, torch.from_numpy(kept), torch.tensor([min(x, m) for x in lens], dtype=torch.int32)

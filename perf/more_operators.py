"""Performance cases of the paged-cache operators: the rotation of queries by position, appending
keys and values to a paged cache with the rotation applied on the way, and the attention of one
new token per sequence over a paged cache.

``run`` computes an operator in its plain form (elementary fp32 torch operations, angles in fp64)
or, where ``own`` is true, through the library's entry points.  Sizes: 128-wide heads, 4 query
heads per kv head, 8 kv heads for the whole block (fewer for a head shard).  Pages are
[page, position, head, 128] or, where ``heads_first``, [page, head, position, 128]; they hold bf16
or, where ``e4m3``, 8-bit values with a scale for each head.
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
THETA = 500000.0
TOP8 = 448.0  # the largest e4m3 value

# context extension: every frequency divided by 4; by bands of wavelength (the block's scaled table);
# a ramp over the pairs, with the rotated part magnified
SCALINGS = {
    "plain": None,
    "linear": dict(factor=4.0),
    "bands": dict(factor=8.0, low=1.0, high=4.0, context=8192.0),
    "ramp": dict(factor=16.0, low=1.0, high=32.0, context=4096.0),
}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the queries of a decode step of 64 sequences: latency
        dict(name="rope_b64_heads32", op="rope", tokens=64, heads=32, rot=128, half=False, scaling="plain", top=4096),
        # the queries of a long prompt, frequencies scaled for a longer context
        dict(name="rope_t8192_heads32_bands", op="rope", tokens=8192, heads=32, rot=128, half=False, scaling="bands",
             top=131072),
        # keys of a ragged batch, half of the head rotated in halves, far positions
        dict(name="rope_t5001_heads8_half64_ramp", op="rope", tokens=5001, heads=8, rot=64, half=True, scaling="ramp",
             top=1000000),
        # a decode step's keys and values of 64 sequences of mixed lengths, small pages: latency
        dict(name="append_b64_t1_page16", op="append", B=64, T=1, length=4096, ragged=True, n_kv=8, page=16,
             e4m3=False, heads_first=False, rot=128, half=False, scaling="plain"),
        # prompts of mixed lengths into an 8-bit cache
        dict(name="append_b8_t2048_page64_e4m3", op="append", B=8, T=2048, length=1000, ragged=True, n_kv=8, page=64,
             e4m3=True, heads_first=True, rot=128, half=True, scaling="linear"),
        # whole prompts of a server batch: the most bytes moved
        dict(name="append_b4_t8192_page128", op="append", B=4, T=8192, length=0, ragged=False, n_kv=8, page=128,
             e4m3=False, heads_first=False, rot=128, half=False, scaling="bands"),
        # one chat user: latency
        dict(name="decode_b1_len700_page16", op="decode", B=1, length=700, ragged=False, n_kv=8, page=16, e4m3=False,
             heads_first=False),
        # a small server batch of mixed lengths
        dict(name="decode_b16_len4096_page16", op="decode", B=16, length=4096, ragged=True, n_kv=8, page=16,
             e4m3=False, heads_first=False),
        # a head shard (2 of the 8 kv heads), pages that are no power of two
        dict(name="decode_b24_len2000_page24_kv2", op="decode", B=24, length=2000, ragged=True, n_kv=2, page=24,
             e4m3=False, heads_first=True),
        # one long-context user with an 8-bit cache
        dict(name="decode_b1_len131000_page64_e4m3", op="decode", B=1, length=131000, ragged=False, n_kv=8, page=64,
             e4m3=True, heads_first=False),
        # a large server batch of mixed lengths with an 8-bit cache
        dict(name="decode_b64_len8192_page32_e4m3", op="decode", B=64, length=8192, ragged=True, n_kv=8, page=32,
             e4m3=True, heads_first=True),
        # a large server batch of full caches: the most work
        dict(name="decode_b64_len8192_page64", op="decode", B=64, length=8192, ragged=False, n_kv=8, page=64,
             e4m3=False, heads_first=False),
    ]


PAGES = (8, 16, 16, 24, 32, 48, 64, 64, 128, 256)


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "decode", "decode", "decode"])
    turn = dict(rot=rng.choice([128, 128, 128, 96, 64, 32, 16]), half=rng.random() < 0.4,
                scaling=rng.choice(list(SCALINGS)))
    if op == "rope":
        heads = rng.choice([32, 32, 16, 8, 5, 1])
        return dict(op=op, tokens=_log_int(rng, 1, min(65536, 8192 * 32 // heads)), heads=heads, **turn,
                    top=_log_int(rng, 16, 1000000))
    cache = dict(ragged=rng.random() < 0.6, n_kv=rng.choice([8, 8, 8, 4, 2, 1]), page=rng.choice(PAGES),
                 e4m3=rng.random() < 0.4, heads_first=rng.random() < 0.4)
    if op == "append":
        T = 1 if rng.random() < 0.3 else _log_int(rng, 2, 8192)
        return dict(op=op, B=_log_int(rng, 1, max(1, min(256, 32768 // T))), T=T, length=_log_int(rng, 1, 4096), **cache,
                    **turn)
    length = _log_int(rng, 1, 131072)
    return dict(op=op, B=_log_int(rng, 1, max(1, min(256, 64 * 8192 // length))), length=length, **cache)


def _spread(n, count, ragged, least):
    """`count` whole numbers: n each, or spread over least .. n."""
    if not ragged:
        return [n] * count
    return [max(least, int(round(n * ((0.37 + 0.6180339887 * (b + 1)) % 1.0)))) for b in range(count)]


def _lengths(case):
    """Positions that each sequence holds before the call."""
    return _spread(case["length"], case["B"], case["ragged"], 1 if case["op"] == "decode" else 0)


def _new(case):
    """New positions of each sequence (the others of the T rows are padding)."""
    return _spread(case["T"], case["B"], case["ragged"] and case["T"] > 1, 1)


def _holds(case):
    """Positions of each sequence that its pages have to hold."""
    if case["op"] == "decode":
        return _lengths(case)
    return [a + n for a, n in zip(_lengths(case), _new(case))]


# -------------------------------------------------------------------------------- the inputs
@functools.lru_cache(maxsize=None)
def _context(n_kv):
    """The library's handle for a block with n_kv kv heads, kept as a server keeps it."""
    from transformer_gqa_attention_gb300 import abi
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ctx = abi.attn_create_shard(z(512 * n_kv, 4096), z(128 * n_kv, 4096), z(128 * n_kv, 4096), z(4096, 512 * n_kv),
                                n_kv)
    torch.cuda.synchronize()
    return ctx


class _Handle:
    """The library's description of a paged cache, freed with the state that holds it."""

    def __init__(self, abi, *args):
        self.abi, self.p = abi, abi.attn_paged_create(*args)

    def __del__(self):
        self.abi.attn_paged_destroy(self.p)


def _rope_plan(case):
    from transformer_gqa_attention_gb300 import abi
    more = SCALINGS[case["scaling"]]
    return abi.attn_rope_init("halves" if case["half"] else "pairs", case["rot"], THETA,
                              case["scaling"] if more else None, **(more or {}))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    def ints(v):
        return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)

    s = dict(case)
    if case["op"] == "rope":
        n, h = case["tokens"], case["heads"]
        # the query columns of a fused projection's rows, which end in keys and values
        s["rows"] = normal(n, (h + 2 * max(1, h // HPG)) * D)
        s["x"] = s["rows"][:, :h * D]
        s["pos"] = ints(rng.integers(0, case["top"], size=n))
        s["out"] = torch.zeros(n, h * D, dtype=torch.bfloat16, device=DEV)
        s["freq"], s["gain"] = _frequencies(case)
        if own:
            s |= dict(ctx=_context(8), plan=_rope_plan(case))
        return s

    B, n, ps = case["B"], case["n_kv"], case["page"]
    need = [-(-h // ps) for h in _holds(case)]
    s["max_pages"] = max(1, max(need) + 1)
    s["n_pages"] = sum(need) + 3
    order, table, at = rng.permutation(s["n_pages"]), np.full((B, s["max_pages"]), -1), 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    s["table"] = ints(table)
    s["lens"] = ints(_lengths(case))
    shape = (s["n_pages"], n, ps, D) if case["heads_first"] else (s["n_pages"], ps, n, D)
    s["k"], s["v"] = normal(*shape), normal(*shape)
    s["k_scale"] = s["v_scale"] = None
    if case["e4m3"]:
        s["k"], s["v"] = ((16.0 * s[c]).to(torch.float8_e4m3fn) for c in "kv")
        s["k_scale"] = torch.rand(n, generator=gen, device=DEV) * 0.05 + 0.05
        s["v_scale"] = torch.rand(n, generator=gen, device=DEV) * 0.05 + 0.05
    if case["op"] == "append":
        # keys and values inside the rows of a fused projection
        s["rows"] = normal(B, case["T"], (HPG + 2) * n * D)
        s["new_k"] = s["rows"][:, :, HPG * n * D:(HPG + 1) * n * D]
        s["new_v"] = s["rows"][:, :, (HPG + 1) * n * D:]
        s["n_new"] = ints(_new(case))
        s["freq"], s["gain"] = _frequencies(case)
    else:
        s["q"] = normal(B, n * HPG * D) * 1.5  # a few keys stand out in each row
        s["h"] = torch.zeros(B, n * HPG * D, dtype=torch.bfloat16, device=DEV)
    if own:
        from transformer_gqa_attention_gb300 import abi
        st = s["k"].stride()
        per_pos, per_head = (st[2], st[1]) if case["heads_first"] else (st[1], st[2])
        s["ctx"] = _context(n)
        s["paged"] = _Handle(abi, s["ctx"], s["k"], s["v"], s["n_pages"], ps, "e4m3" if case["e4m3"] else "bf16", st[0],
                             per_pos, per_head, s["k_scale"], s["v_scale"])
        if case["op"] == "append":
            s["plan"] = _rope_plan(case)
    return s


# ------------------------------------------------------------------------------- plain forms
def _frequencies(case):
    """(radians per position [rot / 2] fp64, factor of the rotated part)."""
    rot, kind = case["rot"], case["scaling"]
    j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    w = THETA ** (-2.0 * j / rot)
    if kind == "plain":
        return w, 1.0
    c = SCALINGS[kind]
    if kind == "linear":
        return w / c["factor"], 1.0
    if kind == "bands":
        turns = c["context"] * w / (2.0 * math.pi)  # of the original context
        keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0.0, 1.0)
        return w * keep + w / c["factor"] * (1.0 - keep), 1.0
    pair = lambda turns: rot * math.log(c["context"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(THETA))  # noqa: E731
    lo, hi = max(math.floor(pair(c["high"])), 0), min(math.ceil(pair(c["low"])), rot - 1)
    slow = ((j - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return w / c["factor"] * slow + w * (1.0 - slow), 0.1 * math.log(c["factor"]) + 1.0


def _turned(x, pos, s):
    """x [..., heads, 128] fp32 rotated by pos [...]."""
    rot = s["rot"]
    angle = pos.double()[..., None] * s["freq"]
    cos = (torch.cos(angle) * s["gain"]).float()[..., None, :]
    sin = (torch.sin(angle) * s["gain"]).float()[..., None, :]
    if s["half"]:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    x = s["x"].float().view(s["tokens"], s["heads"], D)
    s["out"].copy_(_turned(x, s["pos"], s).reshape(s["tokens"], -1))
    return s["out"]


def _by_position(s, c):
    """A pool as [page, position, head, 128] (8-bit values as their bytes)."""
    p = s[c].view(torch.uint8) if s["e4m3"] else s[c]
    return p.transpose(1, 2) if s["heads_first"] else p


def _plain_append(s):
    B, T, n = s["B"], s["T"], s["n_kv"]
    t = torch.arange(T, device=DEV)[None, :]
    live = t < s["n_new"][:, None]
    pos = s["lens"][:, None].long() + t
    page = torch.gather(s["table"].long(), 1, (pos // s["page"]).clamp(max=s["max_pages"] - 1))
    k = _turned(s["new_k"].float().unflatten(-1, (n, D)), pos, s)
    v = s["new_v"].float().unflatten(-1, (n, D))
    for c, x in (("k", k), ("v", v)):
        if s["e4m3"]:
            x = (x / s[c + "_scale"][:, None]).clamp(-TOP8, TOP8).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = x.to(torch.bfloat16)
        _by_position(s, c)[page[live], (pos % s["page"])[live]] = x[live]
    return s["k"], s["v"]


def _plain_decode(s):
    B, n, S = s["B"], s["n_kv"], s["max_pages"] * s["page"]
    k, v = ((_by_position(s, c)[s["table"].long().clamp(min=0)]) for c in "kv")
    if s["e4m3"]:
        k, v = (x.view(torch.float8_e4m3fn) for x in (k, v))
    k, v = (x.float().reshape(B, S, n, D).transpose(1, 2) for x in (k, v))
    if s["e4m3"]:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    q = s["q"].float().view(B, n, HPG, D)
    score = torch.matmul(q, k.transpose(2, 3)) * SCALE
    seen = (torch.arange(S, device=DEV)[None, :] < s["lens"][:, None])[:, None, None, :]
    score = torch.where(seen, score, torch.full((), -math.inf, device=DEV))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    h = torch.matmul(p / p.sum(-1, keepdim=True), v)
    s["h"].copy_(h.reshape(B, -1))
    return s["h"]


def _own(s):
    from transformer_gqa_attention_gb300 import abi
    if s["op"] == "rope":
        abi.attn_rope_apply(s["ctx"], s["plan"], s["x"], s["tokens"], s["heads"], s["x"].stride(0), s["pos"], s["out"],
                            s["out"].stride(0))
        return s["out"]
    if s["op"] == "append":
        abi.attn_paged_append(s["ctx"], s["paged"].p, s["new_k"], s["new_v"], s["B"], s["T"], s["new_k"].stride(0),
                              s["new_k"].stride(1), s["plan"], None, s["table"], s["max_pages"], s["lens"], s["n_new"])
        return s["k"], s["v"]
    abi.attn_paged_decode_attention(s["ctx"], s["paged"].p, s["q"], s["B"], s["table"], s["max_pages"], s["lens"], s["h"])
    return s["h"]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode}[state["op"]](state)


# --------------------------------------------------------------------- what the path cannot avoid
def work(case):
    if case["op"] == "rope":
        values = case["tokens"] * case["heads"] * D
        return dict(bytes=4 * values + 4 * case["tokens"], flops=3.0 * values * case["rot"] / D)
    n, size = case["n_kv"], 1 if case["e4m3"] else 2
    entries = sum(-(-h // case["page"]) for h in _holds(case))
    if case["op"] == "append":
        new = sum(_new(case))
        pages = sum(-(-h // case["page"]) - a // case["page"] for a, h in zip(_lengths(case), _holds(case)))
        return dict(bytes=new * n * D * 2 * (2 + size) + 4 * pages + 8 * case["B"], flops=3.0 * new * n * case["rot"])
    keys = sum(_lengths(case))
    head = n * HPG * D * 2
    return dict(bytes=keys * n * D * 2 * size + 2 * case["B"] * head + 4 * entries + 4 * case["B"],
                flops=4.0 * D * HPG * n * keys)


# ------------------------------------------------------------------------ the definition in 64 bits
def _speeds(case):
    """Radians per position of each pair, pair by pair."""
    rot, c, w = case["rot"], SCALINGS[case["scaling"]], []
    for i in range(rot // 2):
        f = math.exp(-math.log(THETA) * 2 * i / rot)
        if case["scaling"] == "linear":
            f /= c["factor"]
        elif case["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > c["context"] / c["low"]:
                f /= c["factor"]
            elif wave >= c["context"] / c["high"]:
                m = (c["context"] / wave - c["low"]) / (c["high"] - c["low"])
                f = (1 - m) * f / c["factor"] + m * f
        elif case["scaling"] == "ramp":
            edge = [rot / 2 * math.log(c["context"] / (2 * math.pi * t)) / math.log(THETA) for t in (c["high"], c["low"])]
            a, b = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            m = min(max((i - a) / (b - a if b > a else 0.001), 0.0), 1.0)
            f = m * f / c["factor"] + (1 - m) * f
        w.append(f)
    return torch.tensor(w, dtype=torch.float64, device=DEV)


def _rotate64(x, at, case):
    """x [rows, heads, 128] fp64 as complex numbers times e^(i position speed)."""
    half, rot = case["rot"] // 2, case["rot"]
    gain = 1.0 if case["scaling"] != "ramp" else 1.0 + 0.1 * math.log(SCALINGS["ramp"]["factor"])
    angle = torch.outer(at.to(torch.float64), _speeds(case))[:, None, :]
    re = torch.arange(half, device=DEV) if case["half"] else torch.arange(0, rot, 2, device=DEV)
    im = re + (half if case["half"] else 1)
    z = torch.complex(x[:, :, re], x[:, :, im]) * torch.polar(torch.full_like(angle, gain), angle)
    y = x.clone()
    y[:, :, re], y[:, :, im] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    f8 = torch.float64
    if case["op"] == "rope":
        n, h = case["tokens"], case["heads"]
        return _rotate64(s["rows"][:, :h * D].to(f8).reshape(n, h, D), s["pos"], case).reshape(n, h * D)
    B, n, ps, table = case["B"], case["n_kv"], case["page"], s["table"].cpu().numpy()
    pools = {c: s[c].to(f8) for c in "kv"}
    by_pos = {c: p.permute(0, 2, 1, 3) if case["heads_first"] else p for c, p in pools.items()}
    if case["op"] == "append":
        cols = {"k": HPG * n * D, "v": (HPG + 1) * n * D}
        for b, (a, m) in enumerate(zip(_lengths(case), _new(case))):
            at = np.arange(a, a + m)
            page = torch.from_numpy(table[b, at // ps].astype(np.int64)).to(DEV)
            slot = torch.from_numpy(at % ps).to(DEV)
            for c in "kv":
                x = s["rows"][b, :m, cols[c]:cols[c] + n * D].to(f8).reshape(m, n, D)
                if c == "k":
                    x = _rotate64(x, torch.from_numpy(at).to(DEV), case)
                if case["e4m3"]:
                    x = torch.clip(x / s[c + "_scale"].to(f8)[None, :, None], -TOP8, TOP8)
                by_pos[c][page, slot] = x
        return pools["k"], pools["v"]
    out = torch.zeros(B, n, HPG, D, dtype=f8, device=DEV)
    for b, L in enumerate(_lengths(case)):
        pages = torch.from_numpy(table[b, :-(-L // ps)].astype(np.int64)).to(DEV)
        k, v = (by_pos[c][pages].reshape(-1, n, D)[:L] for c in "kv")
        if case["e4m3"]:
            k = k * s["k_scale"].to(f8)[None, :, None]
            v = v * s["v_scale"].to(f8)[None, :, None]
        e = torch.einsum("ghd,sgd->ghs", s["q"][b].to(f8).view(n, HPG, D), k) / D ** 0.5
        out[b] = torch.einsum("ghs,sgd->ghd", torch.softmax(e, -1), v)
    return out.view(B, n * HPG * D)

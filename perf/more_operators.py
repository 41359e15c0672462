"""Cases of the paged-cache operators: appending new tokens' keys and values to a
cache of pages with QK-norm and rotation on the way, and attention of the new
tokens over the pages, also where the streams of a batch share a long prefix.

A case is one call of a layer that generates video (or reads prompts) over kept
keys.  `q_lens` are the new tokens of each stream, packed one behind another,
`pad` rows follow the last one; `k_lens` are the keys that each stream has once
the new ones are in its cache.  The cache is a pool of pages of `page` tokens,
[pages][page][kv_heads][d], or with the heads ahead of a page's tokens in memory
(`heads_first`); a table names the pages of each stream, in order.  `block` is
the mask: 0 every key of the stream, 1 causal, F > 1 causal by frames of F
tokens, the queries being the newest tokens.  `groups` (streams in each group)
and `shared` (tokens) say that the streams of a group have their first tokens in
common: whole pages of them are the same pages, a last one begun is a copy.

`run` computes a case in its plain form, or, where `own` is true, by the calls
of video_dit_long_gb300.  `exact` gives the same in 64 bits.
"""
import torch

own = False

D = 128
AXES = (32, 48, 48)
THETA = 10000.0
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one new token in each of eight running streams: launch latency
        dict(name="append_tokens", op="append", q_lens="1,1,1,1,1,1,1,1", k_lens="1,52360,300,8192,129,26440,5000,4352",
             heads=24, kv_heads=8, page=16, heads_first=False, qk="f16", pad=0),
        # the next frame (432 tokens of the Lite grid) of six streams, and a prompt that starts a seventh
        dict(name="append_frames", op="append", q_lens="432,432,432,432,432,432,77",
             k_lens="432,864,3024,10800,20736,1296,77", heads=24, kv_heads=4, page=48, heads_first=True, qk="bf16", pad=24),
        # the Pro clip (52,360 tokens) read into an empty cache
        dict(name="append_pro", op="append", q_lens="52360", k_lens="52360", heads=24, kv_heads=8, page=64,
             heads_first=False, qk="f16", pad=0),
        # the smallest attention call: one token each of three short streams
        dict(name="tokens_short", op="attention", q_lens="1,1,1", k_lens="77,300,130", heads=24, kv_heads=8, page=16,
             heads_first=False, block=1, qk="f16", pad=0, groups="", shared=""),
        # one new token for each of twelve streams whose caches are from one token to the Pro length
        dict(name="tokens", op="attention", q_lens="1,1,1,1,1,1,1,1,1,1,1,1",
             k_lens="1,52360,300,8192,129,26440,5000,4352,1000,3152,12345,20000", heads=24, kv_heads=4, page=64,
             heads_first=False, block=1, qk="f16", pad=0, groups="", shared=""),
        # two streams that generate a frame at a time over the frames kept so far
        dict(name="next_frame", op="attention", q_lens="432,432", k_lens="3024,10800", heads=24, kv_heads=8, page=16,
             heads_first=True, block=432, qk="f16", pad=0, groups="", shared=""),
        # a serving step: two prompts, the rest of a third, and running streams, 24 key heads
        dict(name="mixed_step", op="attention", q_lens="512,77,300,1,1,1,5,1", k_lens="512,77,1300,4352,1,3152,2000,129",
             heads=24, kv_heads=24, page=32, heads_first=False, block=1, qk="bf16", pad=24, groups="", shared=""),
        # the second half of a long clip (8 of 16 frames of 30 x 54 tokens) over its first, causal by frames
        dict(name="half_clip", op="attention", q_lens="12960", k_lens="25920", heads=24, kv_heads=8, page=128,
             heads_first=False, block=1620, qk="f16", pad=0, groups="", shared=""),
        # thirty-two samples of one conditioning clip (16 frames of the Pro grid), one new token each
        dict(name="shared_tokens", op="attention", q_lens=",".join(["1"] * 32),
             k_lens=",".join(str(25921 + 37 * n) for n in range(32)), heads=24, kv_heads=8, page=64, heads_first=False,
             block=1, qk="f16", pad=0, groups="32", shared="25920"),
        # two prompts of 4,352 and 1,081 tokens with eight and five samples each, five tokens a step, one stream alone
        dict(name="shared_steps", op="attention", q_lens="5,5,5,5,5,5,5,5,5,5,5,5,5,5",
             k_lens="4357,4500,5000,4400,4700,4900,6000,4358,1086,1100,1500,1200,1300,2500", heads=24, kv_heads=4, page=16,
             heads_first=True, block=1, qk="f16", pad=3, groups="8,5,1", shared="4352,1081,0"),
        # six samples of one Lite clip (3,024 tokens) that generate their next frame
        dict(name="shared_frames", op="attention", q_lens="432,432,432,432,432,432",
             k_lens="3456,3888,4320,3456,5184,3456", heads=24, kv_heads=8, page=48, heads_first=False, block=432, qk="bf16",
             pad=0, groups="6", shared="3024"),
    ]


def _loguniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kv_heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 24])
    case = dict(op=rng.choice(["append", "append", "attention", "attention", "shared", "shared"]), heads=24,
                kv_heads=kv_heads, page=rng.choice([16, 16, 32, 48, 64, 64, 112, 128, 256]),
                heads_first=rng.random() < 0.4, qk=rng.choice(["f16", "f16", "bf16"]),
                pad=rng.choice([0, 0, rng.randint(1, 40)]))
    text = lambda v: ",".join(str(x) for x in v)  # noqa: E731
    if case["op"] == "append":
        n = _loguniform(rng, 1, 40)
        q = [_loguniform(rng, 1, max(1, 52360 // n)) for _ in range(n)]
        k = [x + (0 if rng.random() < 0.3 else _loguniform(rng, 1, 4000)) for x in q]
        if n > 2 and rng.random() < 0.3:
            q[1] = 0  # a stream that has nothing new
        return {**case, "q_lens": text(q), "k_lens": text(k)}
    block = rng.choice([0, 1, 1, 1, rng.randint(2, 300), 432, 1620])
    if case["op"] == "attention":
        n = _loguniform(rng, 1, 24)
        new = rng.choice([1, 1, 600, 4000 // n + 1])  # single tokens, or up to that many
        k = [_loguniform(rng, rng.choice([1, 1000]), 52360 // (n if new > 600 else 1 + n // 8)) for _ in range(n)]
        q = [max(1, min(_loguniform(rng, 1, new), x + (3 if rng.random() < 0.1 else 0))) for x in k]
        if n > 2 and rng.random() < 0.2:  # a stream that has nothing new, or nothing at all
            q[1] = 0
            if rng.random() < 0.5:
                k[1] = 0
        groups, shared = [], []
    else:
        groups = [_loguniform(rng, 1, 24) for _ in range(rng.choice([1, 1, 2, 3]))]
        shared = [_loguniform(rng, rng.choice([1, 1000]), 40000 // len(groups)) for _ in groups]
        n, new = sum(groups), rng.choice([1, 1, 7, 60])
        q = [_loguniform(rng, 1, new) for _ in range(n)]
        k = [s + a + rng.choice([0, 1, _loguniform(rng, 1, 1500)])
             for s, a in zip([s for s, g in zip(shared, groups) for _ in range(g)], q)]
        if rng.random() < 0.2:  # a stream whose new tokens begin inside the prefix
            q[0] = min(k[0], q[0] + 200)
    return {**case, "op": "attention", "q_lens": text(q), "k_lens": text(k), "block": block, "groups": text(groups),
            "shared": text(shared)}


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _group_of(case):
    """For each stream the first one of its group and the tokens that the group shares."""
    n, of = len(_ints(case["q_lens"])), []
    for streams, shared in zip(_ints(case.get("groups", "")), _ints(case.get("shared", ""))):
        of += [(len(of), shared)] * streams
    return of + [(s, 0) for s in range(len(of), n)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = dict(case)
    H, Hkv, page, x = case["heads"], case["kv_heads"], case["page"], TYPES[case["qk"]]
    q_lens, k_lens = _ints(case["q_lens"]), _ints(case["k_lens"])
    n, T = len(q_lens), sum(q_lens) + case["pad"]
    # the pages of each stream, scattered over the pool; those that a group shares are the first stream's
    wanted = [-(-k // page) for k in k_lens]
    group = _group_of(case)
    fresh = [w - (0 if first == i else min(w, shared // page)) for i, (w, (first, shared)) in enumerate(zip(wanted, group))]
    n_pages = sum(fresh) + 3
    free = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, max(wanted) + 1), -1, dtype=torch.int32, device="cuda")
    copies, at = [], 0
    for i, (w, f, (first, shared)) in enumerate(zip(wanted, fresh, group)):
        table[i, :w - f] = table[first, :w - f]
        table[i, w - f:w] = free[at:at + f]
        if first != i and shared % page and w > shared // page:
            copies.append((first, i, shared // page))
        at += f

    def pool(dtype):
        if case["heads_first"]:
            return normal(n_pages, Hkv, page, D, dtype=dtype).transpose(1, 2)
        return normal(n_pages, page, Hkv, D, dtype=dtype)

    s["k_cache"], s["v_cache"] = pool(x), pool(torch.bfloat16)
    for first, i, j in copies:  # the page that the shared tokens end in, copied for each stream
        for c in (s["k_cache"], s["v_cache"]):
            c[table[i, j].long()] = c[table[first, j].long()]
    s["table"] = table
    s["cu_q"] = torch.tensor(_offsets(q_lens), dtype=torch.int32, device="cuda")
    s["k_now"] = torch.tensor(k_lens, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        qkv = normal(T, H + 2 * Hkv, D, dtype=torch.bfloat16)  # the layer's fused projection; q, k and v are views of it
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        i = torch.zeros(T, dtype=torch.int64, device="cuda")  # each token's place in its stream: a grid of 30 x 54 a frame
        for c, a, b in zip(_offsets(q_lens), q_lens, k_lens):
            i[c:c + a] = torch.arange(b - a, b, device="cuda")
        s["positions"] = torch.stack((i // 1620, i // 54 % 30, i % 54), 1).to(torch.int32)
        s["q_weight"], s["k_weight"] = normal(D, std=0.2, mean=1.0), normal(D, std=0.2, mean=1.0)
        s["q_out"] = torch.zeros((T, H, D), dtype=x, device="cuda")
    else:
        s["q"] = normal(T, H, D, dtype=x)
    if own:
        from video_dit_long_gb300 import k6attn
        h = s["handle"] = k6attn.Handle.for_packed(H, D, "bf16", AXES, THETA)
        more = {}
        if case.get("groups"):
            more["cu_groups"] = torch.tensor(_offsets(_ints(case["groups"])), dtype=torch.int32, device="cuda")
            more["shared"] = torch.tensor(_ints(case["shared"]), dtype=torch.int32, device="cuda")
        plan = s["plan"] = h.paged_plan(s["cu_q"], s["k_now"], table, T, Hkv, page, n_pages, case.get("block", 1), **more)
        if case["op"] == "attention":
            s["out"] = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.zeros((H, T), dtype=torch.float32, device="cuda")
            s["workspace"] = torch.empty(h.paged_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    if own:
        h = s["handle"]
        if s["op"] == "append":
            h.paged_append(s["plan"], s["q"], s["k"], s["v"], s["positions"], s["q_weight"], s["k_weight"], EPS,
                           q_out=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        h.paged_forward(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["out"], s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    return _append(s) if s["op"] == "append" else _attention(s)


# ------------------------------------------------------------- the plain forms

def _append(s):
    freq = torch.cat([THETA ** (-torch.arange(0, a, 2, dtype=torch.float64, device="cuda") / a) for a in AXES])
    axis = torch.cat([torch.full((a // 2,), n, device="cuda") for n, a in enumerate(AXES)])
    angle = s["positions"].double()[:, axis] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2).to(TYPES[s["qk"]])

    q_lens, k_lens = _ints(s["q_lens"]), _ints(s["k_lens"])
    n = sum(q_lens)
    s["q_out"][:n] = turned(s["q"], s["q_weight"])[:n]
    k = turned(s["k"], s["k_weight"])
    for i, (c, a, b) in enumerate(zip(_offsets(q_lens), q_lens, k_lens)):
        at = torch.arange(b - a, b, device="cuda")
        pages, slots = s["table"][i].long()[at // s["page"]], at % s["page"]
        s["k_cache"][pages, slots] = k[c:c + a]
        s["v_cache"][pages, slots] = s["v"][c:c + a]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attention(s):
    H, Hkv, page = s["heads"], s["kv_heads"], s["page"]
    G = H // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((H, s["q"].shape[0]), dtype=torch.float32, device="cuda")
    q_lens, k_lens = _ints(s["q_lens"]), _ints(s["k_lens"])
    for i, (c, Lq, Lk) in enumerate(zip(_offsets(q_lens), q_lens, k_lens)):
        rows = slice(c, c + Lq)
        if not Lk:
            lse[:, rows] = float("-inf")
        if not Lk or not Lq:
            continue
        pages = s["table"][i, :-(-Lk // page)].long()
        keys = s["k_cache"][pages].reshape(-1, Hkv, D)[:Lk].float()
        values = s["v_cache"][pages].reshape(-1, Hkv, D)[:Lk].float()
        seen = None
        if s["block"]:
            at = torch.arange(Lk - Lq, Lk, device="cuda")
            seen = torch.arange(Lk, device="cuda") < ((torch.div(at, s["block"], rounding_mode="floor") + 1) * s["block"])[:, None]
        for j in range(Hkv):
            hs = slice(j * G, (j + 1) * G)
            x = (s["q"][rows, hs].float().transpose(0, 1) @ keys[:, j].T) * D ** -0.5  # [G][Lq][Lk]
            if seen is not None:
                x.masked_fill_(~seen, float("-inf"))
            m = x.amax(-1, keepdim=True)
            p = x.sub_(m.clamp(min=torch.finfo(torch.float32).min)).exp_()  # a row that sees nothing: 0
            l = p.sum(-1, keepdim=True)
            out[rows, hs] = ((p @ values[:, j]) / l.clamp(min=1e-30)).transpose(0, 1).to(torch.bfloat16)
            lse[hs, rows] = (m + l.log())[..., 0]
    return {"out": out, "lse": lse}


# ------------------------------------------------------------- in 64 bits

def _limits(Lq, Lk, block):
    """Keys that each of the Lq newest tokens of a stream of Lk keys sees."""
    return [Lk if block == 0 else max(0, min(Lk, ((i + Lk - Lq) // block + 1) * block)) for i in range(Lq)]


def exact(case, seed):
    global own
    if case["op"] == "attention" and 512.0 * case["heads"] * _pairs(case) > 4e12:
        return None
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _rows_of(s, i, first, last):
    """Places in the flattened pool of stream i's tokens [first, last)."""
    at = torch.arange(first, last, device="cuda")
    return s["table"][i].long().gather(0, at // s["page"]) * s["page"] + at % s["page"]


def _exact_append(s):
    """The rotation as a complex product by exp(i angle), the caches as flat rows."""
    freq = [THETA ** (-2.0 * i / a) for a in AXES for i in range(a // 2)]
    axis = [n for n, a in enumerate(AXES) for _ in range(a // 2)]
    angle = s["positions"].double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    z = {}
    for n in "qk":
        x = s[n].double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * s[n + "_weight"].double()
        z[n] = torch.view_as_real(torch.view_as_complex(y.unflatten(-1, (D // 2, 2)).contiguous()) * turn).flatten(-2)
    q_lens, k_lens = _ints(s["q_lens"]), _ints(s["k_lens"])
    q = s["q_out"].double()
    q[:sum(q_lens)] = z["q"][:sum(q_lens)]
    k, v = (s[n].double().flatten(0, 1) for n in ("k_cache", "v_cache"))
    for i, (c, a, b) in enumerate(zip(_offsets(q_lens), q_lens, k_lens)):
        to = _rows_of(s, i, b - a, b)
        k.index_copy_(0, to, z["k"][c:c + a])
        v.index_copy_(0, to, s["v"][c:c + a].double())
    return {"q": q, "k_cache": k.view(s["k_cache"].shape), "v_cache": v.view(s["v_cache"].shape)}


def _exact_attention(s):
    """One query head after another, blocks of query rows at a time, over keys fetched one by one."""
    H, G = s["heads"], s["heads"] // s["kv_heads"]
    q_lens, k_lens = _ints(s["q_lens"]), _ints(s["k_lens"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((H, s["q"].shape[0]), dtype=torch.float64, device="cuda")
    for i, (c, Lq, Lk) in enumerate(zip(_offsets(q_lens), q_lens, k_lens)):
        if not Lk:
            lse[:, c:c + Lq] = float("-inf")
            continue
        rows = _rows_of(s, i, 0, Lk)
        last = torch.tensor(_limits(Lq, Lk, s["block"]), dtype=torch.int64, device="cuda")[:, None]
        keys, values = (s[n].flatten(0, 1)[rows].double() for n in ("k_cache", "v_cache"))
        for h in range(H):
            for a in range(0, Lq, 2048):
                r = slice(c + a, c + min(a + 2048, Lq))
                logits = s["q"][r, h].double() @ keys[:, h // G].T / D ** 0.5
                hidden = torch.arange(Lk, device="cuda") >= last[a:a + 2048]
                logits[hidden] = float("-inf")
                lse[h, r] = torch.logsumexp(logits, -1)
                w = torch.exp(logits - lse[h, r][:, None])
                w[hidden] = 0.0
                out[r, h] = w @ values[:, h // G]
    return {"out": out, "lse": lse}


# ------------------------------------------------------------- what a pass cannot do without

def _pairs(case):
    return sum(sum(_limits(a, b, case["block"])) for a, b in zip(_ints(case["q_lens"]), _ints(case["k_lens"])))


def work(case):
    H, Hkv = case["heads"], case["kv_heads"]
    q_lens, k_lens = _ints(case["q_lens"]), _ints(case["k_lens"])
    T = sum(q_lens)
    if case["op"] == "append":  # each row of q, k and v read and written; positions; weights
        return {"bytes": T * (2 * (H + 2 * Hkv) * D * 2 + 12) + 2 * D * 4, "flops": T * (H + Hkv) * D * 7}
    # the keys that some query sees, those of a shared prefix once
    keys, prefix = 0, {}
    for a, b, (first, shared) in zip(q_lens, k_lens, _group_of(case)):
        seen = max(_limits(a, b, case["block"]), default=0)
        prefix[first] = max(prefix.get(first, 0), min(seen, shared))
        keys += max(0, seen - shared)
    keys += sum(prefix.values())
    return {"bytes": 2 * T * H * D * 2 + T * H * 4 + 2 * keys * Hkv * D * 2, "flops": 4.0 * D * H * _pairs(case)}

"""Cases of the packed-sequence operators: per-head QK-norm with multi-axis rotary
positions (forward and backward), and attention over packed sequences with
grouped heads (forward and backward).

A case is one call as a layer of a video diffusion transformer makes it.  Clips
(and prompts, and new tokens of running streams) of different lengths lie one
behind another in one [tokens][heads][d] tensor; `q_lens` and `k_lens` are their
lengths, `pad` rows follow the last one.  `block` is the mask: 0 every key of
the sequence, 1 causal, F > 1 causal by frames of F tokens (a token sees its
own frame and those before it).  Where k is longer than q, the queries are the
newest tokens of the sequence.

`run` computes a case in its plain form, or, where `own` is true, by the calls
of video_dit_long_gb300.  `exact` gives the same in 64 bits.
"""
import numpy as np
import torch

own = False

THETA = 10000.0
EPS = 1e-6
AXES = {128: (32, 48, 48), 64: (16, 24, 24)}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one new token in each of eight running streams, 24 query and 8 key heads: launch latency
        dict(name="norm_rope_tokens", op="norm_rope", tokens=8, heads=24, kv_heads=8, d=128, dtype="bf16", out="f16",
             far=100000, pad=0),
        # the 1024-video-token fp32 configuration with an odd row more: fp32 in and out, d = 64, rotation and norm
        dict(name="norm_rope_f32", op="norm_rope", tokens=1089, heads=4, kv_heads=4, d=64, dtype="f32", out="f32",
             far=0, pad=0),
        # the Pro clip (52,360 tokens), q and k read out of a fused projection, rotated copies in fp16
        dict(name="norm_rope_pro", op="norm_rope", tokens=52360, heads=24, kv_heads=8, d=128, dtype="bf16", out="f16",
             far=0, pad=0),
        # training on one Lite clip: gradients through rotation and norm, and of the norm's weights
        dict(name="norm_rope_bwd_lite", op="norm_rope_backward", tokens=3152, heads=24, kv_heads=8, d=128,
             dtype="bf16", out="f16", far=0, pad=0),
        # the same on the Pro clip, every query head with a key head of its own
        dict(name="norm_rope_bwd_pro", op="norm_rope_backward", tokens=52360, heads=24, kv_heads=24, d=128,
             dtype="bf16", out="f16", far=0, pad=0),
        # the smallest call: three short prompts packed for one causal pass, one of them a single token
        dict(name="attn_short", op="attention", q_lens="77,1,130", k_lens="77,1,130", heads=24, kv_heads=8, block=1,
             qk="bf16", pad=0),
        # one new token for each of twelve streams whose caches are from one token to the Pro length
        dict(name="attn_tokens", op="attention", q_lens="1,1,1,1,1,1,1,1,1,1,1,1",
             k_lens="1,52360,300,8192,129,26440,5000,4352,1000,3152,12345,20000", heads=24, kv_heads=4, block=1,
             qk="f16", pad=0),
        # two streams that generate a frame at a time (432 tokens of the Lite grid) over the frames kept so far
        dict(name="attn_next_frame", op="attention", q_lens="432,432", k_lens="3024,10800", heads=24, kv_heads=8,
             block=432, qk="f16", pad=0),
        # a training batch of clips, images and prompts of different lengths, causal, eight key heads
        dict(name="attn_mixed_causal", op="attention", q_lens="4352,3152,1081,257,77,1", k_lens="4352,3152,1081,257,77,1",
             heads=24, kv_heads=8, block=1, qk="f16", pad=24),
        # one long clip, causal by frames of 30 x 54 tokens (16 frames of the Pro grid)
        dict(name="attn_mid_frames", op="attention", q_lens="25920", k_lens="25920", heads=24, kv_heads=8, block=1620,
             qk="f16", pad=0),
        # the gradients of a small and a ragged batch: full attention over packed clips, 24 key heads
        dict(name="attn_bwd_mixed", op="attention_backward", q_lens="3152,1081,257,77,1", k_lens="3152,1081,257,77,1",
             heads=24, kv_heads=24, block=0, qk="f16", pad=24),
        # the gradients of the long clip, causal by frames
        dict(name="attn_bwd_mid_frames", op="attention_backward", q_lens="25920", k_lens="25920", heads=24, kv_heads=8,
             block=1620, qk="f16", pad=0),
    ]


def _loguniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_backward", "attention", "attention", "attention_backward"])
    kv_heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 24])
    if op.startswith("norm_rope"):
        d = rng.choice([128, 128, 128, 64])
        dtype = "bf16" if d == 128 and rng.random() < 0.8 else "f32"
        return dict(op=op, tokens=_loguniform(rng, 1, 52360), heads=24, kv_heads=kv_heads, d=d, dtype=dtype,
                    out="f32" if dtype == "f32" else rng.choice(["f16", "bf16"]),
                    far=rng.choice([0, _loguniform(rng, 1000, 1000000)]), pad=rng.choice([0, 0, rng.randint(1, 40)]))
    n = _loguniform(rng, 1, 16)
    most = 18000 // n  # tokens of one sequence: a batch, unmasked too, costs less than the long clip
    block = rng.choice([0, 1, 1, rng.randint(2, 300), 432, 1620])
    kind = rng.choice(["packed", "packed", "packed", "step"]) if op == "attention" else rng.choice(["packed"] * 4 + ["step"])
    k_lens = [_loguniform(rng, 1, most) for _ in range(n)]
    if kind == "packed":
        q_lens = list(k_lens)
    else:  # new tokens after cached ones; now and then more queries than keys
        q_lens = [max(1, min(_loguniform(rng, 1, 600), k + (3 if rng.random() < 0.1 else 0))) for k in k_lens]
    if n > 2 and rng.random() < 0.2:  # an empty sequence in the batch
        q_lens[1] = 0
        if rng.random() < 0.5:
            k_lens[1] = 0
    text = lambda v: ",".join(str(x) for x in v)  # noqa: E731
    return dict(op=op, q_lens=text(q_lens), k_lens=text(k_lens), heads=24, kv_heads=kv_heads, block=block,
                qk=rng.choice(["f16", "f16", "bf16"]), pad=rng.choice([0, 0, rng.randint(1, 200)]))


def _lens(text):
    return [int(x) for x in text.split(",")]


def _offsets(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def _limits(Lq, Lk, block):
    """Keys that each of the Lq newest tokens of a sequence of Lk keys sees."""
    if block == 0:
        return np.full(Lq, Lk, np.int64)
    return np.clip(((np.arange(Lq, dtype=np.int64) + (Lk - Lq)) // block + 1) * block, 0, Lk)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = dict(case)
    H, Hkv = case["heads"], case["kv_heads"]
    if case["op"].startswith("norm_rope"):
        d, T = case["d"], case["tokens"] + case["pad"]
        x, y = TYPES[case["dtype"]], TYPES[case["out"]]
        qkv = normal(T, H + 2 * Hkv, d, dtype=x)  # the layer's fused projection; q and k are views of it
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        i = torch.arange(T, device="cuda", dtype=torch.int64)  # row-major grid of 30 x 54 tokens a frame
        s["positions"] = torch.stack((i // 1620 + case["far"], i // 54 % 30, i % 54), 1).to(torch.int32)
        s["q_weight"], s["k_weight"] = normal(d, std=0.2, mean=1.0), normal(d, std=0.2, mean=1.0)
        if case["op"] == "norm_rope_backward":
            gt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
            s["dq_out"], s["dk_out"] = normal(T, H, d, dtype=gt), normal(T, Hkv, d, dtype=gt)
        if own:
            from video_dit_long_gb300 import k6attn
            h = s["handle"] = k6attn.Handle.for_packed(H, d, case["dtype"], AXES[d], THETA)
            if case["op"] == "norm_rope":
                s["q_out"] = torch.empty((T, H, d), dtype=y, device="cuda")
                s["k_out"] = torch.empty((T, Hkv, d), dtype=y, device="cuda")
            else:
                s["dq"], s["dk"] = torch.empty_like(s["dq_out"]), torch.empty_like(s["dk_out"])
                s["dq_weight"], s["dk_weight"] = torch.empty_like(s["q_weight"]), torch.empty_like(s["k_weight"])
                s["workspace"] = torch.empty(h.packed_norm_rope_backward_workspace_bytes(T, Hkv), dtype=torch.uint8,
                                             device="cuda")
        return s
    d = 128
    cu_q, cu_k = _offsets(_lens(case["q_lens"])), _offsets(_lens(case["k_lens"]))
    Tq, Tk = cu_q[-1] + case["pad"], cu_k[-1] + case["pad"]
    x = TYPES[case["qk"]]
    s["q"], s["k"] = normal(Tq, H, d, dtype=x), normal(Tk, Hkv, d, dtype=x)
    s["v"] = normal(Tk, 2 * Hkv, d, dtype=torch.bfloat16)[:, Hkv:]  # a view of the fused projection
    s["cu_q"] = torch.tensor(cu_q, dtype=torch.int32, device="cuda")
    s["cu_k"] = torch.tensor(cu_k, dtype=torch.int32, device="cuda")
    if case["op"] == "attention_backward":
        s["out"], s["lse"] = _attention(s)  # what the forward pass left
        s["dout"] = normal(Tq, H, d, dtype=torch.bfloat16)
    if own:
        from video_dit_long_gb300 import k6attn
        h = s["handle"] = k6attn.Handle.for_packed(H, d, "bf16", AXES[d], THETA)
        plan = s["plan"] = h.packed_plan(s["cu_q"], s["cu_k"], Tq, Tk, Hkv, case["block"])
        if case["op"] == "attention":
            s["out"] = torch.zeros((Tq, H, d), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.zeros((H, Tq), dtype=torch.float32, device="cuda")
            s["workspace"] = torch.empty(h.packed_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
        else:
            s["dq"] = torch.zeros((Tq, H, d), dtype=torch.bfloat16, device="cuda")
            s["dk"] = torch.zeros((Tk, Hkv, d), dtype=torch.bfloat16, device="cuda")
            s["dv"] = torch.zeros((Tk, Hkv, d), dtype=torch.bfloat16, device="cuda")
            s["workspace"] = torch.empty(h.packed_backward_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm_rope":
        return _norm_rope(s)
    if s["op"] == "norm_rope_backward":
        return _norm_rope_backward(s)
    if s["op"] == "attention":
        out, lse = _attention(s)
        return {"out": out, "lse": lse}
    return _attention_backward(s)


def _run_own(s):
    h = s["handle"]
    if s["op"] == "norm_rope":
        h.packed_norm_rope(s["q"], s["k"], s["positions"], s["q_weight"], s["k_weight"], EPS, q_out=s["q_out"],
                           k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "norm_rope_backward":
        h.packed_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["positions"], s["q_weight"],
                                    s["k_weight"], EPS, dq=s["dq"], dk=s["dk"], dq_weight=s["dq_weight"],
                                    dk_weight=s["dk_weight"], workspace=s["workspace"])
        return {"dq": s["dq"], "dk": s["dk"], "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]}
    if s["op"] == "attention":
        h.packed_forward(s["plan"], s["q"], s["k"], s["v"], s["out"], s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    h.packed_backward(s["plan"], s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], s["dq"], s["dk"], s["dv"],
                      workspace=s["workspace"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


# ------------------------------------------------------------- the plain forms

def _cos_sin(positions, d):
    """cos and sin of every pair of a head, [tokens][1][d / 2]; the angles in 64 bits."""
    freq = torch.cat([THETA ** (-torch.arange(0, a, 2, dtype=torch.float64, device="cuda") / a) for a in AXES[d]])
    axis = torch.cat([torch.full((a // 2,), n, device="cuda") for n, a in enumerate(AXES[d])])
    angle = positions.double()[:, axis] * freq
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _norm_rope(s):
    cos, sin = _cos_sin(s["positions"], s["d"])

    def one(x, w):
        x = x.float()
        y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2).to(TYPES[s["out"]])

    return {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"])}


def _norm_rope_backward(s):
    cos, sin = _cos_sin(s["positions"], s["d"])

    def one(g, x, w):
        g, x, t = g.float(), x.float(), g.dtype
        a, b = g[..., 0::2], g[..., 1::2]
        gy = torch.stack((a * cos + b * sin, b * cos - a * sin), -1).flatten(-2)  # the rotation turned back
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        xh, gx = x * r, gy * w
        dx = r * (gx - xh * (gx * xh).mean(-1, keepdim=True))
        return dx.to(t), (gy * xh).sum((0, 1), dtype=torch.float64).float()

    dq, dqw = one(s["dq_out"], s["q"], s["q_weight"])
    dk, dkw = one(s["dk_out"], s["k"], s["k_weight"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _parts(s):
    """(query rows, key rows, mask or None) of each sequence of the batch that has queries or keys."""
    q_lens, k_lens = _lens(s["q_lens"]), _lens(s["k_lens"])
    cq, ck = _offsets(q_lens), _offsets(k_lens)
    for n, (Lq, Lk) in enumerate(zip(q_lens, k_lens)):
        seen = None
        if s["block"]:
            i = torch.arange(Lq, device="cuda") + (Lk - Lq)
            seen = torch.arange(Lk, device="cuda") < ((i // s["block"] + 1) * s["block"])[:, None]
        yield slice(cq[n], cq[n + 1]), slice(ck[n], ck[n + 1]), seen


def _attention(s):
    H, Hkv = s["heads"], s["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((H, s["q"].shape[0]), dtype=torch.float32, device="cuda")
    G = H // Hkv
    for rq, rk, seen in _parts(s):
        for j in range(Hkv):
            hs = slice(j * G, (j + 1) * G)
            q, k, v = s["q"][rq, hs].float().transpose(0, 1), s["k"][rk, j].float(), s["v"][rk, j].float()
            x = (q @ k.T) * 128 ** -0.5  # [G][Lq][Lk]
            if seen is not None:
                x.masked_fill_(~seen, float("-inf"))
            if not k.shape[0]:
                lse[hs, rq] = float("-inf")
                continue
            m = x.amax(-1, keepdim=True)
            m0 = m.clamp(min=torch.finfo(torch.float32).min)  # a row that sees nothing: exp(-inf - finite) = 0
            p = x.sub_(m0).exp_()
            l = p.sum(-1, keepdim=True)
            out[rq, hs] = ((p @ v) / l.clamp(min=1e-30)).transpose(0, 1).to(torch.bfloat16)
            lse[hs, rq] = (m + l.log())[..., 0]
    return out, lse


def _attention_backward(s):
    H, Hkv = s["heads"], s["kv_heads"]
    dq = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    dk = torch.zeros(s["k"].shape, dtype=torch.bfloat16, device="cuda")
    dv = torch.zeros(s["k"].shape, dtype=torch.bfloat16, device="cuda")
    G, scale = H // Hkv, 128 ** -0.5
    for rq, rk, seen in _parts(s):
        for j in range(Hkv):
            hs = slice(j * G, (j + 1) * G)
            q, k, v = s["q"][rq, hs].float().transpose(0, 1), s["k"][rk, j].float(), s["v"][rk, j].float()
            o, do = s["out"][rq, hs].float().transpose(0, 1), s["dout"][rq, hs].float().transpose(0, 1)
            lse = s["lse"][hs, rq][..., None]
            x = (q @ k.T) * scale
            x.sub_(lse.clamp(min=torch.finfo(torch.float32).min)).exp_()  # P
            if seen is not None:
                x.masked_fill_(~seen, 0.0)
            dv[rk, j] = (x.transpose(1, 2) @ do).sum(0).to(torch.bfloat16)
            dp = do @ v.T
            x.mul_(dp.sub_((o * do).sum(-1, keepdim=True)))  # dS
            dq[rq, hs] = ((x @ k) * scale).transpose(0, 1).to(torch.bfloat16)
            dk[rk, j] = ((x.transpose(1, 2) @ q).sum(0) * scale).to(torch.bfloat16)
    return {"dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------- in 64 bits

def _pairs(case):
    return sum(int(_limits(a, b, case["block"]).sum()) for a, b in zip(_lens(case["q_lens"]), _lens(case["k_lens"])))


def exact(case, seed):
    global own
    if case["op"].startswith("attention"):
        Tq, Tk = sum(_lens(case["q_lens"])), sum(_lens(case["k_lens"]))
        if case["heads"] * Tq * Tk * 512.0 * (1 if case["op"] == "attention" else 3) > 4e12:
            return None
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return _exact_norm(s) if case["op"].startswith("norm_rope") else _exact_attention(s)


def _exact_norm(s):
    """The rotation as a complex product by exp(i angle); the backward pass by differentiating that."""
    d = s["d"]
    freq = [THETA ** (-2.0 * i / a) for a in AXES[d] for i in range(a // 2)]
    axis = [n for n, a in enumerate(AXES[d]) for _ in range(a // 2)]
    angle = s["positions"].double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    got = {}
    for n in "qk":
        x, w = s[n].double(), s[n + "_weight"].double()
        back = s["op"] == "norm_rope_backward"
        x.requires_grad_(back)
        w.requires_grad_(back)
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * w
        y = torch.view_as_real(torch.view_as_complex(y.unflatten(-1, (d // 2, 2)).contiguous()) * turn).flatten(-2)
        if back:
            got["d" + n], got["d" + n + "_weight"] = torch.autograd.grad(y, (x, w), s["d" + n + "_out"].double())
        else:
            got[n] = y
    return got


def _exact_attention(s):
    """Every query against every key of the whole batch, blocks of query rows at a time, one query head after another."""
    H, G = s["heads"], s["heads"] // s["kv_heads"]
    q_lens, k_lens = _lens(s["q_lens"]), _lens(s["k_lens"])
    cq, ck = _offsets(q_lens), _offsets(k_lens)
    first, last = np.zeros(s["q"].shape[0], np.int64), np.zeros(s["q"].shape[0], np.int64)
    for n, (Lq, Lk) in enumerate(zip(q_lens, k_lens)):
        first[cq[n]:cq[n + 1]] = ck[n]
        last[cq[n]:cq[n + 1]] = ck[n] + _limits(Lq, Lk, s["block"])
    first, last = torch.from_numpy(first).cuda()[:, None], torch.from_numpy(last).cuda()[:, None]
    at = torch.arange(s["k"].shape[0], device="cuda")
    back = s["op"] == "attention_backward"
    shape = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out, lse = shape(s["q"]), torch.zeros((H, s["q"].shape[0]), dtype=torch.float64, device="cuda")
    dq, dk, dv = shape(s["q"]), shape(s["k"]), shape(s["k"])
    for h in range(H):
        k, v = s["k"][:, h // G].double(), s["v"][:, h // G].double()
        for i in range(0, cq[-1], 4096):
            r = slice(i, min(i + 4096, cq[-1]))
            q = s["q"][r, h].double()
            logits = q @ k.T / 128 ** 0.5
            sees = (at >= first[r]) & (at < last[r])
            if not back:
                logits[~sees] = float("-inf")
                lse[h, r] = torch.logsumexp(logits, -1)
                w = torch.exp(logits - lse[h, r][:, None])
                w[~sees] = 0.0
                out[r, h] = w @ v
                continue
            w = torch.exp(logits - s["lse"][h, r].double()[:, None])
            w[~sees] = 0.0
            do = s["dout"][r, h].double()
            ds = w * (do @ v.T - (do * s["out"][r, h].double()).sum(-1)[:, None])
            dv[:, h // G] += w.T @ do
            dk[:, h // G] += ds.T @ q / 128 ** 0.5
            dq[r, h] = ds @ k / 128 ** 0.5
    return {"dq": dq, "dk": dk, "dv": dv} if back else {"out": out, "lse": lse}


# ------------------------------------------------------------- what a pass cannot do without

def work(case):
    H, Hkv = case["heads"], case["kv_heads"]
    if case["op"].startswith("norm_rope"):
        d = case["d"]
        n = (case["tokens"] + case["pad"]) * (H + Hkv) * d
        e = 4 if case["dtype"] == "f32" else 2
        back = case["op"] == "norm_rope_backward"
        return {"bytes": n * e * (3 if back else 2) + 12 * (case["tokens"] + case["pad"]) + d * 4 * (4 if back else 2),
                "flops": n * (14 if back else 7)}
    Tq, Tk, pairs = sum(_lens(case["q_lens"])), sum(_lens(case["k_lens"])), _pairs(case)
    rows, keys, lse = Tq * H * 256, Tk * Hkv * 256, Tq * H * 4
    if case["op"] == "attention":
        return {"bytes": 2 * rows + 2 * keys + lse, "flops": 4.0 * 128 * H * pairs}
    return {"bytes": 4 * rows + 4 * keys + lse, "flops": 10.0 * 128 * H * pairs}

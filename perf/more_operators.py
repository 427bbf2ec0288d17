"""The cases on which the operators of heads and tokens are measured: the norm
and rotary position of query and key heads (``head_rope``), attention to an
encoder's states (``cross_attention``) and the choice of the next token
(``sample``).

``own`` false: ``run`` is the plain form, elementary torch operations in fp32
(angles and sampling weights in 64 bits: far positions and whole-number
results do not survive fp32).  ``own`` true: ``run`` calls the library.
"""
from __future__ import annotations

import math

import torch

own = False

# Sizes are those of the repository's workloads (32 query and 8 key/value heads
# of 128: 4096 and 1024 channels; the 1280-wide vision encoder at 1601 tokens, here
# as 16 heads of 80; up to four images of 1601 states; a 128256-entry vocabulary;
# prefill of 2048) and ragged ones.


def _rope(name, M, heads, kv_heads, D, rot, layout, scaling, norm, dtype, out):
    return dict(name=name, op="rope", M=M, heads=heads, kv_heads=kv_heads, D=D, rot=rot, layout=layout, scaling=scaling,
                norm=norm, dtype=dtype, out=out)


def _attn(name, B, Lq, Lk, heads, kv_heads, D, mask, lens, shared):
    return dict(name=name, op="attn", B=B, Lq=Lq, Lk=Lk, heads=heads, kv_heads=kv_heads, D=D, mask=mask, lens=lens,
                shared=shared)


def _sample(name, M, V, dtype, top_k, top_p, min_p):
    return dict(name=name, op="sample", M=M, V=V, dtype=dtype, top_k=top_k, top_p=top_p, min_p=min_p)


def listed():
    return [
        # one decoded token: its query and key heads, from the fp32 outputs of the projections
        _rope("rope-decode-1", 1, 32, 8, 128, 128, "half", "llama3", False, "f32", "bf16"),
        # a short ragged prompt, positions on part of narrow heads, pairs side by side
        _rope("rope-ragged-77", 77, 16, 4, 80, 32, "interleaved", "linear", True, "bf16", "f32"),
        # prefill of 2048 tokens, normed heads, from one matrix of queries, keys and values
        _rope("rope-prefill-2048", 2048, 32, 8, 128, 128, "half", "yarn", True, "bf16", "bf16"),
        # one decoded token that sees one image: latency
        _attn("attn-decode-1", 1, 1, 1601, 32, 8, 128, "none", False, False),
        # a decoded token of each of 8 requests, each with images of its own: one read of the states
        _attn("attn-decode-8", 8, 1, 6404, 32, 8, 128, "none", True, False),
        # 16 requests about the same images
        _attn("attn-shared-16", 16, 1, 6404, 32, 8, 128, "none", False, True),
        # the vision encoder, 1601 tokens: every head its own keys, heads of 80
        _attn("attn-vision-1601", 1, 1601, 1601, 16, 16, 80, "none", False, False),
        # prefill of 2048 tokens with four images in the text: a token sees those before it, the first tokens none
        _attn("attn-prefill-2048", 1, 2048, 6404, 32, 8, 128, "images", False, False),
        # the next token of one request
        _sample("sample-1", 1, 128256, "f32", 50, 0.9, 0.0),
        # of 8 requests, from bf16 logits (many equal values), nucleus alone
        _sample("sample-8", 8, 128256, "bf16", 0, 0.95, 0.0),
        # a ragged small vocabulary with every limit
        _sample("sample-ragged-33", 33, 5003, "f32", 200, 0.8, 0.05),
        # of 512 requests: the largest, one read of the logits
        _sample("sample-512", 512, 128256, "f32", 50, 0.95, 0.01),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "sample"])
    if op == "rope":
        while True:
            M, D = _log(rng, 1, 8192), rng.choice([64, 80, 96, 128])
            kv_heads = rng.choice([1, 2, 4, 8])
            heads = kv_heads * rng.choice([1, 3, 4, 5])
            if M * (heads + kv_heads) * D <= 2048 * 40 * 128:
                break
        return _rope("", M, heads, kv_heads, D, rng.choice([D, D, D // 2, D // 4]), rng.choice(["half", "interleaved"]),
                     rng.choice(["none", "linear", "llama3", "yarn"]), rng.random() < 0.5, rng.choice(["f32", "bf16"]),
                     rng.choice(["f32", "bf16"]))
    if op == "attn":
        while True:
            B, Lq, Lk = _log(rng, 1, 16), _log(rng, 1, 2048), _log(rng, 1, 6404)
            D, kv_heads = rng.choice([32, 64, 80, 96, 128]), rng.choice([1, 2, 4, 8, 16])
            heads = kv_heads * rng.choice([1, 1, 3, 4, 5])
            # no dearer than the prefill
            if B * Lq * Lk * heads * D <= 2048 * 6404 * 32 * 128 // 2 and B * heads * Lq * Lk <= 1 << 28:
                break
        shared = B > 1 and rng.random() < 0.2
        return _attn("", B, Lq, Lk, heads, kv_heads, D, rng.choice(["none", "none", "images", "random"]),
                     not shared and rng.random() < 0.5, shared)
    while True:
        M, V = _log(rng, 1, 512), _log(rng, 16, 128256)
        if M * V <= 128 * 128256:
            break
    return _sample("", M, V, rng.choice(["f32", "bf16"]), rng.choice([0, 1, 20, 50, 1000]), rng.choice([1.0, 0.95, 0.8, 0.5]),
                   rng.choice([0.0, 0.0, 0.02, 0.1]))


_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}

# what each kind of long-context scaling is told
_SCALING = {
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, factor=4.0),
    "llama3": dict(base=500000.0, factor=8.0, original_length=8192, low=1.0, high=4.0),
    "yarn": dict(base=1000000.0, factor=4.0, original_length=32768, beta_fast=32.0, beta_slow=1.0),
}


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    if case["op"] == "rope":
        # a token's queries, keys and values as one product leaves them; a long context's positions
        M, H, Hk, D = case["M"], case["heads"], case["kv_heads"], case["D"]
        qkv = normal(M, (H + 2 * Hk) * D).to(_DTYPE[case["dtype"]])
        first = torch.randint(0, 100000, (1,), generator=g, device="cuda")
        return dict(q=qkv[:, :H * D].view(M, H, D), k=qkv[:, H * D:(H + Hk) * D].view(M, Hk, D),
                    positions=first + torch.arange(M, device="cuda"),
                    q_weight=1 + 0.1 * normal(D) if case["norm"] else None,
                    k_weight=1 + 0.1 * normal(D) if case["norm"] else None)
    if case["op"] == "attn":
        B, Lq, Lk, H, Hk, D = (case[n] for n in ("B", "Lq", "Lk", "heads", "kv_heads", "D"))
        Bk = 1 if case["shared"] else B
        q = normal(B, Lq, H, D) * (0.5 + 2 * uniform(H, 1))  # flat and pointed heads
        k, v = normal(Bk, Lk, Hk, D), normal(Bk, Lk, Hk, D) + 0.5 * normal(Hk, D)
        lens = mask = None
        if case["lens"]:
            lens = torch.randint(Lk // 2, Lk + 1, (B,), generator=g, device="cuda").to(torch.int32)
        if case["mask"] == "images":  # key j belongs to the image j // ceil(Lk / 4); a token sees the images before it
            starts = (uniform(B, 4) * (Lq / 2)).sort(dim=1).values
            sees = torch.arange(Lq, device="cuda")[None, :, None] >= starts[:, None, :]
            mask = sees.repeat_interleave(-(-Lk // 4), 2)[:, :, :Lk].contiguous()
        elif case["mask"] == "random":
            mask = uniform(B, Lq, Lk) < 0.7
        return dict(q=q.bfloat16(), k=k.bfloat16(), v=v.bfloat16(), lens=lens, mask=mask)
    M, V = case["M"], case["V"]
    # most tokens unlikely, some tens in question
    logits = normal(M, V) * 2 + torch.where(uniform(M, V) < 40 / V, 8 * uniform(M, V), torch.zeros((), device="cuda"))
    return dict(logits=logits.to(_DTYPE[case["dtype"]]), u=uniform(M), temperature=0.5 + uniform(M))


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if case["op"] == "rope":
        if own:
            import w2_a8_matmul_amd as s3d8

            state["rope"] = s3d8.Rope(case["rot"], layout=case["layout"], scaling=case["scaling"], **_SCALING[case["scaling"]])
        else:
            state["frequencies"], state["factor"] = _plain_frequencies(case["rot"], case["scaling"])
    return state


def run(state):
    if own:
        return _library(state)
    return {"rope": _plain_rope, "attn": _plain_attn, "sample": _plain_sample}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the library


def _library(state):
    import w2_a8_matmul_amd as s3d8

    c = state["case"]
    if c["op"] == "rope":
        return s3d8.head_rope(state["q"], state["k"], state["positions"], state["rope"], q_weight=state["q_weight"],
                              k_weight=state["k_weight"], eps=1e-5, out=c["out"])
    if c["op"] == "attn":
        return s3d8.cross_attention(state["q"], state["k"], state["v"], kv_lens=state["lens"], mask=state["mask"])
    return s3d8.sample(state["logits"], state["u"], temperature=state["temperature"], top_k=c["top_k"], top_p=c["top_p"],
                       min_p=c["min_p"])


# ------------------------------------------------------------------ plain forms


def _plain_frequencies(rot, scaling):
    """Radians per position of each pair, in 64 bits, and the factor on cosine and sine."""
    s = _SCALING[scaling]
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = s["base"] ** (-2 * j / rot)
    if scaling == "linear":
        return f / s["factor"], 1.0
    if scaling == "llama3":  # turns over the original length: few are stretched, many stay
        turns = s["original_length"] * f / (2 * math.pi)
        keep = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        return f * keep + f / s["factor"] * (1 - keep), 1.0
    if scaling == "yarn":
        def pair(turns):  # the pair that makes so many turns over the original length
            return rot * math.log(s["original_length"] / (turns * 2 * math.pi)) / (2 * math.log(s["base"]))
        low, high = max(math.floor(pair(s["beta_fast"])), 0), min(math.ceil(pair(s["beta_slow"])), rot - 1)
        stretch = ((j - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / s["factor"] * stretch + f * (1 - stretch), 0.1 * math.log(s["factor"]) + 1
    return f, 1.0


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    angles = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = ((f(angles) * s["factor"]).float()[:, None, :] for f in (torch.cos, torch.sin))

    def heads(x, weight):
        x = x.float()
        if weight is not None:
            x = x * (x.square().mean(2, keepdim=True) + 1e-5).rsqrt() * weight
        if c["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), 2)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2)
        return torch.cat((turned, x[..., rot:]), 2).to(_DTYPE[c["out"]])

    return heads(s["q"], s["q_weight"]), heads(s["k"], s["k_weight"])


def _plain_attn(s):
    c = s["case"]
    B, Lq, Lk, H, Hk, D = (c[n] for n in ("B", "Lq", "Lk", "heads", "kv_heads", "D"))
    q = s["q"].float().transpose(1, 2)  # [B][H][Lq][D]
    k, v = (t.float().transpose(1, 2).repeat_interleave(H // Hk, 1).expand(B, H, Lk, D) for t in (s["k"], s["v"]))
    scores = torch.matmul(q.contiguous(), k.transpose(2, 3).contiguous()) * (1 / math.sqrt(D))
    seen = s["mask"][:, None] if s["mask"] is not None else None
    if s["lens"] is not None:
        inside = (torch.arange(Lk, device="cuda") < s["lens"][:, None])[:, None, None, :]
        seen = inside if seen is None else seen & inside
    if seen is not None:
        scores = scores.masked_fill(~seen, -math.inf)
    most = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(most == -math.inf, torch.zeros_like(most), most))
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, v.contiguous()) / torch.where(total == 0, torch.ones_like(total), total)
    return o.transpose(1, 2).bfloat16().contiguous()


def _plain_sample(s):
    c = s["case"]
    l = s["logits"].float()
    T = s["temperature"].double()[:, None]
    one = float(1 << 44)  # weights as whole numbers: sums do not depend on their order
    weight = torch.round(torch.exp((l.double() - l.amax(1, keepdim=True).double()) / T) * one).to(torch.int64)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    w = weight.gather(1, order)
    rank = torch.arange(l.shape[1], device="cuda")
    if c["top_k"] > 0:
        w = torch.where(rank < c["top_k"], w, 0)
    if c["top_p"] < 1:
        limit = torch.ceil(c["top_p"] * w.sum(1, keepdim=True).double()).to(torch.int64).clamp(min=1)
        w = torch.where(w.cumsum(1) - w < limit, w, 0)
    w = torch.where(w >= math.ceil(c["min_p"] * one), w, 0)
    kept = torch.zeros_like(w).scatter_(1, order, w)
    upto = kept.cumsum(1)
    total = upto[:, -1:]
    target = torch.floor(s["u"].double()[:, None] * total.double()).to(torch.int64)
    token = (upto <= target).sum(1, keepdim=True)
    return token.to(torch.int32)[:, 0], (kept.gather(1, token).double() / total.double()).float()[:, 0]


# ------------------------------------------------------------------ work


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "rope":
        n = case["M"] * (case["heads"] + case["kv_heads"]) * case["D"]
        return {"bytes": n * (size[case["dtype"]] + size[case["out"]]) + 8 * case["M"], "flops": n * (10 if case["norm"] else 6)}
    if case["op"] == "attn":
        B, Lq, Lk, H, Hk, D = (case[n] for n in ("B", "Lq", "Lk", "heads", "kv_heads", "D"))
        keys = Lk * (0.75 if case["lens"] else 1)  # lengths from half to all, evenly
        share = {"none": 1, "images": 0.75, "random": 0.7}[case["mask"]]
        states = (1 if case["shared"] else B) * keys * Hk * D * 2 * 2
        mask = 0 if case["mask"] == "none" else B * Lq * keys
        return {"bytes": int(2 * B * Lq * H * D * 2 + states + mask), "flops": int(4 * B * Lq * keys * share * H * D)}
    M, V = case["M"], case["V"]
    return {"bytes": M * V * size[case["dtype"]] + 16 * M, "flops": M * V * 4}


# ------------------------------------------------------------------ 64 bits


def _exact_rope(case, s):
    rot, t = case["rot"], _SCALING[case["scaling"]]
    factor, scale = t.get("factor", 1.0), 1.0
    f = []
    for i in range(rot // 2):  # one pair after the other, on the host
        plain = math.exp(-2 * i / rot * math.log(t["base"]))
        mix = 0.0  # share of the stretched frequency
        if case["scaling"] == "linear":
            mix = 1.0
        elif case["scaling"] == "llama3":
            wave = 2 * math.pi / plain
            if wave > t["original_length"] / t["low"]:
                mix = 1.0
            elif wave > t["original_length"] / t["high"]:
                mix = 1 - (t["original_length"] / wave - t["low"]) / (t["high"] - t["low"])
        elif case["scaling"] == "yarn":
            scale = 1 + 0.1 * math.log(factor)
            at = [rot / 2 * math.log(t["original_length"] / (2 * math.pi * b), t["base"]) for b in (t["beta_fast"], t["beta_slow"])]
            first, last = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
            mix = min(1.0, max(0.0, (i - first) / ((last - first) or 0.001)))
        f.append(plain * ((1 - mix) + mix / factor))
    turn = torch.polar(torch.full((case["M"], 1, rot // 2), scale, dtype=torch.float64, device="cuda"),
                       (s["positions"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda"))[:, None])
    both = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + 1e-5) * weight.double()
        y = x.clone()
        first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        both.append(y)
    return both


def _exact_attn(case, s):
    H, Hk, Lk = case["heads"], case["kv_heads"], case["Lk"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        bk = 0 if case["shared"] else b
        n = Lk if s["lens"] is None else int(s["lens"][b])
        for h in range(H):
            k, v = s["k"][bk, :n, h * Hk // H].double(), s["v"][bk, :n, h * Hk // H].double()
            x = s["q"][b, :, h].double() @ k.t().contiguous() / math.sqrt(case["D"])
            if s["mask"] is not None:
                x = torch.where(s["mask"][b, :, :n], x, torch.full_like(x, -math.inf))
            p = torch.softmax(x, 1)
            o[b, :, h] = torch.where(torch.isnan(p).any(1, keepdim=True), torch.zeros_like(p), p) @ v
    return o


def _exact_sample(case, s):
    # the probability of the token, from real weights and no sorting by index: the token itself is None
    M, V = case["M"], case["V"]
    found = torch.empty(M, dtype=torch.float64, device="cuda")
    for m in range(M):
        l = s["logits"][m].double()
        p = torch.softmax((l - l.max()) / s["temperature"][m].double(), 0)
        value, at = torch.sort(p, descending=True, stable=True)
        n = min(case["top_k"] or V, V)
        if case["top_p"] < 1:
            mass = torch.cumsum(value[:n], 0)
            n = min(n, 1 + int((mass < case["top_p"] * mass[-1]).sum()))
        n = min(n, max(1, int((value >= case["min_p"] * value[0]).sum())))
        kept = torch.sort(at[:n]).values
        mass = torch.cumsum(p[kept], 0)
        chosen = min(int((mass <= s["u"][m].double() * mass[-1]).sum()), n - 1)
        found[m] = p[kept[chosen]] / mass[-1]
    return None, found


def exact(case, seed):
    return {"rope": _exact_rope, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](case, _inputs(case, seed))

"""What is measured of three operators of a fine-tuning step: the loss over a large vocabulary
without its logits, AdamW over many tensors with 8- or 32-bit states, and rotary positions.

Every operator stands here twice: in plain torch operations, and as the call a user of the
library makes (`own`).  `exact` computes the same outputs in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

BLOCK = 256  # elements that share one scale of an 8-bit optimizer state


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest configuration's loss: one sequence of 64 tokens, where launches count
        dict(name="ce_small", op="ce", T=64, hidden=256, vocab=1024, counted=1.0, pairs=0, grad=True),
        # the 8B shape's training step: one sequence of 512 tokens, every target counted
        dict(name="ce_sft_512", op="ce", T=512, hidden=4096, vocab=128256, counted=1.0, pairs=0, grad=True),
        # two preference pairs of 512 tokens that share 256, packed [prefix | chosen | rejected]:
        # prefix rows carry no target, the last of each prefix carries two
        dict(name="ce_pairs_1536", op="ce", T=1536, hidden=4096, vocab=128256, counted=1.0, pairs=2, grad=True),
        # log-probs of a reference model, no gradient: a ragged batch over an odd vocabulary
        dict(name="ce_reference_999", op="ce", T=999, hidden=4096, vocab=32003, counted=0.5, pairs=0, grad=False),
        # the 70B shape's training step: 2048 tokens, hidden 8192
        dict(name="ce_sft_70b", op="ce", T=2048, hidden=8192, vocab=128256, counted=1.0, pairs=0, grad=True),
        # the smallest configuration's adapters: 28 small tensors, one launch
        dict(name="adamw32_small", op="adamw", sizes="lora", layers=2, hidden=256, q=256, kv=128, inner=688, r=8, bits=32,
             param="float32", grad="float32", decay=0.0),
        # the 8B shape's adapters (448 tensors, 168 M parameters) with 8-bit states, then 32-bit
        dict(name="adamw8_8b", op="adamw", sizes="lora", layers=32, hidden=4096, q=4096, kv=1024, inner=14336, r=64, bits=8,
             param="float32", grad="float32", decay=0.0),
        dict(name="adamw32_8b", op="adamw", sizes="lora", layers=32, hidden=4096, q=4096, kv=1024, inner=14336, r=64, bits=32,
             param="float32", grad="float32", decay=0.0),
        # tensors of every odd size, in 16 bits throughout, with weight decay
        dict(name="adamw8_ragged", op="adamw", sizes="ragged", count=190, most=400000, of=11, bits=8, param="bfloat16",
             grad="bfloat16", decay=0.01),
        # one new token of the 8B shape, far out in a long context
        dict(name="rope_token", op="rope", T=1, hq=32, hkv=8, d=128, rotary=128, paired=False, scaling="llama3", far=100000,
             type="bfloat16", inverse=False),
        # four sequences of 2048 tokens of the 8B shape, out of the packed q|k|v projection
        dict(name="rope_8192", op="rope", T=8192, hq=32, hkv=8, d=128, rotary=128, paired=False, scaling="llama3", far=2048,
             type="bfloat16", inverse=False),
        # the gradient of a long context: neighbouring pairs, half of each head rotated
        dict(name="rope_long_backward", op="rope", T=32768, hq=64, hkv=8, d=128, rotary=64, paired=True, scaling="yarn",
             far=131072, type="bfloat16", inverse=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["ce", "ce", "adamw", "rope"])
    if op == "ce":
        while True:
            hidden, vocab, T = 8 * _log(rng, 16, 1024), _log(rng, 130, 131071), _log(rng, 1, 4096)
            if T * hidden * vocab <= 2048 * 8192 * 128256:
                break
        pairs = rng.choice([0, 0, 1, 2, 3]) if T >= 9 else 0
        T -= T % (3 * pairs) if pairs else 0
        return dict(op="ce", T=T, hidden=hidden, vocab=vocab, counted=rng.choice([1.0, 0.5, 0.1]), pairs=pairs,
                    grad=rng.random() < 0.75)
    if op == "adamw":
        bits, types = rng.choice([8, 8, 32]), ["float32", "float32", "bfloat16"]
        if rng.random() < 0.5:
            return dict(op="adamw", sizes="lora", layers=_log(rng, 1, 40), hidden=8 * _log(rng, 32, 640), q=64 * _log(rng, 2, 80),
                        kv=64 * _log(rng, 1, 16), inner=8 * _log(rng, 64, 1800), r=rng.choice([8, 16, 24, 32, 64]), bits=bits,
                        param=rng.choice(types), grad=rng.choice(types), decay=rng.choice([0.0, 0.1]))
        return dict(op="adamw", sizes="ragged", count=_log(rng, 1, 700), most=_log(rng, 100, 400000), of=rng.randrange(1 << 20),
                    bits=bits, param=rng.choice(types), grad=rng.choice(types), decay=rng.choice([0.0, 0.01]))
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    return dict(op="rope", T=_log(rng, 1, 16384), hq=hkv * rng.choice([1, 3, 4, 7, 8]), hkv=hkv, d=d,
                rotary=rng.choice([d, d, d // 2, d // 4, d // 2 + 8]), paired=rng.random() < 0.5,
                scaling=rng.choice(["none", "linear", "ntk", "llama3", "yarn"]), far=_log(rng, 1 << 14, 1 << 21),
                type=rng.choice(["bfloat16", "bfloat16", "float32"]), inverse=rng.random() < 0.5)


def _sizes(case):
    """The tensors of an optimizer case, as element counts."""
    if case["sizes"] == "lora":  # A of the seven projections, then B, layer by layer
        h, q, kv, inner, r = (case[k] for k in ("hidden", "q", "kv", "inner", "r"))
        return [r * n for n in (h, h, h, q, h, h, inner, q, kv, kv, h, inner, inner, h)] * case["layers"]
    g = random.Random(case["of"])
    return [_log(g, 1, case["most"]) for _ in range(case["count"])]


def _scaling(case):
    kind = case["scaling"]
    return dict(kind=kind, theta=500000.0, factor=1.0 if kind == "none" else 8.0, original=8192,
                low=1.0, high=32.0 if kind == "yarn" else 4.0)


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "ce":
        T, H, V = case["T"], case["hidden"], case["vocab"]
        w = (normal(V, H) * 0.02).bfloat16()
        targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        # a trained model is sure of some tokens and lost at others: the target's logit lies
        # between 0 and about 20 above the others
        sure = torch.rand(T, 1, generator=g, device="cuda") * 20.0 / (H * 0.0004)
        s["h"] = (normal(T, H) + sure * w[targets.long()].float()).bfloat16()
        s["w"] = w
        s["targets2"] = s["weight2"] = None
        row = torch.arange(T, device="cuda")
        if case["pairs"]:
            n = T // case["pairs"]      # rows of a pair: prefix, chosen and rejected, a third each
            third = n // 3
            at = row % n
            ends = (at == 2 * third - 1) | (at == n - 1)
            targets = torch.where((at < third - 1) | ends, -1, targets).int()
            two = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
            s["targets2"] = torch.where(at == third - 1, two, -1).int()
            push = 0.1 * torch.rand(T, generator=g, device="cuda").mul(0.5).add(0.25)
            s["weight"] = torch.where(at < 2 * third, push, -push)
            s["weight2"] = -push
        else:
            keep = (torch.rand(T, generator=g, device="cuda") < case["counted"]) & ((row + 1) % 512 != 0)
            targets = torch.where(keep, targets, -1).int()
            s["weight"] = torch.where(keep, 1.0 / keep.sum().clamp(min=1), 0.0).float()
        s["targets"] = targets
        return s
    if case["op"] == "adamw":
        sizes = _sizes(case)
        n = sum(sizes)
        blocks = [-(-k // BLOCK) for k in sizes]
        padded = BLOCK * sum(blocks)
        s["p"] = (normal(n) * 0.02).to(getattr(torch, case["param"]))
        rough = torch.exp(normal(n) * 1.5)  # gradients differ by orders of magnitude from weight to weight
        s["g"] = (normal(n) * rough * 1e-3).to(getattr(torch, case["grad"]))
        cut = lambda t: list(t.split(sizes))  # noqa: E731
        s["params"], s["grads"] = cut(s["p"]), cut(s["g"])
        # the states lie one tensor after the other, each from a whole block on
        at = None
        if padded != n:
            before = torch.tensor([b * BLOCK - k for b, k in zip(blocks, sizes)], device="cuda").cumsum(0).roll(1)
            before[0] = 0
            at = torch.arange(n, device="cuda") + torch.repeat_interleave(before, torch.tensor(sizes, device="cuda"))
        s["at"], s["step"] = at, 10 + int(seed) % 1000
        m, v = normal(n) * rough * 3e-4, (rough * 1e-3 * (0.5 + torch.rand(n, generator=g, device="cuda"))).square()
        if at is not None:
            m, v = torch.zeros(padded, device="cuda").index_copy_(0, at, m), torch.zeros(padded, device="cuda").index_copy_(0, at, v)
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _m_codes(m)
            s["v"], s["v_scale"] = _v_codes(v)
        else:
            s["m"], s["v"] = m, v
        return s
    T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
    qkv = normal(T, hq + 2 * hkv, d).to(getattr(torch, case["type"]))
    s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
    S = min(T, case["far"])             # sequences of S tokens, each from a position of its own on
    start = torch.randint(0, case["far"] - S + 1, (-(-T // S),), generator=g, device="cuda")
    row = torch.arange(T, device="cuda")
    s["positions"] = (start[row // S] + row % S).int()
    return s


# ------------------------------------------------------------------ the operators, plainly
def _ce(s):
    """Over pieces of the vocabulary: the row's sum of exp, the logits of its targets and the
    others' share of the gradient; then dh = (w1 + w2) sum_v p_v W_v - w1 W_t1 - w2 W_t2."""
    h, w, T = s["h"].float(), s["w"], s["T"]
    t1 = s["targets"].long()
    live = t1 >= 0
    t2 = s["targets2"].long() if s["targets2"] is not None else torch.full_like(t1, -1)
    pieces = torch.split(w, max(1, (1 << 28) // max(T, 1)))
    logits = lambda piece: h @ piece.float().T  # noqa: E731
    each = torch.stack([torch.logsumexp(logits(x).double(), 1) for x in pieces])
    lse = torch.logsumexp(each, 0)
    at = lambda t: (h.double() * w[t.clamp(min=0)].double()).sum(1)  # noqa: E731
    lse = torch.where(live, lse, 0.0)
    out = {"lse": lse.float(), "logp": torch.where(live, at(t1) - lse, 0.0).float()}
    if s["targets2"] is not None:
        out["logp2"] = torch.where(t2 >= 0, at(t2) - lse, 0.0).float()
    if s["grad"]:
        w1 = torch.where(live, s["weight"], 0.0)
        w2 = torch.where(t2 >= 0, s["weight2"], 0.0) if s["targets2"] is not None else torch.zeros_like(w1)
        first, dh = 0, torch.zeros_like(h)
        for x in pieces:
            col = torch.arange(first, first + x.shape[0], device=h.device)
            p = torch.exp(logits(x).double() - lse[:, None]) * (w1 + w2)[:, None]
            p = p - w1[:, None] * (col == t1[:, None]) - w2[:, None] * (col == t2[:, None])
            dh += p.float() @ x.float()
            first += x.shape[0]
        out["dh"] = dh.bfloat16()
    return out


def _blocks_max(x):
    return x.view(-1, BLOCK).amax(1)


def _m_codes(m):
    """m = scale sign(q) (q / 127)^2, q in -127 .. 127, scale the block's largest |m|."""
    scale = _blocks_max(m.abs())
    q = torch.round(127 * torch.sqrt(m.abs().view(-1, BLOCK) / torch.where(scale > 0, scale, 1)[:, None])).view(-1)
    return (q * torch.sign(m)).to(torch.int8), scale


def _v_codes(v):
    """v = scale (q / 255)^4, q in 0 .. 255, at least 1 where v > 0; scale the block's largest v."""
    scale = _blocks_max(v)
    q = torch.round(255 * torch.sqrt(torch.sqrt(v.view(-1, BLOCK) / torch.where(scale > 0, scale, 1)[:, None]))).view(-1)
    return torch.where(v > 0, q.clamp(min=1), 0).to(torch.uint8), scale


def _m_values(q, scale):
    r = q.float() / 127
    return (r * r.abs()).view(-1, BLOCK).mul(scale[:, None]).view(-1)


def _v_values(q, scale):
    r = (q.float() / 255).square().square()
    return r.view(-1, BLOCK).mul(scale[:, None]).view(-1)


def _adamw(s):
    """m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2, p' = p - lr (m^ / (sqrt v^ + eps) + wd p),
    m^ and v^ without their bias; an 8-bit state is read, used in 32 bits and coded anew."""
    b1, b2, lr, eps, t, wd = 0.9, 0.999, 1e-3, 1e-8, s["step"], s["decay"]
    m = _m_values(s["m"], s["m_scale"]) if s["bits"] == 8 else s["m"]
    v = _v_values(s["v"], s["v_scale"]) if s["bits"] == 8 else s["v"]
    g, p, at = s["g"].float(), s["p"].float(), s["at"]
    if at is not None:
        g = torch.zeros_like(m).index_copy_(0, at, g)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    step = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
    s["p"].copy_(p - lr * ((step if at is None else step[at]) + wd * p))
    if s["bits"] == 8:
        for name, codes, x in (("m", _m_codes, m), ("v", _v_codes, v)):
            q, scale = codes(x)
            s[name].copy_(q)
            s[name + "_scale"].copy_(scale)
        return {"p": s["p"], "m": _m_values(s["m"], s["m_scale"]).bfloat16(), "v": _v_values(s["v"], s["v_scale"]).bfloat16(),
                "m_scale": s["m_scale"], "v_scale": s["v_scale"]}
    s["m"].copy_(m)
    s["v"].copy_(v)
    return {"p": s["p"], "m": s["m"], "v": s["v"]}


def _frequencies(s):
    """Radians a position for each pair, and the factor on cos and sin, in 64 bits."""
    c, d = _scaling(s), s["rotary"]
    theta = c["theta"] * c["factor"] ** (d / (d - 2)) if c["kind"] == "ntk" else c["theta"]
    f = theta ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    if c["kind"] == "linear":
        f = f / c["factor"]
    if c["kind"] in ("llama3", "yarn"):  # turns within the original context say which pairs stay
        keep = ((c["original"] * f / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / c["factor"]
    return f, 0.1 * math.log(c["factor"]) + 1.0 if c["kind"] == "yarn" else 1.0


def _rope(s):
    f, grow = _frequencies(s)
    angle = s["positions"].double()[:, None] * f
    cos, sin = (torch.cos(angle) * grow).float()[:, None], (torch.sin(angle) * grow).float()[:, None]
    if s["inverse"]:  # the gradient of a rotation is the rotation back
        sin = -sin

    def turned(x):
        y, r = x.float(), s["rotary"]
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if s["paired"] else (y[..., :r // 2], y[..., r // 2:r])
        a, b = a * cos - b * sin, b * cos + a * sin
        both = torch.stack((a, b), -1).flatten(-2) if s["paired"] else torch.cat((a, b), -1)
        return torch.cat((both, y[..., r:]), -1).to(x.dtype)

    return {"q": turned(s["q"]), "k": turned(s["k"])}


def run(s):
    if own:
        from layer_streamed_nf4_lut_b200 import model as soup
        if s["op"] == "ce":
            weight = s["weight"] if s["grad"] else None
            weight2 = s["weight2"] if s["grad"] else None
            return soup.linear_ce(s["h"], s["w"], s["targets"], weight, s["targets2"], weight2)
        if s["op"] == "adamw":
            out = {"p": s["p"], "m": s["m"], "v": s["v"]}
            if s["bits"] == 8:
                soup.adamw_multi(s["params"], s["grads"], s["m"], s["v"], lr=1e-3, step=s["step"], weight_decay=s["decay"],
                                 m_scale=s["m_scale"], v_scale=s["v_scale"])
                out["m"], out["v"] = soup.adamw_state_values(s["m"], s["v"], s["m_scale"], s["v_scale"])
                return {**out, "m_scale": s["m_scale"], "v_scale": s["v_scale"]}
            soup.adamw_multi(s["params"], s["grads"], s["m"], s["v"], lr=1e-3, step=s["step"], weight_decay=s["decay"])
            return out
        c = _scaling(s)
        q, k = soup.rope(s["q"], s["k"], s["positions"], theta=c["theta"], rotary_dim=s["rotary"], interleaved=s["paired"],
                         scaling=c["kind"], factor=c["factor"], original_len=c["original"], low_freq_factor=c["low"],
                         high_freq_factor=c["high"], inverse=s["inverse"])
        return {"q": q, "k": k}
    return {"ce": _ce, "adamw": _adamw, "rope": _rope}[s["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without
def _counted(case):
    """Rows of a loss case that have a target, as expected over seeds."""
    T = case["T"]
    if case["pairs"]:
        third = T // case["pairs"] // 3
        return case["pairs"] * max(0, 2 * third - 1)
    return round((T - T // 512) * case["counted"])


def work(case):
    if case["op"] == "ce":
        rows, H, V = max(1, _counted(case)), case["hidden"], case["vocab"]
        two = case["pairs"] > 0
        size = 2 * V * H + 2 * rows * H + case["T"] * (4 + 8 + (8 if two else 0))
        if case["grad"]:
            size += 2 * case["T"] * H + case["T"] * (8 if two else 4)
        return {"bytes": size, "flops": 2 * rows * H * V * (2 if case["grad"] else 1)}
    if case["op"] == "adamw":
        n, wide = sum(_sizes(case)), {"float32": 4, "bfloat16": 2}
        state = 2 * (2 * 1 + 2 * 4 / BLOCK) + 2 * 2 if case["bits"] == 8 else 2 * 2 * 4  # coded state and its values
        return {"bytes": n * (2 * wide[case["param"]] + wide[case["grad"]] + state), "flops": 15 * n}
    heads, n = case["hq"] + case["hkv"], {"float32": 4, "bfloat16": 2}[case["type"]]
    return {"bytes": case["T"] * (2 * heads * case["d"] * n + 4), "flops": 3 * case["T"] * heads * case["rotary"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ce":
        w, out = s["w"].double(), []
        for rows in torch.arange(case["T"], device="cuda").split(256):
            logit = s["h"][rows].double() @ w.T
            lse = torch.logsumexp(logit, 1)
            hot = lambda t: torch.zeros_like(logit).scatter_(1, t.clamp(min=0)[:, None], (t >= 0).double()[:, None])  # noqa: E731
            t1 = s["targets"][rows].long()
            a = hot(t1)
            got = {"lse": torch.where(t1 >= 0, lse, 0.0), "logp": torch.where(t1 >= 0, (logit * a).sum(1) - lse, 0.0)}
            slope = torch.softmax(logit, 1)
            grad = (slope * a.sum(1, keepdim=True) - a) * s["weight"][rows].double()[:, None]
            if s["targets2"] is not None:
                t2 = s["targets2"][rows].long()
                b = hot(t2)
                got["logp2"] = torch.where(t2 >= 0, (logit * b).sum(1) - lse, 0.0)
                grad += (slope * b.sum(1, keepdim=True) - b) * s["weight2"][rows].double()[:, None]
            if case["grad"]:
                got["dh"] = grad @ w
            out.append(got)
        return {k: torch.cat([x[k] for x in out]) for k in out[0]}
    if case["op"] == "adamw":
        wide = lambda t: t if s["at"] is None else torch.zeros(s["m"].numel(), dtype=torch.float64, device="cuda").index_copy_(0, s["at"], t)  # noqa: E731
        g, p = wide(s["g"].double()), s["p"].double()
        m, v = s["m"].double(), s["v"].double()
        if case["bits"] == 8:
            m = torch.sign(m) * (m / 127) ** 2 * s["m_scale"].double().repeat_interleave(BLOCK)
            v = (v / 255) ** 4 * s["v_scale"].double().repeat_interleave(BLOCK)
        m, v = m + 0.1 * (g - m), v + 0.001 * (g * g - v)
        move = m / (1 - 0.9 ** s["step"]) / ((v / (1 - 0.999 ** s["step"])) ** 0.5 + 1e-8)
        move = move if s["at"] is None else move[s["at"]]
        out = {"p": p * (1 - 1e-3 * case["decay"]) - 1e-3 * move, "m": m, "v": v}
        if case["bits"] == 8:
            big = m.abs().view(-1, BLOCK).amax(1)
            top = v.view(-1, BLOCK).amax(1)
            many = lambda t: t.repeat_interleave(BLOCK)  # noqa: E731
            part = (m.abs() / many(big).clamp(min=1e-300)) ** 0.5
            out["m"] = torch.sign(m) * (torch.round(part * 127) / 127) ** 2 * many(big)
            part = (v / many(top).clamp(min=1e-300)) ** 0.25
            out["v"] = (torch.maximum(torch.round(part * 255), (v > 0).double()) / 255) ** 4 * many(top)
            out |= {"m_scale": big, "v_scale": top}
        return out
    c, r = _scaling(case), case["rotary"]
    base = c["theta"] * (c["factor"] ** (r / (r - 2)) if c["kind"] == "ntk" else 1.0)
    rate = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if c["kind"] == "linear":
        rate = [x / c["factor"] for x in rate]
    if c["kind"] in ("llama3", "yarn"):
        stay = [min(1.0, max(0.0, (c["original"] / (2 * math.pi / x) - c["low"]) / (c["high"] - c["low"]))) for x in rate]
        rate = [x / c["factor"] + y * (x - x / c["factor"]) for x, y in zip(rate, stay)]
    grow = 1.0 + 0.1 * math.log(c["factor"]) if c["kind"] == "yarn" else 1.0
    angle = s["positions"].double()[:, None] * torch.tensor(rate, dtype=torch.float64, device="cuda")
    unit = torch.polar(torch.full_like(angle, grow), -angle if case["inverse"] else angle)[:, None]

    def turned(x):
        x = x.double()
        head, tail = x[..., :r], x[..., r:]
        pairs = head.unflatten(-1, (r // 2, 2)) if case["paired"] else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
        both = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        both = both if case["paired"] else both.transpose(-1, -2)
        return torch.cat((both.flatten(-2), tail), -1)

    return {"q": turned(s["q"]), "k": turned(s["k"])}

"""The draft's step in serving, operator by operator: the cases that are measured, and each operator's plain form.

* ``norm``     root-mean-square norm with the residual's addition, out in 8-bit integers with a scale for each token
* ``matmul``   8-bit integer product with scales for each token and channel: hidden states to logits
* ``beam``     selection over beams and vocabulary by cumulative log-probability
* ``reorder``  the draft's states following the selected beams
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence drafting one token: what a step's latency is made of
        dict(name="norm-token", op="norm", M=1, d=4096, dtype="bf16", residual=True),
        # 64 sequences with 5 draft positions each
        dict(name="norm-step", op="norm", M=320, d=4096, dtype="bf16", residual=True),
        # a large batch, or a prompt's rows
        dict(name="norm-batch", op="norm", M=16384, d=4096, dtype="bf16", residual=True),
        # rows that start at no vector boundary, no residual
        dict(name="norm-odd", op="norm", M=257, d=1001, dtype="f32", residual=False),
        # one token through a head of a small vocabulary: the weights' bytes
        dict(name="matmul-token", op="matmul", M=1, K=4096, V=32000, dtype="bf16"),
        # 64 sequences with 5 draft positions: bytes and products about even
        dict(name="matmul-step", op="matmul", M=320, K=4096, V=128256, dtype="bf16"),
        # 256 sequences with 8 draft positions: the products
        dict(name="matmul-batch", op="matmul", M=2048, K=4096, V=151936, dtype="bf16"),
        # nothing a multiple of a tile, logits in 32 bits
        dict(name="matmul-odd", op="matmul", M=37, K=1001, V=3001, dtype="f32"),
        # one sequence growing a tree of four beams
        dict(name="beam-one", op="beam", B=1, W=4, V=32000, K=4, dtype="f32", T=1.0, frozen=False, first=False),
        # a batch of 64 with eight beams
        dict(name="beam-step", op="beam", B=64, W=8, V=128256, K=8, dtype="bf16", T=1.0, frozen=False, first=False),
        # one sequence's small draft cache
        dict(name="reorder-one", op="reorder", L=4, B=1, W=4, K=4, H=4, S=256, D=64, dtype="bf16"),
        # a batch's draft cache, sequences of different lengths
        dict(name="reorder-step", op="reorder", L=8, B=16, W=8, K=8, H=8, S=512, D=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "matmul", "beam", "reorder"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "norm":
        d = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            d = (d + 63) // 64 * 64
        return dict(op=op, M=min(_log(rng, 1, 16384), (1 << 25) // d), d=d, dtype=dtype, residual=rng.random() < 0.6)
    if op == "matmul":
        K = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            K = (K + 63) // 64 * 64
        V = _log(rng, 1000, 152000)
        M = _log(rng, 1, 2048)
        return dict(op=op, M=max(1, min(M, (1 << 40) // (K * V))), K=K, V=V, dtype=dtype)
    if op == "beam":
        V = _log(rng, 64, 152000)
        W = rng.randint(1, 16)
        B = max(1, min(_log(rng, 1, 256), (1 << 25) // (W * V)))
        return dict(op=op, B=B, W=W, V=V, K=min(rng.randint(1, 32), W * V), dtype=dtype, T=rng.choice((0.6, 0.7, 1.0, 1.5)),
                    frozen=rng.random() < 0.3, first=rng.random() < 0.2)
    L, H, D = rng.randint(1, 16), rng.randint(1, 16), rng.choice((8, 40, 64, 80, 128, 256))
    S, W, K = _log(rng, 1, 2048), rng.randint(1, 16), rng.randint(1, 16)
    B = max(1, min(_log(rng, 1, 64), (1 << 27) // (L * H * D * S * W)))
    return dict(op=op, L=L, B=B, W=W, K=K, H=H, S=S, D=D, dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def q8(rows, K):
        # rows start at multiples of 16 bytes, as the product takes them
        buf = torch.zeros(rows, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")
        q = buf[:, :K]
        step = max(1, (1 << 28) // K)
        for i in range(0, rows, step):
            n = min(step, rows - i)
            q[i:i + n] = (randn(n, K) * 32).round_().clamp_(-127, 127).to(torch.int8)
        return q

    if case["op"] == "norm":
        M, d = case["M"], case["d"]
        # hidden states whose rows differ in size, with a few large channels
        big = torch.where(rand(d) < 0.002, 20.0, 1.0)
        x = (randn(M, d) * big * (0.5 + rand(M, 1))).to(dt)
        r = randn(M, d).to(dt) if case["residual"] else None
        return dict(case=case, x=x, residual=r, weight=(1 + 0.1 * randn(d)).to(dt), eps=1e-6)
    if case["op"] == "matmul":
        M, K, V = case["M"], case["K"], case["V"]
        # scales of unit-variance states, and of weights that give logits a deviation of about 3
        return dict(case=case, a=q8(M, K), a_scale=0.02 + 0.02 * rand(M), w=q8(V, K),
                    w_scale=(0.5 + rand(V)) * (3.0 / (0.03 * 1024 * math.sqrt(K))), dtype=dt)
    if case["op"] == "beam":
        B, W, V = case["B"], case["W"], case["V"]
        logits = torch.empty(B, W, V, dtype=dt, device="cuda")
        for b in range(0, B, 16):
            n = min(16, B - b)
            logits[b:b + n] = (randn(n, W, V) * 3).to(dt)
        logits[:, :, rand(V) < 0.01] = -math.inf  # tokens the vocabulary does not allow
        scores = -10 * rand(B, W)
        if case["first"]:  # the first level: one beam holds the context
            scores[:, 0] = 0
            scores[:, 1:] = -math.inf
        frozen = (rand(B, W) < 0.25).to(torch.int32) if case["frozen"] else None
        return dict(case=case, logits=logits, scores=scores, temperature=torch.full((B,), case["T"], device="cuda"), frozen=frozen,
                    pad=2)
    L, B, W, K, H, S, D = (case[k] for k in ("L", "B", "W", "K", "H", "S", "D"))
    src = torch.empty(L, B, W, H, S, D, dtype=dt, device="cuda").normal_(generator=g)
    return dict(case=case, src=src, dst=torch.zeros(L, B, K, H, S, D, dtype=dt, device="cuda"),
                parent=torch.randint(0, W, (B, K), generator=g, device="cuda", dtype=torch.int32),
                lengths=torch.randint(1, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32))


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


# ---- the plain forms


def _norm_plain(s):
    # 64 bits: the rounding to integers has borders everywhere
    t = s["x"].double()
    if s["residual"] is not None:
        t = t + s["residual"].double()
    p = t * s["weight"].double()
    top = p.abs().amax(dim=1, keepdim=True)
    q = torch.where(top > 0, torch.round(p * 127 / top), 0.0)
    rms = torch.sqrt(t.square().mean(dim=1, keepdim=True) + s["eps"])
    scale = (top / (127 * rms)).float()
    out = dict(values=q.float() * scale, scale=scale[:, 0])
    if s["residual"] is not None:
        out["sum"] = t.to(s["x"].dtype)
    return out


def _matmul_plain(s):
    z = s["a"].float() @ s["w"].float().T
    return (z * s["a_scale"][:, None] * s["w_scale"][None, :]).to(s["dtype"])


def _beam_plain(s):
    # 64 bits: candidates of different beams meet at the selection's border
    B, W, V = s["logits"].shape
    K = s["case"]["K"]
    z = s["logits"].double() / s["temperature"].double()[:, None, None]
    top = z.amax(dim=2, keepdim=True)
    key = z - top
    key -= torch.log(torch.exp(key).sum(dim=2, keepdim=True))
    key += s["scores"].double()[:, :, None]
    if s["frozen"] is not None:
        hold = torch.full_like(key, -math.inf)
        hold[:, :, s["pad"]] = s["scores"].double()
        key = torch.where(s["frozen"][:, :, None] != 0, hold, key)
    best, at = torch.sort(key.reshape(B, W * V), dim=1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    none = best == -math.inf
    return dict(parent=torch.where(none, -1, at // V).int(), token=torch.where(none, -1, at % V).int(), score=best.float())


def _reorder_plain(s):
    src, dst, parent = s["src"], s["dst"], s["parent"].long()
    L, B, W, H, S, D = src.shape
    taken = src[:, torch.arange(B, device=src.device)[:, None], parent]
    live = torch.arange(S, device=src.device)[None, :] < s["lengths"][:, None]
    dst.copy_(torch.where(live[None, :, None, None, :, None], taken, dst))
    return dst


_plain = dict(norm=_norm_plain, matmul=_matmul_plain, beam=_beam_plain, reorder=_reorder_plain)


# ---- the framework's calls


def _norm_own(s):
    from speculative_decoding_verification_84_b200 import binding
    r = binding.q8_norm(s["x"], s["weight"], s["eps"], residual=s["residual"])
    # the values that the 8-bit integers stand for
    out = dict(values=torch.mul(r[0], r[1][:, None]), scale=r[1])
    if s["residual"] is not None:
        out["sum"] = r[2]
    return out


def _matmul_own(s):
    from speculative_decoding_verification_84_b200 import binding
    return binding.q8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], s["dtype"])


def _beam_own(s):
    from speculative_decoding_verification_84_b200 import binding
    parent, token, score = binding.beam_select(s["logits"], s["scores"], s["temperature"], s["case"]["K"],
                                               frozen=s["frozen"], pad_token=s["pad"])
    return dict(parent=parent, token=token, score=score)


def _reorder_own(s):
    from speculative_decoding_verification_84_b200 import binding
    return binding.beam_reorder(s["src"], s["parent"], out=s["dst"], lengths=s["lengths"])


_own = dict(norm=_norm_own, matmul=_matmul_own, beam=_beam_own, reorder=_reorder_own)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        M, d = case["M"], case["d"]
        return dict(bytes=M * d * (e * (3 if case["residual"] else 1) + 1) + d * e + 4 * M, flops=6 * M * d)
    if case["op"] == "matmul":
        M, K, V = case["M"], case["K"], case["V"]
        return dict(bytes=(M + V) * K + 4 * (M + V) + M * V * e, flops=2 * M * K * V)
    if case["op"] == "beam":
        B, W, V, K = case["B"], case["W"], case["V"], case["K"]
        rows = 1 if case["first"] else W
        return dict(bytes=B * (rows * V * e + 4 * W + 12 * K), flops=4 * B * rows * V)
    L, B, W, K, H, S, D = (case[k] for k in ("L", "B", "W", "K", "H", "S", "D"))
    # half the positions are live on average, and not every beam is someone's parent
    parents = W * (1 - (1 - 1 / W) ** K)
    return dict(bytes=L * B * H * D * e * (S + 1) / 2 * (parents + K) + 4 * B * (K + 1), flops=0)


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].to(torch.float64)
        if s["residual"] is not None:
            t = torch.add(t, s["residual"])
        y = t * torch.rsqrt((t * t).sum(1) / case["d"] + s["eps"])[:, None] * s["weight"]
        step = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127
        # the integers' borders do not depend on the norm: taken before it, where halves are exact
        p = s["weight"].to(torch.float64) * t
        q = (127 * p / torch.linalg.vector_norm(p, ord=math.inf, dim=1)[:, None]).nan_to_num().round()
        out = dict(values=q * step[:, None], scale=step)
        if s["residual"] is not None:
            out["sum"] = t
        return out
    if case["op"] == "matmul":
        a = s["a"].double().mul_(s["a_scale"].double()[:, None])
        return a @ s["w"].double().mul_(s["w_scale"].double()[:, None]).T
    if case["op"] == "beam":
        z = s["logits"].double().div_(s["temperature"].double().view(-1, 1, 1))
        z = z - torch.logsumexp(z, dim=2, keepdim=True) + s["scores"].double().unsqueeze(2)
        if s["frozen"] is not None:
            idle = s["frozen"] != 0
            z[idle] = -math.inf
            z[..., s["pad"]] = torch.where(idle, s["scores"].double(), z[..., s["pad"]])
        return dict(parent=None, token=None, score=z.flatten(1).topk(case["K"], dim=1).values)
    return None  # a copy: no computed numbers

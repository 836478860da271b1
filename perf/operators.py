"""Measured calls of the operators that stand around an FP8 projection in a layer:

* layer norm, forward (into BF16/FP32, or into the next GEMM's 1x128 E4M3 tiles) and backward;
* a mixture-of-experts layer for a few tokens over FP8 block-scaled expert weights;
* low-rank adapters of many requests beside a shared projection.

`own` selects the library's kernels; otherwise `run` computes the plain form in
elementary torch operations (FP32 arithmetic, one rounding at the end).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the pre-norm of a training step's forward pass, straight into the FP8 projection's operand
        dict(name="norm_tiles_8192", op="norm", M=8192, N=7168, dtype="bf16", tiles=True, bias=True),
        # one token of one request being served: a latency
        dict(name="norm_one_token", op="norm", M=1, N=7168, dtype="bf16", tiles=False, bias=True),
        # an odd width in FP32, rows padded to whole 16-byte units (a head or side network's norm)
        dict(name="norm_odd_f32", op="norm", M=1000, N=1111, dtype="f32", tiles=False, bias=False),
        # the same norm's backward pass in the training step
        dict(name="norm_bwd_8192", op="norm_bwd", M=8192, N=7168, dtype="bf16"),
        # an odd, ragged FP32 backward pass
        dict(name="norm_bwd_odd_f32", op="norm_bwd", M=333, N=2047, dtype="f32"),
        # one token decoded through an expert layer: top-8 of 256 experts, 7168 -> 2048 -> 7168
        dict(name="moe_1", op="moe", T=1, k=8, E=256, H=7168, I=2048, gated=True, absent=0.0),
        # 16 requests decoded together through the ungated up/down pair
        dict(name="moe_16_ungated", op="moe", T=16, k=8, E=64, H=7168, I=2048, gated=False, absent=0.0),
        # 128 requests decoded together, all experts on this GPU: the largest
        dict(name="moe_128", op="moe", T=128, k=8, E=256, H=7168, I=2048, gated=True, absent=0.0),
        # a small layer with ragged counts, some entries on another rank
        dict(name="moe_small", op="moe", T=5, k=3, E=7, H=384, I=256, gated=True, absent=0.3),
        # decoding: 64 requests, 64 adapters, beside a 7168 -> 18432 projection
        dict(name="lora_decode_64", op="lora", T=64, n=64, r=16, K=7168, N=18432, dtype="bf16", none=0.0),
        # prompts of a few adapters in one batch
        dict(name="lora_prompt_4096", op="lora", T=4096, n=8, r=64, K=7168, N=18432, dtype="bf16", none=0.1),
        # ragged: odd token count, a rank that fills no tile, FP32 projection output
        dict(name="lora_ragged_f32", op="lora", T=333, n=5, r=24, K=1032, N=2056, dtype="f32", none=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "moe", "moe", "lora", "lora"])
    if op in ("norm", "norm_bwd"):
        tiles = op == "norm" and rng.random() < 0.4
        N = 128 * _log(rng, 1, 128) if tiles else _log(rng, 33, 16384)
        M = _log(rng, 1, max(1, min(16384, 8192 * 7168 // N)))
        c = dict(op=op, M=M, N=N, dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "norm":
            c.update(tiles=tiles, bias=rng.random() < 0.7)
        return c
    if op == "moe":
        H, I = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 16)
        E = _log(rng, 2, 256)
        return dict(op=op, T=_log(rng, 1, 128), k=rng.randint(1, min(8, E)), E=E, H=H, I=I, gated=rng.random() < 0.6,
                    absent=rng.choice([0.0, 0.0, 0.5]))
    return dict(op=op, T=_log(rng, 1, 4096), n=_log(rng, 1, 128), r=8 * _log(rng, 1, 16), K=8 * _log(rng, 16, 896),
                N=8 * _log(rng, 16, 2304), dtype=rng.choice(["bf16", "bf16", "f32"]), none=rng.choice([0.0, 0.3]))


# ------------------------------------------------------------------ inputs
def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _rows(g, M, N, dt, scale=1.0):
    """[M][N] with rows padded to a multiple of 8 elements, N(0, scale) with a few outlier channels."""
    ld = (N + 7) // 8 * 8
    x = torch.randn((M, ld), generator=g, device="cuda") * scale
    some = torch.randint(0, N, (max(1, N // 1000),), generator=g, device="cuda")
    x[:, some] *= 20.0
    return x.to(dt)[:, :N]


def _routing(case, seed):
    """Zipf(1.1) routing over a seeded order of the experts, k different ones a token (Gumbel top-k);
    `absent`: the share of entries whose expert lives on another rank (id -1)."""
    r = np.random.default_rng([seed, case["T"], case["E"], case["k"]])
    p = (1.0 / np.arange(1, case["E"] + 1) ** 1.1)[r.permutation(case["E"])]
    score = np.log(p)[None, :] + r.gumbel(size=(case["T"], case["E"]))
    ids = np.argsort(-score, axis=1)[:, :case["k"]].astype(np.int32)
    ids[r.random(ids.shape) < case["absent"]] = -1
    return ids


def _fp8_weights(g, E, N, K):
    """E4M3 codes and 128x128 block scales of weights ~ N(0, 0.02): a block's largest magnitude is near 448."""
    w = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        c = torch.randn((min(step, E - e), N, K), generator=g, device="cuda").mul_(112.0).clamp_(-E4M3_MAX, E4M3_MAX)
        w[e:e + step] = c.to(torch.float8_e4m3fn).view(torch.uint8)
    sf = (torch.rand((E, N // 128, K // 128), generator=g, device="cuda") * 0.4 + 0.8) * (0.02 / 112.0)
    return w, sf


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] in ("norm", "norm_bwd"):
        M, N, dt = case["M"], case["N"], _dt(case)
        s["x"] = _rows(g, M, N, dt, 1.5)
        s["x"] += 0.25
        s["gamma"] = 1.0 + 0.1 * torch.randn(N, generator=g, device="cuda")
        s["beta"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case.get("bias") else None
        if case["op"] == "norm_bwd":
            s["dy"] = _rows(g, M, N, dt, 1e-3)
            x = s["x"].double()        # the statistics that the forward pass kept
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
    elif case["op"] == "moe":
        T, E, H, I = case["T"], case["E"], case["H"], case["I"]
        s["x"] = _rows(g, T, H, torch.bfloat16)
        s["ids"] = torch.from_numpy(_routing(case, seed)).cuda()
        s["w"] = torch.softmax(torch.randn((T, case["k"]), generator=g, device="cuda"), 1)
        s["wg"], s["sg"] = _fp8_weights(g, E, I, H) if case["gated"] else (None, None)
        s["wu"], s["su"] = _fp8_weights(g, E, I, H)
        s["wd"], s["sd"] = _fp8_weights(g, E, H, I)
    else:
        T, n, r, K, N = (case[v] for v in ("T", "n", "r", "K", "N"))
        s["x"] = _rows(g, T, K, torch.bfloat16)
        s["a"] = (torch.randn((n, r, K), generator=g, device="cuda") / math.sqrt(K)).bfloat16()
        s["b"] = (torch.randn((n, N, r), generator=g, device="cuda") / math.sqrt(r)).bfloat16()
        s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        s["base"] = torch.randn((T, N), generator=g, device="cuda").to(_dt(case))
        ids = torch.randint(0, n, (T,), generator=g, device="cuda")
        if T == n:
            ids = torch.randperm(n, generator=g, device="cuda")
        ids[torch.rand(T, generator=g, device="cuda") < case["none"]] = n     # group n: no adapter
        s["ids"] = ids
        # the batch's plan, kept for all layers: tokens by group, and the groups' bounds
        s["rows"] = torch.argsort(ids, stable=True).int()
        s["offsets"] = torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=n + 1).cumsum(0)]).int()
    return s


# ------------------------------------------------------------------ one pass
def _tiles(y):
    t = y.view(y.shape[0], -1, 128)
    sf = (t.abs().amax(2) / E4M3_MAX).clamp_min(1e-12)
    q = (t / sf[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view_as(y).to(torch.float8_e4m3fn)
    return q, sf.t()


def _dequant(w, sf):
    """FP32 weights of codes [A][N][K] and block scales [A][N/128][K/128]."""
    A, N, K = w.shape
    v = w.view(torch.float8_e4m3fn).float().view(A, N // 128, 128, K // 128, 128)
    return (v * sf[:, :, None, :, None]).view(A, N, K)


def _norm_plain(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["gamma"]
    if s["beta"] is not None:
        y = y + s["beta"]
    if s["tiles"]:
        return (*_tiles(y), mean, rstd)
    return y.to(s["x"].dtype), mean, rstd


def _norm_bwd_plain(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _moe_plain(s):
    x, ids = s["x"].float(), s["ids"]
    experts = torch.arange(s["E"], device=ids.device)
    used = (ids.reshape(-1, 1) == experts).any(0).nonzero()[:, 0]                 # the experts that any token picks
    share = ((ids[:, :, None] == used) * s["w"][:, :, None]).sum(1)               # [T][A]
    h = x @ _dequant(s["wu"][used], s["su"][used]).transpose(1, 2)                # [A][T][I]
    if s["gated"]:
        gate = x @ _dequant(s["wg"][used], s["sg"][used]).transpose(1, 2)
        h = gate * torch.sigmoid(gate) * h
    y = h @ _dequant(s["wd"][used], s["sd"][used]).transpose(1, 2)                # [A][T][H]
    return (y * share.t()[:, :, None]).sum(0).bfloat16()


def _lora_plain(s):
    n, r = s["n"], s["r"]
    v = s["x"].float() @ s["a"].float().view(n * r, -1).t()                       # every adapter's rank space
    mine = (s["ids"][:, None] == torch.arange(n, device=v.device)) * s["scale"]   # [T][n]
    v = (v.view(-1, n, r) * mine[:, :, None]).view(-1, n * r)
    return (s["base"].float() + v @ s["b"].float().transpose(1, 2).reshape(n * r, -1)).to(s["base"].dtype)


def run(s):
    if own:
        import fine_grained_fp8_x128_b200 as fp8q

        if s["op"] == "norm" and s["tiles"]:
            q, sf, mean, rstd = fp8q.layer_norm_quant(s["x"], s["gamma"], s["beta"], EPS)
            return q.view(torch.float8_e4m3fn), sf[:, :s["M"]], mean, rstd
        if s["op"] == "norm":
            return fp8q.layer_norm(s["x"], s["gamma"], s["beta"], EPS)
        if s["op"] == "norm_bwd":
            return fp8q.layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])
        if s["op"] == "moe":
            return fp8q.moe_few_tokens(s["x"], s["ids"], s["w"], s["wg"], s["sg"], s["wu"], s["su"], s["wd"], s["sd"])
        return fp8q.lora_apply(s["x"], s["rows"], s["offsets"], s["a"], s["b"], s["scale"], s["base"])
    return {"norm": _norm_plain, "norm_bwd": _norm_bwd_plain, "moe": _moe_plain, "lora": _lora_plain}[s["op"]](s)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_norm(s):
    x, N = s["x"].double(), s["N"]
    mean = x.sum(1) / N
    var = ((x - mean[:, None]) ** 2).sum(1) / N
    rstd = 1.0 / torch.sqrt(var + EPS)
    y = (x - mean[:, None]) * rstd[:, None] * s["gamma"].double()[None, :]
    if s["beta"] is not None:
        y += s["beta"].double()[None, :]
    if not s["tiles"]:
        return y, mean, rstd
    t = y.reshape(s["M"], N // 128, 128)
    sf = torch.clamp(t.abs().max(dim=2).values / E4M3_MAX, min=1e-12)
    return (t / sf[:, :, None]).reshape(s["M"], N), sf.t(), mean, rstd


def _exact_norm_bwd(s):
    dy, mean, r = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    xh = (s["x"].double() - mean) * r
    g = dy * s["gamma"].double()[None, :]
    c1, c2 = g.sum(1, keepdim=True) / s["N"], (g * xh).sum(1, keepdim=True) / s["N"]
    return (g - c1 - xh * c2) * r, (dy * xh).sum(0), dy.sum(0)


def _exact_moe(s):
    x, ids = s["x"].double(), s["ids"].cpu().numpy()
    w = s["w"].double()
    y = torch.zeros((s["T"], s["H"]), dtype=torch.float64, device=x.device)

    def mat(codes, sf, e):
        v = codes[e].view(torch.float8_e4m3fn).to(torch.float64)
        return v * sf[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)

    for e in range(s["E"]):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        rows, share = torch.from_numpy(t).to(x.device), w[torch.from_numpy(t), torch.from_numpy(j)]
        h = x[rows] @ mat(s["wu"], s["su"], e).t()
        if s["gated"]:
            gate = x[rows] @ mat(s["wg"], s["sg"], e).t()
            h = h * gate / (1.0 + torch.exp(-gate))
        y.index_add_(0, rows, share[:, None] * (h @ mat(s["wd"], s["sd"], e).t()))
    return y


def _exact_lora(s):
    out = s["base"].double()
    for i in range(s["n"]):
        t = torch.nonzero(s["ids"] == i)[:, 0]
        if len(t):
            v = s["x"][t].double() @ s["a"][i].double().t()
            out[t] += s["scale"][i].double() * (v @ s["b"][i].double().t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "moe": _exact_moe, "lora": _exact_lora}[case["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        e = 4 if case["dtype"] == "f32" else 2
        out = 1 + 4 / 128 if case["tiles"] else e
        return {"bytes": case["M"] * case["N"] * (e + out) + 4 * case["N"] * (2 if case["bias"] else 1) + 8 * case["M"],
                "flops": 8 * case["M"] * case["N"]}
    if case["op"] == "norm_bwd":
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 3 * e * case["M"] * case["N"] + 12 * case["N"] + 8 * case["M"], "flops": 14 * case["M"] * case["N"]}
    if case["op"] == "moe":
        # the experts that are picked, as the mean over a few routings of the same kind
        picked = [_routing(case, 1000 + i) for i in range(8)]
        active = sum(len(np.unique(p[p >= 0])) for p in picked) / 8
        entries = sum(int((p >= 0).sum()) for p in picked) / 8
        mats = (3 if case["gated"] else 2) * case["H"] * case["I"]
        return {"bytes": active * mats * (1 + 4 / 16384) + 4 * case["T"] * case["H"] + 8 * case["T"] * case["k"],
                "flops": 2 * entries * mats}
    T, n, r, K, N = (case[v] for v in ("T", "n", "r", "K", "N"))
    e = 4 if case["dtype"] == "f32" else 2
    some = (1 - case["none"]) * T
    used = n if T == n else n * (1 - (1 - 1 / n) ** some)
    return {"bytes": some * 2 * K + 2 * e * T * N + used * 2 * r * (K + N) + 4 * T, "flops": 2 * some * r * (K + N)}

"""Cases and plain forms of the routed layer's training operators and of its fused dense product.

Operators (shapes as in include/moe.h; all activations and weights bf16 unless said otherwise):

* ``ffn``          one training step of the experts' gated feed-forward block: the forward pass
                   over expert-contiguous rows (both projections, SwiGLU, down projection) and
                   its backward pass.  Outputs y, dxp, dw_gate, dw_up, dw_down.
* ``combine_bwd``  the backward pass of the weighted combine: the gradient of every expert row
                   and of every routing weight.  Outputs dy, dw (fp32).
* ``dense``        out = act(a w^T + bias) + residual.
* ``dense_bwd``    the gradients of act(a w^T + bias) with respect to a, w and bias, from the
                   kept pre-activations (fp32).  Outputs da, dw, dbias (fp32).

Where ``own`` is true, ``run`` calls the library; otherwise it computes the same in plain torch
operations in fp32, rounded once at the end.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # a tiny layer: latency
        dict(name="ffn_tiny", op="ffn", T=64, K=2, E=8, H=256, F=512, skew=0.0),
        # odd widths, a skewed router, experts without rows
        dict(name="ffn_ragged", op="ffn", T=1111, K=3, E=40, H=1032, F=520, skew=1.0),
        # the Qwen3-30B-A3B layer at 4096 tokens: 256 rows an expert on average
        dict(name="ffn_qwen3", op="ffn", T=4096, K=8, E=128, H=2048, F=768, skew=0.0),
        # one rank's 32 of DeepSeek-R1's 256 experts, 2048 tokens' worth of assignments
        dict(name="ffn_r1_share", op="ffn", T=2048, K=8, E=32, H=7168, F=2048, skew=0.3),
        # odd width, few tokens
        dict(name="combine_bwd_ragged", op="combine_bwd", T=515, K=3, H=1032),
        # the DeepSeek-R1 prefill layer
        dict(name="combine_bwd_r1", op="combine_bwd", T=8192, K=8, H=7168),
        # one token through the latent layer's up-projection
        dict(name="dense_one_token", op="dense", M=1, N=7168, K=2048, act="none", bias=True, residual=True),
        # a few decoded tokens through its down-projection
        dict(name="dense_16_tokens", op="dense", M=16, N=2048, K=7168, act="silu", bias=True, residual=False),
        # odd sizes, every part of the epilogue
        dict(name="dense_ragged", op="dense", M=1001, N=1544, K=1032, act="gelu", bias=True, residual=True),
        # the latent layer's up-projection at 4096 tokens, added to the residual stream
        dict(name="dense_latent_up", op="dense", M=4096, N=7168, K=2048, act="none", bias=True, residual=True),
        # odd sizes
        dict(name="dense_bwd_ragged", op="dense_bwd", M=333, N=776, K=520, act="gelu"),
        # the latent layer's down-projection at 4096 tokens with an activation
        dict(name="dense_bwd_latent_down", op="dense_bwd", M=4096, N=2048, K=7168, act="silu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_mult8(rng, lo, hi):
    return 8 * _log_int(rng, lo // 8, hi // 8)


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def draw(rng):
    largest = {c["op"]: max(_cost(x) for x in listed() if x["op"] == c["op"]) for c in listed()}
    op = rng.choice(("ffn", "ffn", "dense", "dense", "combine_bwd", "dense_bwd"))
    while True:
        if op == "ffn":
            c = dict(op=op, T=_log_int(rng, 1, 4096), E=_log_int(rng, 1, 128), H=_log_mult8(rng, 64, 7168),
                     F=_log_mult8(rng, 64, 2048), skew=rng.choice((0.0, 0.3, 1.0)))
            c["K"] = rng.randint(1, min(8, c["E"]))
            if c["E"] * c["H"] * c["F"] > 32 * 7168 * 2048:
                continue
        elif op == "combine_bwd":
            c = dict(op=op, T=_log_int(rng, 1, 8192), K=rng.randint(1, 16), H=_log_mult8(rng, 64, 7168))
        elif op == "dense":
            c = dict(op=op, M=_log_int(rng, 1, 4096), N=_log_mult8(rng, 64, 7168), K=_log_mult8(rng, 64, 7168),
                     act=rng.choice(ACTS), bias=rng.random() < 0.7, residual=rng.random() < 0.6)
        else:
            c = dict(op=op, M=_log_int(rng, 1, 4096), N=_log_mult8(rng, 64, 7168), K=_log_mult8(rng, 64, 7168),
                     act=rng.choice(ACTS))
        if _cost(c) <= largest[op]:
            return c


def _cost(case):
    w = work(case)
    return max(w["flops"] / 1.4e15, w["bytes"] / 6.5e12)


def work(case):
    op = case["op"]
    if op == "ffn":
        rows, E, H, F = case["T"] * case["K"], case["E"], case["H"], case["F"]
        # xp, dy in; y, dxp out; the weights in; their gradients out; the offsets
        return {"bytes": 4 * rows * H * 2 + 2 * 3 * E * H * F * 2 + 4 * (E + 1), "flops": 18 * rows * H * F}
    if op == "combine_bwd":
        T, K, H = case["T"], case["K"], case["H"]
        return {"bytes": T * H * 2 + 2 * T * K * H * 2 + 3 * T * K * 4, "flops": 3 * T * K * H}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "dense":
        extra = (4 * N if case["bias"] else 0) + (2 * M * N if case["residual"] else 0)
        return {"bytes": 2 * (M * K + N * K + M * N) + extra, "flops": 2 * M * N * K}
    # dout (bf16), pre (fp32), a, w in; da, dw, dbias out.  Without an activation the
    # pre-activations are not needed.
    pre = 0 if case["act"] == "none" else 4 * M * N
    return {"bytes": 2 * M * N + pre + 2 * (2 * M * K + 2 * N * K) + 4 * N, "flops": 4 * M * N * K}


def _randn(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def _rows_per_expert(case, seed):
    """Rows of each expert: every token's K assignments drawn with popularity (r + 1)^-skew."""
    rng = np.random.RandomState(seed % (2 ** 31))
    p = (1.0 + np.arange(case["E"])) ** -case["skew"]
    return rng.multinomial(case["T"] * case["K"], rng.permutation(p / p.sum()))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=dict(case))
    e = lambda shape, dt=BF16: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if op == "ffn":
        rows, E, H, F = case["T"] * case["K"], case["E"], case["H"], case["F"]
        n = _rows_per_expert(case, seed)
        s["most"] = int(n.max())
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
        s["xp"], s["dy"] = _randn(g, (rows, H)), _randn(g, (rows, H))
        s["w_gate"], s["w_up"] = _randn(g, (E, F, H), H ** -0.5), _randn(g, (E, F, H), H ** -0.5)
        s["w_down"] = _randn(g, (E, H, F), F ** -0.5)
        # the buffers that a training program keeps for a layer
        s["buf"] = dict(g=e((rows, F), torch.float32), u=e((rows, F), torch.float32), h=e((rows, F)), y=e((rows, H)),
                        dg=e((rows, F)), du=e((rows, F)), dxp=e((rows, H)), dw_gate=e((E, F, H)), dw_up=e((E, F, H)),
                        dw_down=e((E, H, F)))
    elif op == "combine_bwd":
        T, K, H = case["T"], case["K"], case["H"]
        s["dout"], s["y"] = _randn(g, (T, H)), _randn(g, (T * K, H))
        s["row_of_assign"] = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32)
        s["topk_w"] = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), -1)
        s["buf"] = dict(dy=e((T * K, H)), dw=e((T, K), torch.float32))
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["w"] = _randn(g, (M, K)), _randn(g, (N, K), K ** -0.5)
        if op == "dense":
            s["bias"] = torch.randn((N,), generator=g, device="cuda") if case["bias"] else None
            s["residual"] = _randn(g, (M, N)) if case["residual"] else None
            s["buf"] = dict(out=e((M, N)))
        else:
            s["dout"] = _randn(g, (M, N))
            s["pre"] = torch.randn((M, N), generator=g, device="cuda")
            s["buf"] = dict(dpre=e((M, N)), da=e((M, K)), dw=e((N, K)), dbias=e((N,), torch.float32))
    return s


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    from routing_dispatch_grouped_top_b200 import binding as B
    c, b = s["case"], s["buf"]
    op = c["op"]
    if op == "ffn":
        if "ws" not in s:  # dims and workspace: kept by the program for the layer
            s["d"] = B.dims(c["T"], c["H"], c["E"], c["K"], c["F"])
            s["ws"] = B.make_workspace(s["d"])
        d, ws, off = s["d"], s["ws"], s["offsets"]
        B.moe_grouped_gate_up_train(s["xp"], off, s["w_gate"], s["w_up"], d, b["g"], b["u"], b["h"], ws)
        B.moe_grouped_down(b["h"], off, s["w_down"], d, b["y"], ws)
        B.moe_grouped_ffn_backward(s["xp"], b["g"], b["u"], b["h"], s["dy"], off, s["w_gate"], s["w_up"], s["w_down"],
                                   d, b["dg"], b["du"], b["dxp"], b["dw_gate"], b["dw_up"], b["dw_down"], ws)
        return {k: b[k] for k in ("y", "dxp", "dw_gate", "dw_up", "dw_down")}
    if op == "combine_bwd":
        if "d" not in s:
            s["d"] = B.dims(c["T"], c["H"], c["K"], c["K"], 8)
        B.moe_combine_backward(s["dout"], s["y"], s["row_of_assign"], s["topk_w"], s["d"], b["dy"], b["dw"])
        return {"dy": b["dy"], "dw": b["dw"]}
    if "ws" not in s:
        s["ws"] = B.make_dense_workspace(c["M"], c["N"], c["K"])
    if op == "dense":
        B.moe_dense_epilogue(s["a"], s["w"], b["out"], s["ws"], bias=s["bias"], act=c["act"], residual=s["residual"])
        return b["out"]
    B.moe_dense_backward(s["dout"], s["a"], s["w"], s["pre"], b["dpre"], b["da"], b["dw"], b["dbias"], s["ws"],
                         act=c["act"])
    return {"da": b["da"], "dw": b["dw"], "dbias": b["dbias"]}


# ---------------------------------------------------------------------------
# Plain forms (fp32, rounded once at the end)
# ---------------------------------------------------------------------------

def _ffn_plain(s):
    """Every expert's rows padded to the longest group, then batched products."""
    off, most = s["offsets"].long(), s["most"]
    rows, E = s["xp"].shape[0], off.numel() - 1
    row = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(off[1:].contiguous(), row, right=True)
    at = expert * most + row - off[expert]

    def padded(t):
        p = torch.zeros((E * most, t.shape[1]), device="cuda")
        p[at] = t.float()
        return p.view(E, most, -1)

    def packed(t):
        return t.reshape(E * most, -1)[at].to(BF16)

    x, dy = padded(s["xp"]), padded(s["dy"])
    wg, wu, wd = s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    g, u = x @ wg.transpose(1, 2), x @ wu.transpose(1, 2)
    sig = 1.0 / (1.0 + torch.exp(-g))
    h = g * sig * u
    y = packed(h @ wd.transpose(1, 2))
    dw_down = (dy.transpose(1, 2) @ h).to(BF16)
    dh = dy @ wd
    dg = dh * u * sig * (1.0 + g * (1.0 - sig))
    du = dh * g * sig
    dxp = packed(dg @ wg + du @ wu)
    return {"y": y, "dxp": dxp, "dw_gate": (dg.transpose(1, 2) @ x).to(BF16),
            "dw_up": (du.transpose(1, 2) @ x).to(BF16), "dw_down": dw_down}


def _combine_bwd_plain(s):
    T, K = s["topk_w"].shape
    roa = s["row_of_assign"].long()
    dout = s["dout"].float()
    dy = torch.empty_like(s["y"])
    dy[roa] = (s["topk_w"][:, :, None] * dout[:, None, :]).reshape(T * K, -1).to(BF16)
    dw = (s["y"][roa].float().view(T, K, -1) * dout[:, None, :]).sum(-1)
    return {"dy": dy, "dw": dw}


def _erf(x):
    return torch.special.erf(x)


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + _erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    return x


def _dact(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + _erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (x + 0.044715 * x ** 3))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def _dense_plain(s):
    v = s["a"].float() @ s["w"].float().T
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _act(v, s["case"]["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(BF16)


def _dense_bwd_plain(s):
    dpre = s["dout"].float() * _dact(s["pre"], s["case"]["act"])
    return {"da": (dpre @ s["w"].float()).to(BF16), "dw": (dpre.T @ s["a"].float()).to(BF16), "dbias": dpre.sum(0)}


_PLAIN = {"ffn": _ffn_plain, "combine_bwd": _combine_bwd_plain, "dense": _dense_plain, "dense_bwd": _dense_bwd_plain}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    s.pop("buf")
    op = case["op"]
    f64 = torch.float64
    if op == "ffn":
        # expert by expert; the gradients from the derivative of silu written with tanh:
        # sigma(g) = (1 + tanh(g / 2)) / 2
        off = s["offsets"].tolist()
        out = dict(y=torch.empty(s["xp"].shape, dtype=f64), dxp=torch.empty(s["xp"].shape, dtype=f64),
                   dw_gate=torch.empty(s["w_gate"].shape, dtype=f64), dw_up=torch.empty(s["w_up"].shape, dtype=f64),
                   dw_down=torch.empty(s["w_down"].shape, dtype=f64))
        out = {k: v.cuda() for k, v in out.items()}
        for e in range(case["E"]):
            r = slice(off[e], off[e + 1])
            x, dy = s["xp"][r].to(f64), s["dy"][r].to(f64)
            wg, wu, wd = s["w_gate"][e].to(f64), s["w_up"][e].to(f64), s["w_down"][e].to(f64)
            g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
            sigma = (torch.tanh(g / 2) + 1) / 2
            silu = g * sigma
            out["y"][r] = torch.mm(silu * u, wd.t())
            out["dw_down"][e] = torch.mm(dy.t(), silu * u)
            dh = torch.mm(dy, wd)
            dg, du = dh * u * (sigma + silu - silu * sigma), dh * silu
            out["dxp"][r] = torch.mm(torch.cat([dg, du], 1), torch.cat([wg, wu], 0))
            out["dw_gate"][e], out["dw_up"][e] = torch.mm(dg.t(), x), torch.mm(du.t(), x)
        return out
    if op == "combine_bwd":
        T, K = s["topk_w"].shape
        inv = torch.empty_like(s["row_of_assign"]).long()
        inv[s["row_of_assign"].long()] = torch.arange(T * K, device="cuda")  # row -> assignment
        token = inv // K
        dout = s["dout"].to(f64)
        dy = s["topk_w"].to(f64).reshape(-1)[inv][:, None] * dout[token]
        dots = (s["y"].to(f64) * dout[token]).sum(1)
        dw = torch.empty(T * K, dtype=f64, device="cuda")
        dw[inv] = dots
        return {"dy": dy, "dw": dw.view(T, K)}
    if op == "dense":
        v = torch.mm(s["a"].to(f64), s["w"].to(f64).t())
        v = _act64(v + s["bias"].to(f64) if case["bias"] else v, case["act"])
        return v + s["residual"].to(f64) if case["residual"] else v
    dpre = s["dout"].to(f64) * _dact64(s["pre"].to(f64), case["act"])
    return {"da": torch.mm(dpre, s["w"].to(f64)), "dw": torch.mm(dpre.t(), s["a"].to(f64)), "dbias": dpre.sum(0)}


def _act64(x, act):
    half_erfc = lambda z: 0.5 * torch.special.erfc(z)  # noqa: E731
    return {"none": lambda: x, "relu": lambda: x.clamp(min=0), "silu": lambda: x * (torch.tanh(x / 2) + 1) / 2,
            "gelu": lambda: x * half_erfc(-x / math.sqrt(2)),
            "gelu_tanh": lambda: x / (1 + torch.exp(-2 * _z64(x)))}[act]()


def _z64(x):
    return math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)


def _dact64(x, act):
    if act == "gelu_tanh":  # x sigma(2 z(x)): sigma + 2 x z' sigma (1 - sigma)
        sg = 1 / (1 + torch.exp(-2 * _z64(x)))
        return sg + 2 * x * math.sqrt(2 / math.pi) * (1 + 0.134145 * x * x) * sg * (1 - sg)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-x / math.sqrt(2)) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        sg = (torch.tanh(x / 2) + 1) / 2
        return sg + x * sg * (1 - sg)
    return (x > 0).to(x.dtype) if act == "relu" else torch.ones_like(x)

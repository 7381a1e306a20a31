"""The training pass (gated feed-forward block, combine) and the dense product with a fused epilogue
against plain 64-bit formulas.

Tolerances.  u8 = 2^-8 is half a bf16 step relative to a value, u24 = 2^-24 half an fp32 step.  A sum
of n products accumulated in fp32 is off by at most n 2 u24 times the sum of the products' magnitudes
(2 u24: the tensor core may truncate).  Where an operand was rounded to bf16 first, u8 times that sum of
magnitudes is added, and u8 |result| for the rounding of a bf16 result; an error of an operand
itself is carried through by its magnitude.  The fast exponential and divide keep sigma(g) within
2^-19 (|g| < 32).  Every check is element by element against such a bound.  A second check bounds the
2-norm of the error: independent roundings have a relative rms of at most 2^-8 / sqrt(3) = 2.26e-3
each (uniform in the half step at its largest), so `parts` of them at most sqrt(parts) times that.
"""
import math
import re

import pytest
import torch

from routing_dispatch_grouped_top_b200 import binding as B
from routing_dispatch_grouped_top_b200 import build, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U8, U24, SIG = 2.0 ** -8, 2.0 ** -24, 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    B.lib()


def randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def within(name, got, ref, bound, parts=None):
    got, ref = got.to(F64), ref.to(F64)
    assert got.shape == ref.shape
    over = (got - ref).abs() - bound
    assert not torch.isnan(got).any(), f"{name}: NaN"
    assert (over <= 0).all(), f"{name}: {int((over > 0).sum())} of {over.numel()} over the bound, by {over.max():.3e}"
    if parts and ref.numel() >= 4096:
        rel = ((got - ref).norm() / ref.norm()).item()
        assert rel <= math.sqrt(parts) * U8 / math.sqrt(3), f"{name}: relative error {rel:.3e}"


# ---------------------------------------------------------------------------
# Gated feed-forward block
# ---------------------------------------------------------------------------

def ffn_inputs(counts, H, F, seed=0, pad=0):
    """counts: rows of each expert; `pad` rows behind the last one."""
    E, rows = len(counts), sum(counts) + pad
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=DEV)
    return dict(E=E, H=H, F=F, rows=rows, counts=counts, offsets=off, xp=randn((rows, H), seed + 1),
                dy=randn((rows, H), seed + 2), w_gate=randn((E, F, H), seed + 3, H ** -0.5),
                w_up=randn((E, F, H), seed + 4, H ** -0.5), w_down=randn((E, H, F), seed + 5, F ** -0.5))


def ffn_buffers(p, grad=BF, fill=float("nan")):
    f = lambda shape, dt=BF: torch.full(shape, fill, dtype=dt, device=DEV)  # noqa: E731
    E, H, F, R = p["E"], p["H"], p["F"], p["rows"]
    return dict(g=f((R, F), F32), u=f((R, F), F32), h=f((R, F)), y=f((R, H)), dg=f((R, F)), du=f((R, F)),
                dxp=f((R, H)), dw_gate=f((E, F, H), grad), dw_up=f((E, F, H), grad), dw_down=f((E, H, F), grad))


def dims_of(p):
    return B.dims(T=p["rows"], H=p["H"], E=p["E"], K=1, F=p["F"])


def ffn_forward(p, b, ws, d, **kw):
    B.moe_grouped_gate_up_train(p["xp"], p["offsets"], p["w_gate"], p["w_up"], d, b["g"], b["u"], b["h"], ws, **kw)


def ffn_backward(p, b, ws, d, **kw):
    B.moe_grouped_ffn_backward(p["xp"], b["g"], b["u"], b["h"], p["dy"], p["offsets"], p["w_gate"], p["w_up"],
                               p["w_down"], d, b["dg"], b["du"], b["dxp"], b["dw_gate"], b["dw_up"], b["dw_down"], ws,
                               **kw)


def ffn_reference(p):
    """Expert by expert in 64 bits: the results and, under "~name", the bound on each element's error."""
    out = {}
    for e in range(p["E"]):
        r = slice(int(p["offsets"][e]), int(p["offsets"][e + 1]))
        n, H, F = r.stop - r.start, p["H"], p["F"]
        x, dy = p["xp"][r].to(F64), p["dy"][r].to(F64)
        wg, wu, wd = (p[k][e].to(F64) for k in ("w_gate", "w_up", "w_down"))
        g, u = x @ wg.T, x @ wu.T
        eg, eu = (2 * H * U24 * (x.abs() @ w.T.abs()) for w in (wg, wu))
        s = 1 / (1 + torch.exp(-g))
        h = g * s * u
        # |d silu / dg| <= 1.1; sigma's own error
        eh = 1.1 * eg * u.abs() + (g * s).abs() * eu + SIG * h.abs()
        eh_r = eh + U8 * (h.abs() + eh)
        dh = dy @ wd
        edh = 2 * H * U24 * (dy.abs() @ wd.abs())
        ds = s * (1 + g * (1 - s))
        dg, du = dh * u * ds, dh * g * s
        # |d^2 silu / dg^2| <= 0.5; ds is off by sigma's error times 1 + |g|
        edg = edh * (u * ds).abs() + (dh * ds).abs() * eu + (dh * u).abs() * (0.5 * eg + 2 * SIG * (1 + g.abs()))
        edu = edh * (g * s).abs() + dh.abs() * (1.1 * eg + SIG * (g * s).abs())
        edg_r, edu_r = edg + U8 * (dg.abs() + edg), edu + U8 * (du.abs() + edu)
        res = {"g": (g, eg), "u": (u, eu), "h": (h, eh_r), "dg": (dg, edg_r), "du": (du, edu_r)}

        def product(a, ea, b):  # a b with a off by ea, n terms
            k = a.shape[1]
            m = a.abs() @ b.abs()
            return a @ b, ea @ b.abs() + 2 * k * U24 * (m + ea @ b.abs())

        def rounded(v, ev):
            return v, ev + U8 * (v.abs() + ev)

        res["y"] = rounded(*product(h, eh_r, wd.T))
        a, ea = product(dg, edg_r, wg)
        b, eb = product(du, edu_r, wu)
        res["dxp"] = rounded(a + b, ea + eb + 2 * U24 * (a.abs() + b.abs()))
        res["dw_gate"] = product(dg.T, edg_r.T, x)
        res["dw_up"] = product(du.T, edu_r.T, x)
        v, ev = product(h.T, eh_r.T, dy)
        res["dw_down"] = (v.T, ev.T)
        for k, (v, ev) in res.items():
            out.setdefault(k, []).append(v)
            out.setdefault("~" + k, []).append(ev)
    for k in out:
        out[k] = torch.stack(out[k]) if k.lstrip("~").startswith("dw") else torch.cat(out[k])
    return out


FFN_CASES = [  # counts, H, F
    ([5], 8, 8),
    ([1], 64, 64),
    ([64, 64], 64, 128),
    ([0, 1, 15, 16, 17, 0, 63, 64, 65, 0], 136, 72),
    ([127, 128, 129, 0, 255, 256, 257, 3], 264, 520),
    ([0, 0, 0, 700, 0], 1032, 264),
    ([31, 33, 95, 97, 47, 8, 4, 2, 1, 12], 256, 768),
    ([1] * 130, 72, 264),
    ([513, 300], 2048, 776),
    # enough tiles for the CTA pairs in every product: many groups; few long ones, ragged widths
    ([200, 0, 300, 64, 1, 17] * 6, 520, 776),
    ([1300, 2500, 3001], 1032, 1032),
    ([0, 90, 0, 0, 257, 33, 48, 16] * 8, 72, 264),
]


@pytest.mark.parametrize("counts,H,F", FFN_CASES)
def test_ffn_training_step(counts, H, F):
    p = ffn_inputs(counts, H, F, seed=sum(counts) + H)
    b, d = ffn_buffers(p), dims_of(p)
    ws = B.make_workspace(d)
    ffn_forward(p, b, ws, d)
    B.moe_grouped_down(b["h"], p["offsets"], p["w_down"], d, b["y"], ws)
    ffn_backward(p, b, ws, d)
    assert B.read_device_status(ws) == 0
    ref = ffn_reference(p)
    for k in ("g", "u"):
        within(k, b[k], ref[k], ref["~" + k])
    for k in ("h", "dg", "du"):
        within(k, b[k], ref[k], ref["~" + k], parts=1)
    for k in ("y", "dxp"):
        within(k, b[k], ref[k], ref["~" + k], parts=2)
    for k in ("dw_gate", "dw_up", "dw_down"):
        within(k, b[k], ref[k], ref["~" + k] + U8 * (ref[k].abs() + ref["~" + k]), parts=2)


# (the last one: many tiles, the CTA-pair kernels)
@pytest.mark.parametrize("counts,H,F", [FFN_CASES[3], FFN_CASES[4], ([31, 33, 95, 97, 0, 8, 4, 2, 1, 300] * 3, 136, 264)])
def test_ffn_fp32_gradients_and_accumulation(counts, H, F):
    p = ffn_inputs(counts, H, F, seed=7)
    d = dims_of(p)
    ws = B.make_workspace(d)
    b = ffn_buffers(p, grad=F32)
    ffn_forward(p, b, ws, d)
    ffn_backward(p, b, ws, d)
    ref = ffn_reference(p)
    names = ("dw_gate", "dw_up", "dw_down")
    once = {k: b[k].clone() for k in names}
    for k in names:
        within(k, b[k], ref[k], ref["~" + k], parts=1)
    start = {k: randn(b[k].shape, 11, dtype=F32) for k in names}
    for k in names:
        b[k].copy_(start[k])
    ffn_backward(p, b, ws, d, accumulate=True)
    for k in names:  # one fp32 addition
        assert torch.equal(b[k], start[k] + once[k]), k
    assert B.read_device_status(ws) == 0


@pytest.mark.parametrize("copies", [1, 8])   # few tiles, many tiles
def test_ffn_nan_rows_stay_with_their_expert(copies):
    counts = [37, 0, 5, 64, 1, 90] * copies
    p = ffn_inputs(counts, 136, 200, seed=3, pad=9)
    d = dims_of(p)
    ws = B.make_workspace(d)
    clean, dirty = ffn_buffers(p, fill=0.0), ffn_buffers(p, fill=0.0)
    ffn_forward(p, clean, ws, d)
    ffn_backward(p, clean, ws, d)
    bad = 3
    lo, hi, end = int(p["offsets"][bad]), int(p["offsets"][bad + 1]), int(p["offsets"][-1])
    for k, v in (("xp", float("nan")), ("dy", float("inf"))):
        p[k][lo:hi] = v
        p[k][end:] = float("nan")
    for k in ("g", "u", "h", "dg", "du", "dxp"):
        dirty[k][end:] = 7.0
    ffn_forward(p, dirty, ws, d)
    for k in ("g", "u", "h"):  # rows behind the last one hold anything
        assert (dirty[k][end:] == 7.0).all()
        dirty[k][end:] = float("nan")
    ffn_backward(p, dirty, ws, d)
    others = [e for e in range(len(counts)) if e != bad]
    for k in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(clean[k][others], dirty[k][others]), k
        assert not torch.isfinite(dirty[k][bad]).any()
    for k in ("dg", "du", "dxp"):
        assert torch.equal(clean[k][:lo], dirty[k][:lo]) and torch.equal(clean[k][hi:end], dirty[k][hi:end]), k
        assert (dirty[k][end:] == 7.0).all()
    for k in ("dw_gate", "dw_up", "dw_down"):
        assert (clean[k][1] == 0).all()   # an expert without rows
    assert B.read_device_status(ws) == 0


def test_ffn_gradients_against_differences():
    """Central differences of <dy, y> in 64 bits along random directions, against the gradients:
    a check of the formulas that shares nothing with them."""
    p = ffn_inputs([7, 0, 20], 64, 48, seed=5)
    d = dims_of(p)
    ws, b = B.make_workspace(d), ffn_buffers(p, grad=F32)
    ffn_forward(p, b, ws, d)
    ffn_backward(p, b, ws, d)

    def loss(q):
        total = 0.0
        for e in range(p["E"]):
            r = slice(int(p["offsets"][e]), int(p["offsets"][e + 1]))
            g, u = q["xp"][r] @ q["w_gate"][e].T, q["xp"][r] @ q["w_up"][e].T
            total += (p["dy"][r].to(F64) * ((g / (1 + torch.exp(-g)) * u) @ q["w_down"][e].T)).sum().item()
        return total

    q = {k: p[k].to(F64) for k in ("xp", "w_gate", "w_up", "w_down")}
    grads = dict(xp=b["dxp"], w_gate=b["dw_gate"], w_up=b["dw_up"], w_down=b["dw_down"])
    for k, grad in grads.items():
        # a direction with positive overlap, so that the derivative is not a cancelled sum
        v = grad.to(F64).sign() * randn(grad.shape, 13, dtype=F64).abs()
        eps = 1e-4
        diff = (loss({**q, k: q[k] + eps * v}) - loss({**q, k: q[k] - eps * v})) / (2 * eps)
        # each gradient element is within 3 roundings of bf16 operands and result
        assert abs((grad.to(F64) * v).sum().item() - diff) <= 3 * U8 * (grad.to(F64).abs() * v.abs()).sum().item() + 1e-6 * abs(diff)


def test_ffn_parts_streams_graphs_and_repeats():
    p = ffn_inputs([70, 0, 130, 9], 264, 136, seed=21)
    d = dims_of(p)
    ws, want = B.make_workspace(d), ffn_buffers(p)
    ffn_forward(p, want, ws, d)
    ffn_backward(p, want, ws, d)
    names = ("dxp", "dw_gate", "dw_up", "dw_down")
    # one result at a time
    for skip in ({"dxp"}, {"dw_gate", "dw_up"}, {"dw_down"}, set(names) - {"dw_down"}):
        b = ffn_buffers(p)
        ffn_forward(p, b, ws, d)
        ffn_backward(p, {k: None if k in skip else v for k, v in b.items()}, ws, d)
        for k in set(names) - skip:
            assert torch.equal(b[k], want[k]), k
    # another stream, with its own workspace, beside this one
    side, b2 = torch.cuda.Stream(), ffn_buffers(p)
    ws2 = B.make_workspace(d)
    side.wait_stream(torch.cuda.current_stream())
    b = ffn_buffers(p)
    for _ in range(3):
        ffn_forward(p, b, ws, d)
        ffn_forward(p, b2, ws2, d, stream=side)
        ffn_backward(p, b, ws, d)
        ffn_backward(p, b2, ws2, d, stream=side)
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(b[k], want[k]) and torch.equal(b2[k], want[k]), k
    # captured once, replayed on new contents
    b = ffn_buffers(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn_forward(p, b, ws, d)
        ffn_backward(p, b, ws, d)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(b[k], want[k]), k
    xp = p["xp"].clone()
    p["xp"].copy_(randn(xp.shape, 99))
    graph.replay()
    torch.cuda.synchronize()
    got = {k: b[k].clone() for k in names}
    ffn_forward(p, want, ws, d)
    ffn_backward(p, want, ws, d)
    for k in names:
        assert torch.equal(got[k], want[k]), k
    assert B.read_device_status(ws) == 0 and B.read_device_status(ws2) == 0


def test_ffn_without_tokens_and_bad_offsets():
    d = B.dims(T=0, H=64, E=3, K=1, F=40)
    ws = B.make_workspace(d)
    grads = [torch.full((3, 40, 64), 5.0, device=DEV, dtype=BF) for _ in range(2)] + \
            [torch.full((3, 64, 40), 5.0, device=DEV, dtype=BF)]
    empty = torch.empty((0, 64), device=DEV, dtype=BF)
    B.moe_grouped_ffn_backward(empty, None, None, None, empty, torch.zeros(4, dtype=torch.int32, device=DEV), None, None,
                               None, d, None, None, empty, *grads, ws)
    assert all((t == 0).all() for t in grads)
    acc = [torch.full(t.shape, 5.0, device=DEV) for t in grads]
    B.moe_grouped_ffn_backward(empty, None, None, None, empty, None, None, None, None, d, None, None, None, *acc, ws,
                               accumulate=True)
    assert all((t == 5).all() for t in acc)
    # offsets that decrease are reported, and nothing is computed
    p = ffn_inputs([10, 20], 64, 40)
    d = dims_of(p)
    ws, b = B.make_workspace(d), ffn_buffers(p, fill=3.0)
    p["offsets"] = torch.tensor([0, 20, 10], dtype=torch.int32, device=DEV)
    ffn_forward(p, b, ws, d)
    ffn_backward(p, b, ws, d)
    assert B.read_device_status(ws) & B.DEV_BAD_INDEX
    assert all((b[k] == 3.0).all() for k in b)


@pytest.mark.parametrize("E", [3, 60])   # few tiles, many tiles
@pytest.mark.parametrize("off", ["past the end", "negative", "no rows"])
def test_ffn_offsets_of_no_use(E, off):
    p = ffn_inputs([40] * E, 136, 264)
    d = dims_of(p)
    ws = B.make_workspace(d)
    p["offsets"] = p["offsets"].clone()
    if off == "past the end":
        p["offsets"][E] += 1
    elif off == "negative":
        p["offsets"][0] = -1
    else:
        p["offsets"].zero_()
    for grad, accumulate in ((BF, False), (F32, False), (F32, True)):
        b = ffn_buffers(p, grad=grad, fill=3.0)
        ffn_forward(p, b, ws, d)
        ffn_backward(p, b, ws, d, accumulate=accumulate)
        zero = off == "no rows" and not accumulate   # the sum over no rows
        for k in b:
            assert (b[k] == (0.0 if zero and k.startswith("dw") else 3.0)).all(), k
    assert bool(B.read_device_status(ws) & B.DEV_BAD_INDEX) == (off != "no rows")


# Shapes by the kernels that their products take (KERNELS below holds them to it): all on CTA pairs, with more
# tiles than SMs and more than 48 rows a group; few rows a group, so that the rows' gradients (80
# tiles) run on small tiles and all else on pairs; two long groups, whose weight gradients alone are small tiles.
PAIRS = ([200, 0, 300, 64, 1, 17] * 8, 520, 776)
PAIR_GRADS = ([5, 0, 9, 1] * 20, 136, 264)
PAIR_ROWS = ([3000, 4100], 520, 520)


@pytest.mark.parametrize("off", ["past the end", "negative", "decreasing", "no rows"])
def test_ffn_offsets_of_no_use_on_pairs(off):
    E = 160
    p = ffn_inputs([70] * E, 136, 264)
    d = dims_of(p)
    ws = B.make_workspace(d)
    p["offsets"] = p["offsets"].clone()
    if off == "past the end":
        p["offsets"][E] += 1
    elif off == "negative":
        p["offsets"][0] = -1
    elif off == "decreasing":
        p["offsets"][80] = p["offsets"][82]
    else:
        p["offsets"].zero_()
    for grad, accumulate in ((BF, False), (F32, False), (F32, True)):
        b = ffn_buffers(p, grad=grad, fill=3.0)
        ffn_forward(p, b, ws, d)
        ffn_backward(p, b, ws, d, accumulate=accumulate)
        zero = off == "no rows" and not accumulate   # the sum over no rows
        for k in b:
            assert (b[k] == (0.0 if zero and k.startswith("dw") else 3.0)).all(), k
    assert bool(B.read_device_status(ws) & B.DEV_BAD_INDEX) == (off != "no rows")
    # the workspace serves good calls after them
    B.workspace_init(ws)
    p = ffn_inputs([70] * E, 136, 264, seed=1)
    one, two = ffn_buffers(p), ffn_buffers(p)
    for b, w in ((one, ws), (two, B.make_workspace(d))):
        ffn_forward(p, b, w, d)
        ffn_backward(p, b, w, d)
    assert all(torch.equal(one[k], two[k]) for k in one if k != "y")
    assert B.read_device_status(ws) == 0


def test_ffn_nan_rows_stay_with_their_expert_on_pairs():
    """A tile's rows are rounded up to 16: the 75 rows before the bad expert read five of its rows."""
    counts = [137, 0, 75, 64, 161, 190] * 20
    p = ffn_inputs(counts, 136, 264, seed=3, pad=9)
    d = dims_of(p)
    ws = B.make_workspace(d)
    clean, dirty = ffn_buffers(p, fill=0.0), ffn_buffers(p, fill=0.0)
    ffn_forward(p, clean, ws, d)
    ffn_backward(p, clean, ws, d)
    bad, end = [3, 64, 119], int(p["offsets"][-1])   # inside, before the tile of another, the last
    rows = torch.zeros(p["rows"], dtype=torch.bool, device=DEV)
    for e in bad:
        rows[int(p["offsets"][e]):int(p["offsets"][e + 1])] = True
    for k, v in (("xp", float("nan")), ("dy", float("inf"))):
        p[k][rows] = v
        p[k][end:] = float("nan")
    for k in ("g", "u", "h", "dg", "du", "dxp"):
        dirty[k][end:] = 7.0
    ffn_forward(p, dirty, ws, d)
    for k in ("g", "u", "h"):   # rows behind the last one hold anything
        assert (dirty[k][end:] == 7.0).all()
        dirty[k][end:] = float("nan")
    ffn_backward(p, dirty, ws, d)
    others = [e for e in range(len(counts)) if e not in bad]
    good = ~rows
    good[end:] = False
    for k in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(clean[k][others], dirty[k][others]), k
        assert not torch.isfinite(dirty[k][bad]).any()
        assert (clean[k][1] == 0).all()   # an expert without rows
    for k in ("dg", "du", "dxp"):
        assert torch.equal(clean[k][good], dirty[k][good]), k
        assert (dirty[k][end:] == 7.0).all()
    assert B.read_device_status(ws) == 0


@pytest.mark.parametrize("counts,H,F", [PAIRS, PAIR_GRADS, PAIR_ROWS])
def test_ffn_parts_streams_graphs_and_repeats_on_pairs(counts, H, F):
    p = ffn_inputs(counts, H, F, seed=21)
    d = dims_of(p)
    ws, want = B.make_workspace(d), ffn_buffers(p)
    ffn_forward(p, want, ws, d)
    ffn_backward(p, want, ws, d)
    names = ("dxp", "dw_gate", "dw_up", "dw_down")
    ref = ffn_reference(p)
    # some of the results: the same bits, or (two long groups, where a weight gradient without the product
    # before it takes another kernel) the same bounds
    weights = {"dw_gate", "dw_up"}
    for skip in ({"dxp"}, weights, {"dw_down"}, {"dxp"} | weights, {"dxp", "dw_down"}, weights | {"dw_down"}):
        b = ffn_buffers(p)
        ffn_forward(p, b, ws, d)
        ffn_backward(p, {k: None if k in skip else v for k, v in b.items()}, ws, d)
        for k in set(names) - skip:
            within(k, b[k], ref[k], ref["~" + k] + (U8 * (ref[k].abs() + ref["~" + k]) if k != "dxp" else 0))
            assert (counts, H, F) == PAIR_ROWS or torch.equal(b[k], want[k]), k
    # another stream, with its own workspace, beside this one
    side, b, b2, ws2 = torch.cuda.Stream(), ffn_buffers(p), ffn_buffers(p), B.make_workspace(d)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        ffn_forward(p, b, ws, d)
        ffn_forward(p, b2, ws2, d, stream=side)
        ffn_backward(p, b, ws, d)
        ffn_backward(p, b2, ws2, d, stream=side)
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(b[k], want[k]) and torch.equal(b2[k], want[k]), k
    # two graphs of one workspace, replayed in turn, then on new contents
    graphs, bufs = [], []
    for _ in range(2):
        b, graph = ffn_buffers(p), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ffn_forward(p, b, ws, d)
            ffn_backward(p, b, ws, d)
        graphs.append(graph)
        bufs.append(b)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(bufs[0][k], want[k]) and torch.equal(bufs[1][k], want[k]), k
    p["xp"].copy_(randn(p["xp"].shape, 99))
    graphs[1].replay()
    torch.cuda.synchronize()
    ffn_forward(p, want, ws, d)
    ffn_backward(p, want, ws, d)
    for k in names:
        assert torch.equal(bufs[1][k], want[k]), k
    assert B.read_device_status(ws) == 0 and B.read_device_status(ws2) == 0


def kernels_of(fn):
    """The matrix kernels that fn launches, as (kind, mode): "prod" on CTA pairs, "small" on small tiles."""
    fn()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA], acc_events=True) as prof:
        fn()
        torch.cuda.synchronize()
    found = (re.search(r"(prod|small)_kernel<\D*(\d)", e.key) for e in prof.key_averages())
    return {(m[1], int(m[2])) for m in found if m}


KERNELS = [  # the step's products: g and u; dg and du; dxp; dW_gate and dW_up; dW_down
    (PAIRS, {("prod", 0), ("prod", 1), ("prod", 2), ("prod", 3), ("prod", 4)}),
    (([70] * 160, 136, 264), {("prod", 0), ("prod", 1), ("prod", 2), ("prod", 3), ("prod", 4)}),
    (([137, 0, 75, 64, 161, 190] * 20, 136, 264), {("prod", 0), ("prod", 1), ("prod", 2), ("prod", 3), ("prod", 4)}),
    (PAIR_GRADS, {("prod", 0), ("small", 2), ("small", 3), ("prod", 3), ("prod", 4)}),
    (PAIR_ROWS, {("prod", 0), ("prod", 1), ("prod", 2), ("prod", 3), ("prod", 4)}),
]


@pytest.mark.parametrize("shape,want", KERNELS)
def test_ffn_shapes_reach_the_kernels_they_are_meant_for(shape, want):
    p = ffn_inputs(*shape)
    b, d = ffn_buffers(p), dims_of(p)
    ws = B.make_workspace(d)

    def step(**skip):
        ffn_forward(p, b, ws, d)
        ffn_backward(p, {**b, **skip}, ws, d)

    got = kernels_of(step)
    if not got:
        pytest.skip("no kernel records on this machine")
    assert got == want
    if shape == PAIR_ROWS:   # the gradient of w_down alone
        assert kernels_of(lambda: step(dxp=None, dw_gate=None, dw_up=None)) == {("prod", 0), ("small", 4)}


# ---------------------------------------------------------------------------
# Combine
# ---------------------------------------------------------------------------

COMBINE_CASES = [(1, 8, 1), (1, 7168, 8), (37, 264, 3), (300, 1032, 8), (5, 64, 32), (700, 136, 9), (2000, 256, 2),
                 (9000, 72, 4)]


@pytest.mark.parametrize("T,H,K", COMBINE_CASES)
def test_combine_backward(T, H, K):
    d = B.dims(T=T, H=H, E=max(K, 2), K=K, F=8)
    dout, y = randn((T, H), T), randn((T * K, H), H)
    row = inputs.random_bijection(T * K, seed=T).to(DEV)
    w = inputs.random_weights(T, K, seed=K).to(DEV)
    dy, dw = torch.full_like(y, float("nan")), torch.full((T, K), float("nan"), device=DEV)
    B.moe_combine_backward(dout, y, row, w, d, dy, dw)
    gathered = y[row.long()].to(F64).view(T, K, H) * dout.to(F64)[:, None]
    ref_dy = torch.empty((T * K, H), dtype=F64, device=DEV)
    ref_dy[row.long()] = (w.to(F64)[:, :, None] * dout.to(F64)[:, None]).view(T * K, H)
    within("dy", dy, ref_dy, (U8 + 2 * U24) * ref_dy.abs() + 1e-38, parts=1)
    within("dw", dw, gathered.sum(-1), 2 * H * U24 * gathered.abs().sum(-1))
    # each alone, and in place
    dy2, dw2 = torch.empty_like(dy), torch.empty_like(dw)
    B.moe_combine_backward(dout, None, row, w, d, dy2, None)
    B.moe_combine_backward(dout, y, row, w, d, None, dw2)
    assert torch.equal(dy2, dy) and torch.equal(dw2, dw)
    y2 = y.clone()
    B.moe_combine_backward(dout, y2, row, w, d, y2, dw2)
    assert torch.equal(y2, dy) and torch.equal(dw2, dw)


def test_combine_backward_skips_rows_out_of_range():
    T, H, K = 6, 64, 2
    d = B.dims(T=T, H=H, E=4, K=K, F=8)
    dout, y = randn((T, H), 1), randn((T * K, H), 2)
    row = torch.arange(T * K, dtype=torch.int32, device=DEV)
    row[3], row[8] = -1, T * K
    w = torch.ones((T, K), device=DEV)
    dy, dw = torch.full_like(y, 9.0), torch.full((T, K), 9.0, device=DEV)
    B.moe_combine_backward(dout, y, row, w, d, dy, dw)
    assert dw.view(-1)[3] == 0 and dw.view(-1)[8] == 0
    assert (dy[[3, 8]] == 9.0).all()
    keep = [i for i in range(T * K) if i not in (3, 8)]
    assert torch.equal(dy[keep], dout.repeat_interleave(K, 0)[keep])


def test_combine_backward_streams_and_graphs():
    T, H, K = 300, 1032, 3
    d = B.dims(T=T, H=H, E=8, K=K, F=8)
    dout, y = randn((T, H), 1), randn((T * K, H), 2)
    row, w = inputs.random_bijection(T * K, seed=3).to(DEV), inputs.random_weights(T, K, seed=4).to(DEV)
    new = lambda: (torch.empty_like(y), torch.empty((T, K), device=DEV))  # noqa: E731
    want, one, two, rep = new(), new(), new(), new()
    B.moe_combine_backward(dout, y, row, w, d, *want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_combine_backward(dout, y, row, w, d, *one)
    B.moe_combine_backward(dout, y, row, w, d, *two, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_combine_backward(dout, y, row, w, d, *rep)
    graph.replay()
    torch.cuda.synchronize()
    for got in (one, two, rep):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dout.copy_(randn(dout.shape, 9))
    graph.replay()
    B.moe_combine_backward(dout, y, row, w, d, *want)
    torch.cuda.synchronize()
    assert torch.equal(rep[0], want[0]) and torch.equal(rep[1], want[1])


# ---------------------------------------------------------------------------
# Dense product with a fused epilogue
# ---------------------------------------------------------------------------

def act64(x, act):
    return {"none": lambda: x, "relu": lambda: x.clamp(min=0), "silu": lambda: x / (1 + torch.exp(-x)),
            "gelu": lambda: x * 0.5 * torch.special.erfc(-x / math.sqrt(2)),
            "gelu_tanh": lambda: 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))}[act]()


def dact64(x, act):
    x = x.detach().clone().requires_grad_()
    act64(x, act).sum().backward()
    return x.grad


DENSE_CASES = [  # M, N, Kd, act, bias, residual
    (1, 8, 8, "none", False, False), (1, 7168, 2048, "none", True, True), (7, 264, 72, "relu", True, False),
    (16, 2048, 7168, "silu", True, True), (17, 520, 136, "gelu", False, True), (33, 136, 1032, "gelu_tanh", True, True),
    (64, 256, 256, "silu", False, False), (129, 776, 520, "gelu", True, True), (300, 1544, 264, "none", True, True),
    (511, 512, 512, "gelu_tanh", False, False), (1001, 1544, 1032, "gelu", True, True),
    (2, 128, 64, "none", False, True), (130, 1032, 2056, "relu", True, True), (250, 64, 4096, "silu", True, False),
    # enough tiles for the CTA pairs: balanced rows, one and two feature halves, short reductions
    (3001, 2056, 136, "gelu", True, True), (6500, 1288, 264, "relu", True, False), (9000, 520, 72, "silu", False, True),
    (20000, 8, 64, "gelu_tanh", True, True),
]


@pytest.mark.parametrize("M,N,Kd,act,bias,residual", DENSE_CASES)
def test_dense_epilogue(M, N, Kd, act, bias, residual):
    a, w = randn((M, Kd), M), randn((N, Kd), N, Kd ** -0.5)
    bv = randn((N,), 5, dtype=F32) if bias else None
    rv = randn((M, N), 6) if residual else None
    ws = B.make_dense_workspace(M, N, Kd)
    out, pre = torch.full((M, N), float("nan"), device=DEV, dtype=BF), torch.full((M, N), float("nan"), device=DEV)
    B.moe_dense_epilogue(a, w, out, ws, bias=bv, act=act, residual=rv, pre=pre)
    x = a.to(F64) @ w.to(F64).T + (bv.to(F64) if bias else 0)
    ex = 2 * (Kd + 1) * U24 * (a.to(F64).abs() @ w.to(F64).abs().T + (bv.to(F64).abs() if bias else 0))
    ref = act64(x, act) + (rv.to(F64) if residual else 0)
    # |act'| <= 1.13; the activation's own error within SIG
    bound = 1.13 * ex + SIG * x.abs() + 2 * U24 * ref.abs()
    within("pre", pre, x, ex)
    within("out", out, ref, bound + U8 * (ref.abs() + bound), parts=1)
    # without keeping the pre-activations, and in place of the residual
    if residual:
        B.moe_dense_epilogue(a, w, rv, ws, bias=bv, act=act, residual=rv)
        assert torch.equal(rv, out)
    else:
        again = torch.empty_like(out)
        B.moe_dense_epilogue(a, w, again, ws, bias=bv, act=act)
        assert torch.equal(again, out)
    assert B.read_device_status(ws) == 0


@pytest.mark.parametrize("act", list(B.ACTIVATIONS))
@pytest.mark.parametrize("M,N,Kd", [(1, 8, 8), (5, 264, 72), (63, 136, 264), (333, 776, 520), (1000, 264, 1032),
                                    (2050, 64, 136), (6001, 264, 1288), (7000, 1032, 520), (300, 4104, 2056)])
def test_dense_backward(M, N, Kd, act):
    dout, a, w = randn((M, N), 1), randn((M, Kd), 2), randn((N, Kd), 3, Kd ** -0.5)
    pre = randn((M, N), 4, 2.0, dtype=F32)
    if act == "relu":
        pre.view(-1)[:: 7] = 0.0   # the derivative at zero is 0
    ws = B.make_dense_workspace(M, N, Kd)
    f = lambda shape, dt: torch.full(shape, float("nan"), device=DEV, dtype=dt)  # noqa: E731
    ds = (pre > 0).to(F64) if act == "relu" else dact64(pre.to(F64), act)
    dpre = dout.to(F64) * ds
    # act' is within 2^-19 (1 + |x|^2) (products of a few fp32 functions of values below 12)
    slack = 0.0 if act in ("none", "relu") else SIG
    ed = dout.to(F64).abs() * slack * (1 + pre.to(F64) ** 2)
    ed_r = ed + (0 if act in ("none", "relu") else U8) * (dpre.abs() + ed)
    ref_da, ref_dw, ref_db = dpre @ w.to(F64), dpre.T @ a.to(F64), dpre.sum(0)
    m_da, m_dw = ed_r @ w.to(F64).abs(), ed_r.T @ a.to(F64).abs()
    b_da = m_da + 2 * N * U24 * (dpre.abs() @ w.to(F64).abs() + m_da)
    b_dw = m_dw + 2 * M * U24 * (dpre.abs().T @ a.to(F64).abs() + m_dw)
    b_db = ed.sum(0) + 2 * M * U24 * (dpre.abs() + ed).sum(0)
    parts = 1 if act in ("none", "relu") else 2
    for grad in (BF, F32):
        buf, da, dw, db = f((M, N), BF), f((M, Kd), BF), f((N, Kd), grad), f((N,), F32)
        B.moe_dense_backward(dout, a, w, pre, buf, da, dw, db, ws, act=act)
        within("da", da, ref_da, b_da + U8 * (ref_da.abs() + b_da), parts=parts)
        if grad == BF:
            within("dw", dw, ref_dw, b_dw + U8 * (ref_dw.abs() + b_dw), parts=parts)
        else:
            within("dw", dw, ref_dw, b_dw, parts=parts)
        within("dbias", db, ref_db, b_db)
    once_w, once_b = dw.clone(), db.clone()
    start_w, start_b = randn(dw.shape, 8, dtype=F32), randn(db.shape, 9, dtype=F32)
    dw.copy_(start_w)
    db.copy_(start_b)
    B.moe_dense_backward(dout, a, w, pre, buf, None, dw, db, ws, act=act, accumulate=True)
    assert torch.equal(dw, start_w + once_w)
    within("dbias", db, start_b.to(F64) + once_b.to(F64), 2 * 16 * U24 * (start_b.abs() + b_db + dpre.abs().sum(0)))
    # the bias gradient alone
    db2 = f((N,), F32)
    B.moe_dense_backward(dout, None, None, pre, None, None, None, db2, ws, act=act)
    assert torch.equal(db2, once_b)
    assert B.read_device_status(ws) == 0


def test_dense_without_rows():
    ws = B.make_dense_workspace(0, 64, 40)
    e = lambda shape, v=5.0, dt=BF: torch.full(shape, v, device=DEV, dtype=dt)  # noqa: E731
    B.moe_dense_epilogue(e((0, 40)), e((64, 40)), e((0, 64)), ws)
    dw, db = e((64, 40)), e((64,), dt=F32)
    B.moe_dense_backward(e((0, 64)), e((0, 40)), e((64, 40)), None, None, e((0, 40)), dw, db, ws)
    assert (dw == 0).all() and (db == 0).all()
    dw, db = e((64, 40), dt=F32), e((64,), dt=F32)
    B.moe_dense_backward(e((0, 64)), e((0, 40)), e((64, 40)), None, None, None, dw, db, ws, accumulate=True)
    assert (dw == 5).all() and (db == 5).all()


@pytest.mark.parametrize("M,N,Kd", [(5, 264, 72), (333, 776, 520), (6500, 1288, 264)])
def test_dense_streams_graphs_and_repeats(M, N, Kd):
    a, w, bias, res = randn((M, Kd), 1), randn((N, Kd), 2, Kd ** -0.5), randn((N,), 3, dtype=F32), randn((M, N), 4)
    dout = randn((M, N), 5)

    def buffers():
        e = lambda shape, dt=BF: torch.full(shape, float("nan"), device=DEV, dtype=dt)  # noqa: E731
        return dict(out=e((M, N)), pre=e((M, N), F32), dpre=e((M, N)), da=e((M, Kd)), dw=e((N, Kd), F32), db=e((N,), F32))

    def step(b, ws, **kw):
        B.moe_dense_epilogue(a, w, b["out"], ws, bias=bias, act="gelu", residual=res, pre=b["pre"], **kw)
        B.moe_dense_backward(dout, a, w, b["pre"], b["dpre"], b["da"], b["dw"], b["db"], ws, act="gelu", **kw)

    ws, ws2, want = B.make_dense_workspace(M, N, Kd), B.make_dense_workspace(M, N, Kd), buffers()
    step(want, ws)
    side, b, b2 = torch.cuda.Stream(), buffers(), buffers()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        step(b, ws)
        step(b2, ws2, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(b[k], want[k]) and torch.equal(b2[k], want[k]) for k in want)
    graph, b = torch.cuda.CUDAGraph(), buffers()
    with torch.cuda.graph(graph):
        step(b, ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(b[k], want[k]) for k in want)
    a.copy_(randn(a.shape, 9))
    graph.replay()
    torch.cuda.synchronize()
    step(want, ws2)
    assert all(torch.equal(b[k], want[k]) for k in want)
    # without da, or without dw: the other results keep their bits
    for skip in ("da", "dw", "db"):
        b = buffers()
        step({**b, skip: None}, ws)
        assert all(torch.equal(b[k], want[k]) for k in want if k != skip)
    assert B.read_device_status(ws) == 0 and B.read_device_status(ws2) == 0


# ---------------------------------------------------------------------------
# Together: one training step of a routed layer with an output projection
# ---------------------------------------------------------------------------

def test_layer_training_step():
    """Gating, routing, permute, experts, combine and an output projection added to the residual
    stream, forward and backward through the library, against 64-bit autograd of the same layer (on
    the library's expert choices).  The 2-norm bound: the longest chain of bf16 roundings from the
    inputs to a gradient is out, final's gradient, dpre, dout, dy, dg (or h) and the result, eight at
    most, each of relative rms U8 / sqrt(3) at most."""
    T, H, E, K, F, D = 700, 264, 12, 3, 200, 392
    d = B.dims(T=T, H=H, E=E, K=K, F=F)
    x, w_g = randn((T, H), 1), randn((H, E), 2, H ** -0.5, F32)
    w_gate, w_up = randn((E, F, H), 3, H ** -0.5), randn((E, F, H), 4, H ** -0.5)
    w_down, w_out = randn((E, H, F), 5, F ** -0.5), randn((D, H), 6, H ** -0.5)
    bias, stream, dfinal = randn((D,), 7, dtype=F32), randn((T, D), 8), randn((T, D), 9)
    w = B.pack_layer_weights(d, w_g, None, w_gate, w_up, w_down)
    b, ws = B.alloc_layer_buffers(d), B.make_workspace(d)
    wsd = B.make_dense_workspace(T, D, H)
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    TK = T * K
    g, u = e(TK, F, dt=F32), e(TK, F, dt=F32)
    final, pre = e(T, D), e(T, D, dt=F32)
    # forward
    B.moe_gating(x, w["w_g_split"], None, d, b["logits"], ws)
    B.moe_route(b["logits"], d, b["topk_ids"], b["topk_w"])
    B.moe_count_scan(b["topk_ids"], d, b["counts"], b["offsets"], b["part_counts"], b["part_offsets"],
                     b["row_of_assign"], b["assign_of_row"], ws)
    B.moe_permute(x, b["row_of_assign"], b["topk_ids"], b["topk_w"], d, b["xp"])
    B.moe_grouped_gate_up_train(b["xp"], b["offsets"], w_gate, w_up, d, g, u, b["h"], ws)
    B.moe_grouped_down(b["h"], b["offsets"], w_down, d, b["y"], ws)
    B.moe_combine(b["y"], b["row_of_assign"], b["topk_w"], d, b["out"], shared=x)
    B.moe_dense_epilogue(b["out"], w_out, final, wsd, bias=bias, act="silu", residual=stream, pre=pre)
    # backward
    dpre, dout, dw_out, dbias = e(T, D), e(T, H), e(D, H, dt=F32), e(D, dt=F32)
    B.moe_dense_backward(dfinal, b["out"], w_out, pre, dpre, dout, dw_out, dbias, wsd, act="silu")
    dy, dtopk = e(TK, H), e(T, K, dt=F32)
    B.moe_combine_backward(dout, b["y"], b["row_of_assign"], b["topk_w"], d, dy, dtopk)
    dxp, dg, du = e(TK, H), e(TK, F), e(TK, F)
    grads = [e(E, F, H, dt=F32), e(E, F, H, dt=F32), e(E, H, F, dt=F32)]
    B.moe_grouped_ffn_backward(b["xp"], g, u, b["h"], dy, b["offsets"], w_gate, w_up, w_down, d, dg, du, dxp, *grads, ws)
    dx = e(T, H)   # the permute's gradient, plus the shared path's
    B.moe_combine(dxp, b["row_of_assign"], torch.ones((T, K), device=DEV), d, dx, shared=dout)
    assert B.read_device_status(ws) == 0 and B.read_device_status(wsd) == 0

    leaves = dict(x=x, topk=b["topk_w"], w_gate=w_gate, w_up=w_up, w_down=w_down, w_out=w_out, bias=bias)
    q = {k: v.to(F64).requires_grad_() for k, v in leaves.items()}
    ids = b["topk_ids"].long()
    out = q["x"]
    for k in range(K):
        wk = [q[n][ids[:, k]] for n in ("w_gate", "w_up", "w_down")]
        gk, uk = torch.einsum("th,tfh->tf", q["x"], wk[0]), torch.einsum("th,tfh->tf", q["x"], wk[1])
        yk = torch.einsum("tf,thf->th", torch.nn.functional.silu(gk) * uk, wk[2])
        out = out + q["topk"][:, k, None] * yk
    ref_final = torch.nn.functional.silu(out @ q["w_out"].T + q["bias"]) + stream.to(F64)
    ref_final.backward(dfinal.to(F64))
    got = dict(x=dx, topk=dtopk, w_gate=grads[0], w_up=grads[1], w_down=grads[2], w_out=dw_out, bias=dbias)
    limit = math.sqrt(8) * U8 / math.sqrt(3)
    assert ((final.to(F64) - ref_final).norm() / ref_final.norm()).item() <= limit
    for k, v in got.items():
        rel = ((v.to(F64) - q[k].grad).norm() / q[k].grad.norm()).item()
        assert rel <= limit, f"{k}: relative error {rel:.3e}"


def test_workspaces_serve_calls_of_every_shape_in_turn():
    """The tile counters are left at zero: one workspace, calls of different shapes and kinds back to
    back, give the same bits as on fresh workspaces."""
    ws = B.make_dense_workspace(4096, 1024, 1024)
    for i, (M, N, Kd) in enumerate(((3000, 2056, 136), (5, 264, 72), (6500, 1288, 264), (333, 776, 520), (3000, 2056, 136))):
        a, w, dout = randn((M, Kd), i), randn((N, Kd), i + 50), randn((M, N), i + 90)
        res = []
        for s in (ws, B.make_dense_workspace(M, N, Kd)):
            out, da, dw = torch.empty((M, N), dtype=BF, device=DEV), torch.empty_like(a), torch.empty_like(w)
            B.moe_dense_epilogue(a, w, out, s)
            B.moe_dense_backward(dout, a, w, None, None, da, dw, None, s)
            res.append((out, da, dw))
        assert all(torch.equal(p, q) for p, q in zip(*res))
    assert B.read_device_status(ws) == 0


def test_relu_masks_infinite_gradients():
    M, N, Kd = 40, 72, 64
    pre = torch.ones((M, N), device=DEV)
    pre[:, 1::2] = -1.0
    pre[:, 3] = 0.0
    dout = torch.full((M, N), float("inf"), dtype=BF, device=DEV)
    dout[:, 0::2] = 2.0
    dout[5, 7] = float("nan")
    w, a = torch.ones((N, Kd), dtype=BF, device=DEV), torch.ones((M, Kd), dtype=BF, device=DEV)
    dpre, da, dw, db = torch.empty_like(dout), torch.empty_like(a), torch.empty_like(w), torch.empty(N, device=DEV)
    B.moe_dense_backward(dout, a, w, pre, dpre, da, dw, db, B.make_dense_workspace(M, N, Kd), act="relu")
    masked = torch.arange(N, device=DEV) % 2 == 1
    assert torch.equal(dpre, torch.where(masked, 0.0, 2.0).to(BF).expand(M, N))
    assert torch.equal(db, torch.where(masked, 0.0, 2.0 * M))
    assert (da == N).all() and (dw == torch.where(masked, 0.0, 2.0 * M)[:, None]).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_gradient_keeps_fp32_accuracy(act):
    """One row with dout = 1: dbias is act'(pre) itself in fp32, so the activation's gradient is seen
    without the products' roundings.

    Bounds, in u = 2^-23 (an fp32 step, relative): the fast exponential is within 2 + 1.18 |a|, the fast
    divide within 2, an operation and a constant within 1/2.  With e = exp(-|a|) off by err, 1 / (1 + e) is
    off by 2.5 + err e / (1 + e) and e / (1 + e) by 3 + err; sigma(a) and 1 - sigma(a) are these two.
    gelu_tanh's a takes seven operations and constants, its factor k seven.  gelu: the erfc fit's 1.2e-7
    (one u), ten steps and constants of its polynomial on values up to 1.5 and the error of its argument (18 in
    the exponent), the exponent's square (2.5 z^2) and sum, the exponential, divide and products."""
    n = 1 << 17
    pre = torch.linspace(-30.0, 30.0, n, device=DEV).view(1, n)
    x, u = pre.to(F64), 2.0 ** -23
    dout = torch.ones((1, n), dtype=BF, device=DEV)
    ws, db = B.make_dense_workspace(1, n, 8), torch.empty((n,), device=DEV)

    def logistic(a, ea):
        e = torch.exp(-a.abs())
        err = (2 + 1.18 * a.abs() + a.abs() * ea) * u
        big, small, neg = 1 / (1 + e), e / (1 + e), a < 0
        e_big, e_small = big * (2.5 * u + err * small), small * (3 * u + err)
        return (torch.where(neg, small, big), torch.where(neg, big, small), torch.where(neg, e_small, e_big),
                torch.where(neg, e_big, e_small))

    ref = dact64(x, act)
    if act == "silu":     # s (1 + x c)
        s, c, es, ec = logistic(x, 0)
        bound = es * (1 + x * c).abs() + s * x.abs() * ec + s * (1 + (x * c).abs()) * 2 * u
    elif act == "gelu_tanh":   # s + k s c
        a, k = 1.5957691216057308 * (x + 0.044715 * x ** 3), 1.5957691216057308 * x * (1 + 0.134145 * x * x)
        s, c, es, ec = logistic(a, 4)
        ref = s + k * s * c   # (dact64's tanh cancels: 3e-15 off at x = -7, where act' is 5e-15)
        bound = es + k.abs() * (es * c + s * ec) + (s + k.abs() * s * c) * 5 * u
    else:   # cdf + x pdf
        z2 = x * x / 2
        pdf, tail = torch.exp(-z2) / math.sqrt(2 * math.pi), torch.special.erfc(x.abs() / math.sqrt(2)) / 2
        bound = tail * (28 + 4 * z2) * u + (x.abs() * pdf) * (6 + 3 * z2) * u + 2 * u
    B.moe_dense_backward(dout, None, None, pre, None, None, None, db, ws, act=act)
    within("dbias", db, ref[0], bound[0] + 1e-30)
    assert B.read_device_status(ws) == 0


# ---------------------------------------------------------------------------
# Offsets past 32 bits: buffers of more than 2^31 elements
# ---------------------------------------------------------------------------

def test_dense_offsets_past_32_bits():
    M, N, Kd = 330_000, 7168, 64
    a, w, bias = randn((M, Kd), 1), randn((N, Kd), 2, Kd ** -0.5), randn((N,), 3, dtype=F32)
    out, pre = torch.empty((M, N), dtype=BF, device=DEV), torch.empty((M, N), device=DEV)
    ws = B.make_dense_workspace(M, N, Kd)
    B.moe_dense_epilogue(a, w, out, ws, bias=bias, act="relu", pre=pre)
    for r in (slice(0, 300), slice(M - 300, M)):
        x = a[r].to(F64)
        ref, e = x @ w.to(F64).T + bias.to(F64), 2 * (Kd + 1) * U24 * (x.abs() @ w.to(F64).abs().T + bias.abs())
        within("pre", pre[r], ref, e)
        within("out", out[r], ref.clamp(min=0), e + U8 * (ref.abs() + e), parts=1)
    # out serves as its own gradient; relu's dpre is exact
    dpre, da = torch.empty_like(out), torch.empty_like(a)
    dw, db = torch.empty((N, Kd), device=DEV), torch.empty((N,), device=DEV)
    B.moe_dense_backward(out, a, w, pre, dpre, da, dw, db, ws, act="relu")
    r = slice(M - 300, M)
    assert torch.equal(dpre[r], out[r])
    m = out[r].to(F64) @ w.to(F64).abs()
    within("da", da[r], out[r].to(F64) @ w.to(F64), 2 * N * U24 * m + U8 * (1 + 1e-3) * m, parts=None)
    c = slice(N - 16, N)
    d = out[:, c].to(F64)
    within("dw", dw[c], d.T @ a.to(F64), 2 * M * U24 * (d.T @ a.to(F64).abs()))
    within("dbias", db[c], d.sum(0), 2 * M * U24 * d.sum(0))
    assert B.read_device_status(ws) == 0


@pytest.mark.parametrize("counts,H,F", [([1, 298_999, 1000], 64, 7168), ([5] + [0] * 128 + [20], 8192, 2056)])
def test_ffn_offsets_past_32_bits(counts, H, F):
    p = ffn_inputs(counts, H, F)
    d = dims_of(p)
    ws, b = B.make_workspace(d), ffn_buffers(p)
    ffn_forward(p, b, ws, d)
    ffn_backward(p, b, ws, d)
    # the last expert alone
    n, e = counts[-1], len(counts) - 1
    q = dict(p, E=1, rows=n, offsets=torch.tensor([0, n], dtype=torch.int32, device=DEV), xp=p["xp"][-n:],
             dy=p["dy"][-n:], w_gate=p["w_gate"][e:], w_up=p["w_up"][e:], w_down=p["w_down"][e:])
    ref = ffn_reference(q)
    for k in ("g", "u", "h", "dg", "du", "dxp"):
        within(k, b[k][-n:], ref[k], ref["~" + k])
    for k in ("dw_gate", "dw_up", "dw_down"):
        within(k, b[k][e:], ref[k], ref["~" + k] + U8 * (ref[k].abs() + ref["~" + k]))
        if 0 in counts:
            assert (b[k][1:e] == 0).all()
    assert B.read_device_status(ws) == 0


def test_combine_backward_offsets_past_32_bits():
    T, K, H = 40_000, 8, 7168
    d = B.dims(T=T, H=H, E=K, K=K, F=8)
    dout, y = randn((T, H), 1), randn((T * K, H), 2)
    row = torch.arange(T * K, dtype=torch.int32, device=DEV).flip(0).contiguous()
    w = inputs.random_weights(T, K, seed=3).to(DEV)
    dy, dw = torch.empty_like(y), torch.empty((T, K), device=DEV)
    B.moe_combine_backward(dout, y, row, w, d, dy, dw)
    for t in (slice(0, 64), slice(T - 64, T)):
        rows = row.view(T, K)[t].long()
        ref = w[t].to(F64)[:, :, None] * dout[t].to(F64)[:, None]
        within("dy", dy[rows], ref, (U8 + 2 * U24) * ref.abs() + 1e-38, parts=1)
        prod = y[rows].to(F64) * dout[t].to(F64)[:, None]
        within("dw", dw[t], prod.sum(-1), 2 * H * U24 * prod.abs().sum(-1))

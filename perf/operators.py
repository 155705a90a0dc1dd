"""Cases of layer normalisation, the global gradient norm and gradient clipping.

``run`` makes one pass through an operator: with ``own`` false in plain torch
operations, with ``own`` true through the library's entry points
(``capi.fno_layer_norm_fwd`` / ``_bwd``, ``fno_grad_norm``, ``fno_clip_grads``).

Operators (``case["op"]``):

* ``ln_fwd``   y = (x - mean) rstd gamma + beta over the channel axis of
  x [outer][channels][inner], and the statistics mean, rstd [outer][inner];
* ``ln_bwd``   dx, dgamma, dbeta from x, dy and the saved statistics;
* ``norm``     the 2-norm of all gradients together, and the factor
  min(1, max_norm / norm);
* ``clip``     the same, and every gradient times that factor.
"""

import math

import torch

own = False

EPS = 1e-5
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
MOST_BYTES = 1_000_000_000      # that a drawn pass reads and writes
MOST_GRADS = 37_000_000         # elements of the largest drawn set of gradients


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _ln(name, op, dtype, outer, channels, inner):
    return {"name": name, "op": op, "dtype": dtype, "outer": outer, "channels": channels,
            "inner": inner}


def _grads(name, op, dtype, kind, layers, width, modes, hidden, clipped):
    return {"name": name, "op": op, "dtype": dtype, "kind": kind, "layers": layers,
            "width": width, "modes": modes, "hidden": hidden, "clipped": clipped}


def listed():
    return [
        # one sample on a coarse grid: what a single prediction waits for
        _ln("fwd_one_sample_c20_16sq_f32", "ln_fwd", "f32", 1, 20, 16 * 16),
        # the forward benchmark's activations: between two of its blocks
        _ln("fwd_b16_c32_256sq_f32", "ln_fwd", "f32", 16, 32, 256 * 256),
        # a cropped field with odd sides, in half precision
        _ln("fwd_b12_c20_253x191_f16", "ln_fwd", "f16", 12, 20, 253 * 191),
        # scattered points with the features last
        _ln("fwd_rows_20011_c768_bf16", "ln_fwd", "bf16", 20011, 768, 1),
        # the small parity workload's batch
        _ln("bwd_b4_c20_64sq_f32", "ln_bwd", "f32", 4, 20, 64 * 64),
        # the bfloat16 training workload's activations: one layer of its backward
        _ln("bwd_b32_c64_256sq_bf16", "ln_bwd", "bf16", 32, 64, 256 * 256),
        # the three-dimensional workload
        _ln("bwd_b2_c20_128cube_f32", "ln_bwd", "f32", 2, 20, 128 ** 3),
        # scattered points, an odd number of features
        _ln("bwd_rows_4099_c1001_f32", "ln_bwd", "f32", 4099, 1001, 1),
        # every gradient of the training workload's network (R, W, b of four
        # layers, lift and projection): the check for a step that diverges
        _grads("norm_w64_m24_f32", "norm", "f32", "net", 4, 64, 24, 128, True),
        # the small network's gradients, below the limit: nothing is clipped
        _grads("norm_w20_m12_f32", "norm", "f32", "net", 4, 20, 12, 128, False),
        # the benchmark network's gradients, clipped, as the step before the optimiser
        _grads("clip_w32_m16_f32", "clip", "f32", "net", 4, 32, 16, 128, True),
        # many short parameters of odd lengths in bfloat16 (a factorised network)
        _grads("clip_320_ragged_bf16", "clip", "bf16", "ragged", 320, 64, 24, 0, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "norm", "clip"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("norm", "clip"):
        clipped = rng.random() < 0.7
        if rng.random() < 0.5:
            case = _grads("", op, dtype, "net", rng.randint(1, 8), _log(rng, 4, 64),
                          rng.randint(2, 24), _log(rng, 8, 256), clipped)
        else:
            case = _grads("", op, dtype, "ragged", _log(rng, 1, 600), _log(rng, 1, 96),
                          rng.randint(1, 32), 0, clipped)
        while sum(_lengths(case)) > MOST_GRADS:
            case["layers"] = max(1, case["layers"] // 2)
    elif rng.random() < 0.35:
        channels = _log(rng, 4, 8192)
        rows = MOST_BYTES // ((2 if op == "ln_fwd" else 3) * SIZE[dtype] * channels + 16)
        case = _ln("", op, dtype, _log(rng, 1, min(65536, rows)), channels, 1)
    else:
        # from 4 channels on: over two, what is left of dx after its two
        # projections is nothing but rounding
        channels = _log(rng, 4, 128)
        sides = rng.randint(1, 3)
        longest = {1: 4096, 2: 512, 3: 128}[sides]
        inner = 1
        for _ in range(sides):
            side = _log(rng, 4, longest)
            inner *= side - side % 4 if rng.random() < 0.5 else side
        points = MOST_BYTES // ((2 if op == "ln_fwd" else 3) * SIZE[dtype] * channels + 16)
        inner = min(inner, points)
        case = _ln("", op, dtype, _log(rng, 1, min(32, points // inner)), channels, inner)
    del case["name"]
    return case


def _lengths(case):
    """Elements of each gradient."""
    w, m = case["width"], case["modes"]
    if case["kind"] == "net":
        layer = [w * w * (2 * m * m) * 2, w * w, w]
        return [3 * w, w] + layer * case["layers"] + \
            [case["hidden"] * w, case["hidden"], case["hidden"], 1]
    # factors [width][rank] and biases: short, odd lengths, a few empty
    return [(0 if i % 37 == 36 else 1 + (i * 7919 + 13) % (2 * w * m) + (w * m * m if i % 16 == 0
                                                                        else 0))
            for i in range(case["layers"])]


def _elements(case):
    return case["outer"] * case["channels"] * case["inner"]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = TORCH[case["dtype"]]
    if case["op"] in ("norm", "clip"):
        state = _prepare_grads(case, gen, dt)
    else:
        state = _prepare_ln(case, gen, dt)
    state["case"] = case
    if own:
        # the descriptor or the list of tensors, which a program sets up once
        from fourier_neural_spectral_fno_b200 import capi
        state["capi"] = capi
        if case["op"] in ("norm", "clip"):
            state["plan"] = capi.grad_list(state["grads"], state.get("out"))
            state["ws"] = torch.empty(capi.fno_grad_norm_workspace_size(state["plan"]),
                                      dtype=torch.uint8, device="cuda")
        else:
            state["plan"] = capi.layer_norm_desc(case["outer"], case["channels"], case["inner"],
                                                 case["dtype"], EPS)
            state["ws"] = torch.empty(capi.fno_layer_norm_workspace_size(state["plan"]),
                                      dtype=torch.uint8, device="cuda")
    return state


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _prepare_ln(case, gen, dt):
    b, c, n = case["outer"], case["channels"], case["inner"]
    # activations: channels of unlike size and offset, as a network's are
    size = torch.exp(0.5 * _randn(gen, 1, c, 1))
    x = (_randn(gen, b, c, n).mul_(size).add_(0.7 * _randn(gen, 1, c, 1))).to(dt)
    state = {"x": x, "gamma": (1 + 0.2 * _randn(gen, c)).to(dt)}
    if case["op"] == "ln_fwd":
        state["beta"] = (0.2 * _randn(gen, c)).to(dt)
        state["y"] = torch.empty_like(x)
        state["mean"] = torch.empty(b, n, device="cuda")
        state["rstd"] = torch.empty(b, n, device="cuda")
        return state
    # the statistics that the forward has saved
    mean = x.float().mean(1)
    var = (x.float() - mean[:, None]).square_().mean(1)
    state["mean"], state["rstd"] = mean, torch.rsqrt(var + EPS)
    state["dy"] = (0.05 * _randn(gen, b, c, n)).to(dt)
    state["dx"] = torch.empty_like(x)
    state["dgamma"] = torch.empty(c, device="cuda")
    state["dbeta"] = torch.empty(c, device="cuda")
    return state


def _prepare_grads(case, gen, dt):
    lengths = _lengths(case)
    sizes = (1e-3 * torch.exp(_randn(gen, len(lengths)))).tolist()   # each parameter's own size
    grads = [(s * _randn(gen, n)).to(dt) for n, s in zip(lengths, sizes)]
    norm = math.sqrt(sum(n * s * s for n, s in zip(lengths, sizes)))
    state = {"grads": grads, "max_norm": (0.4 if case["clipped"] else 3.0) * max(norm, 1e-6),
             "norm": torch.empty(2, device="cuda")}
    if case["op"] == "clip":
        # the clipped gradients, in slots of one buffer
        starts, end = [], 0
        for n in lengths:
            starts.append(end)
            end += -(-n // 8) * 8
        state["flat"] = torch.zeros(end, dtype=dt, device="cuda")
        state["out"] = [state["flat"][s:s + n] for s, n in zip(starts, lengths)]
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    y = d * rstd * s["gamma"].float()[:, None] + s["beta"].float()[:, None]
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_ln_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()[:, None]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum((0, 2)), "dbeta": dy.sum((0, 2))}


def _plain_norm(s):
    # the sum runs over up to tens of millions of squares: 64 bits
    squares = torch.stack([g.double().square().sum() for g in s["grads"]])
    norm = squares.sum().sqrt()
    factor = torch.clamp(s["max_norm"] / norm, max=1.0)
    return torch.stack([norm, factor]).float()


def _plain_clip(s):
    norm = _plain_norm(s)
    [o.copy_(g.float() * norm[1]) for g, o in zip(s["grads"], s["out"])]
    return {"grads": s["flat"], "norm": norm}


def _own_ln_fwd(s):
    s["capi"].fno_layer_norm_fwd(s["plan"], s["x"], s["gamma"], s["beta"], s["y"], s["mean"],
                                 s["rstd"])
    return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_ln_bwd(s):
    s["capi"].fno_layer_norm_bwd(s["plan"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dy"],
                                 s["dx"], s["dgamma"], s["dbeta"], ws=s["ws"])
    return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def _own_norm(s):
    s["capi"].fno_grad_norm(s["plan"], s["max_norm"], s["norm"], ws=s["ws"])
    return s["norm"]


def _own_clip(s):
    s["capi"].fno_clip_grads(s["plan"], s["max_norm"], s["norm"], ws=s["ws"])
    return {"grads": s["flat"], "norm": s["norm"]}


_run_plain = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "norm": _plain_norm,
              "clip": _plain_clip}
_run_own = {"ln_fwd": _own_ln_fwd, "ln_bwd": _own_ln_bwd, "norm": _own_norm, "clip": _own_clip}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] in ("norm", "clip"):
        n = sum(_lengths(case))
        return {"bytes": n * size * (2 if case["op"] == "clip" else 1) + 8,
                "flops": n * (3 if case["op"] == "clip" else 2)}
    n = _elements(case)
    points, c = case["outer"] * case["inner"], case["channels"]
    if case["op"] == "ln_fwd":
        return {"bytes": 2 * n * size + 8 * points + 2 * c * size, "flops": 7 * n}
    return {"bytes": 3 * n * size + 8 * points + c * size + 8 * c, "flops": 14 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        flat = torch.cat([g.to(torch.float64) for g in s["grads"]])
        norm = torch.linalg.vector_norm(flat)
        factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
        both = torch.stack([norm, factor])
        if case["op"] == "norm":
            return both
        out = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
        at = 0
        for g in s["grads"]:
            out[at:at + g.numel()] = g.to(torch.float64) * factor
            at += -(-g.numel() // 8) * 8
        return {"grads": out, "norm": both}
    x, gamma = s["x"].to(torch.float64), s["gamma"].to(torch.float64)
    if case["op"] == "ln_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        x.sub_(mean.unsqueeze(1)).mul_(rstd.unsqueeze(1)).mul_(gamma.view(-1, 1))
        x.add_(s["beta"].to(torch.float64).view(-1, 1))
        return {"y": x, "mean": mean, "rstd": rstd}
    rstd = s["rstd"].to(torch.float64).unsqueeze(1)
    xh = x.sub_(s["mean"].to(torch.float64).unsqueeze(1)).mul_(rstd)
    dy = s["dy"].to(torch.float64)
    dgamma = torch.einsum("bcn,bcn->c", dy, xh)
    dbeta = dy.sum(dim=(0, 2))
    c1 = torch.einsum("bcn,c->bn", dy, gamma) / case["channels"]
    c2 = torch.einsum("bcn,bcn,c->bn", dy, xh, gamma) / case["channels"]
    dx = dy.mul_(gamma.view(-1, 1)).sub_(c1.unsqueeze(1)).sub_(xh.mul_(c2.unsqueeze(1)))
    return {"dx": dx.mul_(rstd), "dgamma": dgamma, "dbeta": dbeta}

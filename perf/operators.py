"""Cases for the dense operators of the radial and node networks.

Five passes are measured: the linear layer with bias, activation and residual
(forward and VJP), the layer norm (forward and VJP with the weights'
gradients) and the orthogonalised update of a weight matrix. `own` selects
the library's calls; otherwise `run` evaluates the same formulas with
elementary torch operations in float32, rounded once at the end.
"""
import math

import torch

own = False

EPS_NORM = 1e-5
EPS_ORTH = 1e-7
STEPS = 5
COEF = (3.4445, -4.7750, 2.0315)

# the largest listed case bounds what a drawn one may cost (bytes, and
# flops at 50 per byte)
MOST = 2.6e9


def listed():
    return [
        # the first hidden layer on the 256 edges of the smallest graph: 8 radial features, launch latency counts
        dict(name="linear_tiny", op="linear", dtype="f32", rows=256, n_in=8, n_out=64, act="silu", residual=False,
             save=False, pitch=1),
        # a hidden layer of the radial network on the edges of the 5184-atom water box, while training
        dict(name="linear_edges", op="linear", dtype="f32", rows=441172, n_in=64, n_out=64, act="silu",
             residual=True, save=True, pitch=1),
        # the readout's first layer on the 32768 diamond atoms: the l = 0 row of l_max = 3 features (16 rows a node)
        dict(name="linear_nodes", op="linear", dtype="bf16", rows=32768, n_in=128, n_out=512, act="gelu",
             residual=False, save=True, pitch=16),
        # backward of a radial layer on the edges of the 1024-atom, 128-neighbour graph
        dict(name="linear_vjp_edges", op="linear_vjp", dtype="f32", rows=131072, n_in=64, n_out=128, act="silu",
             pitch=1),
        # backward of a square node layer that is wide enough for the matrix cores to count
        dict(name="linear_vjp_wide", op="linear_vjp", dtype="bf16", rows=32768, n_in=512, n_out=512, act="silu",
             pitch=1),
        # backward of a radial layer on every edge of the 32768-atom diamond
        dict(name="linear_vjp_diamond", op="linear_vjp", dtype="bf16", rows=5172508, n_in=64, n_out=64, act="silu",
             pitch=1),
        # the norm before the readout when one small graph is evaluated
        dict(name="norm_tiny", op="norm", dtype="f32", rows=256, cols=64, save=False, pitch=1),
        # the norm of the node network's hidden features, while training
        dict(name="norm_nodes", op="norm", dtype="bf16", rows=32768, cols=512, save=True, pitch=1),
        # backward of the radial network's norm on the water box's edges
        dict(name="norm_vjp_edges", op="norm_vjp", dtype="f32", rows=441172, cols=64, pitch=1),
        # backward on node features of an odd width
        dict(name="norm_vjp_odd", op="norm_vjp", dtype="bf16", rows=5184, cols=777, pitch=1),
        # the channel-mixing blocks of an l_max = 3 layer: one 128 x 128 matrix for each of its 34 paths
        dict(name="orth_mix", op="orth", dtype="f32", mats=34, rows=128, cols=128),
        # two wide node weights, kept in 16 bits
        dict(name="orth_wide", op="orth", dtype="bf16", mats=2, rows=512, cols=1024),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_vjp", "norm", "norm_vjp", "orth"])
    case = dict(op=op, dtype=rng.choice(["f32", "bf16"]))
    if op in ("linear", "linear_vjp"):
        case.update(n_in=_log_int(rng, 4, 1024), n_out=_log_int(rng, 4, 1024), act=rng.choice(["none", "silu", "gelu"]),
                    pitch=rng.choice([1, 1, 1, 4]))
        case["rows"] = _log_int(rng, 1, 4_000_000)
        if op == "linear":
            case.update(residual=rng.random() < 0.5, save=rng.random() < 0.5)
        shrink = "rows"
    elif op in ("norm", "norm_vjp"):
        # below 4 columns the gradient of the input is all cancellation
        case.update(cols=_log_int(rng, 4, 2048), pitch=rng.choice([1, 1, 1, 4]))
        case["rows"] = _log_int(rng, 1, 2_000_000)
        if op == "norm":
            case["save"] = rng.random() < 0.5
        shrink = "rows"
    else:
        case.update(rows=_log_int(rng, 4, 1024), cols=_log_int(rng, 4, 1024), mats=_log_int(rng, 1, 64))
        if rng.random() < 0.25:  # the radial last layer: few rows, one column for each path and channel
            case.update(rows=_log_int(rng, 4, 64), cols=rng.choice([5, 15, 34]) * _log_int(rng, 8, 128))
        shrink = "mats"
    w = work(case)
    cost = max(w["bytes"], w["flops"] / 50) * case.get("pitch", 1)
    if cost > MOST:
        case[shrink] = max(1, int(case[shrink] * MOST / cost))
    return case


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _rows(gen, case, cols):
    """Features [rows][cols] as a view of rows `pitch` times as long."""
    pitch = case.get("pitch", 1)
    return _normal(gen, case["rows"], pitch * cols).to(_dtype(case))[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = _dtype(case), case["op"]
    s = dict(case=case)
    if op in ("linear", "linear_vjp"):
        M, K, N = case["rows"], case["n_in"], case["n_out"]
        s["x"] = _rows(gen, case, K)
        s["W"] = (_normal(gen, K, N) / math.sqrt(K)).to(dt)
        if op == "linear":
            s["b"] = 0.1 * _normal(gen, N)
            s["res"] = _normal(gen, M, N).to(dt) if case["residual"] else None
            s["y"] = torch.empty(M, N, dtype=dt, device="cuda")
            s["z"] = torch.empty(M, N, dtype=dt, device="cuda") if case["save"] else None
        else:
            s["z"] = _normal(gen, M, N).to(dt) if case["act"] != "none" else None
            s["gy"] = _normal(gen, M, N).to(dt)
            s["gx"] = torch.empty(M, K, dtype=dt, device="cuda")
            s["gW"] = torch.empty(K, N, device="cuda")
            s["gb"] = torch.empty(N, device="cuda")
    elif op in ("norm", "norm_vjp"):
        M, C = case["rows"], case["cols"]
        s["x"] = _rows(gen, case, C)
        s["gamma"] = 1.0 + 0.2 * _normal(gen, C)
        if op == "norm":
            s["beta"] = 0.2 * _normal(gen, C)
            s["y"] = torch.empty(M, C, dtype=dt, device="cuda")
            s["mean"] = torch.empty(M, device="cuda") if case["save"] else None
            s["rstd"] = torch.empty(M, device="cuda") if case["save"] else None
        else:
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][:, None]).square().mean(1) + EPS_NORM)
            s["gy"] = _normal(gen, M, C).to(dt)
            s["gx"] = torch.empty(M, C, dtype=dt, device="cuda")
            s["ggamma"] = torch.empty(C, device="cuda")
            s["gbeta"] = torch.empty(C, device="cuda")
    else:
        B, R, C = case["mats"], case["rows"], case["cols"]
        # a gradient's spectrum: a few decaying directions over a floor
        k = max(1, min(R, C) // 8)
        fall = torch.exp(-torch.arange(k, device="cuda") / 4.0)
        s["G"] = (1e-2 * (torch.bmm(_normal(gen, B, R, k) * fall, _normal(gen, B, k, C))
                          + 0.25 * _normal(gen, B, R, C))).to(dt)
        s["X"] = torch.empty_like(s["G"])
    return s


def _act(name, z):
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(name, z):
    if name == "silu":
        t = 1.0 / (1.0 + torch.exp(-z))
        return t * (1.0 + z * (1.0 - t))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2 * math.pi))
    return None


def _plain(s):
    case = s["case"]
    dt, op = _dtype(case), case["op"]
    if op == "linear":
        z = s["x"].float() @ s["W"].float() + s["b"]
        y = _act(case["act"], z)
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(dt), "z": z.to(dt)} if case["save"] else {"y": y.to(dt)}
    if op == "linear_vjp":
        d = s["gy"].float()
        if s["z"] is not None:
            d = d * _act_grad(case["act"], s["z"].float())
        return {"gx": (d @ s["W"].float().t()).to(dt), "gW": s["x"].float().t() @ d, "gb": d.sum(0)}
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt(d.square().mean(1) + EPS_NORM)
        y = (d * rstd[:, None] * s["gamma"] + s["beta"]).to(dt)
        return {"y": y, "mean": mean, "rstd": rstd} if case["save"] else {"y": y}
    if op == "norm_vjp":
        h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = s["gy"].float()
        d = g * s["gamma"]
        gx = s["rstd"][:, None] * (d - d.mean(1, keepdim=True) - h * (d * h).mean(1, keepdim=True))
        return {"gx": gx.to(dt), "ggamma": (g * h).sum(0), "gbeta": g.sum(0)}
    X = s["G"].float()
    X = X / (torch.sqrt(X.square().sum((1, 2), keepdim=True)) + EPS_ORTH)
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.transpose(1, 2).contiguous()
    a, b, c = COEF
    for _ in range(STEPS):
        A = torch.bmm(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    if tall:
        X = X.transpose(1, 2).contiguous()
    return {"X": X.to(dt)}


def _calls(s):
    from equivariant_interatomic_potentials_amd import dense
    case, op = s["case"], s["case"]["op"]
    act = {"none": dense.ETP_ACT_NONE, "silu": dense.ETP_ACT_SILU, "gelu": dense.ETP_ACT_GELU}.get(case.get("act"))

    def workspace(size, *args):  # allocated by the first pass and kept with the outputs
        if "ws" not in s:
            s["ws"] = torch.empty(max(16, size(*args)), dtype=torch.uint8, device="cuda")
        return s["ws"]

    if op == "linear":
        dense.etp_linear(s["x"], s["W"], s["y"], s["b"], act, s["res"], s["z"])
        return {"y": s["y"], "z": s["z"]} if case["save"] else {"y": s["y"]}
    if op == "linear_vjp":
        ws = workspace(dense.etp_linear_vjp_workspace, case["rows"], case["n_in"], case["n_out"], s["x"].dtype)
        dense.etp_linear_vjp(s["x"], s["W"], s["gy"], s["z"], act, s["gx"], s["gW"], s["gb"], ws)
        return {"gx": s["gx"], "gW": s["gW"], "gb": s["gb"]}
    if op == "norm":
        dense.etp_layer_norm(s["x"], s["y"], s["gamma"], s["beta"], EPS_NORM, s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]} if case["save"] else {"y": s["y"]}
    if op == "norm_vjp":
        ws = workspace(dense.etp_layer_norm_vjp_workspace, case["rows"], case["cols"], s["x"].dtype)
        dense.etp_layer_norm_vjp(s["x"], s["mean"], s["rstd"], s["gy"], s["gamma"], s["gx"], s["ggamma"], s["gbeta"],
                                 ws)
        return {"gx": s["gx"], "ggamma": s["ggamma"], "gbeta": s["gbeta"]}
    ws = workspace(dense.etp_orthogonalize_workspace, case["mats"], case["rows"], case["cols"], s["G"].dtype)
    dense.etp_orthogonalize(s["G"], s["X"], STEPS, COEF, EPS_ORTH, ws)
    return {"X": s["X"]}


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "linear":
        M, K, N = case["rows"], case["n_in"], case["n_out"]
        wide = 1 + int(case["residual"]) + int(case["save"])
        return {"bytes": e * (M * K + K * N + wide * M * N) + 4 * N, "flops": 2 * M * K * N}
    if op == "linear_vjp":
        M, K, N = case["rows"], case["n_in"], case["n_out"]
        wide = 1 if case["act"] == "none" else 2
        return {"bytes": e * (2 * M * K + K * N + wide * M * N) + 4 * (K * N + N), "flops": 4 * M * K * N}
    if op == "norm":
        M, C = case["rows"], case["cols"]
        return {"bytes": 2 * e * M * C + 8 * C + (8 * M if case["save"] else 0), "flops": 8 * M * C}
    if op == "norm_vjp":
        M, C = case["rows"], case["cols"]
        return {"bytes": 3 * e * M * C + 12 * C + 8 * M, "flops": 13 * M * C}
    B, n, m = case["mats"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    # a step's three products; the two symmetric ones need half their entries
    return {"bytes": 2 * e * B * n * m, "flops": B * STEPS * (n * (n + 1) * m + n * n * (n + 1) + 2 * n * n * m)}


def exact(case, seed):
    """The operators' definitions in float64 on the inputs that prepare makes."""
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("y", "X", "ggamma", "gbeta",
                                                                                         "gx", "gW", "gb")}
    if op == "linear":
        z = torch.addmm(f["b"], f["x"], f["W"])
        y = {"none": lambda t: t, "silu": lambda t: t * torch.sigmoid(t),
             "gelu": lambda t: t * 0.5 * torch.erfc(-t / math.sqrt(2.0))}[case["act"]](z)
        if case["residual"]:
            y = y + f["res"]
        return {"y": y, "z": z} if case["save"] else {"y": y}
    if op == "linear_vjp":
        d = f["gy"]
        if case["act"] == "silu":
            t = torch.sigmoid(f["z"])
            d = d * (t + f["z"] * t * (1 - t))
        elif case["act"] == "gelu":
            d = d * (0.5 * torch.erfc(-f["z"] / math.sqrt(2.0))
                     + f["z"] * torch.exp(-f["z"] ** 2 / 2) / math.sqrt(2 * math.pi))
        gW = sum(torch.mm(f["x"][i:i + 65536].t().contiguous(), d[i:i + 65536]) for i in range(0, case["rows"], 65536))
        return {"gx": torch.mm(d, f["W"].t().contiguous()), "gW": gW, "gb": torch.sum(d, 0)}
    if op == "norm":
        var, mean = torch.var_mean(f["x"], 1, correction=0)
        rstd = (var + EPS_NORM) ** -0.5
        y = torch.addcmul(f["beta"], (f["x"] - mean[:, None]) * rstd[:, None], f["gamma"])
        return {"y": y, "mean": mean, "rstd": rstd} if case["save"] else {"y": y}
    if op == "norm_vjp":
        C = case["cols"]
        r = f["rstd"][:, None]
        h = f["x"] * r - f["mean"][:, None] * r
        d = f["gy"] * f["gamma"]
        gx = r / C * (C * d - d.sum(1, keepdim=True) - h * (d * h).sum(1, keepdim=True))
        return {"gx": gx, "ggamma": torch.sum(f["gy"] * h, 0), "gbeta": torch.sum(f["gy"], 0)}
    X = f["G"]
    if X.shape[1] > X.shape[2]:
        X = X.mT.contiguous()
    X = X / (torch.linalg.matrix_norm(X)[:, None, None] + EPS_ORTH)
    eye = torch.eye(X.shape[1], dtype=torch.float64, device="cuda")
    for _ in range(STEPS):
        A = X @ X.mT.contiguous()
        X = (COEF[0] * eye + A @ (COEF[1] * eye + COEF[2] * A)) @ X
    return {"X": X.mT.contiguous() if case["rows"] > case["cols"] else X}

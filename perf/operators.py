"""What the training operators are measured on: the linear layer with bias, activation and residual, its backward
pass, the global gradient norm and the AdamW step over many tensors.

A case is a dict of plain values; `prepare` makes its inputs, `run` makes one pass through the operator: in its plain
form where `own` is false, through this library's calls where it is true.  Widths are those of this repository's
workloads (vision width 1024, SwiGLU width 2816, token width 4096, the 2 x 2 merged width 4608 of the projector)."""
import math

import torch

own = False

BLOCK = 256          # elements that share one scale of an 8-bit state
CODE_MAX = 448.0     # largest e4m3 value
CODE_MIN = 2.0 ** -9  # smallest positive e4m3 value
HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "step": 10, "max_norm": 1.0}


# ---------------------------------------------------------------------------------------------- cases
def _linear(name, rows, k, n, act, dtype="bf16", backward=False, bias=True, residual=False, save_z=False):
    return {"name": name, "op": "linear_backward" if backward else "linear", "rows": rows, "in": k, "out": n,
            "act": act, "dtype": dtype, "bias": bias, "residual": residual, "save_z": save_z}


def _step(name, op, layers, width, hidden, vectors, bits, master):
    return {"name": name, "op": op, "layers": layers, "width": width, "hidden": hidden, "vectors": vectors,
            "bits": bits, "master": master}


def listed():
    return [
        # one merged token through the projector's first layer: what a request of one small image waits for
        _linear("linear one token", 1, 4608, 4608, "gelu"),
        # the tokens of one 28 x 28 image, the activation's input kept for the backward pass
        _linear("linear one image", 784, 1024, 2816, "silu", save_z=True),
        # a full batch into the token width, added onto a residual stream
        _linear("linear batch", 16384, 4608, 4096, "none", residual=True),
        # the fp32 configuration at a width that no tile divides (14 x 14 RGB patches: 588)
        _linear("linear fp32 ragged", 777, 588, 1001, "gelu", dtype="f32", residual=True),
        # training the projector on one image
        _linear("backward one image", 784, 1024, 2816, "gelu", backward=True),
        # training it on a batch
        _linear("backward batch", 8192, 4608, 4096, "silu", backward=True),
        _linear("backward fp32 ragged", 777, 588, 1001, "silu", dtype="f32", backward=True),
        # the norm over one projector's few gradients, and over eight blocks' gradients
        _step("norm of a projector", "grad_norm", 0, 1152, 1152, 6, 32, True),
        _step("norm of eight blocks", "grad_norm", 8, 1024, 2816, 18, 32, True),
        # norm scales and biases alone: many small fp32 tensors, where latency counts
        _step("adamw vectors", "adamw", 0, 1024, 0, 65, 32, False),
        # eight blocks of the tower, bf16 with fp32 master copies
        _step("adamw eight blocks", "adamw", 8, 1024, 2816, 18, 32, True),
        # the same weights with 8-bit states
        _step("adamw eight blocks 8-bit", "adamw", 8, 1024, 2816, 18, 8, True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "linear_backward", "grad_norm", "adamw", "adamw"])
    if op.startswith("linear"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        wide = dtype == "bf16"
        case = _linear("", _spread(rng, 1, 8192 if wide else 2048), _spread(rng, 64, 4608 if wide else 1024),
                       _spread(rng, 64, 4608 if wide else 1024), rng.choice(["none", "gelu", "silu"]), dtype,
                       op == "linear_backward", rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5)
    else:
        case = _step("", op, _spread(rng, 1, 7), 8 * _spread(rng, 8, 128), 8 * _spread(rng, 16, 352), rng.randint(0, 40),
                     rng.choice([8, 32]) if op == "adamw" else 32, rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------------------------------------- sizes
def _pad8(n):
    return (n + 7) // 8 * 8


def _matrices(case):
    """Element counts of the bf16 matrices: per block of the tower wqkv, wo, w_gate, w_up, w_down; without blocks the
    two matrices of a projector of the given width."""
    d, f = case["width"], case["hidden"]
    if case["layers"] == 0:
        return [d * d, d * f] if f else []
    return [3 * d * d, d * d, f * d, f * d, d * f] * case["layers"]


def _vectors(case):
    return [case["width"] + (i % 3) for i in range(case["vectors"])]  # odd lengths among them


def _flat(counts):
    """Offsets of tensors laid out in one buffer, each from a multiple of 256 elements on, and the buffer's size."""
    at, offsets = 0, []
    for n in counts:
        offsets.append(at)
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    return offsets, at


def work(case):
    if case["op"] == "linear":
        m, k, n = case["rows"], case["in"], case["out"]
        es = 2 if case["dtype"] == "bf16" else 4
        b = es * (m * k + n * k + m * n * (1 + case["residual"] + case["save_z"])) + 4 * n * case["bias"]
        return {"bytes": b, "flops": 2 * m * k * n}
    if case["op"] == "linear_backward":
        m, k, n = case["rows"], case["in"], case["out"]
        es = 2 if case["dtype"] == "bf16" else 4
        b = es * (2 * m * k + 2 * n * k + m * n * (1 + (case["act"] != "none"))) + 4 * n * case["bias"]
        return {"bytes": b, "flops": 4 * m * k * n}
    big, small = sum(_matrices(case)), sum(_vectors(case))
    if case["op"] == "grad_norm":
        return {"bytes": 2 * big + 4 * small + 4, "flops": 2 * (big + small)}
    state = 2 * 8 if case["bits"] == 32 else 2 * 2 + 2 * 8 / BLOCK
    return {"bytes": (4 + 2 + 8 * case["master"] + state) * big + (8 + 4 + state) * small, "flops": 15 * (big + small)}


# ---------------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, scale, dtype, ld=None):
    """A normal matrix; rows padded to `ld` elements where that is given."""
    if ld is None or ld == shape[-1]:
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)
    return (torch.randn((shape[0], ld), generator=gen, device="cuda") * scale).to(dtype)[:, :shape[1]]


def _e4m3_blocks(v):
    """Power-of-two scale of each block of 256 values, the smallest that brings them to at most 448, and the codes."""
    b = v.reshape(-1, BLOCK)
    top = b.abs().amax(1)
    f, e = torch.frexp(top)
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp_min(-126)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.zeros_like(top))
    return (b / torch.where(top > 0, scale, torch.ones_like(scale))[:, None]).reshape(-1), scale


def _first_moment_codes(m):
    q, scale = _e4m3_blocks(m)
    return q.to(torch.float8_e4m3fn), scale


def _root_codes(v):
    """The second moment is held as codes of its root; a root above zero never becomes zero."""
    q, scale = _e4m3_blocks(v.sqrt())
    c = q.to(torch.float8_e4m3fn)
    low = (q > 0) & (c.to(q.dtype) == 0)
    return torch.where(low, torch.full_like(q, CODE_MIN), c.to(q.dtype)).to(torch.float8_e4m3fn), scale


def _group(gen, counts, case, dtype, grads_only):
    """One buffer for each of the parameters, gradients, master copies and states of the tensors `counts`."""
    offsets, n = _flat(counts)
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for o, c in zip(offsets, counts):
        live[o:o + c] = True
    normal = lambda s: torch.randn(n, generator=gen, device="cuda") * s * live  # noqa: E731
    group = {"counts": counts, "offsets": offsets, "grad": normal(1e-3).to(dtype)}
    if grads_only:
        return group
    master = normal(0.02)
    group["param"] = master.to(dtype)
    if case["master"] and dtype == torch.bfloat16:
        group["master"] = master
    group["decay"] = 0.1 if dtype == torch.bfloat16 else 0.0
    m, v = normal(3e-4), normal(1e-3).square()
    if case["bits"] == 8:
        group["m"], group["m_scale"] = _first_moment_codes(m)
        group["v"], group["v_scale"] = _root_codes(v)
    else:
        group["m"], group["v"] = m, v
    return group


def _cut(group, key):
    """The tensors of a group's buffer (their blocks' scales for a scale buffer)."""
    if key not in group:
        return [None] * len(group["counts"])
    per = BLOCK if key.endswith("scale") else 1
    return [group[key][o // per:o // per + (c + per - 1) // per] for o, c in zip(group["offsets"], group["counts"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"].startswith("linear"):
        m, k, n, dt = case["rows"], case["in"], case["out"], _dtype(case)
        ld = _pad8(k) if case["dtype"] == "bf16" else k
        s = {"case": case, "x": _normal(gen, (m, k), 1.0, dt, ld), "w": _normal(gen, (n, k), 0.02, dt, ld)}
        if case["op"] == "linear":
            s["bias"] = _normal(gen, (n,), 0.02, torch.float32) if case["bias"] else None
            s["residual"] = _normal(gen, (m, n), 1.0, dt) if case["residual"] else None
            s["y"] = torch.empty((m, n), dtype=dt, device="cuda")
            s["z"] = torch.empty_like(s["y"]) if case["save_z"] else None
        else:
            s["z"] = _normal(gen, (m, n), 1.0, dt) if case["act"] != "none" else None
            s["d_y"] = _normal(gen, (m, n), 1.0, dt)
            s["dx"] = torch.empty((m, ld), dtype=dt, device="cuda")[:, :k]
            s["dw"] = torch.empty((n, ld), dtype=dt, device="cuda")[:, :k]
            s["db"] = torch.empty(n, device="cuda") if case["bias"] else None
        if own:
            from vision_transformer_encoder_dsv4v_b200 import dsv4v as A
            act = {"none": A.ACT_NONE, "gelu": A.ACT_GELU, "silu": A.ACT_SILU}[case["act"]]
            kind = A.DSV4V_BF16 if case["dtype"] == "bf16" else A.DSV4V_F32
            s["desc"] = A.make_linear(m, k, n, act, kind, ld_x=ld, ld_w=ld)
            if case["op"] == "linear_backward":
                s["workspace"] = torch.empty(A.dsv4v_linear_backward_workspace_size(s["desc"]), dtype=torch.uint8,
                                             device="cuda")
        return s
    grads_only = case["op"] == "grad_norm"
    groups = []
    for counts, dt in ((_matrices(case), torch.bfloat16), (_vectors(case), torch.float32)):
        if counts:
            groups.append(_group(gen, counts, case, dt, grads_only))
    s = {"case": case, "groups": groups}
    if grads_only:
        s["norm"] = torch.empty((), device="cuda")
    else:
        s["norm"] = sum(g["grad"].double().square().sum() for g in groups).sqrt().float()
    if own:
        from vision_transformer_encoder_dsv4v_b200 import dsv4v as A
        grads = [t for g in groups for t in _cut(g, "grad")]
        if grads_only:
            s["table"] = A.GradTable(grads)
            s["workspace"] = torch.empty(A.dsv4v_grad_norm_workspace_size(s["table"]), dtype=torch.uint8, device="cuda")
        else:
            s["table"] = A.AdamwTable([
                dict(param=p, grad=g, master=w, exp_avg=m, exp_avg_sq=v, exp_avg_scale=ms, exp_avg_sq_scale=vs,
                     weight_decay=group["decay"])
                for group in groups
                for p, g, w, m, v, ms, vs in zip(*(_cut(group, key) for key in (
                    "param", "grad", "master", "m", "v", "m_scale", "v_scale")))])
            s["config"] = A.make_adamw(HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], step=HYPER["step"],
                                       max_grad_norm=HYPER["max_norm"])
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _activation(z, act):
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _derivative(z, act):
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain_linear(s):
    case, dt = s["case"], s["x"].dtype
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _activation(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(dt)] + ([z.to(dt)] if case["save_z"] else [])


def _plain_linear_backward(s):
    case, dt = s["case"], s["x"].dtype
    dz = s["d_y"].float()
    if s["z"] is not None:
        dz = dz * _derivative(s["z"].float(), case["act"])
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    return [dx.to(dt), dw.to(dt)] + ([dz.sum(0)] if case["bias"] else [])


def _plain_grad_norm(s):
    return sum(g["grad"].float().square().sum(dtype=torch.float64) for g in s["groups"]).sqrt().float()


def _plain_adamw(s):
    h = HYPER
    correct1, correct2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    clip = (h["max_norm"] / s["norm"]).clamp_max(1)
    out = []
    for g in s["groups"]:
        eight = "m_scale" in g
        grad = g["grad"].float() * clip
        if eight:
            m = (g["m"].float().reshape(-1, BLOCK) * g["m_scale"][:, None]).reshape(-1)
            v = (g["v"].float().reshape(-1, BLOCK) * g["v_scale"][:, None]).reshape(-1).square()
        else:
            m, v = g["m"], g["v"]
        m = m * h["beta1"] + grad * (1 - h["beta1"])
        v = v * h["beta2"] + (grad * grad) * (1 - h["beta2"])
        p = g["master"] if "master" in g else g["param"].float()
        p = p * (1 - h["lr"] * g["decay"]) - (h["lr"] / correct1) * (m / (v.sqrt() * (1 / math.sqrt(correct2)) + h["eps"]))
        g["param"].copy_(p)
        out.append(g["param"])
        if "master" in g:
            g["master"].copy_(p)
            out.append(g["master"])
        if eight:
            m, m_scale = _first_moment_codes(m)
            v, v_scale = _root_codes(v)
            g["m"].copy_(m), g["v"].copy_(v), g["m_scale"].copy_(m_scale), g["v_scale"].copy_(v_scale)
            out += [g["m"], g["m_scale"], g["v"], g["v_scale"]]
        else:
            g["m"].copy_(m), g["v"].copy_(v)
            out += [g["m"], g["v"]]
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "grad_norm": _plain_grad_norm,
                "adamw": _plain_adamw}[op](state)
    from vision_transformer_encoder_dsv4v_b200 import dsv4v as A
    s = state
    if op == "linear":
        A.dsv4v_linear_forward(s["desc"], s["x"], s["w"], s["bias"], s["residual"], s["z"], s["y"])
        return [s["y"]] + ([s["z"]] if s["z"] is not None else [])
    if op == "linear_backward":
        A.dsv4v_linear_backward(s["desc"], s["x"], s["w"], s["z"], s["d_y"], s["dx"], s["dw"], s["db"], s["workspace"])
        return [s["dx"], s["dw"]] + ([s["db"]] if s["db"] is not None else [])
    if op == "grad_norm":
        A.dsv4v_grad_norm(s["table"], s["norm"], s["workspace"])
        return s["norm"]
    A.dsv4v_adamw_step(s["config"], s["table"], grad_norm=s["norm"])
    return [g[key] for g in s["groups"] for key in ("param", "master", "m", "m_scale", "v", "v_scale") if key in g]


# ---------------------------------------------------------------------------------------------- the definitions, in 64 bits
def _exact_blocks(v):
    """Scale and scaled values of each block, by comparing with powers of two rather than by taking exponents apart."""
    b = v.view(-1, BLOCK)
    top = b.abs().max(dim=1).values
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / CODE_MAX)))
    scale = torch.where(top / scale > CODE_MAX, scale * 2, scale)
    scale = torch.where(top / (scale / 2) <= CODE_MAX, scale / 2, scale).clamp_min(2.0 ** -126)
    scale = torch.where(top > 0, scale, torch.zeros_like(scale))
    return torch.where(scale[:, None] > 0, b / scale[:, None], torch.zeros_like(b)).view(-1), scale


def _nearest_code(q):
    """The e4m3 value nearest to q, |q| <= 448: steps of 2^(e-3) between 2^e and 2^(e+1), of 2^-9 below 2^-6."""
    size = q.abs()
    e = torch.floor(torch.log2(size.clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(q / step) * step


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "linear":
        z = torch.einsum("mk,nk->mn", state["x"].double(), state["w"].double())
        if case["bias"]:
            z += state["bias"].double()
        if case["act"] == "gelu":
            y = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
        elif case["act"] == "silu":
            y = z * torch.special.expit(z)
        else:
            y = z
        y = y + state["residual"].double() if case["residual"] else y
        return [y, z] if case["save_z"] else [y]
    if case["op"] == "linear_backward":
        dz = state["d_y"].double()
        if case["act"] == "gelu":
            z = state["z"].double()
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        elif case["act"] == "silu":
            z = state["z"].double()
            s = torch.special.expit(z)
            dz = dz * (s + z * s * torch.special.expit(-z))
        out = [torch.einsum("mn,nk->mk", dz, state["w"].double()), torch.einsum("mn,mk->nk", dz, state["x"].double())]
        return out + ([torch.einsum("mn->n", dz)] if case["bias"] else [])
    if case["op"] == "grad_norm":
        return torch.linalg.vector_norm(torch.cat([g["grad"].double() for g in state["groups"]]))
    t, b1, b2 = HYPER["step"], HYPER["beta1"], HYPER["beta2"]
    norm = float(state["norm"])
    clip = HYPER["max_norm"] / norm if norm > HYPER["max_norm"] else 1.0
    out = []
    for g in state["groups"]:
        grad = clip * g["grad"].double()
        if case["bits"] == 8:
            per = lambda key: g[key + "_scale"].double().repeat_interleave(BLOCK)  # noqa: E731
            m, v = g["m"].double() * per("m"), (g["v"].double() * per("v")) ** 2
        else:
            m, v = g["m"].double(), g["v"].double()
        m, v = torch.lerp(grad, m, b1), torch.lerp(grad ** 2, v, b2)
        p = g["master" if "master" in g else "param"].double()
        p = p - HYPER["lr"] * (g["decay"] * p + (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + HYPER["eps"]))
        out += [p, p] if "master" in g else [p]
        if case["bits"] == 8:
            qm, sm = _exact_blocks(m)
            qv, sv = _exact_blocks(torch.sqrt(v))
            cv = _nearest_code(qv)
            out += [_nearest_code(qm), sm, torch.where((qv > 0) & (cv == 0), torch.full_like(cv, CODE_MIN), cv), sv]
        else:
            out += [m, v]
    return out

"""The gradient norm and the AdamW step against the fp64 oracle (oracle/dsv4v_optim.py), through the
C ABI.

Tolerances, with u = 2^-24 (half a step of fp32):
  * Norm: squares of 8 values are summed in fp32 (at most 8 u, all of one sign), the rest in fp64, and
    the root is rounded to fp32: 8 u / 2 + u, taken as 6 u.
  * Moments: beta and 1 - beta are rounded (u each), the clip factor and its product (2 u), each product
    and the sum (u each): at most 6 u of |beta m| + |(1 - beta) g| for the first, 8 u of v (a sum of
    positive terms, the clip entering twice) for the second.
  * Parameters: the factor 1 - lr decay, its product and the difference are 3 u of |p|, the update's
    chain (root, two roundings of scalars, sum, quotient, product) 12 u beside the first moment's 6 u:
    4 u |p| + 20 u of the update that |beta m| + |(1 - beta) g| would give.
  * A bf16 parameter is the fp32 result rounded once: half a step more, 2^-8 of it.
  * 8-bit states: one rounding to e4m3, half a step: 2^-4 of the value, or half the smallest code's
    step (2^-10 of the scale); a root that is raised to the smallest code is off by at most that code
    (2^-9).  The kernel starts each step from the stored values, and so does the oracle."""
import numpy as np
import pytest
import torch

from oracle import dsv4v_optim as O
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8)


def norm_of(grads):
    table = A.GradTable(grads)
    out = torch.full((), -1.0, device="cuda")
    ws = torch.empty(A.dsv4v_grad_norm_workspace_size(table), dtype=torch.uint8, device="cuda")
    A.dsv4v_grad_norm(table, out, ws)
    return out


def np64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def normal(n, scale, dtype, seed, offset=0):
    """n normal values; offset: elements that the view starts behind its buffer's (aligned) start."""
    gen = torch.Generator().manual_seed(seed)
    buf = (torch.randn(n + offset, generator=gen) * scale).to(dtype).cuda()
    return buf[offset:]


# ---------------------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("sizes", [[1], [7, 0, 8, 9], [8191, 8192, 8193], [100003, 5, 0, 262144], [0], []])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_grad_norm(sizes, dtype, offset):
    grads = [normal(n, 1.0, dtype, 7 * i + n, offset) for i, n in enumerate(sizes)]
    want = O.grad_norm([np64(g) for g in grads])
    got = float(norm_of(grads))
    assert abs(got - want) <= 6 * U * want


def test_grad_norm_many_tensors_and_types():
    # more tensors than one launch takes (1300 or so), of both types
    grads = [normal(1 + 37 * (i % 11), 1.0, torch.bfloat16 if i % 3 else torch.float32, i) for i in range(3000)]
    want = O.grad_norm([np64(g) for g in grads])
    a, b = norm_of(grads), norm_of(grads)
    assert abs(float(a) - want) <= 6 * U * want
    assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [1e30, 1e-30, 3e38])
def test_grad_norm_where_squares_leave_fp32(scale):
    grads = [torch.tensor([scale, -0.5 * scale, 0.0] + [0.25 * scale] * 5, device="cuda"), torch.zeros(300, device="cuda")]
    want = O.grad_norm([np64(g) for g in grads])
    got = float(norm_of(grads))
    if want > torch.finfo(torch.float32).max:
        assert got == float("inf")
    else:
        assert abs(got - want) <= 6 * U * want


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_grad_norm_of_gradients_that_are_not_finite(bad):
    g = torch.ones(5000, device="cuda", dtype=torch.bfloat16)
    g[4321] = bad
    got = float(norm_of([torch.ones(10, device="cuda"), g]))
    assert np.isnan(got) if np.isnan(bad) else got == float("inf")


# ---------------------------------------------------------------------------------------------- AdamW
def make(n, p_dtype, g_dtype, bits, master, seed, offset=0, decay=0.1):
    t = {"param": normal(n, 0.1, p_dtype, seed, offset), "grad": normal(n, 0.5, g_dtype, seed + 1, offset), "weight_decay": decay}
    if master:
        t["master"] = normal(n, 0.1, torch.float32, seed, offset)
        t["param"].copy_(t["master"])
    m, v = normal(n, 0.2, torch.float32, seed + 2, offset), normal(n, 0.3, torch.float32, seed + 3, offset).square_()
    if bits == 32:
        t["exp_avg"], t["exp_avg_sq"] = m, v
    else:
        blocks = (n + 255) // 256
        for key, x in (("exp_avg", m), ("exp_avg_sq", v.sqrt())):
            scale = torch.tensor(O.block_scales(np64(x)), dtype=torch.float32, device="cuda")
            assert scale.numel() == blocks
            code = (x / scale.repeat_interleave(256)[:n]).to(torch.float8_e4m3fn).view(torch.uint8)
            t[key] = torch.zeros(n + offset, dtype=torch.uint8, device="cuda")[offset:]
            t[key].copy_(code)
            t[key + "_scale"] = scale
    return t


def state_of(t):
    m, v = t["exp_avg"], t["exp_avg_sq"]
    if "exp_avg_scale" not in t:
        return np64(m), np64(v)
    codes = lambda x: x.view(torch.uint8).cpu().numpy().reshape(-1)  # noqa: E731
    return O.decode(codes(m), np64(t["exp_avg_scale"])), O.decode(codes(v), np64(t["exp_avg_sq_scale"])) ** 2


def check_step(tensors, run, step, norm=None, max_norm=0.0, hyper=HYPER):
    """Runs `run` (one step of all the tensors) and holds each of them to the oracle."""
    before = [(np64(t.get("master", t["param"]) if t.get("master") is not None else t["param"]), np64(t["grad"]), *state_of(t))
              for t in tensors]
    run()
    torch.cuda.synchronize()
    for t, (p0, g, m0, v0) in zip(tensors, before):
        h = dict(hyper, decay=t.get("weight_decay", 0.0), norm=norm, max_norm=max_norm)
        p, m, v = O.adamw(p0, g, m0, v0, step, **h)
        clip = min(1.0, max_norm / norm) if norm and max_norm else 1.0
        size = h["beta1"] * np.abs(m0) + (1 - h["beta1"]) * np.abs(g) * clip
        denom = np.sqrt(v / (1 - h["beta2"] ** step)) + h["eps"]
        tol = 4 * U * np.abs(p0) + 20 * U * h["lr"] / (1 - h["beta1"] ** step) * size / denom
        got = np64(t["param"])
        half = 2.0 ** -8 * np.abs(p) if t["param"].dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(got - p) <= tol + half), np.max(np.abs(got - p) - tol - half)
        if t.get("master") is not None:
            w = np64(t["master"])
            assert np.all(np.abs(w - p) <= tol), np.max(np.abs(w - p) - tol)
            assert torch.equal(t["param"], t["master"].to(torch.bfloat16))
        m1, v1 = state_of(t)
        if "exp_avg_scale" not in t:
            assert np.all(np.abs(m1 - m) <= 6 * U * size)
            assert np.all(np.abs(v1 - v) <= 8 * U * v + 2.0 ** -149)
            continue
        sm, sr = np64(t["exp_avg_scale"]), np64(t["exp_avg_sq_scale"])
        for got, want, s, low in ((m1, m, sm, 2.0 ** -10), (np.sqrt(v1), np.sqrt(v), sr, 2.0 ** -9)):
            each = np.repeat(s, 256)[:len(got)]
            assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * (1 + 1e-5) + low * each)
            for b, scale in enumerate(s):
                top = np.abs(want[256 * b:256 * b + 256]).max()
                assert (scale == 0) == (top == 0)
                if top > 0:  # a power of two, the smallest that fits
                    assert np.log2(scale) == np.round(np.log2(scale))
                    assert top / scale <= 448 * (1 + 1e-5) and (top / scale > 224 * (1 - 1e-5) or scale == 2.0 ** -126)
        assert np.all((v1 > 0) == (v > 0))


@pytest.mark.parametrize("n", [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 70001])
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16 f32grad", "master"])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_tensor(n, kind, bits):
    p_dtype = torch.float32 if kind == "f32" else torch.bfloat16
    g_dtype = torch.float32 if kind in ("f32", "bf16 f32grad") else torch.bfloat16
    t = make(n, p_dtype, g_dtype, bits, kind == "master", 11 * n)
    table = A.AdamwTable([t])
    for step in (1, 2, 1000):
        check_step([t], lambda: A.dsv4v_adamw_step(A.make_adamw(step=step, **HYPER), table), step)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 2, 5])
def test_adamw_unaligned_views_keep_their_neighbours(bits, offset):
    t = make(1003, torch.bfloat16, torch.bfloat16, bits, True, 5, offset)
    pad = 16
    kept = {}
    for key in ("param", "master", "exp_avg", "exp_avg_sq"):  # each inside a longer buffer
        big = torch.full((1003 + 2 * pad + offset,), 3, device="cuda").to(t[key].dtype)
        view = big[pad + offset:pad + offset + 1003]
        view.copy_(t[key])
        t[key] = view
        kept[key] = (big, big.clone())
    check_step([t], lambda: A.dsv4v_adamw_step(A.make_adamw(step=3, **HYPER), A.AdamwTable([t])), 3)
    for key, (big, was) in kept.items():
        assert torch.equal(big[:pad + offset].view(torch.uint8), was[:pad + offset].view(torch.uint8)), key
        assert torch.equal(big[pad + offset + 1003:].view(torch.uint8), was[pad + offset + 1003:].view(torch.uint8)), key


def test_adamw_list_longer_than_a_table():
    # more tensors than one launch takes (360 or so), of every kind, empty ones among them
    tensors = [make((37 * i) % 701, torch.float32 if i % 4 == 0 else torch.bfloat16, torch.float32 if i % 4 == 0 else torch.bfloat16,
                    8 if i % 3 == 0 else 32, i % 4 == 2, 1000 + i, decay=0.1 * (i % 2)) for i in range(800)]
    live = [t for t in tensors if t["param"].numel()]
    assert len(live) < len(tensors)
    table = A.AdamwTable(tensors)
    check_step(live, lambda: A.dsv4v_adamw_step(A.make_adamw(step=4, **HYPER), table), 4)


@pytest.mark.parametrize("max_norm", [0.01, 1e6, 0.0])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_clips_by_the_norm(max_norm, bits):
    tensors = [make(n, torch.bfloat16, torch.bfloat16, bits, True, n) for n in (300, 4097)]
    norm = norm_of([t["grad"] for t in tensors])
    table = A.AdamwTable(tensors)
    cfg = A.make_adamw(step=2, max_grad_norm=max_norm, **HYPER)
    check_step(tensors, lambda: A.dsv4v_adamw_step(cfg, table, grad_norm=norm), 2, float(norm), max_norm)


def test_adamw_zero_gradients_and_zero_states():
    for bits in (32, 8):
        t = make(600, torch.float32, torch.float32, bits, False, 3)
        for key in ("grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            if key in t:
                t[key].zero_()
        check_step([t], lambda: A.dsv4v_adamw_step(A.make_adamw(step=1, **HYPER), A.AdamwTable([t])), 1)


def test_adamw_8bit_root_is_never_rounded_to_zero():
    # one element's root is 2^-12 of its block's largest: below half the smallest code
    t = make(256, torch.float32, torch.float32, 8, False, 3, decay=0.0)
    t["grad"].zero_()
    t["exp_avg"].zero_(), t["exp_avg_scale"].zero_(), t["exp_avg_sq"].zero_(), t["exp_avg_sq_scale"].zero_()
    t["grad"][0], t["grad"][1] = 448.0, 448.0 * 2.0 ** -22
    check_step([t], lambda: A.dsv4v_adamw_step(A.make_adamw(step=1, **HYPER), A.AdamwTable([t])), 1)
    assert int(t["exp_avg_sq"][1]) == 1 and int(t["exp_avg_sq"][2]) == 0


def test_adamw_8bit_values_that_are_not_finite_become_nan():
    t = make(512, torch.float32, torch.float32, 8, False, 3)
    t["grad"][5], t["grad"][300] = float("inf"), float("nan")
    other = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in t.items()}
    other["grad"][5], other["grad"][300] = 0.0, 0.0
    A.dsv4v_adamw_step(A.make_adamw(step=1, **HYPER), A.AdamwTable([t]))
    m, v = state_of(t)
    bad = np.zeros(512, bool)
    bad[[5, 300]] = True
    assert np.array_equal(np.isnan(m), bad) and np.array_equal(np.isnan(v), bad)
    # the others are what they would be beside zeros
    A.dsv4v_adamw_step(A.make_adamw(step=1, **HYPER), A.AdamwTable([other]))
    ok = torch.from_numpy(~bad).cuda()
    assert torch.equal(t["param"][ok], other["param"][ok])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_skips_a_step_whose_norm_is_not_finite(bad, bits):
    t = make(3000, torch.bfloat16, torch.bfloat16, bits, True, 3)
    was = {k: v.clone() for k, v in t.items() if torch.is_tensor(v)}
    step = torch.tensor(6, device="cuda")
    norm = torch.tensor(bad, device="cuda")
    for max_norm in (0.0, 1.0):
        A.dsv4v_adamw_step(A.make_adamw(max_grad_norm=max_norm, **HYPER), A.AdamwTable([t]), grad_norm=norm, step_dev=step)
    assert int(step) == 6
    for k, v in was.items():
        assert torch.equal(t[k].view(torch.uint8), v.view(torch.uint8)), k


def test_adamw_device_schedule_in_a_replayed_graph():
    tensors = [make(n, torch.bfloat16, torch.bfloat16, bits, True, n) for n, bits in ((5000, 32), (777, 8))]
    table = A.AdamwTable(tensors)
    grads = A.GradTable([t["grad"] for t in tensors])
    ws = torch.empty(A.dsv4v_grad_norm_workspace_size(grads), dtype=torch.uint8, device="cuda")
    norm, lr, step = torch.zeros((), device="cuda"), torch.zeros((), device="cuda"), torch.zeros((), dtype=torch.int64, device="cuda")
    cfg = A.make_adamw(max_grad_norm=0.5, **dict(HYPER, lr=123.0))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        A.dsv4v_grad_norm(grads, norm, ws)
        A.dsv4v_adamw_step(cfg, table, grad_norm=norm, lr_dev=lr, step_dev=step)
    for i in range(1, 4):
        for t in tensors:
            t["grad"].copy_(normal(t["grad"].numel(), 0.1 * i, torch.bfloat16, i))
        rate = np.float32(1e-2 / i)
        lr.fill_(float(rate))
        want_norm = O.grad_norm([np64(t["grad"]) for t in tensors])
        norm32 = float(np.float32(want_norm))
        check_step(tensors, graph.replay, i, norm32, 0.5, dict(HYPER, lr=float(rate)))
        assert abs(float(norm) - want_norm) <= 6 * U * want_norm
        assert int(step) == i


def test_adamw_beyond_32_bit_offsets():
    # a tensor of over 2^31 elements: its end is stepped like a tensor of its own
    n, tail = 2 ** 31 + 777, 1024 + 777
    t = {"param": torch.zeros(n, dtype=torch.bfloat16, device="cuda"), "grad": torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
         "exp_avg": torch.zeros(n, dtype=torch.uint8, device="cuda"), "exp_avg_sq": torch.zeros(n, dtype=torch.uint8, device="cuda"),
         "exp_avg_scale": torch.zeros((n + 255) // 256, device="cuda"), "exp_avg_sq_scale": torch.zeros((n + 255) // 256, device="cuda")}
    start = n - tail
    assert start % 256 == 0
    t["param"][start:] = normal(tail, 0.1, torch.bfloat16, 1)
    t["grad"][start:] = normal(tail, 0.1, torch.bfloat16, 2)
    last = {k: v[start if not k.endswith("scale") else start // 256:].clone() for k, v in t.items()}
    assert abs(float(norm_of([t["grad"]])) - float(norm_of([last["grad"]]))) <= 12 * U * float(norm_of([last["grad"]]))
    A.dsv4v_adamw_step(A.make_adamw(**HYPER), A.AdamwTable([t]))
    A.dsv4v_adamw_step(A.make_adamw(**HYPER), A.AdamwTable([last]))
    for k, v in last.items():
        assert torch.equal(t[k][start if not k.endswith("scale") else start // 256:].view(torch.uint8), v.view(torch.uint8)), k
    assert not t["param"][:start].any()


# ---------------------------------------------------------------------------------------------- the binding's refusals
def test_tables_refuse_what_the_call_could_not_read():
    ok = lambda: make(300, torch.bfloat16, torch.bfloat16, 8, True, 1)  # noqa: E731
    A.AdamwTable([ok()])
    for change, match in [(dict(grad=torch.zeros(299, device="cuda")), "299 elements"),
                          (dict(grad=torch.zeros(300, device="cuda", dtype=torch.float16)), "float16"),
                          (dict(param=torch.zeros(600, device="cuda")[::2]), "not contiguous"),
                          (dict(exp_avg_scale=None), "no exp_avg_scale"),
                          (dict(exp_avg_scale=torch.zeros(1, device="cuda")), "1 elements"),
                          (dict(exp_avg=torch.zeros(300, device="cuda")), "uint8|float32|fp32 states"),
                          (dict(master=torch.zeros(300, device="cuda", dtype=torch.bfloat16)), "bfloat16")]:
        with pytest.raises(ValueError, match=match):
            A.AdamwTable([dict(ok(), **change)])
    t = ok()
    with pytest.raises(ValueError, match="overlap"):
        A.AdamwTable([t, t])
    with pytest.raises(ValueError, match="not contiguous"):
        A.GradTable([torch.zeros(6, device="cuda")[::2]])
    with pytest.raises(ValueError, match="float16"):
        A.GradTable([torch.zeros(6, device="cuda", dtype=torch.float16)])

"""What the optimizer's operators lose to rounding, on inputs that are made to show it.

u = 2^-24 is half a step of fp32."""
import numpy as np
import pytest
import torch

from oracle import dsv4v_optim as O
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def np64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def norm_of(grads):
    table = A.GradTable(grads)
    out = torch.full((), -1.0, device="cuda")
    ws = torch.empty(A.dsv4v_grad_norm_workspace_size(table), dtype=torch.uint8, device="cuda")
    A.dsv4v_grad_norm(table, out, ws)
    return out


# ---------------------------------------------------------------------------------------------- norm
# One value of 1 and squares just below u behind it: an fp32 sum that holds the 1 loses each of them.  Eight squares take
# eight roundings, at most 8 u of their sum: 4 u of the norm, and u for its own rounding.  Sums of sixteen would lose 15 u
# here, 7.4 u of the norm.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def ones_among_small(n, piece, runs, dtype):
    # pieces of `piece` elements, 256 of them side by side; of each `runs` such rows the first has the ones
    i = torch.arange(n)
    one = (i % piece == 0) & (i // (256 * piece) % runs == 0)
    return torch.where(one, 1.0, 2.0 ** -12 * (1 - 2.0 ** -8)).to(dtype)


def at_offset(g, offset):
    buf = torch.zeros(g.numel() + offset, dtype=g.dtype, device="cuda")
    buf[offset:] = g
    return buf[offset:]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("piece,runs", [(8, 1), (8, 2), (4, 2), (4, 4), (16, 1)])
@pytest.mark.parametrize("offset", [0, 1])
def test_grad_norm_keeps_what_a_large_neighbour_hides(dtype, piece, runs, offset):
    g = at_offset(ones_among_small(8 * 8192, piece, runs, dtype), offset)
    want = O.grad_norm([np64(g)])
    assert abs(float(norm_of([g])) - want) <= 5 * U * want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("piece,runs", [(8, 2), (4, 4)])
@pytest.mark.parametrize("n", [8192, 8193, 50000])
def test_grad_norm_does_not_depend_on_the_address(dtype, piece, runs, n):
    g = ones_among_small(n, piece, runs, dtype)
    got = [norm_of([at_offset(g, offset)]) for offset in range(8)]
    assert all(torch.equal(got[0], x) for x in got[1:])


# ---------------------------------------------------------------------------------------------- AdamW
@pytest.mark.parametrize("decay", [1e-8, 3e-8, 1e-7, 1e-6])
@pytest.mark.parametrize("on_device", [False, True])
def test_adamw_takes_a_small_decay_on_average(decay, on_device):
    # weights from 1 to 2, whose step (2 u) is above lr weight_decay, and updates of a few such steps: each result's
    # rounding is even over a step, so the mean over n weights is off by 2 u / sqrt(12 n) times a few, beside 20 u of
    # the update and of the decay
    n, lr, step = 1 << 20, 2.0 ** -20, 1000
    gen = torch.Generator().manual_seed(0)
    uniform = lambda lo, hi: (lo + (hi - lo) * torch.rand(n, generator=gen)).cuda()  # noqa: E731
    p, m, v = uniform(1, 2), uniform(-0.1, 0.1), uniform(1e-3, 1e-2)
    g = torch.randn(n, generator=gen).cuda()
    want, _, _ = O.adamw(np64(p), np64(g), np64(m), np64(v), step, lr, decay=decay / lr)
    size = np.abs(want - np64(p)).max()
    table = A.AdamwTable([dict(param=p, grad=g, exp_avg=m, exp_avg_sq=v, weight_decay=decay / lr)])
    if on_device:
        count, rate = torch.tensor(step - 1, device="cuda"), torch.tensor(lr, device="cuda")
        A.dsv4v_adamw_step(A.make_adamw(1.0), table, lr_dev=rate, step_dev=count)
    else:
        A.dsv4v_adamw_step(A.make_adamw(lr, step=step), table)
    mean = (np64(p) - want).mean()
    assert abs(mean) <= 6 * 2 * U / np.sqrt(12 * n) + 20 * U * size


# ---------------------------------------------------------------------------------------------- 8-bit states
# Stochastic rounding.  One step is the oracle's, code for code, but for draws that fall between the kernel's fp32 moments
# and the exact ones: the moments are off by a few u, 2^-20 of a code's step, so that hardly one of 10^5 elements differs,
# and then by one code.
def moments(t):
    codes = lambda x: x.view(torch.uint8).cpu().numpy().reshape(-1)  # noqa: E731
    return (O.decode(codes(t["exp_avg"]), np64(t["exp_avg_scale"])),
            O.decode(codes(t["exp_avg_sq"]), np64(t["exp_avg_sq_scale"])) ** 2)


def make8(n, seed, p_dtype=torch.float32, offset=0, master=False, zero=False):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda s, dtype: at_offset((torch.randn(n, generator=gen) * s).to(dtype), offset)  # noqa: E731
    t = {"param": normal(0.1, p_dtype), "grad": normal(0.5, p_dtype), "weight_decay": 0.1, "state_rounding": A.ROUND_STOCHASTIC}
    if master:
        t["master"] = at_offset(t["param"].float().cpu(), offset)
    blocks = (n + 255) // 256
    for key, s in (("exp_avg", 0.2), ("exp_avg_sq", 0.3)):
        t[key] = at_offset(torch.zeros(n, dtype=torch.uint8), offset)
        t[key + "_scale"] = torch.zeros(blocks, device="cuda")
        if not zero:
            x = (torch.randn(n, generator=gen) * s).double().numpy()
            x = np.abs(x) if key == "exp_avg_sq" else x
            scale = O.block_scales(x)
            codes = torch.from_numpy(x / np.repeat(scale, 256)[:n]).float().to(torch.float8_e4m3fn).view(torch.uint8)
            t[key].copy_(codes)
            t[key + "_scale"].copy_(torch.from_numpy(scale))
    return t


HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8)


@pytest.mark.parametrize("n", [1, 7, 8, 255, 257, 2048, 70001])
@pytest.mark.parametrize("kind,offset", [("f32", 0), ("bf16", 0), ("master", 0), ("master", 3)])
@pytest.mark.parametrize("step", [1, 1000, (1 << 33) + 5])
def test_stochastic_codes_are_the_oracles(n, kind, offset, step):
    p_dtype = torch.float32 if kind == "f32" else torch.bfloat16
    tensors = [make8(size, 11 * n + i, p_dtype, offset, kind == "master") for i, size in enumerate((n, 0, 300))]
    before = [(np64(t.get("master", t["param"])), np64(t["grad"]), *moments(t)) for t in tensors]
    A.dsv4v_adamw_step(A.make_adamw(step=step, **HYPER), A.AdamwTable(tensors))
    for i, (t, (p, g, m, v)) in enumerate(zip(tensors, before)):
        if len(p) == 0:
            continue
        p1, m1, v1 = O.adamw(p, g, m, v, step, decay=0.1, **HYPER)
        qm, qr, sm, sr = O.stochastic_codes(m1, v1, step, i)
        assert np.array_equal(np64(t["exp_avg_scale"]), sm) and np.array_equal(np64(t["exp_avg_sq_scale"]), sr)
        for key, want in (("exp_avg", qm), ("exp_avg_sq", qr)):
            got = O.e4m3_values()[t[key].cpu().numpy()]
            off = got != want
            assert off.sum() <= 1 + 1e-4 * len(p), (key, off.sum())
            assert np.all(np.abs(got - want) <= np.abs(want) / 8 + 2.0 ** -9)
        half = 2.0 ** -8 * np.abs(p1) if kind != "f32" else 0.0
        assert np.all(np.abs(np64(t["param"]) - p1) <= half + 4 * U * np.abs(p) + 1e-4 * HYPER["lr"])


def test_stochastic_steps_repeat_and_follow_the_device_count():
    # the same call gives the same codes, whether the host or the device counts, eagerly or replayed
    a, b, c = (make8(5000, 1) for _ in range(3))
    count = torch.zeros((), dtype=torch.int64, device="cuda")
    graph, replayed = torch.cuda.CUDAGraph(), torch.zeros((), dtype=torch.int64, device="cuda")
    cfg, table = A.make_adamw(**HYPER), A.AdamwTable([c])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        A.dsv4v_adamw_step(cfg, table, step_dev=replayed)
    seen = []
    for step in range(1, 5):
        A.dsv4v_adamw_step(A.make_adamw(step=step, **HYPER), A.AdamwTable([a]))
        A.dsv4v_adamw_step(cfg, A.AdamwTable([b]), step_dev=count)
        graph.replay()
        torch.cuda.synchronize()
        for key in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "param"):
            assert torch.equal(a[key], b[key]) and torch.equal(a[key], c[key]), (step, key)
        seen.append(a["exp_avg_sq"].clone())
    assert not torch.equal(seen[0], seen[1])


def test_stochastic_states_that_are_not_finite_become_nan():
    t = make8(512, 3)
    t["grad"][5], t["grad"][300] = float("inf"), float("nan")
    A.dsv4v_adamw_step(A.make_adamw(step=1, **HYPER), A.AdamwTable([t]))
    m, v = moments(t)
    bad = np.zeros(512, bool)
    bad[[5, 300]] = True
    assert np.array_equal(np.isnan(m), bad) and np.array_equal(np.isnan(v), bad)


# Many steps, against fp64 moments that are never taken from the codes.  The rounding keeps the expectation of both
# moments; what is left is its spread.  The second moment's: a step moves v by d = (1 - beta2) |g^2 - v| on average, and a
# draw between codes a gap h <= 17/64 v apart has a variance of at most d h: 2.7e-4 v^2 a step where v falls, which adds up
# to a relative deviation of at most 1.1 over 3000 steps of falling.  The mean over n = 16384 elements is then within
# 5 x 1.1 / 128 = 4.3 % of the exact one.  The first moment keeps about ten steps: 7 steps' variance of at most (1/16)^2 of
# |m| around it, a deviation below 0.17 and 0.7 % for the mean.  The updates are longer by 3/8 of v's relative variance (by
# 3 % in a steady state, 16 % behind a hundredfold fall in the oracle's own run): between 0.95 and 1.25 of the exact ones.
@pytest.mark.parametrize("kind", ["constant", "normal", "sparse"])
def test_stochastic_moments_follow_the_averages(kind):
    n, fall = 16384, 2000
    lr = 2.0 ** -10
    t = make8(n, 5, zero=True)
    t["param"].zero_()
    t["weight_decay"] = 0.0
    table, cfg = A.AdamwTable([t]), A.make_adamw(lr, 0.9, 0.999, 1e-12)
    count = torch.zeros((), dtype=torch.int64, device="cuda")
    M, V = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(1)
    decoded = lambda key: (t[key].view(torch.float8_e4m3fn).double().view(-1, 256) * t[key + "_scale"].double()[:, None]).view(-1)  # noqa: E731
    for step in range(1, 5001):
        size = 1.0 if step <= fall else 0.1
        if kind == "constant":
            g = torch.full((n,), size, device="cuda")
        else:
            g = torch.randn(n, generator=gen, device="cuda") * size
            if kind == "sparse" and step % 10:
                g.zero_()
        t["grad"].copy_(g)
        t["param"].zero_()
        A.dsv4v_adamw_step(cfg, table, step_dev=count)
        g = g.double()
        M.mul_(0.9).add_(g, alpha=0.1)
        V.mul_(0.999).add_(g * g, alpha=0.001)
        if step in (10, 100, 1000, 2000, 2300, 3000, 4000, 5000):
            m, v = decoded("exp_avg"), decoded("exp_avg_sq").square()
            assert abs(float(v.sum() / V.sum()) - 1) <= 0.05, step
            assert abs(float((m - M).mean())) <= 0.01 * float(M.abs().mean()) + 5 * 0.17 / n ** 0.5 * float(M.square().mean().sqrt()), step
            want = lr * (M / (1 - 0.9 ** step)).abs() / (V / (1 - 0.999 ** step)).sqrt()
            ratio = float(t["param"].double().abs().mean() / want.mean())
            assert 0.95 <= ratio <= 1.25, (step, ratio)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [0.0, 0.1])
@pytest.mark.parametrize("n", [13, 600])
def test_adamw_leaves_infinite_weights_infinite(bits, decay, n):
    # p (1 - lr decay) - update, as for a bias that masks with its infinities
    p = torch.randn(n, generator=torch.Generator().manual_seed(1)).cuda()
    p[3], p[9], p[11] = float("-inf"), float("inf"), float("nan")
    was = p.clone()
    t = {"param": p, "grad": torch.ones(n, device="cuda"), "weight_decay": decay}
    dtype = torch.uint8 if bits == 8 else torch.float32
    t["exp_avg"], t["exp_avg_sq"] = torch.zeros(n, dtype=dtype, device="cuda"), torch.zeros(n, dtype=dtype, device="cuda")
    if bits == 8:
        t["exp_avg_scale"], t["exp_avg_sq_scale"] = (torch.zeros((n + 255) // 256, device="cuda") for _ in range(2))
    A.dsv4v_adamw_step(A.make_adamw(1e-2), A.AdamwTable([t]))
    assert p[3] == float("-inf") and p[9] == float("inf") and torch.isnan(p[11])
    rest = torch.isfinite(was)
    want = was[rest] * (1 - 1e-2 * decay) - 1e-2
    assert torch.allclose(p[rest], want, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("count", [3, 500])
def test_roundings_side_by_side(count):
    # tensors of both roundings in one call, more than a launch takes too: each has the codes that its own rounding
    # gives it, and a tensor rounded to nearest those of a call without the others
    make = lambda: [dict(make8(40 + i % 300, i), state_rounding=i % 2) for i in range(count)]  # noqa: E731
    both, nearest = make(), [t for t in make() if not t["state_rounding"]]
    before = [(np64(t["param"]), np64(t["grad"]), *moments(t)) for t in both]
    A.dsv4v_adamw_step(A.make_adamw(step=9, **HYPER), A.AdamwTable(both))
    A.dsv4v_adamw_step(A.make_adamw(step=9, **HYPER), A.AdamwTable(nearest))
    for a, b in zip([t for t in both if not t["state_rounding"]], nearest):
        assert all(torch.equal(a[k], b[k]) for k in ("param", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"))
    off = total = 0
    for i, (t, (p, g, m, v)) in enumerate(zip(both, before)):
        if t["state_rounding"]:
            qm, qr, _, _ = O.stochastic_codes(*O.adamw(p, g, m, v, 9, decay=0.1, **HYPER)[1:], 9, i)
            for key, want in (("exp_avg", qm), ("exp_avg_sq", qr)):
                off += int((O.e4m3_values()[t[key].cpu().numpy()] != want).sum())
                total += len(want)
    assert off <= 1 + 1e-4 * total

"""A training step of a two-layer projector as a program would run it: the Linear layers forward and backward, the
gradient norm, the clipped AdamW step on bf16 weights with fp32 masters, eagerly and as a replayed graph.

Tolerances.  Each step is held to the fp64 oracle from the weights it started with, in the Frobenius norm, by counting
bf16 roundings (at most 2^-8 of a tensor's norm each) along the way: y takes those of h and y; the second layer's
gradients those of h, dw and dx; the first layer's those of z, dz, the incoming gradient, dw and dx besides.  The
optimizer is held to its own gradients by the tolerance of its tests: 4 u of the weight and 20 u of the largest step."""
import numpy as np
import pytest
import torch

from oracle import dsv4v_linear as OL
from oracle import dsv4v_optim as OO
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -8
U = 2.0 ** -24
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)


def np64(t):
    return t.detach().double().cpu().numpy()


def fro(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


class Projector:
    """hidden = gelu(x w1^T + b1), y = hidden w2^T + b2 + residual, with everything a step needs."""

    def __init__(self, rows, width, hidden, out, bits, seed=0):
        gen = torch.Generator().manual_seed(seed)
        bf16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.l1 = A.make_linear(rows, width, hidden, A.ACT_GELU)
        self.l2 = A.make_linear(rows, hidden, out)
        self.x = (torch.randn(rows, width, generator=gen)).bfloat16().cuda()
        self.residual = torch.randn(rows, out, generator=gen).bfloat16().cuda()
        self.target = torch.randn(rows, out, generator=gen).cuda()
        self.z, self.h, self.y = bf16(rows, hidden), bf16(rows, hidden), bf16(rows, out)
        self.dy, self.dh, self.dx = bf16(rows, out), bf16(rows, hidden), bf16(rows, width)
        shapes = {"w1": (hidden, width), "w2": (out, hidden), "b1": (hidden,), "b2": (out,)}
        self.master = {k: (torch.randn(s, generator=gen) * (s[-1] ** -0.5 if len(s) == 2 else 0.1)).cuda() for k, s in shapes.items()}
        self.w = {k: (m.bfloat16() if m.dim() == 2 else m) for k, m in self.master.items()}
        self.g = {k: torch.zeros_like(w) for k, w in self.w.items()}
        self.state = {}
        tensors = []
        for k, w in self.w.items():
            n = w.numel()
            if bits == 8:
                s = dict(exp_avg=torch.zeros(n, dtype=torch.uint8, device="cuda"), exp_avg_sq=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                         exp_avg_scale=torch.zeros((n + 255) // 256, device="cuda"), exp_avg_sq_scale=torch.zeros((n + 255) // 256, device="cuda"))
            else:
                s = dict(exp_avg=torch.zeros(n, device="cuda"), exp_avg_sq=torch.zeros(n, device="cuda"))
            self.state[k] = s
            tensors.append(dict(param=w, grad=self.g[k], master=self.master[k] if w.dim() == 2 else None,
                                weight_decay=0.05 if w.dim() == 2 else 0.0, **s))
        self.table = A.AdamwTable(tensors)
        self.grads = A.GradTable(list(self.g.values()))
        size = max(A.dsv4v_linear_backward_workspace_size(self.l1), A.dsv4v_linear_backward_workspace_size(self.l2))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.norm_ws = torch.empty(A.dsv4v_grad_norm_workspace_size(self.grads), dtype=torch.uint8, device="cuda")
        self.norm = torch.zeros((), device="cuda")
        self.step = torch.zeros((), dtype=torch.int64, device="cuda")
        self.cfg = A.make_adamw(max_grad_norm=0.5, **HYPER)

    def run(self):
        w, g = self.w, self.g
        A.dsv4v_linear_forward(self.l1, self.x, w["w1"], w["b1"], None, self.z, self.h)
        A.dsv4v_linear_forward(self.l2, self.h, w["w2"], w["b2"], self.residual, None, self.y)
        self.dy.copy_((self.y.float() - self.target) / self.y.shape[0])
        A.dsv4v_linear_backward(self.l2, self.h, w["w2"], None, self.dy, self.dh, g["w2"], g["b2"], self.ws)
        A.dsv4v_linear_backward(self.l1, self.x, w["w1"], self.z, self.dh, self.dx, g["w1"], g["b1"], self.ws)
        A.dsv4v_grad_norm(self.grads, self.norm, self.norm_ws)
        A.dsv4v_adamw_step(self.cfg, self.table, grad_norm=self.norm, step_dev=self.step)

    def everything(self):
        out = dict(self.w, **{"master " + k: v for k, v in self.master.items()}, **{"grad " + k: v for k, v in self.g.items()})
        out.update({"y": self.y, "dx": self.dx, "norm": self.norm, "step": self.step})
        out.update({f"{k} {n}": t for k, s in self.state.items() for n, t in s.items()})
        return {k: v.clone() for k, v in out.items()}


def moments(p, k):
    s = p.state[k]
    if "exp_avg_scale" not in s:
        return np64(s["exp_avg"]), np64(s["exp_avg_sq"])
    codes = lambda t: t.cpu().numpy()  # noqa: E731
    return (OO.decode(codes(s["exp_avg"]), np64(s["exp_avg_scale"])),
            OO.decode(codes(s["exp_avg_sq"]), np64(s["exp_avg_sq_scale"])) ** 2)


@pytest.mark.parametrize("rows,width,hidden,out", [(1, 64, 96, 48), (50, 200, 304, 104), (784, 1024, 2816, 1024)])
@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps(rows, width, hidden, out, bits):
    p = Projector(rows, width, hidden, out, bits)
    for step in range(1, 4):
        w = {k: np64(v) for k, v in p.w.items()}
        master = {k: np64(v) for k, v in p.master.items()}
        m0 = {k: moments(p, k) for k in p.w}
        p.run()
        torch.cuda.synchronize()
        assert A.dsv4v_device_error() == 0 and int(p.step) == step
        h, z = OL.forward(np64(p.x), w["w1"], w["b1"], None, "gelu")
        y, _ = OL.forward(h, w["w2"], w["b2"], np64(p.residual))
        assert fro(np64(p.y), y) <= 2 * ROUND
        dh, dw2, db2, _ = OL.backward(h, w["w2"], None, np64(p.dy))
        dx, dw1, db1, _ = OL.backward(np64(p.x), w["w1"], z, dh, "gelu")
        for got, want, roundings in ((p.g["w2"], dw2, 2), (p.g["b2"], db2, 1), (p.g["w1"], dw1, 4), (p.g["b1"], db1, 3), (p.dx, dx, 4)):
            assert fro(np64(got), want) <= roundings * ROUND
        norm = OO.grad_norm([np64(g) for g in p.g.values()])
        assert abs(float(p.norm) - norm) <= 6 * U * norm
        for k in p.w:
            before = (master[k] if p.w[k].dim() == 2 else w[k]).reshape(-1)
            decay = 0.05 if p.w[k].dim() == 2 else 0.0
            after, _, v = OO.adamw(before, np64(p.g[k]).reshape(-1), *m0[k], step, decay=decay, norm=float(p.norm), max_norm=0.5, **HYPER)
            clip = min(1.0, 0.5 / float(p.norm))
            size = HYPER["beta1"] * np.abs(m0[k][0]) + (1 - HYPER["beta1"]) * np.abs(np64(p.g[k]).reshape(-1)) * clip
            denom = np.sqrt(v / (1 - HYPER["beta2"] ** step)) + HYPER["eps"]
            tol = 4 * U * np.abs(before) + 20 * U * HYPER["lr"] / (1 - HYPER["beta1"] ** step) * size / denom
            got = np64(p.master[k] if p.w[k].dim() == 2 else p.w[k]).reshape(-1)
            assert np.all(np.abs(got - after) <= tol), k
            if p.w[k].dim() == 2:
                assert torch.equal(p.w[k], p.master[k].bfloat16())


@pytest.mark.parametrize("bits", [32, 8])
def test_a_replayed_training_step_is_the_eager_one(bits):
    # two captured graphs beside an eager program of the same inputs, replayed in turn
    eager, a, b = (Projector(300, 200, 304, 104, bits) for _ in range(3))
    graphs = []
    for p in (a, b):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.run()
        graphs.append(graph)
    for step in range(4):
        eager.run()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = eager.everything()
        for p in (a, b):
            for k, v in p.everything().items():
                assert torch.equal(v.view(torch.uint8) if v.dim() else v, want[k].view(torch.uint8) if v.dim() else want[k]), (step, k)


def test_blocks_gradients_go_into_the_step():
    # the tower's own backward, then the norm and the step over its weights; the next forward reads the new weights
    D, H, F = 1024, 16, 2816
    cfg, batch = A.make_config(D, H, F, 2, 4096, 1), A.BatchRef([(6, 9), (5, 4)])
    gen = torch.Generator().manual_seed(0)
    shapes = {"norm1_w": (D,), "norm2_w": (D,), "wqkv": (3 * D, D), "wo": (D, D), "w_gate": (F, D), "w_up": (F, D), "w_down": (D, F)}
    layer = {k: (1 + 0.1 * torch.randn(s, generator=gen)).cuda() if len(s) == 1 else (0.02 * torch.randn(s, generator=gen)).bfloat16().cuda()
             for k, s in shapes.items()}
    grad = {k: torch.empty_like(v) for k, v in layer.items()}
    x0 = torch.randn(batch.n_patches, D, generator=gen).bfloat16().cuda()
    d_out = torch.randn(batch.n_patches, D, generator=gen).bfloat16().cuda()
    dx = torch.empty_like(x0)
    ws = torch.empty(max(A.dsv4v_backward_workspace_size(cfg, batch), A.dsv4v_workspace_size(cfg, batch)), dtype=torch.uint8, device="cuda")
    cos = torch.empty(batch.n_patches, D // H // 2, device="cuda")
    sin = torch.empty_like(cos)
    A.dsv4v_rope2d_table(cfg, batch, cos, sin)
    table = A.AdamwTable([dict(param=layer[k], grad=grad[k], exp_avg=torch.zeros(layer[k].numel(), device="cuda"),
                               exp_avg_sq=torch.zeros(layer[k].numel(), device="cuda")) for k in layer])
    grads = A.GradTable([grad[k] for k in layer])
    norm = torch.empty((), device="cuda")
    norm_ws = torch.empty(A.dsv4v_grad_norm_workspace_size(grads), dtype=torch.uint8, device="cuda")
    keys = ("norm1_w", "norm2_w", "wqkv", "wo", "w_gate", "w_up", "w_down")
    before = {k: v.clone() for k, v in layer.items()}
    A.dsv4v_block_backward(cfg, batch, A.block_weights(layer), cos, sin, x0, d_out, dx, A.block_grads(*(grad[k] for k in keys)), ws)
    A.dsv4v_grad_norm(grads, norm, norm_ws)
    A.dsv4v_adamw_step(A.make_adamw(1e-2), table, grad_norm=norm)
    x = x0.clone()
    A.dsv4v_block_forward(cfg, batch, A.block_weights(layer), cos, sin, x, ws)
    assert A.dsv4v_device_error() == 0
    want = OO.grad_norm([np64(g) for g in grad.values()])
    assert abs(float(norm) - want) <= 6 * U * want
    for k, v in layer.items():  # a first step moves every weight that has a gradient by the learning rate, against its sign
        moved, g = np64(v) - np64(before[k]), np64(grad[k])
        after = OO.adamw(np64(before[k]).reshape(-1), g.reshape(-1), 0 * g.reshape(-1), 0 * g.reshape(-1), 1, 1e-2)[0].reshape(v.shape)
        half = 2.0 ** -8 * np.abs(after) if v.dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(np64(v) - after) <= 4 * U * np.abs(np64(before[k])) + 20 * U * 1e-2 + half), k
        assert np.abs(moved).max() > 5e-3
    # the forward after the step is that of the new weights, bit for bit
    torch.cuda.synchronize()
    again = x0.clone()
    A.dsv4v_block_forward(cfg, batch, A.block_weights({k: v.clone() for k, v in layer.items()}), cos, sin, again, ws)
    assert torch.equal(x, again)

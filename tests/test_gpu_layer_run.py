"""The operators around a delta-rule layer as a serving loop and a training step run them together."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import (build, chunk_fwd, decode_tokens, gated_scan_bwd, gated_scan_fwd,
                                           output_gate_rmsnorm, output_gate_rmsnorm_bwd, rmsnorm_bwd, rmsnorm_fwd,
                                           rmsnorm_quant, state_copy, state_dequantize, state_quantize)
from tests import layer_reference as ref
from tests.layer_reference import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_serving():
    """Two requests prefilled into a pool, continued by drafts; one is parked in 8 bits, the other goes on, and the
    parked one resumes in another slot. Every step against the same layer with fp32 states that were never parked,
    the parked request's within what its codes can be off."""
    torch.manual_seed(0)
    H, d, D, T, K = 4, 128, 512, 70, 4
    w_in, w_out = 1 + 0.1 * torch.randn(D, device="cuda"), 1 + 0.1 * torch.randn(d, device="cuda")
    proj = [torch.randn(D, H * d, device="cuda") / D ** 0.5 for _ in range(5)] + [torch.randn(D, H, device="cuda") / D ** 0.5]

    def layer_in(x, res):
        """Norm with the residual in 8 bits, then the projections of what the codes stand for."""
        q8, scales, h = rmsnorm_quant(x, w_in, residual=res)
        y = (q8.float().unflatten(-1, (-1, 128)) * scales[..., None]).flatten(-2)
        plain, _, _ = rmsnorm_fwd(x, w_in, residual=res)
        assert ((y - plain.float()).norm() / plain.float().norm()) < 0.04  # 2^-4 at most of each value
        q, k, v, g, z = ((y @ p).unflatten(-1, (H, d)) for p in proj[:5])
        return [t.bfloat16() for t in (q, k, v)], (g + 3).contiguous(), torch.sigmoid(y @ proj[5]), z.bfloat16(), h

    how = dict(gate="logsigmoid", l2norm_qk=True)
    x, res = torch.randn(2, T, D, device="cuda").bfloat16(), torch.randn(2, T, D, device="cuda").bfloat16()
    (q, k, v), g, beta, z, _ = layer_in(x, res)
    _, state = chunk_fwd(q, k, v, g, beta, d ** -0.5, **how)
    pool = torch.zeros(8, H, d, d, device="cuda")
    state_copy(pool, i32([0, 1]), i32([6, 2]), source=state)
    exact = state.clone()

    def step(slots, rows, pool, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(2, K, D, generator=gen, device="cuda").bfloat16()
        res = torch.randn(2, K, D, generator=gen, device="cuda").bfloat16()
        (q, k, v), g, beta, z, _ = layer_in(x, res)
        q, k, v, g, beta, z = (t[rows].contiguous() for t in (q, k, v, g, beta, z))
        drafts = decode_tokens(q, k, v, g, beta, d ** -0.5, pool, slots=i32(slots), write_state=False, **how)
        accepted = i32([3] * len(rows))
        out = decode_tokens(q, k, v, g, beta, d ** -0.5, pool, slots=i32(slots), counts=accepted, **how)
        assert torch.equal(out[:, :3], drafts[:, :3])
        return output_gate_rmsnorm(out[:, :3].contiguous(), z[:, :3].contiguous(), w_out)

    a, b = step([6, 2], [0, 1], pool, 1), step([0, 1], [0, 1], exact, 1)
    assert torch.equal(a, b) and torch.equal(pool[[6, 2]], exact)
    store = torch.zeros(3, H, d, d, dtype=torch.int8, device="cuda")
    scales = torch.zeros(3, H, d, device="cuda")
    state_quantize(pool, i32([6]), store, scales, i32([1]))
    state_copy(pool, i32([-1]), i32([6]))
    a, b = step([2], [1], pool, 2), step([1], [1], exact, 2)
    assert torch.equal(a, b)
    state_dequantize(store, scales, i32([1]), pool, i32([4]))
    assert ((pool[4] - exact[0]).abs() <= exact[0].abs().amax(-1, keepdim=True) / 254 * (1 + 2.0 ** -12)).all()
    state_quantize(pool, i32([4]), store, scales, i32([2]))
    state_dequantize(store, scales, i32([2]), pool, i32([5]))
    # What was held once is held again within a rounding of its scale.
    assert ((pool[5] - pool[4]).abs() <= 2.0 ** -21 * pool[4].abs()).all()
    a, b = step([4, 2], [0, 1], pool, 3), step([0, 1], [0, 1], exact, 3)
    assert torch.equal(a[1], b[1]) and (a[0] - b[0]).float().norm() / b[0].float().norm() < 0.05
    assert not pool[[0, 1, 3, 6, 7]].any()


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, w):
        y, h, rstd = rmsnorm_fwd(x, w, residual=residual, save_rstd=True)
        ctx.save_for_backward(h, rstd, w)
        return y, h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh):
        h, rstd, w = ctx.saved_tensors
        return rmsnorm_bwd(dy.contiguous(), h, rstd, w, dh=dh.contiguous())


class Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, z, w):
        ctx.save_for_backward(o, z, w)
        return output_gate_rmsnorm(o, z, w)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        return output_gate_rmsnorm_bwd(dout.contiguous(), *ctx.saved_tensors)


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z):
        h, _, carries = gated_scan_fwd(x, z, gate="logsigmoid", write="complement", save_carries=True)
        ctx.save_for_backward(x, z, carries)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        dx, dz, _ = gated_scan_bwd(dh.contiguous(), *ctx.saved_tensors, gate="logsigmoid", write="complement")
        return dx, dz


def test_training():
    """Norm with its residual, the gated recurrence and the output gate in a layer, twice: the gradients under
    autograd against the same layer of elementary operations in 64 bits."""
    gen = torch.Generator().manual_seed(4)
    B, T, H, d = 2, 40, 2, 64
    D = H * d
    leaves = [torch.randn(*s, generator=gen) * f + o for s, f, o in
              (((B, T, D), 1, 0), ((B, T, D), 2, 0), ((D,), 0.1, 1), ((d,), 0.1, 1), ((D, D), D ** -0.5, 0), ((D, D), D ** -0.5, 0))]
    dout, dres = torch.randn(B, T, D, generator=gen), torch.randn(B, T, D, generator=gen)

    def plain_norm(x, res, w):
        h = x + res
        return w * h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt(), h

    def plain_gate(o, z, w):
        return w * o * (o.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * torch.sigmoid(z)

    def plain_scan(x, z):
        a, h, out = torch.sigmoid(z), 0.0, []
        for t in range(T):
            h = a[:, t] * h + (1 - a[:, t]) * x[:, t]
            out.append(h)
        return torch.stack(out, 1)

    def run(norm, scan, gate, cast, device):
        x, res, w, wo, pa, pb = (cast(t).to(device).requires_grad_() for t in leaves)
        y, r = x, res
        for _ in range(2):
            y, r = norm(y, r, w)
            h = scan((y @ pa).contiguous(), (y @ pb + 1).contiguous())
            y = gate(h.unflatten(-1, (H, d)).contiguous(), (y @ pa).unflatten(-1, (H, d)).contiguous(), wo).flatten(-2)
        loss = (y * cast(dout).to(device)).sum() + (r * cast(dres).to(device)).sum()
        return y, r, torch.autograd.grad(loss, (x, res, w, wo, pa, pb))

    got = run(Norm.apply, Scan.apply, Gate.apply, lambda t: t.float(), "cuda")
    want = run(plain_norm, plain_scan, plain_gate, lambda t: t.double(), "cpu")
    for a, b in zip((*got[:2], *got[2]), (*want[:2], *want[2])):
        a, b = f64(a), f64(b)
        # fp32 through two layers of some hundred roundings each, and matrix products of 128 terms (torch's, in
        # fp32): 2^-24 times a few hundred of the values' size.
        assert np.linalg.norm(a - b) <= 2.0 ** -14 * np.linalg.norm(b)
    assert ref.U == 2.0 ** -24

"""GPU test of the operators in include/cbk_nn.h inside torch.autograd functions: their own calls' bits, and
a refusal outside of one."""
import pytest

from test_gpu_nn import acts, compress, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 30, 400])
def test_autograd_functions_around_the_operators(T):
    import torch
    import fly_decode_amd as cbk

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, t):
            ctx.t = t
            return cbk.linear(t, x)

        @staticmethod
        def backward(ctx, dy):
            return cbk.linear_dx(ctx.t, dy), None

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate, up):
            ctx.save_for_backward(x)
            ctx.pair = gate, up
            return cbk.ffn_gated(gate, up, x)

        @staticmethod
        def backward(ctx, dh):
            return cbk.ffn_gated_bwd(*ctx.pair, *ctx.saved_tensors, dh, projections=False)[0], None, None

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, head, labels):
            loss, lse = cbk.xent(head, x, labels)
            ctx.save_for_backward(x, labels, lse)
            ctx.head = head
            return loss

        @staticmethod
        def backward(ctx, dloss):
            x, labels, lse = ctx.saved_tensors
            return cbk.xent_bwd(ctx.head, x, labels, lse, dloss.contiguous()), None, None

    K, F, V = 128, 320, 500
    gate, up, down, head = (compress(cbk, weights(torch, *s, 900, 140 + i, 0.1)) for i, s in enumerate(((F, K), (F, K), (K, F), (V, K))))
    x = acts(torch, T, K, 145).cuda().requires_grad_()
    labels = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(146)).cuda()
    h = Block.apply(x, gate, up)
    y = Linear.apply(h, down)
    Loss.apply(y, head, labels).sum().backward()

    with torch.no_grad():
        loss, lse = cbk.xent(head, y, labels)
        dy = cbk.xent_bwd(head, y, labels, lse, torch.ones(T, device="cuda"))
        dx = cbk.ffn_gated_bwd(gate, up, x, cbk.linear_dx(down, dy))[0]
    assert torch.equal(x.grad.view(torch.int16), dx.view(torch.int16))
    with pytest.raises(ValueError, match="no_grad"):
        cbk.ffn_gated(gate, up, x)

"""An expert MLP of the user's own (two matrices and GELU, where the layer's experts are SwiGLU) on the
layer's routing, from the grouped products:

* ``train_step``: forward and backward on packed rows (the dispatch's exact offsets), the weight
  gradients added to fp32 accumulators;
* ``serve``: the same MLP with 8-bit weights and activations on the dispatch's padded rows
  (``moe_segments``), for any number of tokens down to one (the products' kernel is chosen by the rows of
  the buffer, so that a few tokens on padded rows take the kernel of many).

    python examples/expert_mlp.py [--tokens T]

prints how far both are from the same MLP in plain torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_layer_10_gb300 as moe  # noqa: E402

gelu = torch.nn.functional.gelu


class ExpertMLP:
    """E experts W2 gelu(W1 x), top k of a linear router, T tokens a step.  W1 [E, f, d], W2 [E, d, f]."""

    def __init__(self, T, d, f, E, k, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)

        self.T, self.d, self.f, self.E, self.k = T, d, f, E, k
        self.W_r = normal(d, E, std=d ** -0.5)
        self.W1 = normal(E, f, d, std=d ** -0.5).bfloat16()
        self.W2 = normal(E, d, f, std=f ** -0.5).bfloat16()
        self.dW1 = torch.zeros(E, f, d, device="cuda")
        self.dW2 = torch.zeros(E, d, f, device="cuda")
        self.cfg = moe.config(T=T, d=d, f=f, E=E, k=k)
        self.buf = moe.Buffers.allocate(self.cfg)
        n, rows = T * k, self.buf.rows
        fp32 = dict(dw_dtype=torch.float32, accumulate=1)
        self.up, self.down = moe.grouped_config(n, d, f, E, **fp32), moe.grouped_config(n, f, d, E, **fp32)
        self.up8, self.down8 = moe.grouped_config(rows, d, f, E), moe.grouped_config(rows, f, d, E)
        self.ws = moe.grouped_workspace(self.up)
        self.quantised = None

    def route(self, x):
        """Experts and gates of every slot, and the dispatch: rows sorted by expert."""
        T, E, k = self.T, self.E, self.k
        i32 = dict(dtype=torch.int32, device="cuda")
        idx, gates = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
        counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        row_of_slot, token_of_row = torch.empty(T, k, **i32), torch.empty(T * k, **i32)
        x_perm = torch.empty(self.buf.rows, self.d, dtype=torch.bfloat16, device="cuda")
        moe.moe_route(self.cfg, x, self.W_r, None, idx, gates, None, self.buf.ws)
        moe.moe_dispatch(self.cfg, idx, x, counts, offsets, row_of_slot, token_of_row, x_perm, self.buf.ws)
        return idx, gates, offsets, row_of_slot, token_of_row, x_perm

    def train_step(self, x, dy):
        """y, and for its gradient dy the input gradient (of the experts' path) and the gates'; the weight
        gradients are added to dW1 and dW2."""
        _, gates, offsets, row_of_slot, token_of_row, _ = self.route(x)
        n, token = self.T * self.k, token_of_row.long()
        begin, end = offsets[:-1], offsets[1:]   # packed groups: one array serves as both
        gate = torch.empty(n, device="cuda")
        gate[row_of_slot.flatten().long()] = gates.flatten()

        def rows(width):
            return torch.empty(n, width, dtype=torch.bfloat16, device="cuda")

        xp, a, o = x[token], rows(self.f), rows(self.d)
        moe.moe_grouped_mm(self.up, begin, end, xp, self.W1, a, self.ws)
        h = gelu(a.float()).bfloat16()
        moe.moe_grouped_mm(self.down, begin, end, h, self.W2, o, self.ws)
        y = torch.zeros(self.T, self.d, device="cuda").index_add_(0, token, o.float() * gate[:, None])

        dyp = dy[token]
        dgate = (dyp.float() * o.float()).sum(1)
        do = (dyp.float() * gate[:, None]).bfloat16()
        dh, dxp = rows(self.f), rows(self.d)
        moe.moe_grouped_mm_dw(self.down, begin, end, do, h, self.dW2, self.ws)
        moe.moe_grouped_mm_dx(self.down, begin, end, do, self.W2, dh, self.ws)
        da = torch.ops.aten.gelu_backward(dh.float(), a.float()).bfloat16()
        moe.moe_grouped_mm_dw(self.up, begin, end, da, xp, self.dW1, self.ws)
        moe.moe_grouped_mm_dx(self.up, begin, end, da, self.W1, dxp, self.ws)
        dx = torch.zeros(self.T, self.d, device="cuda").index_add_(0, token, dxp.float())
        dgates = dgate[row_of_slot.flatten().long()].view(self.T, self.k)
        return y.bfloat16(), dx.bfloat16(), dgates

    def quantise(self):
        """8-bit codes and scales of the weights, one scale an output channel (once, before serving)."""
        self.quantised = []
        for W in (self.W1, self.W2):
            codes = torch.empty(W.shape, dtype=torch.int8, device="cuda")
            scales = torch.empty(W.shape[:2], device="cuda")
            moe.moe_quantize_rows_i8(W, codes, scales)
            self.quantised += [codes, scales]

    def serve(self, x):
        """y with 8-bit weights and activations (one scale a row, found as it comes)."""
        _, gates, _, _, _, x_perm = self.route(x)
        q1, s1, q2, s2 = self.quantised
        begin, end = (torch.empty(self.E, dtype=torch.int32, device="cuda") for _ in range(2))
        moe.moe_segments(self.cfg, begin, end, self.buf.ws)

        def product(cfg, v, q, s, out):
            codes = torch.empty(v.shape, dtype=torch.int8, device="cuda")
            scales = torch.empty(v.shape[0], device="cuda")
            moe.moe_quantize_rows_i8(v, codes, scales)
            moe.moe_grouped_mm_i8(cfg, begin, end, codes, scales, q, s, out, self.ws)
            return out

        rows = self.buf.rows
        a = product(self.up8, x_perm, q1, s1, torch.zeros(rows, self.f, dtype=torch.bfloat16, device="cuda"))
        h = gelu(a.float()).bfloat16()
        o = product(self.down8, h, q2, s2, torch.zeros(rows, self.d, dtype=torch.bfloat16, device="cuda"))
        y = torch.empty(self.T, self.d, dtype=torch.bfloat16, device="cuda")
        moe.moe_combine(self.cfg, o, gates, y, self.buf.ws)
        return y

    def plain(self, x, idx, gates, W1=None, W2=None):
        """The same MLP in plain torch, fp32, for the experts and gates given."""
        W1, W2 = (self.W1.float(), self.W2.float()) if W1 is None else (W1, W2)
        y = torch.zeros(self.T, self.d, device="cuda")
        for e in range(self.E):
            t, j = (idx == e).nonzero(as_tuple=True)
            y = y.index_add(0, t, gelu(x[t] @ W1[e].T) @ W2[e].T * gates[t, j, None])
        return y


def far(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def main(argv=None):
    """{what: relative difference from plain torch} of a training step and of serving."""
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=512)
    T = p.parse_args(argv).tokens
    m = ExpertMLP(T, d=256, f=512, E=8, k=2)
    x, dy = (torch.randn(T, m.d, device="cuda").bfloat16() for _ in range(2))
    idx, gates = m.route(x)[:2]
    y, dx, dgates = m.train_step(x, dy)
    m.quantise()
    y8 = m.serve(x)
    assert moe.moe_check_error(m.ws) == 0 and moe.moe_check_error(m.buf.ws) == 0
    leaves = [t.float().requires_grad_() for t in (x, gates, m.W1, m.W2)]
    ref = m.plain(leaves[0], idx.long(), leaves[1], leaves[2], leaves[3])
    ref.backward(dy.float())
    rdx, rdg, rd1, rd2 = (t.grad for t in leaves)
    return {"y": far(y, ref), "dx": far(dx, rdx), "dgates": far(dgates, rdg), "dW1": far(m.dW1, rd1),
            "dW2": far(m.dW2, rd2), "y (8-bit)": far(y8, ref)}


if __name__ == "__main__":
    for what, off in main().items():
        print(f"{what:10s} {off:.2e} off plain torch")

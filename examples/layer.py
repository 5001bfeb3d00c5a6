"""One selective-scan layer from this package's operators, trained and served.

    residual, x -> addnorm -> in_proj -> (x, z) -> sconv -> x_proj -> sscan
                -> gatenorm(z) -> out_proj -> next layer's x

The projections are torch matrix products; everything between them is this
package's.  ``train`` fits the layer to a random target on a batch of sequences with the
forward and gradient operators; ``serve`` runs packed prompts of different
lengths through the cached forms and then decodes token by token, and
checks that both give what one call over the whole sequences gives.

    python examples/layer.py [--dtype f32|bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_recurrence_gb300 as lr  # noqa: E402


class Layer:
    """Weights of a layer and its forward, gradient, prompt and single-token forms."""

    def __init__(self, width=256, inner=512, states=16, rank=16, conv=4, dtype=torch.float32, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std: torch.randn(s, generator=g, device=device) * std  # noqa: E731
        self.inner, self.states, self.rank, self.dtype = inner, states, rank, dtype
        self.w = {
            "norm": torch.ones(width, device=device),
            "in_proj": r(2 * inner, width, std=width ** -0.5),
            "conv": r(inner, conv, std=conv ** -0.5), "conv_bias": r(inner, std=0.1),
            "x_proj": r(rank + 2 * states, inner, std=inner ** -0.5),
            "dt_proj": r(inner, rank, std=rank ** -0.5), "dt_bias": r(inner, std=0.5) - 3.0,
            "A": -torch.arange(1, states + 1, device=device).float().repeat(inner, 1), "D": torch.ones(inner, device=device),
            "gate_norm": torch.ones(inner, device=device),
            "out_proj": r(width, inner, std=inner ** -0.5),
        }

    def _mm(self, name):
        return self.w[name].to(self.dtype)

    def _split(self, proj):
        """Step sizes before their projection, B and C, of proj [.., rank + 2 states, time]."""
        return (t.contiguous() for t in proj.split([self.rank, self.states, self.states], -2))

    # ---- whole batches --------------------------------------------------------

    def forward(self, x, residual):
        """x [batch, L, width] in the layer's dtype, residual [batch, L, width] float32.
        Returns the layer's output, the new residual and what the gradients need."""
        w, (b, L, d) = self.w, x.shape
        h, res = lr.addnorm_fwd(x.view(-1, d), residual.view(-1, d), w["norm"])
        xz = torch.matmul(self._mm("in_proj"), h.view(b, L, d).transpose(1, 2))
        xc, z = xz[:, :self.inner], xz[:, self.inner:]
        u, _ = lr.sconv_fwd(xc, w["conv"], w["conv_bias"])
        low, B, C = self._split(torch.matmul(self._mm("x_proj"), u))
        raw = torch.matmul(self._mm("dt_proj"), low).float() + w["dt_bias"][:, None]
        delta = torch.nn.functional.softplus(raw).to(self.dtype)
        y, _ = lr.sscan_fwd(u, delta, w["A"], B, C, w["D"])
        g = lr.gatenorm_fwd(y, z, w["gate_norm"])
        out = torch.matmul(self._mm("out_proj"), g).transpose(1, 2).contiguous()
        return out, res.view(b, L, d), (h, res, xc, z, u, low, B, C, raw, delta, y, g)

    def backward(self, saved, dout, dresidual):
        """Gradients for upstream gradients of the output and of the new residual:
        a dict over the weights, and (dx, dresidual)."""
        w, (h, res, xc, z, u, low, B, C, raw, delta, y, g) = self.w, saved
        b, L, d = dout.shape
        gw = {}
        do = dout.transpose(1, 2)  # [b, width, L]
        gw["out_proj"] = torch.einsum("bwl,bdl->wd", do.float(), g.float())
        dg = torch.matmul(self._mm("out_proj").t(), do).contiguous()
        gate = lr.gatenorm_bwd(y, z, w["gate_norm"], dg)
        gw["gate_norm"] = gate["dweight"]
        s = lr.sscan_bwd(u, delta, w["A"], B, C, w["D"], None, gate["dy"])
        gw["A"], gw["D"] = s["dA"], s["dD"]
        draw = s["ddelta"].float() * torch.sigmoid(raw)
        gw["dt_bias"] = draw.sum((0, 2))
        gw["dt_proj"] = torch.einsum("bdl,brl->dr", draw, low.float())
        dlow = torch.matmul(w["dt_proj"].t(), draw)
        dproj = torch.cat([dlow, s["dB"], s["dC"]], 1)
        gw["x_proj"] = torch.einsum("bpl,bdl->pd", dproj, u.float())
        du = (s["du"].float() + torch.matmul(w["x_proj"].t(), dproj)).to(self.dtype)
        c = lr.sconv_bwd(xc, w["conv"], w["conv_bias"], None, du)
        gw["conv"], gw["conv_bias"] = c["dweight"], c["dbias"]
        dxz = torch.cat([c["dx"], gate["dz"]], 1)
        hv = h.view(b, L, d)
        gw["in_proj"] = torch.einsum("bpl,bld->pd", dxz.float(), hv.float())
        dh = torch.matmul(self._mm("in_proj").t(), dxz).transpose(1, 2).reshape(-1, d).contiguous()
        a = lr.addnorm_bwd(res, w["norm"], dh, dresidual.reshape(-1, d).contiguous())
        gw["norm"] = a["dweight"]
        return gw, (a["dx"].view(b, L, d), a["dresidual"].view(b, L, d))

    # ---- requests over a cache -------------------------------------------------

    def cache(self, rows, device="cuda"):
        """Cache rows for `rows` requests: the convolution's last inputs and the scan's states."""
        k = self.w["conv"].shape[1] - 1
        return (torch.zeros(rows, self.inner, k, dtype=self.dtype, device=device),
                torch.zeros(rows, self.inner, self.states, device=device))

    def prompt(self, x, residual, cu_seqlens, slots, has_state, cache):
        """Packed prompts x [tokens, width]: outputs [tokens, width], the new residual, caches advanced in place."""
        w, tables = self.w, dict(cu_seqlens=cu_seqlens, slots=slots, has_state=has_state)
        h, res = lr.addnorm_fwd(x, residual, w["norm"])
        xz = torch.matmul(self._mm("in_proj"), h.t())
        xc, z = xz[:self.inner], xz[self.inner:]
        u = lr.sconv_prompt(xc, w["conv"], w["conv_bias"], state=cache[0], **tables)
        low, B, C = self._split(torch.matmul(self._mm("x_proj"), u))
        raw = torch.matmul(self._mm("dt_proj"), low)
        y = lr.sscan_prompt(u, raw, w["A"], B, C, w["D"], state=cache[1], delta_bias=w["dt_bias"], delta_softplus=True, **tables)
        g = lr.gatenorm_fwd(y[None], z[None], w["gate_norm"])[0]
        return torch.matmul(self._mm("out_proj"), g).t().contiguous(), res

    def step(self, x, residual, slots, cache):
        """One token of every request, x [requests, width]."""
        w = self.w
        h, res = lr.addnorm_fwd(x, residual, w["norm"])
        xz = torch.matmul(h, self._mm("in_proj").t())
        xc, z = xz[:, :self.inner], xz[:, self.inner:]
        u = lr.sconv_step(xc, w["conv"], w["conv_bias"], state=cache[0], slots=slots)
        low, B, C = (t.contiguous() for t in torch.matmul(u, self._mm("x_proj").t()).split([self.rank, self.states, self.states], 1))
        raw = torch.matmul(low, self._mm("dt_proj").t())
        y = lr.sscan_step(u, raw, w["A"], B, C, w["D"], state=cache[1], slots=slots, delta_bias=w["dt_bias"],
                          delta_softplus=True)
        g = lr.gatenorm_step(y, z, w["gate_norm"])
        return torch.matmul(g, self._mm("out_proj").t()), res


def train(layer, steps=30, batch=2, length=96, rate=0.02, seed=1):
    """Adam-free gradient descent (momentum) on a random target; returns the losses."""
    width = layer.w["norm"].shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(batch, length, width, generator=g, device="cuda").to(layer.dtype)
    residual = torch.randn(batch, length, width, generator=g, device="cuda")
    target = torch.randn(batch, length, width, generator=g, device="cuda") * 0.1
    losses, speed = [], {k: torch.zeros_like(v) for k, v in layer.w.items()}
    for _ in range(steps):
        out, _, saved = layer.forward(x, residual)
        err = out.float() - target
        losses.append(float((err * err).mean()))
        dout = (2 * err / batch / length).to(layer.dtype)
        grads, _ = layer.backward(saved, dout, torch.zeros_like(residual))
        for k, v in grads.items():
            speed[k].mul_(0.9).add_(v)
            if k != "A":
                layer.w[k].sub_(rate * speed[k])
    return losses


def serve(layer, lengths=(33, 0, 7, 120), decode=5, seed=2):
    """Prompts of `lengths` tokens, packed, then `decode` single tokens each; returns the
    largest difference from the whole sequences in one call, over the outputs' size."""
    width = layer.w["norm"].shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = len(lengths)
    xs = [torch.randn(n + decode, width, generator=g, device="cuda").to(layer.dtype) for n in lengths]
    table = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    slots, cache = table(list(range(rows + 1, 1, -1))), layer.cache(rows + 2)
    packed = torch.cat([x[:n] for x, n in zip(xs, lengths)])
    out, _ = layer.prompt(packed, torch.zeros_like(packed, dtype=torch.float32), table(cu), slots,
                          table([False] * rows, torch.bool), cache)
    got = [[out[cu[i]:cu[i + 1]]] for i in range(rows)]
    for t in range(decode):
        x = torch.stack([x[n + t] for x, n in zip(xs, lengths)])
        y, _ = layer.step(x, torch.zeros_like(x, dtype=torch.float32), slots, cache)
        for i in range(rows):
            got[i].append(y[i:i + 1])
    worst = 0.0
    for i, x in enumerate(xs):
        want, _, _ = layer.forward(x[None], torch.zeros_like(x[None], dtype=torch.float32))
        diff = (torch.cat(got[i]).float() - want[0].float()).abs().max()
        worst = max(worst, float(diff / want.float().abs().max()))
    if lr.get_last_error() != lr.SSCAN_OK:
        raise RuntimeError("a request table was out of range")
    return worst


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="bf16")
    a = ap.parse_args()
    layer = Layer(dtype={"f32": torch.float32, "bf16": torch.bfloat16}[a.dtype])
    losses = train(layer)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    print(f"serving: packed prompts and decoded tokens within {serve(layer):.2e} of whole sequences")


if __name__ == "__main__":
    main()

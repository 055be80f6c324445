"""A gated feed-forward layer with int8 weights and activations, and the tuning of its channel scales.

    h -> quantise by token -> act(h Wg^T) * (h Wu^T) -> quantise by token -> . Wd^T -> out

The weights are rounded once to int8 with one scale a channel; every product then runs on int8 data.  Tuning keeps the
int8 weights and moves the gate's and the other projection's scales along their gradients, so that the gated values come
closer to those of the float32 layer.

    python examples/int8_feed_forward.py [--hidden 4096] [--inner 11008] [--tokens 512] [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_dequant_dot_amd as loom  # noqa: E402


class Int8FeedForward:
    """The layer: packed int8 weights [channels][k / 4] and float32 scales [channels] for the three projections."""

    def __init__(self, gate, up, down, act="silu"):
        # the row quantiser serves weights too: one scale a row
        (self.gate, self.gate_scale), (self.up, self.up_scale), (self.down, self.down_scale) = (
            loom.quantize_rows(w) for w in (gate, up, down))
        self.act = act

    def gated(self, h, dtype=torch.bfloat16):
        q, scale = loom.quantize_rows(h)
        return q, scale, loom.i8_gated_projection(self.gate, self.gate_scale, self.up, self.up_scale, q, scale,
                                                  act=self.act, dtype=dtype)

    def __call__(self, h):
        _, _, y = self.gated(h, h.dtype)
        q, scale = loom.quantize_rows(y)
        return loom.i8_matmul(self.down, self.down_scale, q, scale, dtype=h.dtype)

    def tune(self, h, target, rate):
        """One step on the scales towards target = the gated values wanted; returns the mean squared error before it."""
        q, scale, y = self.gated(h, torch.float32)
        d = y - target
        _, d_gate, d_up = loom.i8_gated_projection_backward(self.gate, self.gate_scale, self.up, self.up_scale, q,
                                                            scale, d, act=self.act, want_d_x=False)
        # steps relative to each scale, of the size `rate` for the channel with the steepest slope
        for s, g in ((self.gate_scale, d_gate), (self.up_scale, d_up)):
            slope = g * s
            s.mul_(1 - rate * slope / slope.abs().max().clamp_min(1e-30))
        return d.square().mean()


def main(hidden=4096, inner=11008, tokens=512, steps=8, seed=0):
    """Builds the layer, compares it with float32, tunes it -> (relative error of the layer, errors of the steps)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    gate, up = (torch.randn(inner, hidden, generator=g, device="cuda") / hidden ** 0.5 for _ in range(2))
    down = torch.randn(hidden, inner, generator=g, device="cuda") / inner ** 0.5
    h = torch.randn(tokens, hidden, generator=g, device="cuda")
    layer = Int8FeedForward(gate, up, down)
    gated = torch.nn.functional.silu(h @ gate.t()) * (h @ up.t())
    wanted = gated @ down.t()
    got = layer(h)
    error = ((got - wanted).norm() / wanted.norm()).item()
    # scales that are off by a few percent, as after rounding to fewer bits, and their way back
    layer.gate_scale *= 1 + 0.05 * torch.randn(inner, generator=g, device="cuda")
    layer.up_scale *= 1 + 0.05 * torch.randn(inner, generator=g, device="cuda")
    losses = [layer.tune(h, gated, 0.02) for _ in range(steps)]
    return error, [x.item() for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("hidden", 4096), ("inner", 11008), ("tokens", 512), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    error, losses = main(a.hidden, a.inner, a.tokens, a.steps)
    print(f"layer against float32: relative error {error:.4f}")
    print("mean squared error of the gated values over the steps:", " ".join(f"{x:.3e}" for x in losses))

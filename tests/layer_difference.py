"""A difference of the diagonal recurrence's loss along a direction of one input, with what fp32
arithmetic and the curvature of the loss may put between it and the gradient."""
from __future__ import annotations

import torch

import layer_oracle as lo

INPUTS = {"v": "dv", "beta": "dbeta", "decay": "ddecay", "state": "dstate_in"}
# The largest change of a value: the loss is a line in v, beta and the state, not in the decay.
STEP = {"v": 1.0, "beta": 2.0 ** -4, "decay": 2.0 ** -7, "state": 1.0}


def inputs(seed, gate):
    x = lo.glr_inputs(seed, 2, 150, 2, 32, gate, "fp32")
    x["decay"] = x["decay"].clamp(0.05, 0.95)
    return x


def loss(x, out, state):
    return ((out.double() * x["dout"].double()).sum() + (state.double() * x["dstate"].double()).sum()).item()


def definition(x, reverse):
    """(loss, how far an fp32 forward pass may be off)"""
    o, ob, s, sb = lo.glr(x["v"], x["beta"], x["decay"], x["state"], reverse)
    u = lo.U  # out and state are rounded once more
    off = ((ob + u * (o.abs() + ob)) * x["dout"].double().abs()).sum() + ((sb + u * (s.abs() + sb)) * x["dstate"].double().abs()).sum()
    return loss(x, o, s), off.item()


def along_gradient(x, name, reverse):
    """Inputs to both sides of x[name] along its own gradient, where the loss changes most: (x+, x-, the
    step between as it is in fp32, the difference of the losses, the bound of |<gradient, step> - difference|
    in fp32, and of the difference alone)."""
    ref = lo.glr_grad(x["v"], x["beta"], x["decay"], x["dout"], x["state"], x["dstate"], reverse)
    grad, bound = ref[INPUTS[name]]
    way = (grad / grad.abs().max() * STEP[name]).float()
    hi, lo_ = {**x, name: x[name] + way}, {**x, name: x[name] - way}
    step = hi[name].double() - lo_[name].double()
    (l1, e1), (l0, e0) = definition(hi, reverse), definition(lo_, reverse)
    bends = abs((grad * step).sum().item() - (l1 - l0))  # by the definition itself: the loss is no line
    rounds = ((bound + lo.U * (grad.abs() + bound)) * step.abs()).sum().item()
    return hi, lo_, step, l1 - l0, bends + rounds + e1 + e0, e1 + e0

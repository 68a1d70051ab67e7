"""fp64 restatement of the layers around the weight matrices, and their gradients.

Written from the formulas alone; shares no code with the CUDA path:

  layer norm   mean, var over the width;  h = (x - mean) / sqrt(var + eps);  y = h gain + bias
  linear       z = x W^T + b;  y = act(z) + residual
  gradients    by the chain rule, each as one expression in fp64
"""
from __future__ import annotations

import numpy as np
from scipy.special import expit, ndtr

ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")


def act(z, name):
    z = np.asarray(z, np.float64)
    if name == "none":
        return z
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "relu2":
        return np.where(z < 0, 0.0, z) ** 2
    if name == "gelu":
        return z * ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * expit(z)
    raise ValueError(name)


def act_slope(z, name):
    z = np.asarray(z, np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "relu2":
        return 2 * np.where(z < 0, 0.0, z)
    if name == "gelu":
        return ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        c = np.sqrt(2 / np.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = expit(z)
        return s + z * s * (1 - s)
    raise ValueError(name)


def layer_norm(x, gain=None, bias=None, eps=1e-5):
    """(y, mean, rstd)"""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if gain is not None:
        y = y * np.asarray(gain, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, gain=None, skip=None):
    """(dx, dgain, dbias) for the statistics given."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    h = (x - mean) * rstd
    q = dy if gain is None else dy * np.asarray(gain, np.float64)
    dx = rstd * (q - q.mean(axis=1, keepdims=True) - h * (q * h).mean(axis=1, keepdims=True))
    if skip is not None:
        dx = dx + np.asarray(skip, np.float64)
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


def linear(x, w, bias=None, act_name="none", residual=None):
    """(y, z)"""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = act(z, act_name)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, z


def linear_backward(dy, x, w, in_act="none", in_preact=None, skip=None):
    """(dx, dw, db)"""
    dy = np.asarray(dy, np.float64)
    dx = dy @ np.asarray(w, np.float64)
    if in_act != "none":
        dx = dx * act_slope(in_preact, in_act)
    if skip is not None:
        dx = dx + np.asarray(skip, np.float64)
    return dx, dy.T @ np.asarray(x, np.float64), dy.sum(axis=0)

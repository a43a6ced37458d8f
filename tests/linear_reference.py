"""Plain 64-bit forms of the product's epilogue and its gradient, on the CPU (not
collected by pytest), from the definitions in include/zeroshard.h; nothing here
calls the library."""
import math

import torch

F64 = torch.float64
C = 2 * math.sqrt(2 / math.pi)


def logistic_argument(x, act):
    """w of act(x) = x / (1 + exp(-w)), and its slope."""
    if act == "gelu":
        return C * (x + 0.044715 * x ** 3), C * (1 + 3 * 0.044715 * x * x)
    return x, torch.ones_like(x)


def activate(x, act):
    if act == "relu":
        return torch.clamp(x, min=0)
    if act in ("gelu", "silu"):
        return x * torch.sigmoid(logistic_argument(x, act)[0])
    return x


def slope(x, act):
    """(act'(x), a bound that a relative error of its parts scales with)."""
    if act == "relu":
        s = (x > 0).to(F64)
        return s, s
    if act in ("gelu", "silu"):
        w, dw = logistic_argument(x, act)
        p, q = torch.sigmoid(w), torch.sigmoid(-w)
        return p + x * p * q * dw, p * (1 + (x * q * dw).abs())
    return torch.ones_like(x), torch.ones_like(x)

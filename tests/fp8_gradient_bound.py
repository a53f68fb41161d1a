"""How far an 8-bit layer's products may be from those of the unrounded operands, as a share of the norm.

e4m3 keeps four bits: an element's rounding is at most 2^-4 of it, spread evenly, so 2^-4 / sqrt(3) of it in the mean of
squares at most; a product of two rounded factors, sqrt(2) of that.  The roundings are independent, so a sum's error has
the root of the sum of squares of its terms' errors, and for factors of mean zero the sum itself has that of its terms:
over a matrix the ratio of the norms is at most sqrt(2 / 3) 2^-4 = 0.051.  Twice 2^-9 for the result's bf16 and the
elements far below their block's largest."""
import torch

ROUNDING = (2 / 3) ** 0.5 * 2.0 ** -4 + 2 * 2.0 ** -9


def layer64(x, w, dy):
    """(y, dx, dw) in 64 bits."""
    x, w, dy = x.double(), w.double(), dy.double()
    return x @ w, dy @ w.T, x.T @ dy


def near(got: torch.Tensor, ref: torch.Tensor) -> bool:
    return got.shape == ref.shape and bool((got - ref).norm() <= ROUNDING * ref.norm())

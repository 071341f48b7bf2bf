"""How far a sliding-window output may be off in the norm, per kernel.

The elementwise bound of window_ref holds for any order of rounding and grows
with the number of positions; over long windows a kernel could lose a thousand
times its usual error within it.  In the norm, errors of random sign add as
their squares, and what each kernel keeps can be told apart.  With n positions,
relative to the output's norm:

  scores    one sum over the head dim, by matrix instructions of 16 dims that
            truncate: between 0 and 1 unit in the last place (2^-23.5 of the sum
            on average) lost each time, half of it on average, from a sum that
            has 2/3 of its final size on average: 2^-24.5 2/3 = 2.8e-8 per
            instruction; 32 of them at head dim 512 are 9e-7, 4 (the cluster
            kernel's chains) 1.1e-7
  weights   exp2 2^-22 and its argument's rounding, together below 4e-7
  P         two bf16 parts, each rounded to nearest: at most 2^-18 of a weight,
            2^-18 / sqrt(3) = 2.2e-6 in the mean square; fp32 or three parts:
            2^-24 and less
  O         on the tensor cores 8 truncating additions a tile of 128 positions,
            2.8e-8 each as above: 1.8e-6 for the 8 tiles between two folds

  cluster kernel                        sqrt(1.1^2 + 4^2) e-7 = 4.2e-7 < 2^-20
  tensor cores, folded (any length)     sqrt(0.9^2 + 0.4^2 + 2.2^2 + 1.8^2) e-6 = 3.0e-6 < 2^-18
  tensor cores, prompt rows over windows that do not fold: the library's 2^-17

(P in one bf16 part is off by 2^-9 / sqrt(3) = 1.1e-3, in two truncated parts
by 2^-16 on average; an O that is never folded by 2^-17 and more from 50 tiles
on.)"""
import torch

CLUSTER = 2.0 ** -20
FOLDED = 2.0 ** -18
UNFOLDED = 2.0 ** -17


def off(out, ref):
    """|out - ref| / |ref|, per stream and KV head alike: of the whole tensor."""
    out, ref = out.double(), ref.double()
    return float(torch.linalg.vector_norm(out - ref) / torch.linalg.vector_norm(ref))

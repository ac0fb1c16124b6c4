"""How exact the fp32 states of the bf16 linear-attention calls are, as a norm.

A state is X = sum_s w_s b_s c_s^T with b, c of independent zero-mean values, so an error of its terms enters its norm
like the terms themselves: relative errors of at most d per term give a relative L2 error of at most d. With
e = 2^-24, per term: w_s c_s rounded once (e), split into three bf16 parts, each of which leaves at most 2^-8 of what
is left (2^-24 = e), and w_s = exp2 within 4 e of an argument that is off by 2 e of itself (x 2^-x < 0.54: 2 e at
most): 8 e. A token that lies c chunks of 32 back passes c carries, each an exp2 and a product (5 e), which its
weight outruns where the head forgets. Every addition is off by at most e of a partial sum, whose norm is at most the
state's; they are independent: e times the root of their number, three (parts) for each token that still counts,
which is 1 / (1 - lam^2) tokens for a decay lam, and 16 for what is not a token's.

Two parts instead of three leave 2^-16 at most and, over many values, 2.0e-6 to 2.6e-6 as a root mean square: above
the bound (test_mixer_states.py). A run of tokens that a first pass sums on its own is one more carry, that far back.
"""

import math

E32 = 2.0 ** -24


def state_bound(n, g):
    """Relative L2 error that a state of n tokens at log decay g < 0 may have."""
    counting = min(n, 1.0 / (1.0 - math.exp(2 * g)))
    carries = 0 if n <= 32 else max(1.0, counting / 32)
    return E32 * (8 + 5 * carries + math.sqrt(3 * counting + 16))

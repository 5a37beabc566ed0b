"""The division by the repetition in adjust_logits, for every size of either
number: within the last bit of the exact quotient, which rounded to 53 bits and
then to 24 is next to or equal to the one rounded once.  Quotients come from the
reciprocal, q = v y with up to 1.5 u (u = 2^-23) of its size off, and a remainder
that corrects it to 2^-150 / v: half of u at v = 2^-125 (with the last rounding's
half: one number off), and below that up to 2^-22.5, as a v whose remainder is
not rounded to 0 is above 2^-127.6: 2.8 of the least u, and half: three numbers
off.  Repetitions past 2^+-100 are scaled by a power of two, the quotient back:
exact, or a second rounding of a subnormal one, whose two halves make one number
at most."""
import numpy as np
import pytest
import torch

from tests.test_adjust_logits import DEV


def ordered(x):
    """fp32 numbers as whole numbers in their order."""
    i = x.view(np.int32).astype(np.int64)
    return np.where(i < 0, -(i & 0x7fffffff), i)


@pytest.mark.gpu
def test_quotients_of_every_size():
    from weight_streaming_expert_gb300 import adjust_logits
    rng = np.random.default_rng(5)
    V = 20000
    sizes = rng.uniform(-149, 128, V - 3000)
    logits = np.concatenate([np.exp2(sizes), np.exp2(rng.uniform(-8, 5, 2990)), [0.0, 2.0 ** -149, 2.0 ** -126, 3.4e38, np.inf,
                             2.0 ** -80, 2.0 ** 100, 1.0, 1e-30, 1e30]]).astype(np.float32)
    reps = np.array([2.0 ** -149, 3e-40, 2.0 ** -130, 2.0 ** -128 * 1.7, 2.0 ** -126, 1.3e-20, 2.0 ** -20, 2.0 ** -20 * 1.01, 0.1,
                     0.7, 1.0, 1.05, 1.1, 1.3, 2.0, 3.0, 1e3, 2.0 ** 20, 1.2e6, 1e18, 2.0 ** 126 * 1.9, 2.0 ** 127 * 1.3, 3.4e38],
                    dtype=np.float32)
    M = len(reps)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    got = adjust_logits(torch.from_numpy(logits).to(DEV).expand(M, -1), history=i32(list(range(V))),
                        spans=i32([[0, V, V]] * M), repetition=torch.from_numpy(reps).to(DEV)).cpu().numpy()
    for m in range(M):
        with np.errstate(over="ignore"):
            want = (logits.astype(np.float64) / np.float64(reps[m])).astype(np.float32)
        want[logits == 0] = 0  # of 0 the product with the repetition
        off = np.abs(ordered(got[m]) - ordered(want))
        off = np.where(logits < 2.0 ** -125, off - 2, off)
        assert off.max() <= 1, (reps[m], logits[off.argmax()], got[m][off.argmax()], want[off.argmax()])

"""Times of calls in GPU tests."""

import torch


def least_us(f, calls=4, times=5):
    """Least time of a call among others, in us."""
    for _ in range(3):
        f()
    best = float("inf")
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(calls):
            f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / calls * 1e3)
    return best

"""Shared by the tests of cross attention, the 8-bit cache and group norm:
seeded inputs, widening, and the error bounds."""
import numpy as np

# A rounding to a format is off by at most half a step, relative to the value.
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
# ... and by half of the smallest subnormal in absolute terms.
HALF_SUB = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def randn(seed, *shape, dtype="bf16", sd=1.0, device="cuda"):
    """Seeded N(0, sd^2) of a dtype, drawn on the host."""
    import torch
    x = np.random.default_rng(seed).standard_normal(shape) * sd
    return torch.from_numpy(x).to(torch_dtype(dtype)).to(device)


def f64(t):
    import torch
    return t.detach().to("cpu").to(torch.float64).numpy()


def bits(t):
    import torch
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def attention_bound(ref, mag, dtype, n_keys, vmax, kv8=False):
    """|o - ref| for one element. Each probability is rounded once (half a
    step, relative), so the weighted sum is off by at most that share of mag =
    sum p |v|; float32 scores (|s| up to some tens, d = 128 products added),
    ex2.approx (2^-22) and float32 sums add less than 2^-12 of mag; the output
    is rounded once. In fp16 a probability is kept at least 2^7 above its
    share of the row's largest, so its subnormal rounding is at most 2^-25 /
    2^7 of it for each key. Over the 8-bit cache P is fp16 whatever the output,
    times the value scale: the rounding is 2^-32 of the largest scale, and a
    code is at most 448 of which the block's largest value has 224 or more."""
    h = HALF_STEP[dtype]
    sub = n_keys * vmax * 2.0 ** -32 * (2.0 if kv8 else 1.0) if dtype == "fp16" or kv8 else 0.0
    return (h + 2.0 ** -12) * mag + h * np.abs(ref) + HALF_SUB[dtype] + sub


def check_attention(got, ref, mag, dtype, n_keys, vmax, what="", kv8=False):
    assert np.isfinite(got).all(), what
    bound = attention_bound(ref, mag, dtype, n_keys, vmax, kv8)
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), (what, float(np.abs(got - ref).max()), float((np.abs(got - ref) / bound).max()))

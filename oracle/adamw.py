"""AdamW on one tensor from its definition in 64 bits (numpy), and the rounding of its 8-bit states."""
import numpy as np

BLOCK, CODE_MAX, SCALE_MIN = 128, 448.0, 2.0 ** -100


def step(p, g, m, v, t, lr, betas, eps, decay, grad_scale=1.0):
    """(p, m, v) after step t."""
    b1, b2 = betas
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - lr * decay) - lr / (1 - b1 ** t) * m / (np.sqrt(v) / np.sqrt(1 - b2 ** t) + eps)
    return p, m, v


def mix(x):
    """On uint32 arrays or ints."""
    x = np.asarray(x, dtype=np.uint32)
    with np.errstate(over="ignore"):
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x85A308D3)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0xB7E15163)
        return x ^ (x >> np.uint32(16))


def noise(seed, t, tensor, index):
    """(for m, for v, for p), 16 bits each, of the elements `index` (uint64)."""
    low = lambda x: np.uint32(int(x) & 0xFFFFFFFF)  # noqa: E731
    key = mix(low(int(mix(low(int(mix(low(seed))) + t))) + tensor))
    i = np.asarray(index, dtype=np.uint64)
    with np.errstate(over="ignore"):
        r = mix((i & np.uint64(0xFFFFFFFF)).astype(np.uint32) * np.uint32(0x9E3779B9) + (i >> np.uint64(32)).astype(np.uint32) * np.uint32(0x2E1B2139) + key)
        return r >> np.uint32(16), r & np.uint32(0xFFFF), (r * np.uint32(0x2E1B2139)) >> np.uint32(16)


def spacing(x, significant, least):
    """Between neighbours around x of a type of so many significant bits whose smallest normal value is `least`."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), least))) - (significant - 1))


def stochastic(x, bits, significant, least):
    """x rounded away from zero with the probability of what lies below, by 16 random bits."""
    step = spacing(x, significant, least)
    size = np.abs(x) / step
    return np.copysign(np.floor(size + bits / 65536.0) * step, x)


def scales(x):
    """One per block."""
    x = np.concatenate([np.abs(x), np.zeros(-len(x) % BLOCK)]).reshape(-1, BLOCK)
    return np.maximum(x.max(axis=1) / CODE_MAX, SCALE_MIN)


def spread(s, n):
    return np.repeat(s, BLOCK)[:n]

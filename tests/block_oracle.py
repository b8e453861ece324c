"""Plain definitions in 64 bits of the operators that tokens pass through in a block: the oracle of their tests."""
import numpy as np
import torch

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Philox4x32 with 10 rounds (Salmon et al. 2011): four words from four and two, whole numbers of Python."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = M0 * c[0], M1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xffffffff, (a >> 32) ^ c[3] ^ k[1], a & 0xffffffff]
        k = [(k[0] + W0) & 0xffffffff, (k[1] + W1) & 0xffffffff]
    return c


def keep(count, p, seed, offset=0):
    """Whether elements offset, offset + 1, ... are kept."""
    seed &= (1 << 64) - 1
    threshold, bits = round(p * 65536), []
    for block in range(offset // 8, -(-(offset + count) // 8)):
        for word in philox([block & 0xffffffff, block >> 32, 0, 0], [seed & 0xffffffff, seed >> 32]):
            bits += [word & 0xffff, word >> 16]
    return torch.tensor(bits[offset % 8:offset % 8 + count], dtype=torch.int64) >= threshold


def scale_of(p):
    t = round(p * 65536)
    return 65536 / (65536 - t) if t < 65536 else 0.0


def sort(ids, experts, align, rows):
    """place, source, offsets as numpy arrays, pair by pair."""
    flat = np.asarray(ids).reshape(-1)
    place, source = np.full(flat.shape, -1, np.int32), np.full(rows, -1, np.int32)
    counts = np.bincount(flat[(flat >= 0) & (flat < experts)], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)]).astype(np.int32)
    following = offsets[:-1].copy()
    for p, e in enumerate(flat):
        if 0 <= e < experts:
            place[p], source[following[e]] = following[e], p
            following[e] += 1
    return place.reshape(np.shape(ids)), source, offsets


def rotary(x, positions, freqs, sections, pairing, inverse=False):
    """x [tokens, heads, dim], positions [axes, tokens]; the result, and the sum of its terms' magnitudes."""
    x, pairs = x.double(), sum(sections)
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(x.device)
    a = (positions.double()[axis] * freqs[:, None]).T[:, None]
    c, s = a.cos(), -a.sin() if inverse else a.sin()
    at = torch.arange(pairs, device=x.device)
    first, second = (at, pairs + at) if pairing == "halves" else (2 * at, 2 * at + 1)
    u, v = x[..., first], x[..., second]
    out, size = x.clone(), x.abs()
    out[..., first], out[..., second] = u * c - v * s, v * c + u * s
    size[..., first], size[..., second] = (u * c).abs() + (v * s).abs(), (v * c).abs() + (u * s).abs()
    return out, size

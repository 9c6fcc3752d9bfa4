"""Plain forms in 64 bits of the operators around a serving step, and batches to run them on."""
import math

import torch

BS = 16
BF16, E4M3, E5M2 = 0, 1, 2
PER_TENSOR, PER_HEAD, PER_TOKEN_HEAD = 0, 1, 2
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
TOP = {E4M3: 448.0, E5M2: 57344.0}
# half a step of the formats relative to the value, and of their least step
HALF = {E4M3: 2.0 ** -4, E5M2: 2.0 ** -3, BF16: 2.0 ** -8}
LEAST = {E4M3: 2.0 ** -10, E5M2: 2.0 ** -17, BF16: 2.0 ** -134}


def decode(codes, fmt):
    return codes.double() if fmt == BF16 else codes.view(F8[fmt]).to(torch.float32).double()


def encode(x, fmt):
    """Binary32 values to codes, saturating."""
    return x.clamp(-TOP[fmt], TOP[fmt]).to(F8[fmt]).view(torch.uint8)


# ------------------------------------------------------------------ norm and rotation

def rotated(x, weight, eps, pos, inv_freq, axis, interleaved):
    """(z, size): the rows of x [N][H][dh] normed and rotated, and |y_a| + |y_b| of each dim's pair.
    pos [A][N], inv_freq [pairs] in radians, axis [pairs] or None."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
    n = len(inv_freq)
    z, size = y.clone(), y.abs()
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    p = pos.double()[axis.long() if axis is not None else torch.zeros_like(i)]  # [pairs][N]
    t = (p * inv_freq.to(p)[:, None]).T[:, None]
    z[..., a] = y[..., a] * torch.cos(t) - y[..., b] * torch.sin(t)
    z[..., b] = y[..., a] * torch.sin(t) + y[..., b] * torch.cos(t)
    size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return z, size


# ------------------------------------------------------------------ pages

class Pool:
    """The pool's rules, in Python: the lowest free pages first, all or nothing."""

    def __init__(self, n):
        self.n, self.refs = n, [0] * n

    def free(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def alloc(self, tables, old, new):
        want = [max(0, -(-z // BS) - -(-a // BS)) for a, z in zip(old, new)]
        ids = self.free()
        if sum(want) > len(ids):
            return False
        at = 0
        for row, a, w in zip(tables, old, want):
            for i in range(w):
                row[-(-a // BS) + i] = ids[at]
                self.refs[ids[at]] = 1
                at += 1
        return True

    def give(self, tables, old, new):
        for row, a, z in zip(tables, old, new):
            for i in range(-(-z // BS), -(-a // BS)):
                self.refs[row[i]] -= 1
                row[i] = -1

    def fork(self, tables, lens, parents, mb):
        ids, at = self.free(), 0
        out, out_lens, copies = [], [], []
        if sum(1 for s in parents if s >= 0 and lens[s] % BS) > len(ids):
            return None
        for s in parents:
            row, n, c = [-1] * mb, 0, [-1, -1]
            if s >= 0:
                n = lens[s]
                for i in range(n // BS):
                    row[i] = tables[s][i]
                    self.refs[row[i]] += 1
                if n % BS:
                    c = [tables[s][n // BS], ids[at]]
                    row[n // BS] = ids[at]
                    at += 1
            out.append(row)
            out_lens.append(n)
            copies.append(c)
        for c in copies:
            if c[1] >= 0:
                self.refs[c[1]] = 1
        return out, out_lens, copies

    def words(self):
        bits = [0] * ((self.n + 31) // 32)
        for i in self.free():
            bits[i // 32] |= 1 << i % 32
        return [0, len(self.free()), 0, 0] + self.refs + [x - (1 << 32) if x >> 31 else x for x in bits]

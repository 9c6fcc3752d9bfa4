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


# ------------------------------------------------------------------ trees

def way_up(parents, j):
    """Node j, its parent, and so on."""
    out = [j]
    while parents[out[-1]] >= 0:
        out.append(parents[out[-1]])
    return out


def random_parents(n, g, kind="tree"):
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [-1] * n
    return [-1] * min(n, 1) + [int(torch.randint(-1 if j % 7 == 0 else max(0, j - 12), j, (1,), generator=g)) for j in range(1, n)]


class TreeBatch:
    """Sequences of (tokens in all, of them nodes) over a shuffled pool whose spare rows and pages hold `junk`."""

    def __init__(self, seqs, hq, hkv, dh, fmt=E4M3, gran=PER_HEAD, window=0, kind="tree", seed=0, dev="cuda", amp=1.0, junk=0x7F,
                 spare=3, qf8=False):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.hq, self.hkv, self.dh, self.fmt, self.gran, self.window = seqs, hq, hkv, dh, fmt, gran, window
        B = len(seqs)
        self.lens, self.nodes = [s[0] for s in seqs], [s[1] for s in seqs]
        pages = [(n + BS - 1) // BS for n in self.lens]
        mb = max(pages + [1]) + 1
        self.nb = sum(pages) + spare
        ids = torch.randperm(self.nb, generator=g).tolist()
        bt = torch.full((B, mb), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            bt[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
            at += n
        self.parents = [random_parents(n, g, kind) for n in self.nodes]
        N = sum(self.nodes)
        self.cu = torch.tensor([0] + torch.tensor(self.nodes).cumsum(0).tolist(), dtype=torch.int32)
        self.q = (torch.randn(N, hq, dh, generator=g) * amp).to(torch.bfloat16).to(dev)
        shape = (self.nb, hkv, BS, dh)
        vals = [torch.randn(shape, generator=g) * torch.exp(torch.rand(hkv, 1, 1, generator=g) * 2 - 1) for _ in range(2)]
        self.qs = self.ks = self.vs = None
        if fmt == BF16:
            self.kc, self.vc = (v.to(torch.bfloat16).to(dev) for v in vals)
            self.K, self.V = (c.double() for c in (self.kc, self.vc))
        else:
            if gran == PER_TOKEN_HEAD:
                s = [torch.exp(torch.rand(self.nb, hkv, BS, generator=g) * 6 - 3) * (5.0 / TOP[fmt]) for _ in range(2)]
                wide = [x[..., None] for x in s]
            else:
                s = [torch.exp(torch.rand(hkv if gran == PER_HEAD else 1, generator=g)) * (5.0 / TOP[fmt]) for _ in range(2)]
                wide = [x.view(-1, 1, 1) for x in s]
            self.kc, self.vc = (encode(v / w, fmt).to(dev) for v, w in zip(vals, wide))
            self.ks, self.vs = (x.float().contiguous().to(dev) for x in s)
            self.K, self.V = (decode(c, fmt) * w.double().to(dev) for c, w in zip((self.kc, self.vc), wide))
            if qf8:
                n = hq if gran == PER_HEAD else 1
                self.qs = (torch.rand(n, generator=g) + 0.5).mul(3.0 * amp / TOP[fmt]).to(dev)
        # rows past the sequences, and pages of nobody
        t = torch.arange(mb * BS)
        used = torch.zeros(self.nb, BS, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            used[bt[b, t[:n] // BS].long(), t[:n] % BS] = True
        if junk is not None:
            un = ~used.to(dev)
            for c in (self.kc, self.vc):
                c.view(torch.uint8).permute(0, 2, 1, 3)[un] = junk
            if gran == PER_TOKEN_HEAD and fmt != BF16:
                for s in (self.ks, self.vs):
                    s.permute(0, 2, 1)[un] = math.nan
        self.bt, self.sl, self.cu_d = bt.to(dev), torch.tensor(self.lens, dtype=torch.int32, device=dev), self.cu.to(dev)
        self.par = torch.tensor([p for ps in self.parents for p in ps], dtype=torch.int32, device=dev)
        self.dev = dev

    def query(self):
        if self.qs is None:
            return self.q.double()
        s = self.qs.view(1, -1, 1)
        return decode(encode(self.q.float() / s, self.fmt), self.fmt) * s.double()

    def reference(self, bad=()):
        """(out, bound) in 64 bits: what every row is, and how far an output may be from it.  `bad`: pages masked out.

        The bound: the output's rounding, half a step of bf16; the weights' roundings (FP8: three E5M2 parts, within 2^-9 of
        the weight or 2^-24 of the row's largest; bf16: 2^-17); the logits' errors, which change each weight by their size:
        the query's two E4M3 parts, off by 2^-18 of the row's largest, and sums in binary32, 2^-19 of the sum of magnitudes;
        2^-19 for exp2, the sums of weights and the merge."""
        q = self.query()
        out, bound = torch.zeros_like(q), torch.zeros_like(q)
        G, bt = self.hq // self.hkv, self.bt.cpu()
        for b, (L, n) in enumerate(zip(self.lens, self.nodes)):
            if n == 0:
                continue
            t = torch.arange(L)
            blk = bt[b, t // BS].long()
            ok = (blk >= 0) & (blk < self.nb) & ~torch.isin(blk, torch.tensor(list(bad), dtype=torch.int64))
            K, V = (c[blk.clamp(0, self.nb - 1).to(self.dev), :, (t % BS).to(self.dev)] for c in (self.K, self.V))
            P = L - n
            see = torch.zeros(n, L, dtype=torch.bool)
            for j in range(n):
                way = way_up(self.parents[b], j)
                lo = max(0, P + len(way) - self.window) if self.window else 0
                see[j, lo:P] = True
                see[j, [P + i for i in (way[:self.window] if self.window else way)]] = True
            see = (see & ok).to(self.dev)
            a, z = int(self.cu[b]), int(self.cu[b + 1])
            for h in range(self.hkv):  # the group's rows at once
                k, v = K[:, h], V[:, h]
                qq = q[a:z, h * G:(h + 1) * G].reshape(-1, self.dh)
                seen = see.repeat_interleave(G, 0)
                x = torch.nan_to_num(qq @ k.T / math.sqrt(self.dh), nan=0.0).masked_fill(~seen, -math.inf)
                p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)  # a row that sees nothing: zeros
                v0 = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
                k0 = torch.nan_to_num(k, nan=0.0)
                o, w = p @ v0, p @ v0.abs()
                d = 2.0 ** -19 * (qq.abs() @ k0.abs().T).amax(1, keepdim=True) / math.sqrt(self.dh)
                if self.fmt == BF16:
                    e, least = 2.0 ** -17, 2.0 ** -100
                else:
                    e, least = 2.0 ** -9, 2.0 ** -24
                    if self.qs is None:
                        d = d + 2.0 ** -18 * qq.abs().amax(1, keepdim=True) * k0.abs().sum(1).max() / math.sqrt(self.dh)
                top = p.amax(1, keepdim=True)
                bd = 2.0 ** -8 * o.abs() + (e + 2 * d + 2.0 ** -19) * w + least * top * (seen.double() @ v0.abs()) + 1e-30
                out[a:z, h * G:(h + 1) * G] = o.view(n, G, self.dh)
                bound[a:z, h * G:(h + 1) * G] = bd.view(n, G, self.dh)
        return out, bound


class OnGpu:
    """A batch's call, on memory of its own whose contents say nothing."""

    def __init__(self, kvq, b):
        self.kvq, self.b = kvq, b
        self.ws = kvq.new_tree_workspace(b.hq, b.hkv, b.dh, b.dev).fill_(0xFF)
        self.out = torch.full_like(b.q, 7.0)
        self.st = torch.zeros(1, dtype=torch.int32, device=b.dev)

    def call(self, **kw):
        b = self.b
        a = dict(parents=b.par, block_tables=b.bt, seq_lens=b.sl, cu_q_lens=b.cu_d, q=b.q, out=self.out, q_scale=b.qs,
                 flags=self.kvq.KVQ_Q_FP8 if b.qs is not None else 0, dev_status=self.st, workspace=self.ws) | kw
        self.kvq.kvq_tree_attn(k_cache=b.kc, v_cache=b.vc, k_scale=b.ks, v_scale=b.vs, scale_granularity=b.gran, fmt=b.fmt,
                               sliding_window=b.window, **a)
        return self.out

    def check(self, status=0, bad=(), what=""):
        torch.cuda.synchronize()
        assert int(self.st.item()) == status, what
        ref, bound = self.b.reference(bad)
        err = (self.out.double() - ref).abs()
        worst = float((err / bound).max()) if err.numel() else 0.0
        assert bool((err <= bound).all()), f"{what}: {worst:.2f} of the bound, error {float(err.max()):.3e}"
        return worst


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

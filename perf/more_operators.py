"""The operators around a serving step over the paged caches, as measured cases.

  rope    queries and keys normed per head and rotated by their positions, K and V
          quantized into their pages, in one pass
  tree    attention of trees of drafted tokens over the cache: a node sees its
          sequence's tokens before the tree and its own ancestors
  commit  the rows of the accepted path moved together behind the tokens before the
          tree, in every layer's caches
  fork    beams: the last step's pages let go, the tables forked from their parents
          (full pages shared, the last one copied), pages taken for the next tokens

Caches hold pages of 16 tokens: [num_blocks][Hkv][16][dh] FP8 codes or bf16, or
[num_blocks][Hkv][9 dh] bytes of the 4-bit cache.  A page pool is int32 words: four of
a header (the second: how many pages are free), a count of each page's holders, then a
bit for each free page.
"""
import math

import torch

own = False

BS = 16  # tokens of a page
DEV = "cuda"
PER_TENSOR, PER_HEAD = 0, 1
FMT = {"bf16": 0, "e4m3": 1, "e5m2": 2}  # the framework's numbers of the formats
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6
HEADER = 4  # words before a pool's counts


# ---------------------------------------------------------------- the cases

def _rope(name, tokens, hq, hkv, dh, fmt="e4m3", per_head=True, axes=1, pairs=0, interleaved=False, norm=True, far=4096):
    c = dict(op="rope", tokens=tokens, hq=hq, hkv=hkv, dh=dh, fmt=fmt, per_head=per_head, axes=axes,
             pairs=pairs or dh // 2, interleaved=interleaved, norm=norm, far=far)
    return dict(c, name=name) if name else c


def _tree(name, batch, low, high, nodes, hq, hkv, dh, fmt="e4m3", per_head=True, window=0):
    c = dict(op="tree", batch=batch, low=low, high=high, nodes=nodes, hq=hq, hkv=hkv, dh=dh, fmt=fmt,
             per_head=per_head, window=window)
    return dict(c, name=name) if name else c


def _commit(name, batch, low, high, nodes, caches, hkv, dh, kind="e4m3"):
    c = dict(op="commit", batch=batch, low=low, high=high, nodes=nodes, caches=caches, hkv=hkv, dh=dh, kind=kind)
    return dict(c, name=name) if name else c


def _fork(name, beams, width, low, high, grow, caches, hkv, dh, kind="e4m3"):
    c = dict(op="fork", beams=beams, width=width, low=low, high=high, grow=grow, caches=caches, hkv=hkv, dh=dh, kind=kind)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a batch, far into its sequences; a long prompt; an image's patches
        # behind text, with positions in time, height and width, before a layer kept in bf16
        _rope("rope_step", 32, 32, 8, 128, far=131072),
        _rope("rope_long", 32768, 32, 8, 128, per_head=False, norm=False, far=0),
        _rope("rope_image", 4100, 16, 16, 64, fmt="bf16", axes=3, pairs=24, interleaved=True, far=900),
        # a few drafts of two short sequences; a batch's trees; a large tree over a long context;
        # a batch of mixed lengths with a window; a layer kept in bf16
        _tree("tree_tiny", 2, 37, 100, 5, 8, 2, 64, per_head=False),
        _tree("tree_batch", 32, 2049, 2049, 16, 32, 8, 128),
        _tree("tree_long", 1, 32768, 32768, 64, 32, 8, 128),
        _tree("tree_mixed", 128, 17, 16384, 24, 32, 8, 128, fmt="e5m2", window=4096),
        _tree("tree_bf16", 16, 700, 4096, 30, 28, 4, 128, fmt="bf16"),
        # two sequences' trees in a small model's 4-bit caches; a batch's in a large model's
        _commit("commit_small", 2, 37, 100, 7, 4, 2, 64, kind="fp4"),
        _commit("commit_batch", 32, 512, 2049, 24, 32, 8, 128),
        # two beams' widths: a single short prompt's, and those of a batch of longer ones
        _fork("fork_small", 6, 6, 37, 100, 1, 4, 2, 64, kind="fp4"),
        _fork("fork_batch", 64, 4, 512, 2049, 5, 8, 8, 128),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(("rope", "rope", "tree", "tree", "tree", "commit", "fork"))
    hq, hkv, dh = rng.choice(((32, 8, 128), (8, 2, 64), (16, 16, 64), (28, 4, 128), (64, 8, 128),
                              (40, 8, 128), (6, 2, 64), (4, 4, 128)))
    per_head = rng.random() < 0.6
    if op == "rope":
        axes = rng.choice((1, 1, 1, 2, 3))
        pairs = rng.choice((dh // 2, dh // 2, dh // 4, 8 * rng.randint(1, dh // 16)))
        return _rope("", _log(rng, 1, 16384), hq, hkv, dh, rng.choice(("e4m3", "e4m3", "e5m2", "bf16")), per_head, axes,
                     pairs, rng.random() < 0.3, rng.random() < 0.7, _log(rng, 2, 1000000))
    if op == "tree":
        nodes = _log(rng, 1, 128)
        high = max(nodes + 1, _log(rng, 8, 32768))
        batch = _log(rng, 1, max(1, min(128, 400000 // high, (1 << 21) // (high * nodes) + 1)))
        return _tree("", batch, max(nodes, high // 5), high, nodes, hq, hkv, dh, rng.choice(("e4m3", "e4m3", "e5m2", "bf16")),
                     per_head, _log(rng, 1, 4096) if rng.random() < 0.3 else 0)
    kind = rng.choice(("e4m3", "bf16", "fp4"))
    high = _log(rng, 20, 2049)
    if op == "commit":
        nodes = min(high - 1, _log(rng, 1, 64))
        return _commit("", _log(rng, 1, 32), max(nodes, high // 3), high, nodes, 2 * rng.randint(1, 12), hkv, dh, kind)
    width = rng.randint(1, 8)
    return _fork("", width * _log(rng, 1, 8), width, max(1, high // 3), high, rng.randint(1, 40), 2 * rng.randint(1, 3), hkv, dh, kind)


# ---------------------------------------------------------------- inputs

def _spread(n, low, high):
    """n lengths spread over the logarithm between low and high; the middle one is the highest."""
    return [high if b == n // 2 else round(low * (high / low) ** ((b + 1) * 0.6180339887498949 % 1.0)) for b in range(n)]


def _nodes(case):
    """Nodes of each sequence's tree: at least half of the case's."""
    return [case["nodes"] if b == 0 else max(1, round(case["nodes"] * (0.5 + 0.5 * ((b + 1) * 0.7548776662466927 % 1.0))))
            for b in range(case["batch"])]


def _tables(lens, h):
    """Block tables of sequences of these lengths in a shuffled pool without a page to spare; its pages."""
    pages = (lens + BS - 1) // BS
    total, mb = int(pages.sum()), int(pages.max())
    bt = torch.full((len(lens), mb), -1, dtype=torch.int32)
    bt[torch.arange(mb)[None, :] < pages[:, None]] = torch.randperm(total, generator=h).to(torch.int32)
    return bt, total


def _pages(kind, caches, blocks, hkv, dh, g):
    """Caches of some layers with anything in them, one after another in one tensor."""
    if kind == "bf16":
        return torch.randn(caches, blocks, hkv, BS, dh, generator=g, device=DEV, dtype=torch.bfloat16)
    tail = (9 * dh,) if kind == "fp4" else (BS, dh)
    return torch.randint(0, 127, (caches, blocks, hkv) + tail, generator=g, device=DEV, dtype=torch.uint8)


def _inv_freq(pairs):
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)


def _turns(inv_freq):
    """A frequency as the framework takes it: turns a position, times 2^64."""
    return (inv_freq / (2 * math.pi) * 2.0 ** 64).round().to(torch.int64)


def _axes(case):
    """The axis whose position turns each pair: the pairs shared out in runs, the first axis' the longest."""
    n, a = case["pairs"], case["axes"]
    return torch.tensor([min(a - 1, max(0, i - (n - n // a * (a - 1))) // max(1, n // a) + (i >= n - n // a * (a - 1)))
                         for i in range(n)], dtype=torch.uint8)


def _prepare_rope(case, g, h):
    N, hq, hkv, dh, fmt = case["tokens"], case["hq"], case["hkv"], case["dh"], case["fmt"]
    # one projection's output, whose heads q, k and v are slices of
    qkv = torch.randn(N, (hq + 2 * hkv) * dh, generator=g, device=DEV, dtype=torch.bfloat16)
    q, k, v = (t.view(N, -1, dh) for t in qkv.split((hq * dh, hkv * dh, hkv * dh), 1))
    if case["axes"] > 1:  # text, then patches row by row
        w = max(1, int(math.sqrt(N)))
        i = torch.arange(N)
        pos = torch.stack([i // max(1, N // 2), i // w, i % w])[:case["axes"]] + case["far"]
    elif case["far"]:
        pos = torch.randint(0, case["far"], (1, N), generator=h)
    else:
        pos = torch.arange(N)[None]
    blocks = (N + BS - 1) // BS + 1
    page = torch.randperm(blocks, generator=h)[torch.arange(N) // BS]
    slots = page * BS + torch.arange(N) % BS
    inv = _inv_freq(case["pairs"])
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]
    n = hkv if case["per_head"] else 1
    s = (5.0 + torch.rand(2, n, generator=g, device=DEV)) / TOP.get(fmt, 1.0)
    norm = [torch.rand(dh, generator=g, device=DEV).add_(0.5).to(torch.bfloat16) if case["norm"] else None for _ in range(2)]
    return {"q": q, "k": k, "v": v, "pos": pos.to(torch.int32).to(DEV), "inv_freq": inv.to(DEV), "turns": _turns(inv).to(DEV),
            "axis": _axes(case).to(DEV) if case["axes"] > 1 else None, "q_weight": norm[0], "k_weight": norm[1],
            "slots": slots.to(DEV), "k_scale": s[0].contiguous(), "v_scale": s[1].contiguous(),
            "kc": torch.zeros(blocks, hkv, BS, dh, device=DEV, dtype=torch.bfloat16).to(dt),
            "vc": torch.zeros(blocks, hkv, BS, dh, device=DEV, dtype=torch.bfloat16).to(dt),
            "q_out": torch.zeros(N, hq, dh, dtype=torch.bfloat16, device=DEV)}


def _parents(n, h):
    """A tree's parents, each before its node; a few nodes begin a tree of their own."""
    j = torch.arange(n)
    u = torch.rand(n, generator=h)
    p = (j * (0.3 + 0.7 * u)).floor().long().clamp(min=0)
    p = torch.where(j > 0, torch.minimum(p, j - 1), p - 1)
    return torch.where((torch.rand(n, generator=h) < 0.05) & (j > 0), torch.full_like(p, -1), p)


def _prepare_tree(case, g, h):
    hq, hkv, dh, fmt, B = case["hq"], case["hkv"], case["dh"], case["fmt"], case["batch"]
    nq = torch.tensor(_nodes(case))
    lens = torch.maximum(torch.tensor(_spread(B, case["low"], case["high"])), nq)
    bt, total = _tables(lens, h)
    amp = torch.exp(torch.rand(2, hkv, generator=g, device=DEV) * 2 - 1)
    s = amp * (5.0 / TOP.get(fmt, 5.0))
    if not case["per_head"]:
        s = s.amax(1, keepdim=True)

    def pages(a, sc):
        x = torch.randn(total, hkv, BS, dh, generator=g, device=DEV, dtype=torch.bfloat16) * a[:, None, None].to(torch.bfloat16)
        if fmt == "bf16":
            return x
        x = (x.float() / sc[:, None, None]).clamp(-TOP[fmt], TOP[fmt])
        return x.to(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).view(torch.uint8)

    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(nq, 0)])
    N = int(cu[-1])
    # one scratch buffer for every call, as a serving loop keeps it
    return {"kc": pages(amp[0], s[0]), "vc": pages(amp[1], s[1]), "k_scale": s[0].contiguous(), "v_scale": s[1].contiguous(),
            "q": torch.randn(N, hq, dh, generator=g, device=DEV, dtype=torch.bfloat16),
            "parents": torch.cat([_parents(int(n), h) for n in nq]).to(torch.int32).to(DEV), "cu": cu.to(torch.int32).to(DEV),
            "nq": nq.to(DEV), "nq_max": int(nq.max()), "bt": bt.to(DEV), "lens": lens.to(torch.int32).to(DEV),
            "out": torch.zeros(N, hq, dh, dtype=torch.bfloat16, device=DEV),
            "ws": torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)}


def _prepare_commit(case, g, h):
    B = case["batch"]
    nq = torch.tensor(_nodes(case))
    lens = torch.maximum(torch.tensor(_spread(B, case["low"], case["high"])), nq)
    bt, total = _tables(lens, h)
    # accepted paths: the first node, then some past the places that the path moves to
    most = max(1, min(8, case["nodes"] // 2))
    taken = torch.minimum((torch.rand(B, generator=h) * most).long() + 1, (nq // 2).clamp(min=1))
    key = torch.rand(B, case["nodes"], generator=h)
    j = torch.arange(case["nodes"])
    key[(j < taken[:, None]) | (j >= nq[:, None])] = 2.0
    nodes = torch.sort(torch.argsort(key, 1)[:, :most].masked_fill(j[:most] >= taken[:, None] - 1, 1 << 20), 1)[0]
    path = torch.cat([torch.zeros(B, 1, dtype=torch.int64), nodes], 1)[:, :most]
    path = torch.where(j[:most] < taken[:, None], path, torch.full_like(path, -1))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(nq, 0)])
    caches = _pages(case["kind"], case["caches"], total, case["hkv"], case["dh"], g)
    return {"caches": caches, "list": list(caches.unbind(0)), "bt": bt.to(DEV), "lens": lens.to(torch.int32).to(DEV),
            "cu": cu.to(torch.int32).to(DEV), "path": path.to(torch.int32).to(DEV), "taken": taken.to(torch.int32).to(DEV),
            "new_lens": torch.zeros(B, dtype=torch.int32, device=DEV)}


def _prepare_fork(case, g, h):
    n, w = case["beams"], case["width"]
    # the beams of a prompt share its pages, then have some of their own
    prompt = torch.tensor(_spread(n // w, case["low"], case["high"])).repeat_interleave(w)
    lens = prompt + (torch.rand(n, generator=h) * 30).long()
    pages, shared = (lens + BS - 1) // BS, prompt // BS
    mb = (case["high"] + 30 + case["grow"]) // BS + 2
    slot = torch.arange(mb)[None, :]
    first = torch.arange(n) // w * w
    used = slot < pages[:, None]
    mine = used & ((slot >= shared[:, None]) | (torch.arange(n) == first)[:, None])
    # what the prompts hold, three pages of each beam's own, and as many and the next tokens' once forked
    total = int(pages.new_tensor(_spread(n // w, case["low"], case["high"])).add_(BS).floor_divide_(BS).sum()) + n * (case["grow"] // BS + 8)
    total += -total % 32
    bt = torch.full((n, mb), -1, dtype=torch.int64)
    bt[mine] = torch.randperm(total, generator=h)[:int(mine.sum())]
    bt = torch.where(used & ~mine, bt[first], bt)
    pool = torch.zeros(HEADER + total + total // 32, dtype=torch.int64)
    pool[HEADER:HEADER + total] = torch.bincount(bt[used], minlength=total)
    pool = _with_bits(pool.to(torch.int32).to(DEV), total)
    parents = (torch.rand(n, generator=h) * w).long() + first
    caches = _pages(case["kind"], case["caches"], total, case["hkv"], case["dh"], g)
    return {"caches": caches, "list": list(caches.unbind(0)), "bt": bt.to(torch.int32).to(DEV), "lens": lens.to(torch.int32).to(DEV),
            "parents": parents.to(torch.int32).to(DEV), "pool": pool, "total": total,
            "tables": torch.full((n, mb), -1, dtype=torch.int32, device=DEV), "have": torch.zeros(n, dtype=torch.int32, device=DEV),
            "out_lens": torch.zeros(n, dtype=torch.int32, device=DEV), "none": torch.zeros(n, dtype=torch.int32, device=DEV),
            "copies": torch.full((n, 2), -1, dtype=torch.int32, device=DEV)}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    make = {"rope": _prepare_rope, "tree": _prepare_tree, "commit": _prepare_commit, "fork": _prepare_fork}[case["op"]]
    return make(case, g, h) | {"case": case, "gran": PER_HEAD if case.get("per_head") else PER_TENSOR}


# ---------------------------------------------------------------- plain forms

def _normed(x, weight):
    x = x.float()
    return x if weight is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _rotated(x, cos, sin, interleaved):
    n = cos.shape[-1]
    head, tail = x[..., :2 * n], x[..., 2 * n:]
    a, b = (head[..., ::2], head[..., 1::2]) if interleaved else (head[..., :n], head[..., n:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.cat([torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1), tail], -1)


def _angles(st):
    """cos, sin [N][1][pairs] in 64 bits: far positions take more than a binary32 angle has."""
    pos = st["pos"].double()
    at = pos[st["axis"].long()].t() if st["axis"] is not None else pos[0][:, None]
    a = at * st["inv_freq"]
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def _run_rope(st):
    case = st["case"]
    cos, sin = (t.float() for t in _angles(st))
    q = _rotated(_normed(st["q"], st["q_weight"]), cos, sin, case["interleaved"])
    k = _rotated(_normed(st["k"], st["k_weight"]), cos, sin, case["interleaved"])
    st["q_out"].copy_(q)
    page, row = st["slots"] // BS, st["slots"] % BS
    _put(st["kc"], page, row, k, st["k_scale"], case["fmt"])
    _put(st["vc"], page, row, st["v"].float(), st["v_scale"], case["fmt"])
    return {"q": st["q_out"], "k": st["kc"], "v": st["vc"]}


def _put(cache, page, row, x, scale, fmt):
    if fmt == "bf16":
        cache[page, :, row] = x.to(torch.bfloat16)
        return
    x = (x / scale[:, None]).clamp(-TOP[fmt], TOP[fmt])
    cache.view(torch.uint8)[page, :, row] = x.to(cache.dtype).view(torch.uint8)


def _gather(st, cache, scale):
    """Every sequence's tokens, padded: binary32 [B][hkv][T][dh]."""
    fmt = st["case"]["fmt"]
    if fmt != "bf16":
        cache = cache.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2)
    v = cache.float()[st["bt"].clamp(min=0).long()]  # [B][blocks][hkv][16][dh]
    B, mb, hkv, _, dh = v.shape
    v = v.transpose(1, 2).reshape(B, hkv, mb * BS, dh)
    return v if fmt == "bf16" else v * scale.view(1, -1, 1, 1)


def _ancestors(parents):
    """[B][M][M] whether node j has node i on its way up, itself included, of parents [B][M]: the
    inverse of I - (parent of), a triangle of zeros and ones, is the sum of its powers."""
    M = parents.shape[1]
    up = (parents[..., None] == torch.arange(M, device=DEV)).double()
    eye = torch.eye(M, dtype=torch.float64, device=DEV).expand_as(up)
    return torch.linalg.solve_triangular(eye - up, eye, upper=False, unitriangular=True) > 0.5


def _run_tree(st):
    case, cu = st["case"], st["cu"].long()
    lens, nq, M = st["lens"].long(), st["nq"], st["nq_max"]
    hq, hkv, dh, W = case["hq"], case["hkv"], case["dh"], case["window"]
    G, B = hq // hkv, lens.shape[0]
    K, V = _gather(st, st["kc"], st["k_scale"]), _gather(st, st["vc"], st["v_scale"])
    j = torch.arange(M, device=DEV)
    row = (cu[:-1, None] + j).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][row].float().view(B, M, hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * M, dh)
    x = torch.matmul(q, K.transpose(2, 3)).mul_(1.0 / math.sqrt(dh)).view(B, hkv, G, M, -1)
    anc = _ancestors(torch.where(j < nq[:, None], st["parents"][row], torch.full_like(row, -1)))
    depth = anc.sum(-1) - 1
    first = lens - nq  # position of the trees' first nodes
    t = torch.arange(K.shape[2], device=DEV)
    node = (t - first[:, None]).clamp(0, M - 1)[:, None, :].expand(-1, M, -1)  # the node of each token [B][M][T]
    drafted = (t >= first[:, None])[:, None]
    seen = torch.where(drafted, torch.gather(anc, 2, node), torch.ones_like(drafted)) & (t < lens[:, None])[:, None]
    if W:
        place = torch.where(drafted, first[:, None, None] + torch.gather(depth[:, None].expand(-1, M, -1), 2, node), t)
        seen = seen & (place > (first[:, None] + depth)[..., None] - W)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    den = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, G * M, -1), V).view(B, hkv, G, M, dh) / den
    st["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, M, hq, dh)[j < nq[:, None]])
    return {"out": st["out"]}


def _move(c, src, dst, kind):
    """Rows (page, row of the page) of every cache, read before any is written."""
    if kind == "fp4":  # a page's codes, then its scales
        dh = c.shape[-1] // 9
        _move(c[..., :8 * dh].view(*c.shape[:3], BS, dh // 2), src, dst, "")
        _move(c[..., 8 * dh:].view(*c.shape[:3], BS, dh // 16), src, dst, "")
    else:
        c[:, dst[0], :, dst[1]] = c[:, src[0], :, src[1]]


def _run_commit(st):
    cu, lens, path, taken = st["cu"].long(), st["lens"].long(), st["path"].long(), st["taken"].long()
    B, P = path.shape
    first = lens - (cu[1:] - cu[:-1])
    i = torch.arange(P, device=DEV)
    moved = i < taken[:, None]
    stay = (lens - 1)[:, None].expand(-1, P)  # where nothing moves: the last row, onto itself
    src = torch.where(moved, first[:, None] + path, stay)
    dst = torch.where(moved, first[:, None] + i, stay)
    b = torch.arange(B, device=DEV)[:, None]
    bt = st["bt"].long()
    at = [(bt[b, p // BS].reshape(-1), (p % BS).reshape(-1)) for p in (src, dst)]
    _move(st["caches"], at[0], at[1], st["case"]["kind"])
    st["new_lens"].copy_(first + taken)
    return {"caches": st["caches"], "lens": st["new_lens"]}


def _with_bits(pool, total):
    """The pool with its free pages counted and marked."""
    free = (pool[HEADER:HEADER + total] == 0).view(-1, 32).long()
    bits = (free << torch.arange(32, device=pool.device)).sum(1)
    pool[HEADER + total:] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    pool[1] = free.sum()
    return pool


def _held(pool, total, ids, by):
    """`by` holders more of each page of ids (-1: none)."""
    counts = torch.zeros(total + 1, dtype=torch.int32, device=DEV)
    counts.scatter_add_(0, torch.where(ids >= 0, ids, torch.full_like(ids, total)).reshape(-1).long(),
                        torch.full((ids.numel(),), by, dtype=torch.int32, device=DEV))
    pool[HEADER:HEADER + total] += counts[:total]


def _take(pool, total, wanted):
    """The lowest free pages, one for each True of `wanted` in its order, -1 elsewhere."""
    held = (pool[HEADER:HEADER + total] != 0).to(torch.int8)
    lowest = torch.sort(held, stable=True)[1].to(torch.int32)  # free pages first, ascending
    rank = torch.cumsum(wanted.reshape(-1), 0).view(wanted.shape) - 1
    return torch.where(wanted, lowest[rank.clamp(min=0, max=total - 1)], torch.full_like(rank, -1, dtype=torch.int32))


def _count(lens):
    return (lens.long() + BS - 1) // BS


def _run_fork(st):
    case, pool, total, tables = st["case"], st["pool"], st["total"], st["tables"]
    slot = torch.arange(tables.shape[1], device=DEV)
    # the last step's pages go back
    held = slot < _count(st["have"])[:, None]
    _held(pool, total, torch.where(held, tables, torch.full_like(tables, -1)), -1)
    tables.masked_fill_(held, -1)
    # each row from its parent: full pages are shared, a last one that is not full is copied
    src, lens = st["bt"][st["parents"].long()], st["lens"][st["parents"].long()]
    full = (lens // BS)[:, None]
    part = (slot == full) & (lens % BS > 0)[:, None]
    new = _take(pool, total, part)
    tables.copy_(torch.where(slot < full, src, new))
    st["copies"].copy_(torch.stack([torch.where(part, t, torch.full_like(t, -1)).amax(1) for t in (src, new)], 1))
    _held(pool, total, tables, 1)
    st["out_lens"].copy_(lens)
    pair = torch.where(st["copies"][:, :1] >= 0, st["copies"], torch.full_like(st["copies"], total - 1)).long()
    st["caches"][:, pair[:, 1]] = st["caches"][:, pair[:, 0]]
    # and pages for the next tokens
    more = lens + case["grow"]
    new = _take(pool, total, (slot >= _count(lens)[:, None]) & (slot < _count(more)[:, None]))
    tables.copy_(torch.maximum(tables, new))
    _held(pool, total, new, 1)
    _with_bits(pool, total)
    st["have"] = more
    return {"tables": tables, "lens": st["out_lens"], "copies": st["copies"], "pool": pool, "caches": st["caches"]}


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if own:
        import fp8_quantized_paged_gb300 as kvq
        if case["op"] == "rope":
            kvq.kvq_rope_write(st["q"], st["k"], st["v"], st["pos"], st["turns"], st["axis"], st["q_weight"], st["k_weight"], EPS,
                               case["interleaved"], st["slots"], st["kc"], st["vc"], st["k_scale"], st["v_scale"], st["gran"],
                               FMT[case["fmt"]], st["q_out"])
            return {"q": st["q_out"], "k": st["kc"], "v": st["vc"]}
        if case["op"] == "tree":
            kvq.kvq_tree_attn(st["q"], st["cu"], st["parents"], st["kc"], st["vc"], st["bt"], st["lens"], st["k_scale"], st["v_scale"],
                              st["gran"], FMT[case["fmt"]], case["window"], st["ws"], st["out"])
            return {"out": st["out"]}
        if case["op"] == "commit":
            kvq.kvq_tree_commit(st["list"], st["cu"], st["bt"], st["lens"], st["path"], st["taken"], st["new_lens"])
            return {"caches": st["caches"], "lens": st["new_lens"]}
        kvq.kvq_pages_free(st["pool"], st["tables"], st["have"], st["none"])
        kvq.kvq_pages_fork(st["pool"], st["bt"], st["lens"], st["parents"], st["tables"], st["out_lens"], st["copies"])
        kvq.kvq_copy_pages(st["list"], st["copies"])
        st["have"] = st["out_lens"] + case["grow"]
        kvq.kvq_pages_alloc(st["pool"], st["tables"], st["out_lens"], st["have"])
        return {"tables": st["tables"], "lens": st["out_lens"], "copies": st["copies"], "pool": st["pool"], "caches": st["caches"]}
    return {"rope": _run_rope, "tree": _run_tree, "commit": _run_commit, "fork": _run_fork}[case["op"]](st)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, hkv, dh = case["op"], case["hkv"], case["dh"]
    if op == "rope":
        N, hq, e = case["tokens"], case["hq"], 2 if case["fmt"] == "bf16" else 1
        # the rows in, q and the cache's rows out; a slot and the positions of each token
        return {"bytes": N * (dh * (4 * hq + 2 * hkv * (2 + e)) + 8 + 4 * case["axes"]), "flops": 0}
    if op == "tree":
        hq, W, e = case["hq"], case["window"], 2 if case["fmt"] == "bf16" else 1
        bytes_, pairs = 0, 0
        for n, m in zip(_spread(case["batch"], case["low"], case["high"]), _nodes(case)):
            before = max(n, m) - m
            bytes_ += 2 * ((min(before, W) if W else before) + m) * hkv * dh * e + 4 * m * hq * dh
            pairs += m * min(before + 3, W or before + 3)  # a few ancestors each
        return {"bytes": bytes_, "flops": 4 * pairs * hq * dh}
    row = {"fp4": dh * 9 // 16, "e4m3": dh, "bf16": 2 * dh}[case["kind"]] * hkv
    if op == "commit":
        most = max(1, min(8, case["nodes"] // 2))
        rows = sum(min((most + 1) / 2, max(1, m // 2)) - 1 for m in _nodes(case))
        return {"bytes": 2 * case["caches"] * rows * row + 32 * case["batch"], "flops": 0}
    lens = [n + 15 for n in _spread(case["beams"] // case["width"], case["low"], case["high"]) for _ in range(case["width"])]
    # entries and counts read and written, twice: let go and taken; a page each copied
    return {"bytes": sum(2 * 16 * (n // BS + 2) for n in lens) + 2 * case["caches"] * len(lens) * BS * row, "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits

def _step(a, lowest, bits, top):
    """a >= 0 to the nearest value of `bits` explicit significand bits (ties to even) with least exponent
    `lowest`, at most `top`."""
    e = torch.floor(torch.log2(torch.clamp(a, min=2.0 ** lowest)))
    e = torch.where(torch.exp2(e) > a, e - 1, e).clamp(min=lowest)
    u = torch.exp2(e - bits)
    return torch.clamp(torch.round(a / u) * u, max=top)


def _exact_rope(case, st):
    n, N = case["pairs"], case["tokens"]
    axis = st["axis"].long() if st["axis"] is not None else torch.zeros(n, dtype=torch.int64, device=DEV)
    turn = torch.exp(1j * st["pos"].double()[axis].T * st["inv_freq"])[:, None]  # [N][1][pairs]

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
        first = (torch.arange(n, device=DEV) * 2) if case["interleaved"] else torch.arange(n, device=DEV)
        second = first + (1 if case["interleaved"] else n)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    def held(x, s):
        cache = torch.zeros(st["kc"].shape, dtype=torch.float64, device=DEV)
        if case["fmt"] != "bf16":
            x = x / s.double().view(1, -1, 1)
            x = torch.sign(x) * _step(x.abs(), *((-6, 3, 448.0) if case["fmt"] == "e4m3" else (-14, 2, 57344.0)))
        cache[st["slots"] // BS, :, st["slots"] % BS] = x
        return cache

    return {"q": turned(st["q"], st["q_weight"]), "k": held(turned(st["k"], st["k_weight"]), st["k_scale"]),
            "v": held(st["v"].double(), st["v_scale"])}


def _exact_tree(case, st):
    cu, lens, parents = st["cu"].tolist(), st["lens"].tolist(), st["parents"].tolist()
    G, W, fmt, out = case["hq"] // case["hkv"], case["window"], case["fmt"], []
    eight = torch.arange(256, dtype=torch.uint8, device=DEV)
    eight = None if fmt == "bf16" else eight.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).double()
    for b, L in enumerate(lens):
        at = torch.arange(L, device=DEV)
        pages = st["bt"][b, at // BS].long()
        K, V = ((st[n + "c"][pages, :, at % BS].double() if eight is None else
                 eight[st[n + "c"][pages, :, at % BS].long()] * st[n + "_scale"].double().view(1, -1, 1)) for n in "kv")
        m = cu[b + 1] - cu[b]
        hide = torch.zeros(m, L, dtype=torch.bool)
        hide[:, L - m:] = True
        for j in range(m):
            way = []
            i = j
            while i >= 0:
                way.append(i)
                i = parents[cu[b] + i]
            hide[j, [L - m + i for i in (way[:W] if W else way)]] = False
            if W:
                hide[j, :max(0, min(L - m, L - m + len(way) - W))] = True
        hide = hide.to(DEV)
        q = st["q"][cu[b]:cu[b + 1]].double()
        o = []
        for g in range(case["hkv"]):
            x = torch.einsum("nhd,td->hnt", q[:, g * G:(g + 1) * G], K[:, g]) / math.sqrt(case["dh"])
            o.append(torch.einsum("hnt,td->nhd", torch.softmax(x.masked_fill(hide, -math.inf), -1), V[:, g]))
        out.append(torch.cat(o, 1))
    return {"out": torch.cat(out)}


def exact(case, seed):
    if case["op"] in ("commit", "fork"):  # whole numbers and bits moved
        return None
    return (_exact_rope if case["op"] == "rope" else _exact_tree)(case, prepare(case, seed))

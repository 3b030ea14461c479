"""The operators around a speculative decoding step over the paged FP8 latent cache, as
workloads to be timed and compared: rotary positions, the fused cache write (latent norm,
rotary positions, quantisation), reading the cache back, attention for a tree of drafted
tokens, and the acceptance of drafted tokens from given random numbers.

``run`` computes each operator in its plain form (elementary torch operations in float32 or
wider) or, where ``own`` is true, calls this library. ``exact`` computes the same outputs
from the operators' definitions in float64.
"""
import math
import random

import numpy as np
import torch

own = False

D, DV, ROPE, PAGE = 576, 512, 64, 64
SM_SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 32 sequences: the heads' RoPE parts, taken from the query
        # projection's rows (192 a head) to the absorbed query (576 a head); positions far
        # into a context that YaRN stretched 40 times
        dict(name="rope 32 tokens", op="rope", n=32, H=12, width=192, factor=40.0, orig=4096,
             interleaved=True, top=163840),
        # a prefill chunk, half layout, plain frequencies
        dict(name="rope 8192 tokens", op="rope", n=8192, H=12, width=192, factor=1.0, orig=0,
             interleaved=False, top=40960),
        # one decode step's rows out of a fused query/latent projection (2,112 a row)
        dict(name="append 32 rows", op="append", n=32, stride=2112, factor=40.0, orig=4096,
             interleaved=True, top=163840, pages=64),
        # a prefill chunk's rows, dense
        dict(name="append 8192 rows", op="append", n=8192, stride=576, factor=1.0, orig=0,
             interleaved=False, top=40960, pages=256),
        # a batch's short shared prefixes read back before an up-projection
        dict(name="gather 8 x 333", op="gather", B=8, lo=200, hi=466, skip=37, f32=False),
        # eight long histories read back whole
        dict(name="gather 8 x 32768", op="gather", B=8, lo=32768, hi=32768, skip=0, f32=False),
        # one user's small draft tree over a short context: latency
        dict(name="tree 1 x 8 nodes 1K", op="tree", B=1, n=8, H=12, lo=1024, hi=1024, empty=False),
        # the verify workload's batch with a 16-node tree on a 32K prefix
        dict(name="tree 8 x 16 nodes 32K", op="tree", B=8, n=16, H=12, lo=32784, hi=32784, empty=False),
        # the batched decode workload's lengths with 32-node trees
        dict(name="tree 32 x 32 nodes 4K-16K", op="tree", B=32, n=32, H=12, lo=4096, hi=16384, empty=False),
        # chains of three drafts of a draft model with its own probabilities, eight users
        dict(name="accept 8 x 3 drafts", op="accept", B=8, n=4, V=129280, tree=False, drafted=True, cut=False),
        # a large batch of longer chains
        dict(name="accept 64 x 7 drafts", op="accept", B=64, n=8, V=129280, tree=False, drafted=True, cut=False),
        # draft trees without draft probabilities; target rows cut to their largest entries
        dict(name="accept 32 trees of 16", op="accept", B=32, n=16, V=129280, tree=True, drafted=False, cut=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "gather", "tree", "accept"])
    if op in ("rope", "append"):
        factor, orig = rng.choice([(1.0, 0), (4.0, 0), (40.0, 4096), (8.0, 8192)])
        c = dict(op=op, n=_log(rng, 1, 8192), factor=factor, orig=orig, interleaved=rng.random() < 0.5,
                 top=_log(rng, 1000, 1000000))
        if op == "rope":
            return dict(c, H=rng.randint(1, 12), width=rng.choice([64, 192]))
        return dict(c, stride=rng.choice([576, 640, 2112]), pages=-(-c["n"] // PAGE) * 2)
    if op == "gather":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 8 * 32768 // B)
        f32 = rng.random() < 0.4
        hi = max(1, hi // 2) if f32 else hi
        lo = rng.randint(max(1, hi // 2), hi)
        return dict(op=op, B=B, lo=lo, hi=hi, skip=rng.randint(0, min(100, lo // 2)), f32=f32)
    if op == "tree":
        B, n, H = _log(rng, 1, 64), _log(rng, 1, 64), rng.randint(1, 16)
        top = min(40960, 32 * 16384 // B, 32 * 32 * 12 * 10240 // (B * n * H))
        hi = _log(rng, n + 64, max(n + 65, top))
        return dict(op=op, B=B, n=n, H=H, lo=rng.randint(n + 1, hi), hi=hi, empty=rng.random() < 0.25)
    B, n = _log(rng, 1, 64), rng.randint(2, 32)
    V = _log(rng, 1000, min(163840, 64 * 8 * 129280 // (B * n)))
    tree = rng.random() < 0.5
    return dict(op=op, B=B, n=n, V=V, tree=tree, drafted=not tree and rng.random() < 0.7, cut=rng.random() < 0.5)


def _lens(c):
    """The sequences' lengths, spread evenly over [lo, hi] (the last one empty where asked)."""
    B = c["B"]
    lens = [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) for b in range(B)]
    if c.get("empty") and B > 1:
        lens[-1] = 0
    return lens


# ----------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _frequencies(c):
    """Radians per position of the 32 pairs: base 10000, all divided by `factor` (linear) or,
    with an original length, blended between the two by YaRN's ramp (32 to 1 rotations)."""
    base = 10000.0
    plain = [base ** (-2.0 * j / ROPE) for j in range(ROPE // 2)]
    if c["factor"] == 1.0:
        return plain
    if not c["orig"]:
        return [f / c["factor"] for f in plain]

    def pair_of(rotations):
        return ROPE * math.log(c["orig"] / (rotations * 2 * math.pi)) / (2 * math.log(base))

    low = max(0, math.floor(pair_of(32.0)))
    high = min(ROPE - 1, math.ceil(pair_of(1.0)))
    ramp = [min(1.0, max(0.0, (j - low) / max(high - low, 0.001))) for j in range(ROPE // 2)]
    return [f / c["factor"] * r + f * (1 - r) for f, r in zip(plain, ramp)]


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["orig"] else 1.0


def _codes(rows, g):
    """N(0, 1) latent rows as e4m3 codes at the scale 0.0125 (row by row in chunks)."""
    codes = torch.empty(rows, D, dtype=torch.uint8, device=DEV)
    for r in range(0, rows, 1 << 17):
        x = torch.randn(min(1 << 17, rows - r), D, generator=g, device=DEV)
        codes[r:r + x.shape[0]] = (x * 80.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes


def _paged(lens, g):
    """A pool holding the sequences on randomly ordered pages, its page table, the lengths."""
    pages = [-(-n // PAGE) for n in lens]
    order = torch.randperm(sum(pages), generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    pool = _codes(max(1, at) * PAGE, g).view(-1, PAGE, D)
    return pool, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def _parents(n, r):
    """A draft tree's parents: each node hangs below one of the four nodes before it."""
    return [-1] + [r.randint(max(0, j - 4), j - 1) for j in range(1, n)]


def prepare(case, seed):
    c, g, r = case, _gen(seed), random.Random(seed)
    s = dict(case=c)
    if c["op"] == "rope":
        # the query projection's rows; the rotated part is the last 64 of each head
        x = torch.randn(c["n"], c["H"], c["width"], generator=g, device=DEV).bfloat16()
        q = torch.zeros(c["n"], c["H"], D, dtype=torch.bfloat16, device=DEV)
        s.update(x=x[..., c["width"] - ROPE:], out=q[..., DV:],
                 positions=torch.randint(0, c["top"], (c["n"],), generator=g, device=DEV))
    elif c["op"] == "append":
        rows = c["pages"] * PAGE
        x = torch.randn(c["n"], c["stride"], generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn(c["n"], 1, generator=g, device=DEV))  # rows of differing norms
        slots = torch.randperm(rows, generator=g, device=DEV)[:c["n"]]
        slots[15::16] = -1  # padding
        s.update(x=x.bfloat16()[:, c["stride"] - D:], slots=slots, kv_scale=0.0125,
                 weight=(1 + 0.2 * torch.randn(DV, generator=g, device=DEV)).bfloat16(),
                 pool=_codes(rows, g).view(-1, PAGE, D),
                 positions=torch.randint(0, c["top"], (c["n"],), generator=g, device=DEV))
    elif c["op"] == "gather":
        lens = _lens(c)
        starts = [min(c["skip"], n) for n in lens]
        ends = np.cumsum([0] + [n - a for n, a in zip(lens, starts)])
        pool, table, seq = _paged(lens, g)
        s.update(pool=pool, table=table, lens=seq, kv_scale=0.0125, n=int(ends[-1]),
                 starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                 cu=torch.tensor(ends, dtype=torch.int64, device=DEV))
    elif c["op"] == "tree":
        B, n, lens = c["B"], c["n"], _lens(c)
        pool, table, seq = _paged(lens, g)
        masks = []
        for _ in range(B):
            seen = []
            for j, a in enumerate(_parents(n, r)):
                seen.append((seen[a] if a >= 0 else 0) | (1 << j))
            masks.append([m - (1 << 64) if m >> 63 else m for m in seen])
        s.update(pool=pool, table=table, lens=seq, kv_scale=0.0125,
                 mask=torch.tensor(masks, dtype=torch.int64, device=DEV),
                 q=torch.randn(B, n, c["H"], D, generator=g, device=DEV).bfloat16())
    else:
        B, n, V = c["B"], c["n"], c["V"]
        parents = [_parents(n, r) if c["tree"] else list(range(-1, n - 1)) for _ in range(B)]
        par = torch.tensor(parents, device=DEV)
        logits = 5.0 * torch.randn(B, n, V, generator=g, device=DEV)  # a few tokens hold most of a row
        guess = torch.softmax(logits + 0.7 * torch.randn(B, n, V, generator=g, device=DEV), -1)
        guess = torch.take_along_dim(guess, par[:, 1:, None].clamp(min=0), 1)  # node j's draft row
        tokens = torch.zeros(B, n, dtype=torch.int32, device=DEV)
        tokens[:, 1:] = torch.multinomial(guess.reshape(-1, V), 1, generator=g).view(B, n - 1).int()
        p = torch.softmax(logits, -1)
        if c["cut"]:  # as top-k renormalisation leaves them
            p[p < p.topk(min(V, 200), -1).values[..., -1:]] = 0.0
            p /= p.sum(-1, keepdim=True)
        s.update(p=p, tokens=tokens, u=torch.rand(B, n + 1, generator=g, device=DEV),
                 parents=par.int() if c["tree"] else None, q=guess if c["drafted"] else None)
    if own:  # what a serving program sets up once: rotary tables, the cache's view, a workspace
        import mla_latent_kv_attention_gb300 as mla
        if c["op"] in ("rope", "append"):
            s["rope"] = mla.mla_rope_init(10000.0, factor=c["factor"], original_positions=c["orig"],
                                          amplitude=_amplitude(c), interleaved=c["interleaved"])
        elif c["op"] in ("gather", "tree"):
            s["kv"] = mla.KVCache(s["pool"], s["table"], s["lens"], s["kv_scale"])
        if c["op"] == "tree":
            s["ws"] = mla.workspace(mla.MLA_OP_VERIFY_TREE, c["B"], c["H"], c["n"], DEV)
    return s


# ------------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


_run_own = {}
_run_plain = {}


def _own(op):
    def keep(f):
        _run_own[op] = f
        return f
    return keep


def _plain(op):
    def keep(f):
        _run_plain[op] = f
        return f
    return keep


@_own("rope")
def _(s):
    import mla_latent_kv_attention_gb300 as mla
    return mla.mla_rope(s["rope"], s["x"], s["positions"], out=s["out"])


@_own("append")
def _(s):
    import mla_latent_kv_attention_gb300 as mla
    mla.mla_cache_append_rope(s["pool"], s["x"], s["slots"], s["kv_scale"], s["rope"], s["positions"],
                              norm_weight=s["weight"], eps=EPS)
    return s["pool"].view(torch.float8_e4m3fn)


@_own("gather")
def _(s):
    import mla_latent_kv_attention_gb300 as mla
    return mla.mla_cache_gather(s["kv"], s["cu"], s["n"], starts=s["starts"],
                                dtype=torch.float32 if s["case"]["f32"] else torch.bfloat16)


@_own("tree")
def _(s):
    import mla_latent_kv_attention_gb300 as mla
    return mla.mla_verify_tree(s["kv"], s["q"], s["mask"], SM_SCALE, ws=s["ws"])


@_own("accept")
def _(s):
    import mla_latent_kv_attention_gb300 as mla
    return mla.mla_accept_drafts(s["p"], s["tokens"], s["u"], parents=s["parents"], draft_probs=s["q"])


def _turn(x, positions, c):
    """float32 x [..., 64] rotated by its positions [n] (angles in float64)."""
    f = torch.tensor(_frequencies(c), dtype=torch.float64, device=DEV)
    angle = positions.double().view(-1, *([1] * (x.dim() - 1))) * f
    cos, sin = ((t * _amplitude(c)).float() for t in (angle.cos(), angle.sin()))
    if c["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


@_plain("rope")
def _(s):
    s["out"].copy_(_turn(s["x"].float(), s["positions"], s["case"]))
    return s["out"]


@_plain("append")
def _(s):
    x = s["x"].float()
    c, pe = x[:, :DV], x[:, DV:]
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    y = torch.cat((c, _turn(pe, s["positions"], s["case"])), -1)
    y = (y * (1.0 / s["kv_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = s["slots"] >= 0
    s["pool"].view(-1, D)[s["slots"][keep]] = y[keep]
    return s["pool"].view(torch.float8_e4m3fn)


def _rows(table, b, pos):
    """Flat cache rows of positions pos of sequences b."""
    return table[b, pos // PAGE].long() * PAGE + pos % PAGE


@_plain("gather")
def _(s):
    row = torch.arange(s["n"], device=DEV)
    b = torch.searchsorted(s["cu"], row, right=True) - 1
    at = _rows(s["table"], b, row - s["cu"][b] + s["starts"][b])
    y = s["pool"].view(-1, D)[at].view(torch.float8_e4m3fn).float() * s["kv_scale"]
    return y if s["case"]["f32"] else y.bfloat16()


@_plain("tree")
def _(s):
    B, n, H, _ = s["q"].shape
    top = s["case"]["hi"]
    pos = torch.arange(top, device=DEV).expand(B, top)
    have = pos < s["lens"][:, None]
    at = _rows(s["table"], torch.arange(B, device=DEV)[:, None], torch.where(have, pos, 0))
    k = s["pool"].view(-1, D)[torch.where(have, at, 0)].view(torch.float8_e4m3fn).float() * s["kv_scale"]
    node = pos - (s["lens"][:, None] - n)  # the tree's node whose key sits there, if >= 0
    bit = (s["mask"][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
    seen = have[:, None, :] & ((node[:, None, :] < 0) | (bit == 1))
    x = torch.matmul(s["q"].float().view(B, n * H, D), k.transpose(1, 2)) * SM_SCALE
    x = x.view(B, n, H, top).masked_fill_(~seen[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x.sub_(m.clamp(min=-1e30)))
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w.view(B, n * H, top), k[..., :DV]).view(B, n, H, DV) / total.clamp(min=1e-30)
    return out.bfloat16(), (m + torch.log(total)).squeeze(-1)


def _weight(w):
    """Probabilities as whole multiples of 2^-43, so that sums do not depend on their order."""
    return (torch.where(w > 0, w, 0.0).clamp(max=1.0) * 2.0 ** 43).round().long()


@_plain("accept")
def _(s):
    p, tokens, u, q = s["p"], s["tokens"].long(), s["u"], s["q"]
    B, n, V = p.shape
    j = torch.arange(n, device=DEV)
    batch = torch.arange(B, device=DEV)[:, None]
    par = (j - 1).expand(B, n) if s["parents"] is None else s["parents"].long()
    drafted = (tokens >= 0) & (tokens < V) & (par >= 0) & (par < j)
    par, tok = torch.where(drafted, par, 0), torch.where(drafted, tokens, 0)
    target = p[batch, par, tok]
    if q is None:  # a node is taken when its parent's number falls into its share
        sibling = (par[:, :, None] == par[:, None, :]) & drafted[:, :, None] & drafted[:, None, :] & (j[None, :] < j[:, None])
        again = (sibling & (tok[:, :, None] == tok[:, None, :])).any(-1)
        share = torch.where(drafted & ~again, _weight(target), 0)
        below = (sibling * share[:, None, :]).sum(-1)
        mark = (u[batch, par] * 2.0 ** 43).long()
        taken = drafted & (mark >= below) & (mark < below + share)
    else:  # a draft is taken with probability target / draft
        taken = drafted & (u[batch, par] * q[batch, (j - 1).clamp(min=0), tok] < target)
    up = torch.eye(n, dtype=torch.float64, device=DEV).repeat(B, 1, 1)
    up[batch, j, par] += (drafted & (j > 0)).double()
    above = torch.linalg.matrix_power(up, n) > 0  # node and its ancestors
    kept = above[:, :, 0] & ~(above & (~taken & (j > 0))[:, None, :]).any(-1)
    depth = above.sum(-1) - 1
    last = torch.where(kept, depth, -1).argmax(-1)
    count = depth.gather(1, last[:, None])
    chain = above[torch.arange(B, device=DEV), last]
    path = torch.full((B, n + 1), -1, device=DEV).scatter_(1, torch.where(chain, depth, n), j.expand(B, n))[:, :n]
    # the token after the last node kept: from what the refused drafts leave of its row
    row = p[batch[:, 0], last]
    if q is None:
        refused = drafted & (par == last[:, None]) & (j > 0)
        left = torch.cat((row, row[:, :1]), 1).scatter_(1, torch.where(refused, tok, V), 0.0)[:, :V]
    else:
        more = torch.cat((drafted[:, 1:], drafted[:, :1] & False), 1).gather(1, last[:, None])
        left = torch.where(more, (row - q[batch[:, 0], last.clamp(max=n - 2)]).clamp(min=0), row)
    w, whole = _weight(left), _weight(row)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, whole)
    cum = w.cumsum(-1)
    total = cum[:, -1:]
    mark = (u[:, n:] * 2.0 ** 31).long()
    at = (total >> 31) * mark + (((total & (2 ** 31 - 1)) * mark) >> 31)  # floor(total * u)
    new = torch.where(total > 0, (cum <= at).sum(-1, keepdim=True), -1)
    out = torch.where((j < count) & (j < n - 1), tokens.gather(1, torch.cat((path[:, 1:], path[:, :1]), 1).clamp(min=0)), -1)
    out = torch.where(j == count, new, out)
    return out.int(), path.int(), count[:, 0].int()


# ------------------------------------------------------------------------- what it has to do

def work(case):
    c = case
    if c["op"] == "rope":
        pairs = c["n"] * c["H"] * ROPE // 2
        return dict(bytes=pairs * 8 + 8 * c["n"], flops=6 * pairs)
    if c["op"] == "append":
        n = c["n"] - c["n"] // 16
        return dict(bytes=n * (2 * D + D + 8) + 8 * c["n"] + 2 * DV, flops=n * (4 * DV + 6 * ROPE // 2 + D))
    if c["op"] == "gather":
        n = sum(m - min(c["skip"], m) for m in _lens(c))
        pages = sum(-(-m // PAGE) for m in _lens(c))
        return dict(bytes=n * D * (5 if c["f32"] else 3) + 4 * pages + 16 * c["B"], flops=n * D)
    if c["op"] == "tree":
        keys, rows = sum(_lens(c)), c["B"] * c["n"] * c["H"]
        # the prefix is seen whole, of the nodes' own keys about half
        pairs = sum(max(0, m - c["n"] // 2) for m in _lens(c)) * c["n"] * c["H"]
        return dict(bytes=keys * D + rows * (2 * D + 2 * DV + 4) + 8 * c["B"] * c["n"] + keys // 16,
                    flops=2 * pairs * (D + DV))
    # one row of the target (and of the drafts) a sequence, the nodes' own entries
    row = c["B"] * c["V"]
    return dict(bytes=4 * row * (2 if c["drafted"] else 1) + c["B"] * c["n"] * (4 * 5 + 8), flops=4 * row)


# --------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "gather": _exact_gather,
            "tree": _exact_tree, "accept": _exact_accept}[case["op"]](s)


def _exact_turn(x, positions, c):
    """x [n, ..., 64] in float64 as complex numbers times amplitude * e^(i position f)."""
    f = np.array(_frequencies(c))
    phase = positions.cpu().numpy().astype(np.float64)[:, None] * f[None, :]
    w = torch.from_numpy(_amplitude(c) * np.exp(1j * phase)).to(x.device)
    w = w.view(w.shape[0], *([1] * (x.dim() - 2)), ROPE // 2)
    if c["interleaved"]:
        return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (ROPE // 2, 2)).contiguous()) * w).flatten(-2)
    z = torch.complex(x[..., :ROPE // 2].contiguous(), x[..., ROPE // 2:].contiguous()) * w
    return torch.cat((z.real, z.imag), -1)


def _exact_rope(s):
    return _exact_turn(s["x"].double(), s["positions"], s["case"])


def _exact_append(s):
    x = s["x"].double()
    norm = torch.sqrt((x[:, :DV] ** 2).sum(-1, keepdim=True) / DV + EPS)
    y = torch.cat((x[:, :DV] / norm * s["weight"].double(), _exact_turn(x[:, DV:], s["positions"], s["case"])), -1)
    pool = s["pool"].view(torch.float8_e4m3fn).to(torch.float64)
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            pool[slot // PAGE, slot % PAGE] = (y[i] / s["kv_scale"]).clamp(-448, 448)
    return pool


def _exact_cache(s, b, lo, hi):
    """Rows lo .. hi - 1 of sequence b in float64."""
    pages = s["table"][b, :-(-hi // PAGE)].long()
    k = s["pool"][pages].reshape(-1, D)[lo:hi]
    return k.view(torch.float8_e4m3fn).to(torch.float64) * s["kv_scale"]


def _exact_gather(s):
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    return torch.cat([_exact_cache(s, b, starts[b], lens[b]) for b in range(len(lens))])


def _exact_tree(s):
    B, n, H, _ = s["q"].shape
    out = torch.zeros(B, n, H, DV, dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, H), -math.inf, dtype=torch.float64, device=DEV)
    masks = s["mask"].tolist()
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        k = _exact_cache(s, b, 0, L)
        x = torch.einsum("jhd,kd->jhk", s["q"][b].double(), k) * SM_SCALE
        hide = torch.tensor([[not (masks[b][j] >> i) & 1 for i in range(n)] for j in range(n)], device=DEV)
        x[:, :, L - n:] = torch.where(hide[:, None, :], -math.inf, x[:, :, L - n:])
        lse[b] = torch.logsumexp(x, -1)
        out[b] = torch.einsum("jhk,kd->jhd", torch.exp(x - lse[b][..., None]), k[:, :DV])
    return out, lse


def _exact_accept(s):
    """Node by node on the host, sums in float64."""
    B, n, V = s["p"].shape
    tokens, u = s["tokens"].tolist(), s["u"].double().tolist()
    out, path, count = (np.full((B, n), -1, np.int32), np.full((B, n), -1, np.int32), np.zeros(B, np.int32))
    for b in range(B):
        par = list(range(-1, n - 1)) if s["parents"] is None else s["parents"][b].tolist()
        at = k = 0
        path[b, 0] = 0
        while True:
            row = s["p"][b, at].double().cpu().numpy()
            kids = [j for j in range(1, n) if par[j] == at]
            if s["q"] is None:
                acc, took = 0.0, None
                for j in (j for i, j in enumerate(kids) if tokens[b][j] not in [tokens[b][k2] for k2 in kids[:i]]):
                    if acc <= u[b][at] < acc + row[tokens[b][j]]:
                        took = j
                    acc += row[tokens[b][j]]
            else:
                took = next((j for j in kids if u[b][at] * float(s["q"][b, j - 1, tokens[b][j]]) < row[tokens[b][j]]), None)
            if took is None:
                break
            out[b, k], k, at = tokens[b][took], k + 1, took
            path[b, k] = at
        left = row.copy()
        if s["q"] is None:
            left[[tokens[b][j] for j in kids]] = 0.0
        elif kids:
            left = np.maximum(left - s["q"][b, at].double().cpu().numpy(), 0.0)
        left = left if left.sum() > 0 else row
        out[b, k], count[b] = np.searchsorted(np.cumsum(left), u[b][n] * left.sum(), side="right"), k
    return out, path, count

"""Operators around a latent cache with a scale for each block of positions, as workloads to be
timed and compared: rotary positions with several axes, the cache write that chooses the blocks'
scales, attention over such a cache (decode, speculative verify, draft trees, prefill), and reading
it back.

``run`` computes each operator in its plain form (elementary torch operations in float32 or wider)
or, where ``own`` is true, calls this library. ``exact`` computes the same outputs from the
operators' definitions in float64.

A cached row is 576 e4m3 codes: 512 of the latent, 64 RoPE dims. ``block`` positions share one
float32 scale, a power of two; a value is its code times its block's scale. Writing rows raises a
block's scale to the smallest power of two that brings its largest entry to 448 or less, never
lowers it while the block holds earlier positions, and rewrites their codes to the new scale.
"""
import math
import random

import numpy as np
import torch

own = False

D, DV, ROPE, PAIRS = 576, 512, 64, 32
SM_SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
LOWEST, HIGHEST = -60, 60  # exponents of a block's scale
DEV = "cuda"


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 32 sequences of text and images: the heads' RoPE parts, out of the
        # query projection's rows (192 a head) into the absorbed query (576 a head)
        dict(name="turn 32 tokens", op="turn", n=32, H=12, width=192, factor=40.0, orig=4096, pairs=True,
             sections="8 12 12", mixed=False, top=163840),
        # a prefill chunk of image and video tokens, half layout, the axes' pairs in turn
        dict(name="turn 8192 tokens", op="turn", n=8192, H=12, width=192, factor=1.0, orig=0, pairs=False,
             sections="12 10 10", mixed=True, top=40960),
        # one decode step's rows out of a fused query/latent projection (2,112 a row), most of them
        # into blocks begun earlier
        dict(name="write 32 x 1 rows", op="write", B=32, new=1, lo=500, hi=2000, block=16, page=64, stride=2112,
             factor=40.0, orig=4096, pairs=True, sections="8 12 12", mixed=False, top=163840),
        # a prefill chunk on a 32,768-position prefix, a scale for each page
        dict(name="write 1 x 8192 rows", op="write", B=1, new=8192, lo=40960, hi=40960, block=64, page=64,
             stride=576, factor=1.0, orig=0, pairs=False, sections="12 10 10", mixed=True, top=40960),
        # one user, short context: latency
        dict(name="decode 1 x 1K", op="attend", kind="decode", B=1, n=1, H=12, lo=1024, hi=1024, block=16, page=64,
             empty=False, f32=False),
        # the batched decode workload's batch
        dict(name="decode 32 x 4K-16K", op="attend", kind="decode", B=32, n=1, H=12, lo=4096, hi=16384, block=16,
             page=64, empty=False, f32=False),
        # one very long history
        dict(name="decode 1 x 142000", op="attend", kind="decode", B=1, n=1, H=12, lo=142000, hi=142000, block=64,
             page=64, empty=False, f32=False),
        # four speculative positions on a 32K prefix, a scale for every position
        dict(name="verify 8 x 4 on 32K", op="attend", kind="verify", B=8, n=4, H=12, lo=32772, hi=32772, block=1,
             page=64, empty=False, f32=False),
        # draft trees of 16 nodes on the same prefix
        dict(name="tree 8 x 16 nodes on 32K", op="attend", kind="tree", B=8, n=16, H=12, lo=32784, hi=32784,
             block=32, page=64, empty=False, f32=False),
        # the causal prefill workload: an 8,192-position chunk on a 32,768-position prefix
        dict(name="prefill 8192 on 32K", op="attend", kind="prefill", B=1, n=8192, H=12, lo=40960, hi=40960,
             block=64, page=64, empty=False, f32=False),
        # a batch's short shared prefixes read back before an up-projection
        dict(name="read 8 x 333", op="read", B=8, lo=200, hi=466, skip=37, block=16, page=64, f32=False),
        # eight long histories read back whole
        dict(name="read 8 x 32768", op="read", B=8, lo=32768, hi=32768, skip=0, block=64, page=64, f32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _positions_of(rng):
    factor, orig = rng.choice([(1.0, 0), (4.0, 0), (40.0, 4096), (8.0, 8192)])
    axes = rng.randint(1, 4)
    cut = sorted(rng.sample(range(1, PAIRS), axes - 1))
    sections = [b - a for a, b in zip([0] + cut, cut + [PAIRS])]
    return dict(factor=factor, orig=orig, pairs=rng.random() < 0.5, sections=" ".join(map(str, sections)),
                mixed=rng.random() < 0.5, top=_log(rng, 1000, 1000000))


def draw(rng):
    op = rng.choice(["turn", "write", "attend", "attend", "attend", "read"])
    blocks = dict(block=2 ** rng.randint(0, 6), page=rng.choice([64, 64, 128, 192]))
    if op == "turn":
        return dict(op=op, n=_log(rng, 1, 8192), H=rng.randint(1, 12), width=rng.choice([64, 192]),
                    **_positions_of(rng))
    if op == "write":
        B = _log(rng, 1, 128)
        new = _log(rng, 1, 8192 // B)
        hi = new + _log(rng, 1, max(2, 40960 // B))
        return dict(op=op, B=B, new=new, lo=rng.randint(new, hi), hi=hi, stride=rng.choice([576, 640, 2112]),
                    **blocks, **_positions_of(rng))
    if op == "read":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 8 * 32768 // B)
        f32 = rng.random() < 0.4
        hi = max(1, hi // 2) if f32 else hi
        lo = rng.randint(max(1, hi // 2), hi)
        return dict(op=op, B=B, lo=lo, hi=hi, skip=rng.randint(0, min(100, lo // 2)), f32=f32, **blocks)
    kind = rng.choice(["decode", "decode", "verify", "tree", "prefill"])
    H = rng.randint(1, 16)
    if kind == "prefill":
        B, n = 1, _log(rng, 1, 4096)
        hi = n + _log(rng, 1, 32768)
        return dict(op=op, kind=kind, B=B, n=n, H=H, lo=hi, hi=hi, empty=False, f32=False, **blocks)
    n = {"decode": 1, "verify": rng.randint(1, 4), "tree": _log(rng, 1, 64)}[kind]
    B = _log(rng, 1, 64)
    top = min(142000, 32 * 16384 // B, 8192 * 12 * 36864 // (B * n * H))
    hi = _log(rng, n + 64, max(n + 65, top))
    return dict(op=op, kind=kind, B=B, n=n, H=H, lo=rng.randint(n + 1, hi), hi=hi, empty=rng.random() < 0.25,
                f32=kind == "verify" and rng.random() < 0.3, **blocks)


def _lens(c):
    """The sequences' lengths, spread evenly over [lo, hi] (the last one empty where asked)."""
    B = c["B"]
    lens = [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) for b in range(B)]
    if c.get("empty") and B > 1:
        lens[-1] = 0
    return lens


# ----------------------------------------------------------------------------- the inputs

def _frequencies(c):
    """Radians per position of the 32 pairs: base 10000, all divided by `factor` (linear) or,
    with an original length, blended between the two by YaRN's ramp (32 to 1 rotations)."""
    base = 10000.0
    plain = [base ** (-2.0 * j / ROPE) for j in range(PAIRS)]
    if c["factor"] == 1.0:
        return plain
    if not c["orig"]:
        return [f / c["factor"] for f in plain]

    def pair_of(rotations):
        return ROPE * math.log(c["orig"] / (rotations * 2 * math.pi)) / (2 * math.log(base))

    low = max(0, math.floor(pair_of(32.0)))
    high = min(ROPE - 1, math.ceil(pair_of(1.0)))
    ramp = [min(1.0, max(0.0, (j - low) / max(high - low, 0.001))) for j in range(PAIRS)]
    return [f / c["factor"] * r + f * (1 - r) for f, r in zip(plain, ramp)]


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["orig"] else 1.0


def _sections(c):
    return [int(w) for w in c["sections"].split()]


def _axes(c):
    """The axis of each pair: section after section, or (mixed) the axes in turn while they have
    pairs left."""
    left = _sections(c)
    if not c["mixed"]:
        return [a for a, k in enumerate(left) for _ in range(k)]
    axes = []
    while len(axes) < PAIRS:
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                axes.append(a)
    return axes


def _places(c, g):
    """Positions [axes, n] of n tokens: text (the axes alike) and images (rows of patches)."""
    n = c["n"] if c["op"] == "turn" else c["B"] * c["new"]
    axes = len(_sections(c))
    at = torch.randint(0, c["top"], (n,), generator=g, device=DEV).expand(axes, n).clone()
    picture = torch.rand(n, generator=g, device=DEV) < 0.7
    at[1:] += torch.randint(0, 64, (axes - 1, n), generator=g, device=DEV) * picture
    return at


def _blocks(rows, block, g):
    """Rows of differing norms as codes and block scales, as the cache write leaves them."""
    codes = torch.empty(rows, D, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows // block, device=DEV)
    for r in range(0, rows, 1 << 17):  # (a multiple of every block)
        m = min(1 << 17, rows - r)
        x = torch.randn(m, D, generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device=DEV))
        top = x.view(m // block, -1).abs().amax(-1)
        s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
        x /= s.repeat_interleave(block)[:, None]
        codes[r:r + m] = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[r // block:(r + m) // block] = s
    return codes, scales


def _paged(c, g):
    """A pool holding the sequences on randomly ordered pages, its scales and its page table."""
    lens, page = _lens(c), c["page"]
    pages = [-(-n // page) for n in lens]
    order = torch.randperm(sum(pages), generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    at = max(1, at)
    codes, scales = _blocks(at * page, c["block"], g)
    return dict(pool=codes.view(at, page, D), scales=scales.view(at, -1), table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def _parents(n, r):
    """A draft tree's parents: each node hangs below one of the four nodes before it."""
    return [-1] + [r.randint(max(0, j - 4), j - 1) for j in range(1, n)]


def prepare(case, seed):
    c, r = case, random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "turn":
        # the query projection's rows; the turned part is the last 64 of each head
        x = torch.randn(c["n"], c["H"], c["width"], generator=g, device=DEV).bfloat16()
        q = torch.zeros(c["n"], c["H"], D, dtype=torch.bfloat16, device=DEV)
        s.update(x=x[..., c["width"] - ROPE:], out=q[..., DV:], at=_places(c, g))
    else:
        s.update(_paged(c, g))
    if c["op"] == "write":
        n = c["B"] * c["new"]
        x = torch.randn(n, c["stride"], generator=g, device=DEV)
        x[:, -ROPE:] *= torch.exp(0.5 + 0.7 * torch.randn(n, 1, generator=g, device=DEV))  # (not normalised)
        s.update(x=x.bfloat16()[:, c["stride"] - D:], at=_places(c, g),
                 weight=(1 + 0.2 * torch.randn(DV, generator=g, device=DEV)).bfloat16(),
                 cu=torch.arange(c["B"] + 1, device=DEV) * c["new"])
    elif c["op"] == "read":
        lens = _lens(c)
        starts = [min(c["skip"], n) for n in lens]
        ends = np.cumsum([0] + [n - a for n, a in zip(lens, starts)])
        s.update(n=int(ends[-1]), starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                 cu=torch.tensor(ends, dtype=torch.int64, device=DEV))
    elif c["op"] == "attend":
        B, n, H = c["B"], c["n"], c["H"]
        q = torch.randn(B, n, H, D, generator=g, device=DEV).bfloat16()
        if c["kind"] == "tree":
            masks = []
            for _ in range(B):
                seen = []
                for j, a in enumerate(_parents(n, r)):
                    seen.append((seen[a] if a >= 0 else 0) | (1 << j))
                masks.append([m - (1 << 64) if m >> 63 else m for m in seen])
            s["mask"] = torch.tensor(masks, dtype=torch.int64, device=DEV)
        s["q"] = q[:, 0] if c["kind"] == "decode" else q[0] if c["kind"] == "prefill" else q
    if own:  # what a serving program sets up once: rotary tables, the cache's view, a workspace
        import mla_latent_kv_attention_gb300 as mla
        if c["op"] in ("turn", "write"):
            s["rope"] = mla.mla_rope_init(10000.0, factor=c["factor"], original_positions=c["orig"],
                                          amplitude=_amplitude(c), interleaved=c["pairs"])
            s["axes"] = mla.mla_rope_axes_init(_sections(c), interleaved=c["mixed"])
        if c["op"] != "turn":
            s["kv"] = mla.KVCache(s["pool"], s["table"], s["lens"], 1.0, scales=s["scales"])
        if c["op"] == "attend":
            op = {"decode": mla.MLA_OP_DECODE, "verify": mla.MLA_OP_VERIFY, "tree": mla.MLA_OP_VERIFY_TREE,
                  "prefill": mla.MLA_OP_PREFILL}[c["kind"]]
            s["ws"] = mla.workspace(op, c["B"], c["H"], c["n"], DEV)
    return s


# ------------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_turn(s):
    import mla_latent_kv_attention_gb300 as mla
    return mla.mla_rope(s["rope"], s["x"], s["at"], out=s["out"], axes=s["axes"])


def _own_write(s):
    import mla_latent_kv_attention_gb300 as mla
    mla.mla_cache_append_scaled(s["kv"], s["x"], s["cu"], s["rope"], s["at"], axes=s["axes"],
                                norm_weight=s["weight"], eps=EPS)
    return s["pool"].view(torch.float8_e4m3fn), s["scales"]


def _own_attend(s):
    import mla_latent_kv_attention_gb300 as mla
    c = s["case"]
    if c["kind"] == "tree":
        return mla.mla_verify_tree(s["kv"], s["q"], s["mask"], SM_SCALE, ws=s["ws"])
    call = {"decode": mla.mla_decode, "prefill": mla.mla_prefill,
            "verify": mla.mla_verify_f32 if c["f32"] else mla.mla_verify}[c["kind"]]
    return call(s["kv"], s["q"], SM_SCALE, ws=s["ws"])


def _own_read(s):
    import mla_latent_kv_attention_gb300 as mla
    return mla.mla_cache_gather(s["kv"], s["cu"], s["n"], starts=s["starts"],
                                dtype=torch.float32 if s["case"]["f32"] else torch.bfloat16)


def _turn(x, at, c):
    """float32 x [n, ..., 64] turned to positions at [axes, n] (angles in float64)."""
    f = torch.tensor(_frequencies(c), dtype=torch.float64, device=DEV)
    place = at.double()[torch.tensor(_axes(c), device=DEV)].T  # [n, 32]
    angle = (place * f).view(place.shape[0], *([1] * (x.dim() - 2)), PAIRS)
    cos, sin = ((t * _amplitude(c)).float() for t in (angle.cos(), angle.sin()))
    if c["pairs"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x[..., :PAIRS], x[..., PAIRS:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _plain_turn(s):
    s["out"].copy_(_turn(s["x"].float(), s["at"], s["case"]))
    return s["out"]


def _plain_write(s):
    c = s["case"]
    G, page, new = c["block"], c["page"], c["new"]
    x = s["x"].float()
    lat, pe = x[:, :DV], x[:, DV:]
    lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    y = torch.cat((lat, _turn(pe, s["at"], c)), -1)
    row = torch.arange(x.shape[0], device=DEV)
    b = torch.searchsorted(s["cu"], row, right=True) - 1
    pos = s["lens"][b].long() - (s["cu"][b + 1] - row)
    flat = s["table"][b, pos // page].long() * page + pos % page
    block, place = flat // G, flat % G
    codes, scales = s["pool"].view(-1, G, D), s["scales"].view(-1)
    # the scale a block needs for its new rows, and how many earlier ones it holds
    top = torch.zeros_like(scales).scatter_reduce_(0, block, y.abs().amax(-1), "amax")
    first = torch.full_like(scales, G, dtype=torch.int64).scatter_reduce_(0, block, place, "amin")
    m, e = torch.frexp(top)
    need = torch.where(m <= 0.875, e - 9, e - 8).clamp(LOWEST, HIGHEST)
    need = torch.ldexp(torch.ones_like(top), torch.where(top > 0, need, LOWEST))
    touched = torch.unique(block)
    was = scales[touched]
    now = torch.where(first[touched] > 0, torch.maximum(was, need[touched]), need[touched])
    kept = codes[touched]
    moved = (kept.view(torch.float8_e4m3fn).float() * (was / now)[:, None, None]).to(torch.float8_e4m3fn)
    earlier = torch.arange(G, device=DEV)[None, :] < first[touched][:, None]
    codes[touched] = torch.where(earlier[:, :, None], moved.view(torch.uint8), kept)
    scales[touched] = now
    y = (y / scales[block][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes.view(-1, D)[flat] = y
    return s["pool"].view(torch.float8_e4m3fn), s["scales"]


def _rows(s, b, pos):
    """float32 cached rows at positions pos of sequences b."""
    page = s["case"]["page"]
    flat = s["table"][b, pos // page].long() * page + pos % page
    k = s["pool"].view(-1, D)[flat].view(torch.float8_e4m3fn).float()
    return k.mul_(s["scales"].view(-1)[flat // s["case"]["block"]][..., None])


def _plain_read(s):
    row = torch.arange(s["n"], device=DEV)
    b = torch.searchsorted(s["cu"], row, right=True) - 1
    y = _rows(s, b, row - s["cu"][b] + s["starts"][b])
    return y if s["case"]["f32"] else y.bfloat16()


def _softmax_rows(q, k, seen):
    """q [B, R, 576] float32, k [B, L, 576], seen [B, R, L]: outputs and log-sum-exps."""
    x = torch.matmul(q, k.transpose(1, 2)).mul_(SM_SCALE).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = x.sub_(m.clamp(min=-1e30)).exp_()
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w, k[..., :DV]).div_(total.clamp(min=1e-30))
    return out, (m + torch.log(total)).squeeze(-1)


def _plain_attend(s):
    c = s["case"]
    B, n, H, top = c["B"], c["n"], c["H"], c["hi"]
    q = s["q"].float().view(B, n, H, D)
    pos = torch.arange(top, device=DEV).expand(B, top)
    have = pos < s["lens"][:, None]
    k = _rows(s, torch.arange(B, device=DEV)[:, None], torch.where(have, pos, 0))
    k = torch.where(have[..., None], k, 0.0)
    outs, lses = [], []
    for j0 in range(0, n, 512):  # (a prefill's scores in pieces)
        j = torch.arange(j0, min(n, j0 + 512), device=DEV)
        node = (pos - (s["lens"][:, None] - n))[:, None, :]  # the new position whose key sits there, if >= 0
        if c["kind"] == "tree":
            bit = (s["mask"][:, j, None] >> node.clamp(0, 63)) & 1
            seen = have[:, None, :] & ((node < 0) | (bit == 1))
        else:
            seen = have[:, None, :] & (node <= j[:, None])
        part = q[:, j0:j0 + 512].reshape(B, -1, D)
        out, lse = _softmax_rows(part, k, seen.repeat_interleave(H, 1))
        outs.append(out.view(B, -1, H, DV))
        lses.append(lse.view(B, -1, H))
    out, lse = torch.cat(outs, 1), torch.cat(lses, 1)
    shape = s["q"].shape[:-1]
    out, lse = out.view(*shape, DV), lse.view(shape)
    return (out if c["f32"] else out.bfloat16()), lse


_run_own = dict(turn=_own_turn, write=_own_write, attend=_own_attend, read=_own_read)
_run_plain = dict(turn=_plain_turn, write=_plain_write, attend=_plain_attend, read=_plain_read)


# ------------------------------------------------------------------------- what it has to do

def work(case):
    c = case
    G = c.get("block")
    if c["op"] == "turn":
        pairs = c["n"] * c["H"] * PAIRS
        return dict(bytes=pairs * 8 + 8 * c["n"] * len(_sections(c)), flops=6 * pairs)
    if c["op"] == "write":
        n = c["B"] * c["new"]
        return dict(bytes=n * (2 * D + D + 8 * len(_sections(c))) + 8 * c["B"] + 2 * DV + 4 * -(-n // G),
                    flops=n * (4 * DV + 6 * PAIRS + 2 * D))
    if c["op"] == "read":
        n = sum(m - min(c["skip"], m) for m in _lens(c))
        pages = sum(-(-m // c["page"]) for m in _lens(c))
        return dict(bytes=n * D * (5 if c["f32"] else 3) + 4 * (n // G + pages) + 16 * c["B"], flops=n * D)
    keys, rows = sum(_lens(c)), c["B"] * c["n"] * c["H"]
    # the prefix is seen whole, of the new positions' own keys about half
    pairs = sum(max(0, m - c["n"] // 2) for m in _lens(c)) * c["n"] * c["H"]
    return dict(bytes=keys * D + 4 * (keys // G + keys // c["page"]) + rows * (2 * D + (4 if c["f32"] else 2) * DV + 4),
                flops=2 * pairs * (D + DV))


# --------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"turn": _exact_turn, "write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _exact_turned(x, at, c):
    """x [n, ..., 64] in float64 as complex numbers times amplitude * e^(i position f)."""
    at = at.cpu().numpy().astype(np.float64)
    phase = np.stack([at[a] * f for a, f in zip(_axes(c), _frequencies(c))], -1)
    w = torch.from_numpy(_amplitude(c) * np.exp(1j * phase)).to(x.device)
    w = w.view(w.shape[0], *([1] * (x.dim() - 2)), PAIRS)
    if c["pairs"]:
        return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (PAIRS, 2)).contiguous()) * w).flatten(-2)
    z = torch.complex(x[..., :PAIRS].contiguous(), x[..., PAIRS:].contiguous()) * w
    return torch.cat((z.real, z.imag), -1)


def _exact_turn(s):
    return _exact_turned(s["x"].double(), s["at"], s["case"])


def _exact_write(s):
    c = s["case"]
    G, page, new = c["block"], c["page"], c["new"]
    x = s["x"].double()
    norm = torch.sqrt((x[:, :DV] ** 2).sum(-1, keepdim=True) / DV + EPS)
    y = torch.cat((x[:, :DV] / norm * s["weight"].double(), _exact_turned(x[:, DV:], s["at"], c)), -1)
    pool = s["pool"].view(torch.float8_e4m3fn).to(torch.float64).view(-1, D)
    scales = s["scales"].double().view(-1).tolist()
    table, tops = s["table"].tolist(), y.abs().amax(-1).tolist()
    for b, L in enumerate(_lens(c)):
        pos = L - new
        while pos < L:  # block by block of the sequence
            end = min(L, (pos // G + 1) * G)
            row = b * new + pos - (L - new)
            top = max(tops[row:row + end - pos])
            power = LOWEST
            while power < HIGHEST and top > 448.0 * 2.0 ** power:
                power += 1
            flat = table[b][pos // page] * page + pos % page
            block, k = flat // G, pos % G
            scale = 2.0 ** power
            if k > 0:
                scale = max(scale, scales[block])
                pool[flat - k:flat] *= scales[block] / scale
            scales[block] = scale
            pool[flat:flat + end - pos] = (y[row:row + end - pos] / scale).clamp(-448, 448)
            pos = end
    return pool.view(s["pool"].shape), torch.tensor(scales, dtype=torch.float64, device=DEV).view(s["scales"].shape)


def _exact_rows(s, b, lo, hi):
    """Rows lo .. hi - 1 of sequence b in float64."""
    c = s["case"]
    pages = s["table"][b, :-(-hi // c["page"])].long()
    k = s["pool"][pages].view(torch.float8_e4m3fn).to(torch.float64)
    k = k.view(len(pages), -1, c["block"], D) * s["scales"][pages].double()[:, :, None, None]
    return k.reshape(-1, D)[lo:hi]


def _exact_read(s):
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    return torch.cat([_exact_rows(s, b, starts[b], lens[b]) for b in range(len(lens))])


def _exact_attend(s):
    c = s["case"]
    B, n, H = c["B"], c["n"], c["H"]
    q = s["q"].view(B, n, H, D)
    out = torch.zeros(B, n, H, DV, dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, H), -math.inf, dtype=torch.float64, device=DEV)
    masks = s["mask"].tolist() if c["kind"] == "tree" else None
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        k = _exact_rows(s, b, 0, L)
        for j0 in range(0, n, 256):
            m = min(256, n - j0)
            x = torch.einsum("jhd,kd->jhk", q[b, j0:j0 + m].double(), k) * SM_SCALE
            if masks is not None:
                hide = torch.tensor([[not (masks[b][j] >> i) & 1 for i in range(n)] for j in range(n)], device=DEV)
                x[:, :, L - n:] = torch.where(hide[:, None, :], -math.inf, x[:, :, L - n:])
            else:
                last = L - n + j0 + torch.arange(m, device=DEV)
                x.masked_fill_((torch.arange(L, device=DEV) > last[:, None])[:, None, :], -math.inf)
            lse[b, j0:j0 + m] = torch.logsumexp(x, -1)
            out[b, j0:j0 + m] = torch.einsum("jhk,kd->jhd", torch.exp(x - lse[b, j0:j0 + m][..., None]), k[:, :DV])
    return out.view(*s["q"].shape[:-1], DV), lse.view(s["q"].shape[:-1])

"""The operators of the 4-bit expert layer, measured: routing with gate weights, quantization to
microscaled 4-bit floating point, the products of such operands (dense, and per expert over routed
rows), and the weighted combination of the experts' outputs.

Each case runs one operator once, on inputs drawn from a seed. `run` computes the operator with
elementary torch operations, or, where `own` is true, through this package's entry points.

Formats. A row of d values is cut into blocks; a block shares one 8-bit scale s and every value is a
4-bit e2m1 number q (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) that stands for q * s * g, g a
float32 scale of the whole matrix (1 where there is none):
  "e8m0_32"  blocks of 32, s = 2^(floor(log2 max|x / g|) - 2), a power of two in 2^-127 .. 2^127
  "e4m3_16"  blocks of 16, s = max|x| / (6 g) rounded to e4m3 (at least 2^-9, at most 448)
and q = x / (s g) rounded to the nearest e2m1 number, ties to the even code, saturating at 6; a
block of zeros has s = 2^-127 (e8m0) or 0 (e4m3). Two codes a byte, the even column in the low bits.
Scales lie in tiles of 128 rows x 4 blocks (512 bytes), tiles row-major: row r, block b of a tile at
byte 16 (r % 32) + 4 (r / 32) + b, both sides padded with zeros to whole tiles.

Routed rows lie in segments (one an expert, each starting at a multiple of 128): seg[0 .. E] the
starts, seg[E + 1 .. 2E] the token counts, perm the token of each row (-1: none).
"""
import math

import torch

own = False

_BLOCK = {"e8m0_32": 32, "e4m3_16": 16}
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_contexts = {}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # routing: one decoding step's few tokens; the 64-expert top-6 layer's calibration batch; a wide
        # router with balance bias and groups, an odd token count, half-width logits
        dict(name="route_decode", op="route", n=4, E=64, k=6, score="sigmoid", bias=True, groups=8, top_groups=4,
             rank="top2", renormalise=True, dtype="f32"),
        dict(name="route_e64", op="route", n=32768, E=64, k=6, score="softmax", bias=False, groups=1, top_groups=1,
             rank="max", renormalise=True, dtype="f32"),
        dict(name="route_wide", op="route", n=9973, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             rank="top2", renormalise=True, dtype="bf16"),
        # quantization: the 64-expert layer's tokens straight into their experts' segments; a small batch
        # of float32 activations of the 28672-wide projection under a matrix scale
        dict(name="quantize_e64_routed", op="quantize", n=32768, d=2048, E=64, k=6, fmt="e8m0_32", dtype="bf16",
             scaled=False),
        dict(name="quantize_small", op="quantize", n=33, d=28672, E=0, k=0, fmt="e4m3_16", dtype="f32", scaled=True),
        # products: one token through the 28672 -> 8192 projection; a prompt-sized batch of it; the 16-expert
        # top-2 layer's down projections on an odd batch
        dict(name="matmul_decode", op="matmul", n=1, d_in=28672, d_out=8192, E=0, k=0, fmt="e4m3_16", out="bf16",
             scaled=True),
        dict(name="matmul_dense", op="matmul", n=16384, d_in=28672, d_out=8192, E=0, k=0, fmt="e4m3_16", out="bf16",
             scaled=True),
        dict(name="matmul_e16_down", op="matmul", n=4099, d_in=512, d_out=1024, E=16, k=2, fmt="e8m0_32", out="f32",
             scaled=False),
        # gate and up projections with SiLU(gate) * up: the 64-expert layer on a whole batch and on a few tokens
        dict(name="act_e64", op="act", n=32768, d_in=2048, d_out=1408, E=64, k=6, fmt="e8m0_32", scaled=False),
        dict(name="act_decode", op="act", n=5, d_in=2048, d_out=1408, E=64, k=6, fmt="e4m3_16", scaled=True),
        # combination: the 64-expert layer's outputs with an always-active part; a few tokens
        dict(name="combine_e64", op="combine", n=32768, d=2048, E=64, k=6, dtype="f32", out="bf16", add=True),
        dict(name="combine_decode", op="combine", n=5, d=2048, E=64, k=6, dtype="f32", out="bf16", add=False),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    return 128 * _log_uniform(rng, lo // 128, hi // 128)


def draw(rng):
    op = rng.choice(["route", "route", "quantize", "quantize", "matmul", "matmul", "matmul", "act", "act", "combine"])
    fmt = rng.choice(["e8m0_32", "e4m3_16"])
    if op == "route":
        groups, size = rng.choice([1, 1, 2, 4, 8]), rng.randint(2, 48)
        E = groups * size
        top_groups = rng.randint(1, groups)
        return dict(op="route", n=_log_uniform(rng, 1, 40000), E=E, k=rng.randint(1, min(10, top_groups * size)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, rank=rng.choice(["max", "top2"]), renormalise=rng.random() < 0.7,
                    dtype=rng.choice(["f32", "bf16"]))
    E = rng.choice([0, 0, 8, 16, 40, 64])
    k = rng.randint(1, 6) if E else 0
    if op == "quantize":
        return dict(op="quantize", n=_log_uniform(rng, 1, 20000), d=_width(rng, 128, 4096), E=E, k=k, fmt=fmt,
                    dtype=rng.choice(["bf16", "f32"]), scaled=rng.random() < 0.5)
    if op == "combine":
        return dict(op="combine", n=_log_uniform(rng, 1, 20000), d=_width(rng, 128, 4096), E=E or 16, k=k or 2,
                    dtype=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]), add=rng.random() < 0.5)
    if op == "act":
        return dict(op="act", n=_log_uniform(rng, 1, 16000), d_in=_width(rng, 256, 2048), d_out=_width(rng, 128, 1408),
                    E=E, k=k, fmt=fmt, scaled=rng.random() < 0.5)
    if E:
        return dict(op="matmul", n=_log_uniform(rng, 1, 16000), d_in=_width(rng, 128, 2048),
                    d_out=_width(rng, 128, 2048), E=E, k=k, fmt=fmt, out=rng.choice(["bf16", "f32"]),
                    scaled=rng.random() < 0.5)
    return dict(op="matmul", n=_log_uniform(rng, 1, 12000), d_in=_width(rng, 128, 16384),
                d_out=_width(rng, 128, 8192), E=0, k=0, fmt=fmt, out=rng.choice(["bf16", "f32"]),
                scaled=rng.random() < 0.5)


# ------------------------------------------------------------------------------ formats, in plain torch
def _steps(a):
    """Index of the e2m1 level nearest to a >= 0 (ties to the even index)."""
    up = lambda t: (a > t).to(torch.uint8)     # a tie stays below
    at = lambda t: (a >= t).to(torch.uint8)    # a tie goes up
    return up(0.25) + at(0.75) + up(1.25) + at(1.75) + up(2.5) + at(3.5) + up(5.0)


def _block_scale(top, g, fmt):
    """The block scales for the blocks' largest magnitudes (both in float64)."""
    t = top / g
    if fmt == "e8m0_32":
        e = (torch.frexp(t).exponent - 3).clamp(-127, 127)           # floor(log2 t) - 2
        e = torch.where(t > 0, e, torch.full_like(e, -127))
        return torch.ldexp(torch.ones_like(t), e)
    t = t / 6
    e = (torch.frexp(t).exponent - 1).clamp_min(-6)
    step = torch.ldexp(torch.ones_like(t), e - 3)
    s = (torch.round(t / step) * step).clamp(2.0 ** -9, 448.0)
    return torch.where(t > 0, s, torch.zeros_like(s))


def _quantize(x, g, fmt):
    """(codes uint8 [R, d], block scales float64 [R, d / block]) of x [R, d]; g broadcasts over rows."""
    R, d = x.shape
    v = x.double().view(R, d // _BLOCK[fmt], _BLOCK[fmt])
    s = _block_scale(v.abs().amax(-1), g, fmt)
    a = v.abs() / (s * g).clamp_min(1e-300)[..., None]
    c = _steps(a)
    c = torch.where(v < 0, c + 8, c)
    c = torch.where(c == 8, torch.zeros_like(c), c)                  # no negative zero
    return c.view(R, d), s


def _to_bytes(s, fmt):
    """The scales' 8-bit encodings."""
    if fmt == "e8m0_32":
        return (torch.frexp(s).exponent + 126).to(torch.uint8)
    return s.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _from_bytes(b, fmt):
    if fmt == "e8m0_32":
        return torch.ldexp(torch.ones(b.shape, dtype=torch.float64, device=b.device), b.int() - 127)
    return b.view(torch.float8_e4m3fn).double()


def _tile(b):
    """Scale bytes [R, nb] -> the tiled layout, flat."""
    R, nb = b.shape
    p = torch.nn.functional.pad(b, (0, -nb % 4, 0, -R % 128))
    return p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile(t, R, nb):
    rt, kt = (R + 127) // 128, (nb + 3) // 4
    return t.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:R, :nb].contiguous()


def _pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _decode(packed, tiled, fmt, g=None):
    """float32 values [R, d] of packed codes [R, d / 2] and tiled scales; g: matrix scale, per row or one."""
    R, d = packed.shape[0], 2 * packed.shape[1]
    table = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float32, device=packed.device)
    q = torch.stack((packed & 15, packed >> 4), -1).view(R, d)
    s = _from_bytes(_untile(tiled, R, d // _BLOCK[fmt]), fmt).float()
    v = table[q.int()].view(R, d // _BLOCK[fmt], _BLOCK[fmt]) * s[..., None]
    v = v.view(R, d)
    return v if g is None else v * g


# ------------------------------------------------------------------------------ inputs
_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _tokens(n, d, gen):
    """Activations: per-channel variances, a low-rank part and one percent outlier channels."""
    dev = gen.device
    x = torch.randn((n, d), generator=gen, device=dev) * (0.5 + 1.5 * torch.rand(d, generator=gen, device=dev)).sqrt()
    x += torch.randn((n, 8), generator=gen, device=dev) @ (0.3 * torch.randn((8, d), generator=gen, device=dev))
    out = torch.randperm(d, generator=gen, device=dev)[: max(1, d // 100)]
    x[:, out] *= 20
    return x


def _route_inputs(n, E, k, gen):
    """ids [n, k] of a skewed router, and the segments and permutation that group them by expert."""
    dev = gen.device
    p = (torch.randperm(E, generator=gen, device=dev) + 1).float() ** -1.1
    ids = (torch.randn((n, E), generator=gen, device=dev) + p.log()).topk(k, dim=1).indices.int()
    flat = ids.view(-1).long()
    counts = torch.bincount(flat, minlength=E)
    starts = torch.cumsum((counts + 127) // 128 * 128, 0)
    seg = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), starts, counts))
    rows = (n * k + 127) // 128 * 128 + 128 * E
    order = torch.sort(flat, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    perm = torch.full((rows,), -1, dtype=torch.int32, device=dev)
    e = flat[order]
    perm[seg[e] + torch.arange(n * k, device=dev) - first[e]] = (order // k).int()
    return ids, seg, perm, rows


def _operand(x, fmt, scaled, batch=1):
    """x [R, d] in the format: packed codes, tiled scales and the matrix scales (None without them)."""
    g = None
    if scaled:
        g = (x.view(batch, -1).abs().amax(1) / (6 * 448.0)).float()
    per_row = 1.0 if g is None else g.double().repeat_interleave(x.shape[0] // batch)[:, None]
    c, s = _quantize(x, per_row, fmt)
    return _pack(c), _tile(_to_bytes(s, fmt)), g


def _zero_rows(x, perm):
    """The rows of x in segment order, zeros where perm is -1."""
    return torch.where((perm >= 0)[:, None], x[perm.clamp_min(0).long()], torch.zeros((), dtype=x.dtype, device=x.device))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev, op, n = gen.device, case["op"], case["n"]
    st = dict(case)
    if op == "route":
        E = case["E"]
        p = (torch.randperm(E, generator=gen, device=dev) + 1).float() ** -1.1
        st["logits"] = (torch.randn((n, E), generator=gen, device=dev) + p.log()).to(_DTYPE[case["dtype"]])
        st["b"] = 0.1 * torch.randn(E, generator=gen, device=dev) if case["bias"] else None
        st["ids"] = torch.zeros((n, case["k"]), dtype=torch.int32, device=dev)
        st["weights"] = torch.zeros((n, case["k"]), device=dev)
        st["counts"] = torch.zeros(E, dtype=torch.int32, device=dev)
        return st
    E, k = case["E"], case["k"]
    st["rows"], st["seg"], st["perm"] = n, None, None
    if E:
        st["ids"], st["seg"], st["perm"], st["rows"] = _route_inputs(n, E, k, gen)
    rows = st["rows"]
    if op == "quantize":
        d, nb = case["d"], case["d"] // _BLOCK[case["fmt"]]
        x = _tokens(n, d, gen).to(_DTYPE[case["dtype"]])
        st["x"] = x
        st["g"] = (x.float().abs().amax() / (6 * 448.0)).view(1) if case["scaled"] else None
        st["codes"] = torch.zeros((rows, d // 2), dtype=torch.uint8, device=dev)
        st["scales"] = torch.zeros(((rows + 127) // 128 * 128, (nb + 3) // 4 * 4), dtype=torch.uint8, device=dev)
        st["values"] = torch.zeros((rows, d), dtype=torch.float32 if case["scaled"] else torch.bfloat16, device=dev)
        return st
    if op == "combine":
        d = case["d"]
        st["z"] = torch.randn((rows, d), generator=gen, device=dev).to(_DTYPE[case["dtype"]])
        w = torch.rand((n, k), generator=gen, device=dev) + 0.1
        st["weights"] = w / w.sum(1, keepdim=True)
        st["extra"] = torch.randn((n, d), generator=gen, device=dev).to(_DTYPE[case["out"]]) if case["add"] else None
        st["y"] = torch.zeros((n, d), dtype=_DTYPE[case["out"]], device=dev)
        return st
    d_in, d_out, fmt, B = case["d_in"], case["d_out"], case["fmt"], max(E, 1)
    x = _tokens(n, d_in, gen).to(torch.bfloat16)
    if E:
        x = _zero_rows(x, st["perm"])
    st["xq"], st["xs"], st["xg"] = _operand(x, fmt, case["scaled"])
    del x
    for name in ("w",) if op == "matmul" else ("w", "u"):
        w = (0.02 * torch.randn((B * d_out, d_in), generator=gen, device=dev)).to(torch.bfloat16)
        st[name + "q"], st[name + "s"], st[name + "g"] = _operand(w, fmt, case["scaled"], B)
    out = torch.bfloat16 if op == "act" else _DTYPE[case["out"]]
    st["y"] = torch.zeros((rows, d_out), dtype=out, device=dev)
    return st


# ------------------------------------------------------------------------------ the plain forms
def _plain_route(st):
    x, E, k = st["logits"].double(), st["E"], st["k"]
    score = torch.softmax(x, 1) if st["score"] == "softmax" else 1 / (1 + torch.exp(-x))
    choice = score if st["b"] is None else score + st["b"].double()
    if st["groups"] > 1:
        by = choice.view(-1, st["groups"], E // st["groups"])
        best = torch.sort(by, dim=2, descending=True).values
        rank = best[..., 0] if st["rank"] == "max" else best[..., :2].sum(2)
        kept = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, : st["top_groups"]]
        mask = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(mask[..., None], by, torch.full_like(by, -math.inf)).view(-1, E)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if st["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device=x.device)
    counts.index_add_(0, ids.reshape(-1), torch.ones(ids.numel(), dtype=torch.int32, device=x.device))
    return ids.int(), w.float(), counts


def _scale_values(tiled, rows, d, fmt):
    """The block scales as the float32 values that they stand for."""
    return _from_bytes(_untile(tiled.view(-1), rows, d // _BLOCK[fmt]), fmt).float()


def _plain_quantize(st):
    x, fmt = st["x"], st["fmt"]
    if st["perm"] is not None:
        x = _zero_rows(x, st["perm"])
    g = 1.0 if st["g"] is None else st["g"].double()
    c, s = _quantize(x, g, fmt)
    packed, tiled = _pack(c), _tile(_to_bytes(s, fmt))
    v = _decode(packed, tiled, fmt, st["g"])
    return v.to(st["values"].dtype), tiled


def _plain_product(st, act):
    x = _decode(st["xq"], st["xs"], st["fmt"], st["xg"])
    E, N, d_in = max(st["E"], 1), st["d_out"], st["d_in"]
    if st["seg"] is None:
        x, of = x[None], torch.zeros(1, dtype=torch.int64, device=x.device)
    else:                                                # tiles of 128 rows, each of one expert
        x = x.view(-1, 128, d_in)
        of = torch.searchsorted(st["seg"][:E], 128 * torch.arange(x.shape[0], device=x.device), right=True) - 1

    def times(name):
        g = st[name + "g"]
        w = _decode(st[name + "q"], st[name + "s"], st["fmt"], None if g is None else g.repeat_interleave(N)[:, None])
        return torch.bmm(x, w.view(E, N, d_in)[of].transpose(1, 2)).view(-1, N)

    y = times("w")
    if act:
        y = y * torch.sigmoid(y) * times("u")
    return y.to(st["y"].dtype)


def _positions(st):
    """The packed row of each (token, slot): its expert's segment start plus its rank there."""
    flat = st["ids"].view(-1).long()
    order = torch.sort(flat, stable=True).indices
    e = flat[order]
    counts = st["seg"][st["E"] + 1:]
    first = torch.cumsum(counts, 0) - counts
    pos = torch.empty_like(flat)
    pos[order] = st["seg"][e] + torch.arange(flat.numel(), device=flat.device) - first[e]
    return pos.view(st["ids"].shape)


def _plain_combine(st):
    y = (st["z"][_positions(st)].float() * st["weights"][..., None]).sum(1)
    if st["extra"] is not None:
        y = y + st["extra"].float()
    return y.to(st["y"].dtype)


# ------------------------------------------------------------------------------ one pass
def _context():
    from post_quantization_expert_b200 import clha as L
    dev = torch.cuda.current_device()
    if dev not in _contexts:
        _contexts[dev] = L.Context(dev)
    return L, _contexts[dev]


def run(st):
    op = st["op"]
    if not own:
        if op == "route":
            return _plain_route(st)
        if op == "quantize":
            v, tiled = _plain_quantize(st)
            return v, _scale_values(tiled, st["rows"], st["d"], st["fmt"])
        return _plain_combine(st) if op == "combine" else _plain_product(st, op == "act")
    L, ctx = _context()
    if op == "route":
        L.clha_route_gated(ctx, st["logits"], st["n"], st["E"], st["k"], st["ids"], st["weights"], st["counts"],
                           score=L.SCORE_SOFTMAX if st["score"] == "softmax" else L.SCORE_SIGMOID, bias=st["b"],
                           n_groups=st["groups"], top_groups=st["top_groups"],
                           group_rank=L.GROUP_MAX if st["rank"] == "max" else L.GROUP_TOP2,
                           renormalise=st["renormalise"])
        return st["ids"], st["weights"], st["counts"]
    if op == "combine":
        L.clha_combine(ctx, st["z"], st["rows"], st["d"], st["ids"], st["weights"], st["n"], st["k"], st["E"],
                       st["seg"], st["perm"], st["y"], add=st["extra"])
        return st["y"]
    fmt = L.FP4_E8M0_32 if st["fmt"] == "e8m0_32" else L.FP4_E4M3_16
    if op == "quantize":
        L.clha_fp4_quantize(ctx, st["x"], st["n"], st["d"], fmt, st["codes"], st["scales"], tensor_scale=st["g"],
                            perm=st["perm"], rows=st["rows"], seg=st["seg"], E=max(st["E"], 1))
        L.clha_fp4_dequantize(ctx, st["codes"], st["scales"], st["rows"], st["d"], fmt, st["values"],
                              tensor_scale=st["g"])
        return st["values"], _scale_values(st["scales"], st["rows"], st["d"], st["fmt"])
    if op == "act":
        L.clha_fp4_expert_act(ctx, fmt, st["xq"], st["xs"], st["rows"], st["d_in"], st["wq"], st["ws"], st["uq"],
                              st["us"], st["d_out"], st["y"], x_scale=st["xg"], g_scale=st["wg"], u_scale=st["ug"],
                              seg=st["seg"], E=max(st["E"], 1))
    else:
        L.clha_fp4_matmul(ctx, fmt, st["xq"], st["xs"], st["rows"], st["d_in"], st["wq"], st["ws"], st["d_out"],
                          st["y"], x_scale=st["xg"], w_scale=st["wg"], seg=st["seg"], E=max(st["E"], 1))
    return st["y"]


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, n = case["op"], case["n"]
    size = {"f32": 4, "bf16": 2}
    if op == "route":
        return {"bytes": n * case["E"] * size[case["dtype"]] + n * case["k"] * 8 + case["E"] * 8,
                "flops": n * case["E"] * 4}
    E, k = case["E"], case["k"]
    real = n * k if E else n                             # rows with a token
    per_byte = 0.5 + 1 / _BLOCK[case["fmt"]] if "fmt" in case else 0.0
    if op == "quantize":
        d = case["d"]
        return {"bytes": n * d * size[case["dtype"]] + real * d * (per_byte + (4 if case["scaled"] else 2)),
                "flops": real * d * 4}
    if op == "combine":
        d, out = case["d"], size[case["out"]]
        return {"bytes": real * d * size[case["dtype"]] + n * d * out * (2 if case["add"] else 1),
                "flops": 2 * real * d}
    d_in, d_out = case["d_in"], case["d_out"]
    mats = 2 if op == "act" else 1
    used = E * (1 - (1 - k / E) ** n) if E else 1        # experts that get a token
    out = 2 if op == "act" else size[case["out"]]
    return {"bytes": (real * d_in + used * mats * d_in * d_out) * per_byte + real * d_out * out,
            "flops": 2 * real * d_in * d_out * mats}


# ------------------------------------------------------------------------------ the definitions in 64 bits
def _exact_operand(packed, tiled, fmt, R, d):
    """Values without the matrix scale, float64 [R, d], byte by byte from the layout's definition."""
    dev, blk = packed.device, _BLOCK[fmt]
    r, b = torch.arange(R, device=dev)[:, None], torch.arange(d // blk, device=dev)[None]
    tiles = (d // blk + 3) // 4
    byte = tiled.view(-1)[((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4].double()
    if fmt == "e8m0_32":
        s = torch.pow(2.0, byte - 127)
    else:
        e, m = torch.floor(byte / 8), byte % 8
        s = torch.where(e > 0, (8 + m) * torch.pow(2.0, e - 10), m * 2.0 ** -9)
    out = torch.empty((R, d), dtype=torch.float64, device=dev)
    for half in (0, 1):
        c = ((packed.int() >> (4 * half)) & 15).double()
        sign, c = torch.where(c >= 8, -1.0, 1.0), c % 8
        e, m = torch.floor(c / 2), c % 2
        out[:, half::2] = sign * torch.where(e > 0, (2 + m) * torch.pow(2.0, e - 2), m * 0.5)
    return (out.view(R, d // blk, blk) * s[..., None]).view(R, d)


def _exact_quantize(st):
    fmt, blk = st["fmt"], _BLOCK[st["fmt"]]
    x = st["x"].double()
    if st["perm"] is not None:
        x = torch.cat((x, torch.zeros_like(x[:1])))[st["perm"].long()]        # -1: the row of zeros
    R, d = x.shape
    x = (x if st["g"] is None else x / st["g"].double()).view(R, -1, blk)
    top = x.abs().amax(2, keepdim=True)
    if fmt == "e8m0_32":
        p = torch.floor(torch.log2(top.clamp_min(1e-300)))
        p = torch.where(torch.pow(2.0, p) > top, p - 1, torch.where(torch.pow(2.0, p + 1) <= top, p + 1, p))
        s = torch.pow(2.0, torch.where(top > 0, p - 2, torch.full_like(p, -127)).clamp(-127, 127))
    else:
        grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                            [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                            dtype=torch.float64, device=x.device)             # every e4m3 number, code order
        mid = (grid[1:] + grid[:-1]) / 2
        t = (top / 6).contiguous()
        at = torch.searchsorted(mid, t)                                       # the midpoints below t
        tie = mid[at.clamp_max(len(mid) - 1)] == t
        at = torch.where(tie, at + at % 2, at)                                # on a midpoint: the even code
        s = torch.where(top > 0, grid[at.clamp_min(1)], torch.zeros_like(t))
    a = x.abs() / torch.where(s > 0, s, torch.ones_like(s))
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = (torch.round(a / step) * step).clamp_max(6.0)
    v = (torch.sign(x) * q * s).view(R, d)
    return (v if st["g"] is None else v * st["g"].double()), s.view(R, -1)


def exact(case, seed):
    st = prepare(case, seed)
    op, E = st["op"], st.get("E", 0)
    if op == "route":
        x = st["logits"].double()
        s = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) if st["score"] == "softmax" else torch.sigmoid(x)
        c = s if st["b"] is None else s + st["b"].double()
        if st["groups"] > 1:
            by = c.view(x.shape[0], st["groups"], -1)
            top = by.topk(min(2, by.shape[2]) if st["rank"] == "top2" else 1, 2).values.sum(2)
            worst = top.topk(st["top_groups"], 1).values[:, -1:]
            c = by.masked_fill((top < worst)[..., None], -math.inf).view(x.shape)
        w = torch.gather(s, 1, c.topk(st["k"], 1).indices)
        return None, (w / w.sum(1, keepdim=True) if st["renormalise"] else w), None
    if op == "quantize":
        return _exact_quantize(st)
    if op == "combine":
        z, ids, seg = st["z"].double(), st["ids"].long(), st["seg"]
        hit = torch.nn.functional.one_hot(ids, E).sum(1)                       # [n, E]
        before = torch.cumsum(hit, 0) - hit                                    # earlier tokens of each expert
        row = seg[ids] + before.gather(1, ids)
        y = sum(st["weights"][:, j, None].double() * z[row[:, j]] for j in range(st["k"]))
        return y if st["extra"] is None else y + st["extra"].double()
    d_in, N, rows = st["d_in"], st["d_out"], st["rows"]
    x = _exact_operand(st["xq"], st["xs"], st["fmt"], rows, d_in)
    xg = 1.0 if st["xg"] is None else st["xg"].double()
    y = torch.zeros((rows, N), dtype=torch.float64, device=x.device)
    seg = st["seg"].tolist() if st["seg"] is not None else [0, rows, rows]
    for e in range(max(E, 1)):
        r = slice(seg[e], seg[e] + seg[max(E, 1) + 1 + e])
        parts = []
        for name in ("w", "u") if op == "act" else ("w",):
            q = st[name + "q"].view(max(E, 1), N, -1)[e]
            s = st[name + "s"].view(max(E, 1), -1)[e]
            wg = 1.0 if st[name + "g"] is None else st[name + "g"][e].double()
            parts.append(x[r] @ _exact_operand(q, s, st["fmt"], N, d_in).T * xg * wg)
        y[r] = parts[0] * torch.sigmoid(parts[0]) * parts[1] if op == "act" else parts[0]
    return y

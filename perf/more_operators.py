"""The operators around the attention of a decoder layer with an 8-bit checkpoint: their cases, plain forms and work.

Three operators, each called as a serving program calls it:

* ``norm``: the residual's addition, the RMS norm and the rounding of its result to FP8 E4M3 with one scale per 128
  values, in one pass (``msa.add_norm_quant``); without a weight it only rounds, as in front of the output projection;
* ``linear``: a projection of such rows with FP8 weights that carry one scale per 128 x 128 block
  (``msa.fp8_linear``);
* ``rope``: head norms, rotary embedding in a checkpoint's own layout (half or interleaved pairs, a part of the head,
  frequencies scaled for long contexts) and the insert into the paged cache, on the packed rows that the projection
  wrote (``msa.qkv_rope_insert``).

``own`` selects the framework's kernels; otherwise ``run`` computes the plain forms in elementary torch
operations.
"""
import math
import random

import torch

own = False

BLOCK, DIM, GROUP = 128, 128, 128    # tokens per cache block, head size, values per 8-bit scale
FP8_MAX = 448.0
KV_SCALE = 6.0 / 448.0               # K/V per-tensor scale: six standard deviations on E4M3's largest value
EPS, THETA = 1e-6, 10000.0
FACTOR, TRAINED, FAST, SLOW = 4.0, 32768, 32.0, 1.0      # a context stretched to four times the trained length
LOW, HIGH = 1.0, 4.0


# ---------------------------------------------------------------------------------------------- cases --
def _norm(name, tokens, width, residual="bf16", norm=True, out="fp8"):
    c = {"op": "norm", "tokens": tokens, "width": width, "residual": residual, "norm": norm, "out": out}
    return dict(c, name=name) if name else c


def _linear(name, tokens, n, k, out="bf16"):
    c = {"op": "linear", "tokens": tokens, "n": n, "k": k, "out": out}
    return dict(c, name=name) if name else c


def _rope(name, tokens, kv="bf16", kv_heads=4, group=16, layout="half", rotary=128, scaling="none", norm=True):
    c = {"op": "rope", "tokens": tokens, "kv": kv, "kv_heads": kv_heads, "group": group, "layout": layout,
         "rotary": rotary, "scaling": scaling, "norm": norm}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one chat's token on its way into a layer: the smallest call, where latency counts
        _norm("norm 1 token", 1, 4096),
        # a decode step of 64 requests
        _norm("norm 64 decode", 64, 4096),
        # an odd number of rows of a width that ends inside a scale's group, the residual stream kept in 32 bits,
        # both results wanted (a layer whose router reads the rows unrounded)
        _norm("norm 333 x 5008 f32 residual", 333, 5008, residual="f32", out="both"),
        # a chunk of prompts
        _norm("norm 8191 prompt", 8191, 4096),
        # the attention's output of 32 requests with 8 positions, 64 heads, rounded for the output projection
        _norm("quant 256 x 8192", 256, 8192, residual="none", norm=False),
        # one token through the query, key and value projection of one tensor-parallel rank of eight
        _linear("linear 1 x 1280 x 4096", 1, 1280, 4096),
        # a decode step of 64 requests through the packed projection: 64 + 2 * 4 query, key and value heads and
        # 2 * 4 index heads of 128
        _linear("linear 64 x 10240 x 4096", 64, 10240, 4096),
        # speculative verification, 32 requests with 8 positions, through the output projection
        _linear("linear 256 x 4096 x 8192", 256, 4096, 8192),
        # a chunk of prompts through the packed projection
        _linear("linear 8191 x 10240 x 4096", 8191, 10240, 4096),
        # logits of 64 requests over a vocabulary of odd size, in 32 bits
        _linear("linear 64 x 100003 x 4096 f32", 64, 100003, 4096, out="f32"),
        # one new token for each of 64 requests, interleaved pairs in half of the head
        _rope("rope 64 decode", 64, layout="interleaved", rotary=64),
        # a chunk of prompts into an FP8 cache, the frequencies stretched by parts
        _rope("rope 8191 prompt fp8", 8191, kv="fp8", rotary=64, scaling="parts"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "rope"))
    if op == "norm":
        width = 16 * _log(rng, 8, 512)
        norm = rng.random() < 0.75
        return _norm(None, _log(rng, 1, min(8191, 8191 * 4096 // width)), width,
                     rng.choice(("bf16", "f32", "none")) if norm else "none", norm, rng.choice(("fp8", "fp8", "bf16", "both")))
    if op == "linear":
        n, k = _log(rng, 64, 16384), 16 * _log(rng, 16, 512)
        if rng.random() < 0.5:
            n = max(128, n // 128 * 128)
        return _linear(None, _log(rng, 1, min(8191, 8191 * 10240 * 4096 // (n * k))), n, k, rng.choice(("bf16", "bf16", "f32")))
    g = rng.choice((1, 2, 4))
    return _rope(None, _log(rng, 1, 8190), rng.choice(("bf16", "fp8")), g, rng.choice((4, 8, 16)),
                 rng.choice(("half", "interleaved")), rng.choice((32, 64, 96, 128)),
                 rng.choice(("none", "linear", "parts", "waves")), rng.random() < 0.7)


def _groups(n):
    return (n + GROUP - 1) // GROUP


def work(case):
    t = case["tokens"]
    if case["op"] == "norm":
        n = t * case["width"]
        b = 2.0 * n
        b += {"none": 0.0, "bf16": 4.0, "f32": 8.0}[case["residual"]] * n              # in and out
        b += 4.0 * case["width"] if case["norm"] else 0.0
        if case["out"] != "bf16":
            b += n + 4.0 * t * _groups(case["width"])
        if case["out"] != "fp8":
            b += 2.0 * n
        return {"bytes": b, "flops": 6.0 * n}
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        b = 1.0 * t * k + 1.0 * n * k + 4.0 * (t + _groups(n)) * _groups(k) + (4.0 if case["out"] == "f32" else 2.0) * t * n
        return {"bytes": b, "flops": 2.0 * t * n * k}
    g, h = case["kv_heads"], case["kv_heads"] * case["group"]
    kv = 2.0 if case["kv"] == "bf16" else 1.0
    b = t * DIM * (2.0 * (h + 2 * g) + 2.0 * h + kv * 2 * g) + t * 12.0
    return {"bytes": b, "flops": 10.0 * t * (h + g) * DIM}


# --------------------------------------------------------------------------------------------- inputs --
def _e4m3(x):
    return x.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _quant_rows(x):
    """fp32 [T, K] -> (uint8 E4M3 codes, fp32 scales [T, ceil(K / 128)])."""
    T, K = x.shape
    g = _groups(K)
    v = torch.nn.functional.pad(x, (0, g * GROUP - K)).reshape(T, g, GROUP)
    s = v.abs().amax(-1) / FP8_MAX
    y = torch.where(s[..., None] > 0, v / s.clamp(min=1e-38)[..., None], torch.zeros_like(v))
    return _e4m3(y).reshape(T, g * GROUP)[:, :K].contiguous().view(torch.uint8), s


def _quant_weight(n, k, gen):
    """A weight of N(0, 0.02) values with blocks of unequal size, as (uint8 codes [n, k], fp32 scales)."""
    gn, gk = _groups(n), _groups(k)
    codes = torch.empty((n, k), dtype=torch.uint8, device="cuda")
    scales = torch.empty((gn, gk), dtype=torch.float32, device="cuda")
    size = 0.02 * torch.exp(0.3 * torch.randn((gn, gk), generator=gen, device="cuda"))
    step = max(1, 16384 * 4096 // (GROUP * gk * GROUP))              # blocks of rows at a time
    for at in range(0, gn, step):
        m = min(step, gn - at)
        x = torch.randn((m, GROUP, gk, GROUP), generator=gen, device="cuda")
        x *= size[at:at + m, None, :, None]
        s = x.abs().amax((1, 3)) / FP8_MAX
        scales[at:at + m] = s
        y = _e4m3(x / s[:, None, :, None]).view(torch.uint8).reshape(m * GROUP, gk * GROUP)
        rows = min(n, (at + m) * GROUP) - at * GROUP
        codes[at * GROUP:at * GROUP + rows] = y[:rows, :k]
    return codes, scales


def prepare(case, seed):
    rng = random.Random(seed * 7919 + 29)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    s = {"case": dict(case), "flags": torch.zeros(1, dtype=torch.int32, device="cuda")}
    T = case["tokens"]
    if case["op"] == "norm":
        W = case["width"]
        # the stream of a deep layer: a few channels far larger than the others
        channels = torch.exp(0.5 * rand(W)) * torch.where(torch.rand(W, generator=gen, device="cuda") < 0.004, 20.0, 1.0)
        s["x"] = (rand(T, W) * channels).to(torch.bfloat16)
        if case["residual"] != "none":
            kind = torch.bfloat16 if case["residual"] == "bf16" else torch.float32
            s["residual"] = (3.0 * rand(T, W) * channels).to(kind)
            s["residual_out"] = torch.empty_like(s["residual"])
        if case["norm"]:
            s["weight"] = 1.0 + 0.1 * rand(W)
        if case["out"] != "fp8":
            s["out"] = torch.empty((T, W), dtype=torch.bfloat16, device="cuda")
        if case["out"] != "bf16":
            s["codes"] = torch.empty((T, W), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((T, _groups(W)), dtype=torch.float32, device="cuda")
    elif case["op"] == "linear":
        s["a"], s["a_scales"] = _quant_rows(rand(T, case["k"]) * torch.exp(0.4 * rand(case["k"])))
        s["w"], s["w_scales"] = _quant_weight(case["n"], case["k"], gen)
        kind = torch.float32 if case["out"] == "f32" else torch.bfloat16
        s["out"] = torch.empty((T, case["n"]), dtype=kind, device="cuda")
    else:
        G, H = case["kv_heads"], case["kv_heads"] * case["group"]
        # one packed row per token, as the projection writes it: queries, keys, values
        s["packed"] = (2.0 * rand(T, H + 2 * G, DIM)).to(torch.bfloat16)
        for n in ("wq", "wk"):
            s[n] = 1.0 + 0.1 * rand(DIM)
        t = torch.arange(T, device="cuda")
        if T > 1024:                      # a prompt's chunk fills pages
            p = rng.randint(0, 100000) + t
            pages = _groups(T)
            perm = torch.randperm(pages, generator=gen, device="cuda")
            s["slots"] = perm[t // BLOCK] * BLOCK + t % BLOCK
        else:                             # decode tokens lie in a page each
            p = torch.randint(0, 131072, (T,), generator=gen, device="cuda")
            pages = T
            perm = torch.randperm(pages, generator=gen, device="cuda")
            s["slots"] = perm[t] * BLOCK + p % BLOCK
        s["positions"], s["pages"] = p.to(torch.int32), pages
        kind = torch.bfloat16 if case["kv"] == "bf16" else torch.uint8
        s["k_cache"] = torch.zeros((pages, G, BLOCK, DIM), dtype=kind, device="cuda")
        s["v_cache"] = torch.zeros((pages, G, BLOCK, DIM), dtype=kind, device="cuda")
        s["q_out"] = torch.empty((T, H, DIM), dtype=torch.bfloat16, device="cuda")
    return s


def _packed(s):
    """Queries, keys and values as views of the packed rows."""
    G = s["case"]["kv_heads"]
    return s["packed"][:, :-2 * G], s["packed"][:, -2 * G:-G], s["packed"][:, -G:]


# ----------------------------------------------------------------------------------------- plain forms --
def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    outs = {}
    if c["residual"] != "none":
        h = h + s["residual"].float()
        outs["residual"] = h.to(s["residual"].dtype)
    y = h
    if c["norm"]:
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    if c["out"] != "fp8":
        outs["out"] = y.to(torch.bfloat16)
    if c["out"] != "bf16":
        codes, outs["scales"] = _quant_rows(y)
        outs["codes"] = codes.view(torch.float8_e4m3fn)
    return outs


def _dequant(codes, scales, rows_per_scale):
    x = codes.view(torch.float8_e4m3fn).float()
    s = scales.repeat_interleave(GROUP, 1)[:, :x.shape[1]]
    if rows_per_scale > 1:
        s = s.repeat_interleave(rows_per_scale, 0)[:x.shape[0]]
    return x * s


def _plain_linear(s):
    y = torch.matmul(_dequant(s["a"], s["a_scales"], 1), _dequant(s["w"], s["w_scales"], GROUP).t())
    return y.to(s["out"].dtype)


def _frequencies(rotary, scaling):
    """(angles per position in fp64 [rotary / 2], the factor on cosine and sine)."""
    i = torch.arange(rotary // 2, dtype=torch.float64, device="cuda")
    f = THETA ** (-2.0 * i / rotary)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / FACTOR, 1.0
    if scaling == "parts":
        # pairs that turn more than FAST times over the trained length keep their frequency, those below SLOW turns
        # are slowed down by the factor, and a ramp over the pairs lies between
        at = [rotary * math.log(TRAINED / (turns * 2.0 * math.pi)) / (2.0 * math.log(THETA)) for turns in (FAST, SLOW)]
        lo, hi = max(0, math.floor(at[0])), min(rotary - 1, math.ceil(at[1]))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f / FACTOR * ramp + f * (1.0 - ramp), 0.1 * math.log(FACTOR) + 1.0
    # the same by wavelength, a ramp over the number of turns between LOW and HIGH
    turns = TRAINED * f / (2.0 * math.pi)
    keep = ((turns - LOW) / (HIGH - LOW)).clamp(0.0, 1.0)
    return f / FACTOR * (1.0 - keep) + f * keep, 1.0


def _rotated(x, w, positions, c):
    y = x.float()
    if c["norm"]:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    R = c["rotary"]
    f, gain = _frequencies(R, c["scaling"])
    angle = positions.double()[:, None] * f
    cos, sin = (gain * angle.cos()).float()[:, None], (gain * angle.sin()).float()[:, None]
    z = y.clone()
    if c["layout"] == "half":
        a, b = y[..., :R // 2], y[..., R // 2:R]
        z[..., :R // 2], z[..., R // 2:R] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        z[..., 0:R:2], z[..., 1:R:2] = a * cos - b * sin, a * sin + b * cos
    return z.to(torch.bfloat16)


def _held(kind, x):
    """What a cache holds of bf16 values."""
    return x if kind == "bf16" else _e4m3(x.float() / KV_SCALE).view(torch.uint8)


def _cache_view(c, x):
    return x if c["kv"] == "bf16" else x.view(torch.float8_e4m3fn)


def _plain_rope(s):
    c = s["case"]
    q, k, v = _packed(s)
    page, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    s["k_cache"][page, :, off] = _held(c["kv"], _rotated(k, s["wk"], s["positions"], c))
    s["v_cache"][page, :, off] = _held(c["kv"], v)
    return _rotated(q, s["wq"], s["positions"], c), _cache_view(c, s["k_cache"]), _cache_view(c, s["v_cache"])


# ------------------------------------------------------------------------------------- the framework's --
def _own_call(s):
    """The marshalled call a decode loop keeps for its buffers and issues every step, on the stream that is current
    here, and its outputs."""
    from block_sparse_attention_07_gb300 import msa
    c = s["case"]
    if c["op"] == "norm":
        call = msa.add_norm_quant(s["x"], s.get("weight"), residual=s.get("residual"), residual_out=s.get("residual_out"),
                                  out=s.get("out"), codes=s.get("codes"), scales=s.get("scales"), eps=EPS, prepare=True)
        outs = {}
        if "residual" in s:
            outs["residual"] = s["residual_out"]
        if "out" in s:
            outs["out"] = s["out"]
        if "codes" in s:
            outs["scales"], outs["codes"] = s["scales"], s["codes"].view(torch.float8_e4m3fn)
        return call, outs
    if c["op"] == "linear":
        return msa.fp8_linear(s["a"], s["a_scales"], s["w"], s["w_scales"], s["out"], s["flags"], prepare=True), s["out"]
    G, H = c["kv_heads"], c["kv_heads"] * c["group"]
    d = msa.make_dims(1, 1, H, G, G, max_blocks_per_seq=s["pages"], num_pages=s["pages"])
    scale = 1.0 if c["kv"] == "bf16" else KV_SCALE
    cache = msa.KVCache(msa.BF16 if c["kv"] == "bf16" else msa.FP8_E4M3, s["k_cache"], s["v_cache"], None, None, scale, scale)
    layout = msa.ROPE_HALF if c["layout"] == "half" else msa.ROPE_INTERLEAVED
    rope = {"none": lambda: msa.make_rope(c["rotary"], THETA, layout),
            "linear": lambda: msa.make_rope(c["rotary"], THETA, layout, msa.ROPE_LINEAR, FACTOR),
            "parts": lambda: msa.make_rope(c["rotary"], THETA, layout, msa.ROPE_BY_PARTS, FACTOR, TRAINED, SLOW, FAST),
            "waves": lambda: msa.make_rope(c["rotary"], THETA, layout, msa.ROPE_BY_TURNS, FACTOR, TRAINED, LOW, HIGH)}[c["scaling"]]()
    nr = msa.make_norm_rope(s["wq"], s["wk"], eps=EPS) if c["norm"] else None
    q, k, v = _packed(s)
    return msa.qkv_rope_insert(d, q, k, v, None, None, s["positions"], s["slots"], nr, rope, s["q_out"], None, cache,
                               None, s["flags"], prepare=True), (
        s["q_out"], _cache_view(c, s["k_cache"]), _cache_view(c, s["v_cache"]))


def run(s):
    if own:
        # A kept call launches on the stream it was made for, on the tensors it was made for: it holds them, so that none
        # of their addresses is another's, and is made again where the state has others. (The stream's handle alone:
        # torch.cuda.current_stream() makes an object around it, 4 us on the host, as long as the smallest launches.)
        if "kept" not in s:
            s["kept"] = s["flags"].device.index, {}
        device, calls = s["kept"]
        stream = torch._C._cuda_getCurrentRawStream(device)
        kept = calls.get(stream)
        if kept is not None:
            call, outputs, held = kept
            for name, x in held:
                if s[name] is not x:
                    kept = None
        if kept is None:
            held = [(n, x) for n, x in s.items() if isinstance(x, torch.Tensor)]
            call, outputs, held = calls[stream] = (*_own_call(s), held)
        call()
        return outputs
    op = s["case"]["op"]
    return _plain_norm(s) if op == "norm" else _plain_linear(s) if op == "linear" else _plain_rope(s)


# ---------------------------------------------------------------------------------------------- exact --
def _e4m3_table():
    """fp64 value of every E4M3 code, from its bit fields."""
    byte = torch.arange(256, device="cuda")
    sign, e, m = 1.0 - 2.0 * (byte >> 7), (byte >> 3) & 15, (byte & 7).double()
    table = sign * torch.where(e > 0, (1.0 + m / 8.0) * torch.pow(2.0, (e - 7).double()), m * 2.0 ** -9)
    table[127] = table[255] = math.nan
    return table


def _exact_linear(s):
    """Group by group: the products of the codes, times the two scales of the group."""
    T, N, K = s["case"]["tokens"], s["case"]["n"], s["case"]["k"]
    table = _e4m3_table()
    y = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    for g in range(_groups(K)):
        lo, hi = g * GROUP, min(K, (g + 1) * GROUP)
        a = table[s["a"][:, lo:hi].long()] * s["a_scales"][:, g:g + 1].double()
        w = table[s["w"][:, lo:hi].long()]
        by_row = s["w_scales"][:, g].double()[torch.arange(N, device="cuda") // GROUP]
        y += (a @ w.T) * by_row
    return y


def _exact_norm(s):
    c = s["case"]
    y = s["x"].double()
    outs = {}
    if c["residual"] != "none":
        y = y + s["residual"].double()
        outs["residual"] = y
    if c["norm"]:
        y = y * (y.square().sum(-1, keepdim=True) / c["width"] + EPS).rsqrt() * s["weight"].double()
    if c["out"] != "fp8":
        outs["out"] = y
    if c["out"] != "bf16":
        scales = torch.stack([part.abs().amax(-1) for part in y.split(GROUP, 1)], 1) / FP8_MAX
        outs["scales"] = scales
        # the values in units of their scale, before their rounding to 8 bits
        outs["codes"] = torch.cat([part / scales[:, i:i + 1] for i, part in enumerate(y.split(GROUP, 1))], 1)
    return outs


def _exact_rope(s):
    """A complex number turned by its angle, one per pair."""
    c = s["case"]
    R = c["rotary"]
    pairs = [THETA ** (-2.0 * i / R) for i in range(R // 2)]
    gain = 1.0
    if c["scaling"] == "linear":
        pairs = [f / FACTOR for f in pairs]
    elif c["scaling"] == "parts":
        place = lambda turns: R / 2.0 * math.log(TRAINED / (2.0 * math.pi * turns), THETA)
        first, last = max(0, math.floor(place(FAST))), min(R - 1, math.ceil(place(SLOW)))
        slow = [min(1.0, max(0.0, (i - first) / max(last - first, 0.001))) for i in range(R // 2)]
        pairs = [f * (1.0 - r + r / FACTOR) for f, r in zip(pairs, slow)]
        gain = 1.0 + 0.1 * math.log(FACTOR)
    elif c["scaling"] == "waves":
        kept = [min(1.0, max(0.0, (TRAINED * f / (2.0 * math.pi) - LOW) / (HIGH - LOW))) for f in pairs]
        pairs = [f * (r + (1.0 - r) / FACTOR) for f, r in zip(pairs, kept)]
    angle = s["positions"].double()[:, None] * torch.tensor(pairs, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, gain), angle)[:, None]
    q, k, v = _packed(s)
    got = []
    for x, w in ((q, "wq"), (k, "wk")):
        y = x.double()
        if c["norm"]:
            y = y * (y.square().sum(-1, keepdim=True) / DIM + EPS).rsqrt() * s[w].double()
        head = y[..., :R]
        if c["layout"] == "half":
            z = torch.complex(head[..., :R // 2], head[..., R // 2:]) * turn
            z = torch.cat((z.real, z.imag), -1)
        else:
            z = torch.view_as_real(torch.view_as_complex(head.reshape(*head.shape[:-1], R // 2, 2).contiguous()) * turn).flatten(-2)
        got.append(torch.cat((z, y[..., R:]), -1))
    caches = []
    for x in (got[1], v.double()):
        cache = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
        cache[s["slots"] // BLOCK, :, s["slots"] % BLOCK] = x if c["kv"] == "bf16" else (x / KV_SCALE).clamp(-448, 448)
        caches.append(cache)
    return got[0], caches[0], caches[1]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "rope": _exact_rope}[case["op"]](s)

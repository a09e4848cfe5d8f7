"""Cases that measure the windowed-session operators of the quantised, paged KV cache.

Three families, as one decode session with a bounded window uses them:

* attention with a sliding window and a few first tokens that stay visible
  (sinks) over the paged cache, for the step's queries ("decode") and for a
  chunk of a prompt ("prefill");
* rotary positions with several axes applied to a step's queries and keys on
  their way into the quantised cache ("rotary");
* the pages themselves: a step's new pages and the pages that left the window
  ("turn"), forking sequences ("fork") and compacting the pool ("compact").

With ``own`` false, run() computes plain torch; with ``own`` true it makes the
calls a user makes of ``long_context_quantized_b200``.
"""
import math

import torch

own = False

BLOCK = 256
DIM = 128
#: bytes of one token of one kv-head in the pool
TOKEN_BYTES = {"k8v4": 202, "k8v8": 260, "f8": 260, "k4v4": 136, "bf16": 512}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request at the longest context, a short window: a launch's latency
        {"name": "decode: 1k window, one request", "op": "decode", "fmt": "k8v4", "batch": 1, "lo": 262144, "hi": 262144,
         "hq": 40, "hkv": 8, "n_q": 1, "window": 1024, "sinks": 4},
        # the two concurrent requests of the ragged workload
        {"name": "decode: 4k window, two requests", "op": "decode", "fmt": "k8v4", "batch": 2, "lo": 65536, "hi": 90112,
         "hq": 32, "hkv": 4, "n_q": 1, "window": 4096, "sinks": 4},
        # a serving batch, short sequences (down to one token) among long ones
        {"name": "decode: 4k window, 64 requests", "op": "decode", "fmt": "k8v4", "batch": 64, "lo": 1, "hi": 32769,
         "hq": 32, "hkv": 4, "n_q": 1, "window": 4096, "sinks": 64},
        # draft verification: four queries with their own windows, int8 cache
        {"name": "decode: 32k window, four drafts", "op": "decode", "fmt": "k8v8", "batch": 1, "lo": 180228, "hi": 180228,
         "hq": 32, "hkv": 4, "n_q": 4, "window": 32768, "sinks": 128},
        # the last 1024-token chunk of a long prompt
        {"name": "prefill: chunk of 1024, 4k window", "op": "prefill", "fmt": "k8v4", "batch": 1, "lo": 180224, "hi": 180224,
         "hq": 32, "hkv": 4, "n_q": 1024, "window": 4096, "sinks": 64},
        # a whole prompt at once, from its first token
        {"name": "prefill: prompt of 8192, 2k window", "op": "prefill", "fmt": "k8v4", "batch": 1, "lo": 8192, "hi": 8192,
         "hq": 32, "hkv": 4, "n_q": 8192, "window": 2048, "sinks": 4},
        # a decode step of two requests: latency
        {"name": "rotary: one token, two requests", "op": "rotary", "fmt": "k8v4", "dtype": "bf16", "batch": 2, "n_new": 1,
         "hq": 32, "hkv": 4, "rot": 128, "axes": 3, "pairs": False, "far": 180224},
        # a prompt chunk of text and image tokens
        {"name": "rotary: chunk of 1024", "op": "rotary", "fmt": "k8v4", "dtype": "bf16", "batch": 1, "n_new": 1024,
         "hq": 32, "hkv": 4, "rot": 128, "axes": 3, "pairs": False, "far": 179200},
        # a long video prompt at once, int8 cache
        {"name": "rotary: 16k video tokens", "op": "rotary", "fmt": "k8v8", "dtype": "bf16", "batch": 1, "n_new": 16384,
         "hq": 40, "hkv": 8, "rot": 128, "axes": 3, "pairs": False, "far": 1000},
        # the pages of a decode step: one new token a row, the pages that left the window
        {"name": "pages: turn of 64 requests", "op": "turn", "rows": 64, "lo": 4096, "hi": 32768, "window": 4096, "sinks": 4,
         "blocks": 8192},
        # sampling eight continuations of each of four prompts
        {"name": "pages: fork 4 into 32", "op": "fork", "fmt": "k8v4", "layers": 16, "hkv": 4, "parents": 4, "children": 32,
         "lo": 5000, "hi": 45003, "blocks": 720},
        # the fragmented pool packed to its front
        {"name": "pages: compact 180 of 720", "op": "compact", "fmt": "k8v4", "layers": 16, "hkv": 4, "rows": 8, "live": 400,
         "moves": 180, "blocks": 720},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "rotary", "rotary", "turn", "fork", "compact"])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "decode":
        batch = _log(rng, 1, 64)
        group = rng.choice([1, 4, 5, 8])
        hi = _log(rng, 64, 262144 // (1 + batch // 8))
        return {"op": op, "fmt": rng.choice(["k8v4", "k8v8", "f8", "k4v4", "bf16"]), "batch": batch,
                "lo": max(4, hi // rng.choice([1, 2, 9])), "hi": hi, "hq": hkv * group, "hkv": hkv, "n_q": rng.choice([1, 1, 2, 4]),
                "window": _log(rng, 16, 32768 if batch <= 4 else 8192), "sinks": rng.choice([0, 1, 4, 37, 128, 300])}
    if op == "prefill":
        n_q = _log(rng, 16, 2048)
        batch = rng.choice([1, 1, 2, 3])
        hi = n_q + rng.choice([0, _log(rng, 1, 60000)])
        return {"op": op, "fmt": "k8v4", "batch": batch, "lo": max(n_q, hi - rng.randrange(1, 700)), "hi": hi,
                "hq": hkv * rng.choice([1, 4, 8]), "hkv": hkv, "n_q": n_q, "window": _log(rng, 16, 8192),
                "sinks": rng.choice([0, 4, 65, 128])}
    if op == "rotary":
        n_new = _log(rng, 1, 8192)
        return {"op": op, "fmt": rng.choice(["k8v4", "k8v8", "f8", "k4v4", "bf16"]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "batch": rng.choice([1, 2, 5]) if n_new < 3000 else 1, "n_new": n_new, "hq": hkv * rng.choice([1, 4, 5]), "hkv": hkv,
                "rot": rng.choice([128, 128, 64, 32, 96]), "axes": rng.choice([1, 2, 3, 4]), "pairs": rng.random() < 0.4,
                "far": _log(rng, 1, 260000)}
    if op == "turn":
        rows = _log(rng, 1, 200)
        hi = _log(rng, 300, 60000)
        return {"op": op, "rows": rows, "lo": max(1, hi // 3), "hi": hi, "window": _log(rng, 16, 16384),
                "sinks": rng.choice([0, 4, 300]), "blocks": rows * (hi // BLOCK + 2) + rng.randrange(1, 500)}
    layers = rng.choice([1, 3, 8])
    fmt = rng.choice(["k8v4", "k8v8", "f8", "k4v4", "bf16"])
    if op == "fork":
        parents = rng.choice([1, 2, 5])
        hi = _log(rng, 20, 12000)
        children = parents * rng.choice([1, 3, 6])
        return {"op": op, "fmt": fmt, "layers": layers, "hkv": hkv, "parents": parents, "children": children,
                "lo": max(1, hi // 2), "hi": hi, "blocks": parents * (hi // BLOCK + 1) + children + rng.randrange(1, 40)}
    blocks = rng.randrange(40, 500)
    live = rng.randrange(10, blocks - 8)
    return {"op": op, "fmt": fmt, "layers": layers, "hkv": hkv, "rows": rng.randrange(1, 9), "live": live,
            "moves": rng.randrange(1, min(live, blocks - live) + 1), "blocks": blocks}


def _lengths(c, rows):
    """Lengths from lo to hi in a scattered order, the same for every seed."""
    step = max(1, rows - 1)
    return [c["lo"] + (c["hi"] - c["lo"]) * (b * 37 % rows if rows % 37 else b) // step for b in range(rows)] if rows > 1 else [c["hi"]]


# ------------------------------------------------------------------ inputs
def _f16(x):
    """fp32 -> fp16, saturated."""
    return x.clamp(max=65504.0).half()


def _scale(amax, top):
    """The format's fp16 scale: the fp32 quotient (by way of 64 bits, which rounds the same), then fp16."""
    return _f16((amax.double() / top).float())


def _divide(x, s):
    """fp32 x / s with 0 where s is 0 (by way of 64 bits, which rounds the same)."""
    return torch.where(s == 0, torch.zeros_like(x), (x.double() / s.double()).float())


def _nibbles(codes):
    c = codes.to(torch.int32) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _quantise8(x):
    s = _scale(x.abs().amax(-1), 127.0)
    return _divide(x, s.float()[..., None]).round().clamp(-127, 127).to(torch.int8), s


def _quantise_f8(x):
    s = _scale(x.abs().amax(-1), 448.0)
    return _divide(x, s.float()[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _quantise4(x):
    g = x.reshape(*x.shape[:-1], DIM // 32, 32)
    s = _scale(g.abs().amax(-1), 7.0)
    return _nibbles(_divide(g, s.float()[..., None]).round().clamp(-7, 7).reshape(x.shape)), s


def _quantise_e8(x):
    g = x.reshape(*x.shape[:-1], DIM // 32, 32)
    m, e = torch.frexp((g.abs().amax(-1).double() / 7.0).float())
    e = torch.where(m == 0, torch.full_like(e, -126), torch.where(m == 0.5, e - 1, e)).clamp(-126, 127)
    codes = (g.double() / torch.exp2(e.double())[..., None]).float().round().clamp(-7, 7)
    return _nibbles(codes.reshape(x.shape)), (e + 127).to(torch.uint8)


def _quantise(fmt, k, v):
    """Rows [..., 128] in fp32 -> the pool's codes and scales of K and of V."""
    if fmt == "bf16":
        return k.bfloat16(), None, v.bfloat16(), None
    pair = {"k8v4": (_quantise8, _quantise4), "k8v8": (_quantise8, _quantise8), "f8": (_quantise_f8, _quantise_f8),
            "k4v4": (_quantise_e8, _quantise_e8)}[fmt]
    kc, ks = pair[0](k)
    vc, vs = pair[1](v)
    return kc, ks, vc, vs


PLANES = ("k_codes", "k_scales", "v_codes", "v_scales")


def _pool(fmt, blocks, hkv, gen, layers=None):
    """Pool planes filled with quantised normal values, 256 tokens a block (with a layer axis if asked)."""
    n = blocks * (layers or 1)
    parts = []
    for at in range(0, n, 256):
        m = min(256, n - at)
        k, v = (torch.randn((m, hkv, BLOCK, DIM), generator=gen, device="cuda") for _ in range(2))
        parts.append(_quantise(fmt, k, v))
    planes = {}
    for name, columns in zip(PLANES, zip(*parts)):
        if columns[0] is not None:
            t = torch.cat(columns)
            planes[name] = t.reshape(layers, blocks, *t.shape[1:]) if layers else t
    return planes


def _table(lengths, blocks, width, gen):
    """Each row's pages, a shuffled choice of the pool's; -1 behind them."""
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lengths):
        m = -(-n // BLOCK)
        table[b, :m] = order[at:at + m]
        at += m
    return table, order[:at]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * (seed + 1))
    s = {"case": c}
    if c["op"] in ("decode", "prefill"):
        lengths = [max(n, c["n_q"]) for n in _lengths(c, c["batch"])]
        width = max(-(-n // BLOCK) for n in lengths)
        blocks = sum(-(-n // BLOCK) for n in lengths)
        s["planes"] = _pool(c["fmt"], blocks, c["hkv"], gen)
        s["table"], _ = _table(lengths, blocks, width, gen)
        s["lens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        s["max_len"] = max(lengths)
        s["q"] = torch.randn((c["batch"], c["n_q"], c["hq"], DIM), generator=gen, device="cuda").bfloat16()
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "rotary":
        pages = -(-(c["n_new"] + 100) // BLOCK) + 1
        s["planes"] = _pool(c["fmt"], pages * c["batch"], c["hkv"], gen)
        s["table"], _ = _table([pages * BLOCK] * c["batch"], pages * c["batch"], pages, gen)
        # rows start inside a page; their rotary positions start at the far context
        s["before"] = torch.randint(0, 100, (c["batch"],), generator=gen, device="cuda", dtype=torch.int32)
        n = torch.arange(c["n_new"], device="cuda", dtype=torch.int32)
        grid = torch.stack([n // 64, n // 8 % 8, n % 8, n], dim=-1)[:, :c["axes"]] if c["axes"] > 1 else n[:, None]
        s["positions"] = (c["far"] + s["before"][:, None, None] + grid[None]).contiguous()
        half = c["rot"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        s["axis"] = [min(i * c["axes"] // half, c["axes"] - 1) for i in range(half)]
        s["axis_at"] = torch.tensor(s["axis"], device="cuda")
        # the heads of a fused projection's output: q, k and v are strided views
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        qkv = torch.randn((c["batch"], c["n_new"], c["hq"] + 2 * c["hkv"], DIM), generator=gen, device="cuda").to(dtype)
        s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=2)
        s["q_out"] = torch.empty((c["batch"], c["n_new"], c["hq"], DIM), dtype=dtype, device="cuda")
    elif c["op"] == "turn":
        # every fourth row is about to begin a page
        lengths = [max(1, n // BLOCK * BLOCK if b % 4 == 0 else n) for b, n in enumerate(_lengths(c, c["rows"]))]
        width = max(lengths) // BLOCK + 2
        s["table0"], _ = _table(lengths, c["blocks"], width, gen)
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        ahead = torch.randint(0, 300, (c["rows"],), generator=gen, device="cuda", dtype=torch.int32)
        s["from_new"], s["to_new"] = lens, lens + 1
        s["from_old"], s["to_old"] = torch.full_like(lens, c["sinks"]), (lens + 1 - c["window"]).clamp(min=0)
        # what left the window in earlier steps is gone already
        page = torch.arange(width, device="cuda")[None]
        gone = (page * BLOCK >= c["sinks"]) & ((page + 1) * BLOCK <= (s["to_old"] - ahead)[:, None])
        s["table0"].masked_fill_(gone, -1)
        s["refs0"] = torch.zeros(c["blocks"], dtype=torch.int32, device="cuda")
        s["refs0"][s["table0"][s["table0"] >= 0].long()] = 1
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
    elif c["op"] == "fork":
        lengths = _lengths(c, c["parents"])
        rows = c["parents"] + c["children"]
        s["planes"] = _pool(c["fmt"], c["blocks"], c["hkv"], gen, c["layers"])
        s["table0"], _ = _table(lengths + [0] * c["children"], c["blocks"], max(lengths) // BLOCK + 2, gen)
        s["refs0"] = torch.zeros(c["blocks"], dtype=torch.int32, device="cuda")
        s["refs0"][s["table0"][s["table0"] >= 0].long()] = 1
        s["lens0"] = torch.tensor(lengths + [0] * c["children"], dtype=torch.int32, device="cuda")
        s["src"] = (torch.arange(c["children"], device="cuda") % c["parents"]).to(torch.int32)
        s["dst"] = torch.arange(c["parents"], rows, device="cuda", dtype=torch.int32)
        s["table"], s["refs"], s["lens"] = s["table0"].clone(), s["refs0"].clone(), s["lens0"].clone()
    else:
        s["planes"] = _pool(c["fmt"], c["blocks"], c["hkv"], gen, c["layers"])
        # `live` pages, `moves` of them behind the first `live`
        low = torch.randperm(c["live"], generator=gen, device="cuda")[:c["live"] - c["moves"]]
        high = c["live"] + torch.randperm(c["blocks"] - c["live"], generator=gen, device="cuda")[:c["moves"]]
        ids = torch.cat([low, high])
        ids = ids[torch.randperm(c["live"], generator=gen, device="cuda")].to(torch.int32)
        width = -(-c["live"] // c["rows"]) + 3
        s["table0"] = torch.full((c["rows"], width), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(c["live"], device="cuda")
        s["table0"][at % c["rows"], at // c["rows"]] = ids
        s["refs0"] = torch.zeros(c["blocks"], dtype=torch.int32, device="cuda")
        s["refs0"][ids.long()] = 1
        # some first pages are shared by the next row
        shared = torch.arange(c["rows"], device="cuda")
        s["table0"][shared, width - 1] = s["table0"][(shared + 1) % c["rows"], 0]
        s["refs0"].index_add_(0, s["table0"][:, width - 1].clamp(min=0).long(), (s["table0"][:, width - 1] >= 0).int())
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the framework keeps: the layers' views, the rotary plan, the workspaces."""
    import long_context_quantized_b200 as nf
    c = s["case"]
    if "planes" in s:
        fmt = {"k8v4": nf.NF_KV_K8V4, "k8v8": nf.NF_KV_K8V8, "f8": nf.NF_KV_F8, "k4v4": nf.NF_KV_K4V4, "bf16": nf.NF_KV_BF16}[c["fmt"]]
        if "layers" in c:
            s["layers"] = nf.KVLayers([nf.KVLayer(fmt, *[s["planes"][n][i] if n in s["planes"] else None for n in PLANES])
                                       for i in range(c["layers"])])
        else:
            s["kv"] = nf.KVLayer(fmt, *[s["planes"].get(n) for n in PLANES])
    if c["op"] == "decode":
        s["workspace"] = torch.zeros(nf.nf_decode_attn_window_workspace_size(c["batch"], c["n_q"], c["hq"], c["hkv"], s["max_len"]),
                                     dtype=torch.uint8, device="cuda")
    elif c["op"] == "rotary":
        s["rope"] = nf.Rope(s["inv_freq"], s["axis"], c["axes"], layout=nf.NF_ROPE_PAIRS if c["pairs"] else nf.NF_ROPE_HALVES)
    elif c["op"] in ("fork", "compact"):
        s["workspace"] = torch.zeros(nf.nf_kv_pages_workspace_size(c["blocks"], c.get("children", 0)), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass
def run(state):
    return {"decode": _attend, "prefill": _attend, "rotary": _rotary, "turn": _turn, "fork": _fork, "compact": _compact}[
        state["case"]["op"]](state)


def _signed(nib):
    return nib - 16 * (nib > 7)


def _open4(codes):
    """Nibble bytes [..., 64] -> codes [..., 128] in fp32."""
    w = codes.to(torch.int32)
    return torch.stack([_signed(w & 15), _signed(w >> 4)], dim=-1).reshape(*codes.shape[:-1], DIM).float()


def _values(fmt, codes, scales, is_k):
    """The fp32 values that codes and scales stand for."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "f8":
        return codes.view(torch.float8_e4m3fn).float() * scales.float()[..., None]
    if fmt == "k4v4":
        return _open4(codes) * torch.exp2(scales.float() - 127.0).repeat_interleave(32, dim=-1)
    if fmt == "k8v8" or is_k:
        return codes.float() * scales.float()[..., None]
    return _open4(codes) * scales.float().repeat_interleave(32, dim=-1)


def _attend(s):
    c = s["case"]
    if own:
        import long_context_quantized_b200 as nf
        if c["op"] == "decode":
            nf.nf_decode_attn_window(s["kv"], s["q"], s["table"], s["lens"], s["max_len"], c["window"], c["sinks"], DIM ** -0.5,
                                     s["out"], None, s["workspace"])
        else:
            nf.nf_prefill_attn_window(s["kv"], s["q"], s["table"], s["lens"], s["max_len"], c["window"], c["sinks"], DIM ** -0.5,
                                      s["out"])
        return s["out"]
    n_q, hkv = c["n_q"], c["hkv"]
    lens = s["lens"].long()
    # the positions that some query may see: the last ones, and before them the sinks
    last = min(c["window"] + n_q - 1, s["max_len"])
    recent = lens[:, None] - last + torch.arange(last, device="cuda")
    first = torch.arange(min(c["sinks"], s["max_len"]), device="cuda")[None].expand(c["batch"], -1)
    pos = torch.cat([first, recent], dim=1)
    there = torch.cat([first < recent[:, :1], recent >= 0], dim=1)
    at = (lens[:, None] - n_q + torch.arange(n_q, device="cuda"))[:, :, None]
    seen = there[:, None] & (pos[:, None] <= at) & ((pos[:, None] > at - c["window"]) | (pos[:, None] < c["sinks"]))
    pos = pos.clamp(min=0)
    block = torch.gather(s["table"].long(), 1, pos // BLOCK).clamp(min=0)[:, :, None]
    slot, head = (pos % BLOCK)[:, :, None], torch.arange(hkv, device="cuda")
    p = s["planes"]
    take = lambda name: p[name][block, head, slot] if name in p else None  # noqa: E731
    k = _values(c["fmt"], take("k_codes"), take("k_scales"), True)
    v = _values(c["fmt"], take("v_codes"), take("v_scales"), False)
    q = s["q"].float().reshape(c["batch"], n_q, hkv, c["hq"] // hkv, DIM)
    scores = torch.einsum("bjhgd,bnhd->bhgjn", q, k) * DIM ** -0.5
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = w.sum(-1)
    o = torch.einsum("bhgjn,bnhd->bjhgd", w, v)
    total = total.permute(0, 3, 1, 2)[..., None]
    o = torch.where(total > 0, o / total.clamp(min=1e-30), torch.zeros_like(o))
    return o.reshape(c["batch"], n_q, c["hq"], DIM).bfloat16()


def _turned(x, cos, sin, rot, pairs):
    """The rows x [..., heads, 128] in 64 bits, their first `rot` channels turned."""
    x = x.double()
    half = rot // 2
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _rotary(s):
    c = s["case"]
    if own:
        import long_context_quantized_b200 as nf
        nf.nf_rope_append_quant(s["kv"], s["rope"], s["positions"], s["q"], s["k"], s["v"], s["table"], s["before"], s["q_out"])
        return [s["q_out"]] + [s["planes"][n] for n in PLANES if n in s["planes"]]
    # far angles, and codes next to a border: 64 bits up to the rotated values
    angle = (s["positions"][..., s["axis_at"]].double() * s["inv_freq"].double())[:, :, None]
    cos, sin = torch.cos(angle), torch.sin(angle)
    q = _turned(s["q"], cos, sin, c["rot"], c["pairs"]).to(s["q"].dtype)
    k = _turned(s["k"], cos, sin, c["rot"], c["pairs"]).float()
    new = dict(zip(PLANES, _quantise(c["fmt"], k, s["v"].float())))
    pos = s["before"].long()[:, None] + torch.arange(c["n_new"], device="cuda")
    block = torch.gather(s["table"].long(), 1, pos // BLOCK)[:, :, None]
    at = (block, torch.arange(c["hkv"], device="cuda"), (pos % BLOCK)[:, :, None])
    return [q] + [s["planes"][n].index_put_(at, new[n]) for n in PLANES if n in s["planes"]]


def _turn(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    table, refs = s["table"], s["refs"]
    if own:
        import long_context_quantized_b200 as nf
        nf.nf_kv_reserve(refs, table, s["from_new"], s["to_new"])
        nf.nf_kv_release(refs, table, s["from_old"], s["to_old"])
        return [table, refs]
    page = torch.arange(table.shape[1], device="cuda")[None]
    # the rows' new pages: the lowest free ones, row by row
    want = (page >= s["from_new"][:, None] // BLOCK) & (page * BLOCK < s["to_new"][:, None]) & (table < 0)
    free = torch.nonzero(refs == 0)[:, 0]
    rank = (torch.cumsum(want.flatten(), 0) - 1).reshape(want.shape).clamp(min=0, max=max(0, free.numel() - 1))
    table = torch.where(want, free[rank].int(), table)
    refs = refs + torch.bincount(table[want].long(), minlength=refs.numel()).int()
    # the pages that left the window
    gone = (page * BLOCK >= s["from_old"][:, None]) & ((page + 1) * BLOCK <= s["to_old"][:, None]) & (table >= 0)
    refs = refs - torch.bincount(table[gone].long(), minlength=refs.numel()).int()
    return [table.masked_fill(gone, -1), refs]


def _fork(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    s["lens"].copy_(s["lens0"])
    table, refs, lens = s["table"], s["refs"], s["lens"]
    p = s["planes"]
    if own:
        import long_context_quantized_b200 as nf
        nf.nf_kv_fork(s["layers"], refs, table, s["src"], s["dst"], lens, s["workspace"])
        return [table, refs, lens] + [p[n] for n in PLANES if n in p]
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src].long()
    page = torch.arange(table.shape[1], device="cuda")[None]
    rows = torch.where(page < (n // BLOCK)[:, None], table[src], torch.full_like(table[src], -1))
    # full pages are shared; a page that the parent still writes is copied to the lowest free ones
    cut = n % BLOCK != 0
    fresh = torch.nonzero(refs == 0)[:, 0][(torch.cumsum(cut, 0) - 1).clamp(min=0)]
    tail = table[src].gather(1, (n // BLOCK)[:, None])[:, 0].long()
    refs = refs + torch.bincount(rows[rows >= 0].long(), minlength=refs.numel()).int()
    refs = refs + torch.bincount(fresh[cut], minlength=refs.numel()).int()
    rows = torch.where((page == (n // BLOCK)[:, None]) & cut[:, None], fresh[:, None].int(), rows)
    table = table.index_copy(0, dst, rows)
    lens = lens.index_copy(0, dst, lens[src])
    return [table, refs, lens] + [p[n_].index_copy_(1, fresh[cut], p[n_][:, tail[cut]]) for n_ in PLANES if n_ in p]


def _compact(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    table, refs = s["table"], s["refs"]
    p = s["planes"]
    if own:
        import long_context_quantized_b200 as nf
        nf.nf_kv_compact(s["layers"], refs, table, s["workspace"])
        return [table, refs] + [p[n] for n in PLANES if n in p]
    used = refs > 0
    live = used.sum()
    ids = torch.arange(refs.numel(), device="cuda")
    src, dst = torch.nonzero(used & (ids >= live))[:, 0], torch.nonzero(~used & (ids < live))[:, 0]
    to = ids.index_copy(0, src, dst)
    refs = refs.index_copy(0, dst, refs[src]).index_fill(0, src, 0)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
    return [table, refs] + [p[n].index_copy_(1, dst, p[n][:, src]) for n in PLANES if n in p]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] in ("decode", "prefill"):
        read = flops = 0
        for n in (max(n, c["n_q"]) for n in _lengths(c, c["batch"])):
            start = max(0, n - c["n_q"] - c["window"] + 1)
            read += (n - start + min(c["sinks"], start)) * c["hkv"] * TOKEN_BYTES[c["fmt"]]
            for j in range(c["n_q"]):
                at = n - c["n_q"] + j
                begin = max(0, at - c["window"] + 1)
                flops += (at + 1 - begin + min(c["sinks"], begin)) * c["hq"] * DIM * 4
        return {"bytes": read + 2 * c["batch"] * c["n_q"] * c["hq"] * DIM * 2, "flops": flops}
    if c["op"] == "rotary":
        rows, size = c["batch"] * c["n_new"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": rows * ((2 * c["hq"] + 2 * c["hkv"]) * DIM * size + c["hkv"] * TOKEN_BYTES[c["fmt"]] + 4 * c["axes"]),
                "flops": rows * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    if c["op"] == "turn":
        width = max(_lengths(c, c["rows"])) // BLOCK + 2
        # the table and the counts restored and gone through once
        return {"bytes": (c["rows"] * width * 3 + c["blocks"] * 3) * 4, "flops": 0}
    page = BLOCK * c["hkv"] * TOKEN_BYTES[c["fmt"]] * c["layers"]
    if c["op"] == "fork":
        cut = sum(_lengths(c, c["parents"])[i % c["parents"]] % BLOCK != 0 for i in range(c["children"]))
        width = max(_lengths(c, c["parents"])) // BLOCK + 2
        return {"bytes": 2 * cut * page + (c["parents"] + c["children"]) * width * 3 * 4 + c["blocks"] * 12, "flops": 0}
    return {"bytes": 2 * c["moves"] * page + c["blocks"] * 12 + (c["live"] + 4 * c["rows"]) * 12, "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_nibbles(b):
    b = b.to(torch.int64)
    lo, hi = b % 16, b // 16
    both = torch.stack((lo, hi), -1).flatten(-2)
    return torch.where(both >= 8, both - 16, both).double()


def _exact_rows(fmt, codes, scales, k):
    if fmt == "bf16":
        return codes.double()
    if fmt == "k4v4":
        return (_exact_nibbles(codes).unflatten(-1, (4, 32)) * torch.pow(2.0, scales.double() - 127)[..., None]).flatten(-2)
    if fmt == "k8v4" and not k:
        return (_exact_nibbles(codes).unflatten(-1, (4, 32)) * scales.double()[..., None]).flatten(-2)
    if fmt == "f8":
        codes = codes.view(torch.float8_e4m3fn)
    return codes.double() * scales.double()[..., None]


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] in ("decode", "prefill"):
        # every query against every key of its sequence, under the mask
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        group = c["hq"] // c["hkv"]
        for b, length in enumerate(s["lens"].tolist()):
            ids = s["table"][b, : -(-length // BLOCK)].long()
            t = torch.arange(length, device="cuda")
            for h in range(c["hkv"]):
                rows = {n: s["planes"][n][ids, h].flatten(0, 1)[:length] if n in s["planes"] else None for n in PLANES}
                k = _exact_rows(c["fmt"], rows["k_codes"], rows["k_scales"], True)
                v = _exact_rows(c["fmt"], rows["v_codes"], rows["v_scales"], False)
                for j0 in range(0, c["n_q"], 512):
                    j = torch.arange(j0, min(j0 + 512, c["n_q"]), device="cuda")
                    at = (length - c["n_q"] + j)[:, None]
                    hidden = (t > at) | ((t <= at - c["window"]) & (t >= c["sinks"]))
                    for g in range(h * group, (h + 1) * group):
                        x = s["q"][b, j, g].double() @ k.T / math.sqrt(DIM)
                        out[b, j, g] = torch.softmax(x.masked_fill_(hidden, -math.inf), -1) @ v
        return out
    if c["op"] == "rotary":
        pos = s["positions"].double()[..., s["axis_at"]]
        z = torch.polar(torch.ones_like(pos), pos * s["inv_freq"].double())[:, :, None]

        def turn(x):
            x = x.double().clone()
            part = x[..., :c["rot"]]
            part = part.unflatten(-1, (-1, 2)) if c["pairs"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z)
            x[..., :c["rot"]] = (y if c["pairs"] else y.transpose(-1, -2)).flatten(-2)
            return x

        k, v = turn(s["k"]), s["v"].double()
        planes = {n: t.double() for n, t in s["planes"].items() if t.dtype == torch.float16 or c["fmt"] == "bf16"}
        if c["fmt"] == "bf16":
            new = {"k_codes": k, "v_codes": v}
        elif c["fmt"] == "k4v4":
            new = {}
        else:
            top = 448.0 if c["fmt"] == "f8" else 127.0
            new = {"k_scales": k.abs().amax(-1) / top,
                   "v_scales": v.unflatten(-1, (4, 32)).abs().amax(-1) / 7.0 if c["fmt"] == "k8v4" else v.abs().amax(-1) / top}
        for b, before in enumerate(s["before"].tolist()):
            for name, x in new.items():
                for i0 in range(0, c["n_new"], BLOCK):
                    at = before + torch.arange(i0, min(i0 + BLOCK, c["n_new"]), device="cuda")
                    planes[name][s["table"][b, at // BLOCK].long(), :, at % BLOCK] = x[b, i0:i0 + BLOCK]
        return [turn(s["q"])] + [planes.get(n) for n in PLANES if n in s["planes"]]
    return None

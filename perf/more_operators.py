"""Cases for what the paged 4-bit cache needs around decoding: rotary positions with several
axes (alone, and within the append), attention of prompts and chunks over the pages,
attention weights accumulated per cached token, and the eviction that goes by them.

``run`` computes an operator in elementary torch operations (``own`` false) or through
the package's calls (``own`` true); ``exact`` gives the same outputs from the definitions
in 64 bits.

A page holds 64 tokens of one KV head: 4-bit codes of the keys and of the values, and per
token and 32-channel group a binary16 scale and offset, x ~ offset + scale * code.  The
keys and the values of even slots count up from the group's minimum; the values of odd
slots count down from its maximum (negative scale).
"""

import math
import random

import torch

own = False

_DEV = torch.device("cuda" if torch.cuda.is_available() else "cpu")
_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
PAGE = 64
GROUP = 32


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------

def listed():
    plain = dict(base=1000000.0, scaling="none", factor=1.0, original_ctx=0, low=1.0, high=32.0)
    parts = dict(base=500000.0, scaling="parts", factor=8.0, original_ctx=8192, low=1.0, high=4.0)
    own10k = dict(base=10000.0, scaling="none", factor=1.0, original_ctx=0, low=1.0, high=32.0)
    return [
        # q and k heads of a 32K-token video prompt (time, height, width in blocks of pairs): memory bandwidth
        dict(name="rope_video_32k", op="rope", T=32768, H=40, D=128, axes="16,24,24", order="blocks", freq="shared",
             layout="half", dtype="fp16", max_pos=32768, **plain),
        # an image's patches, each axis with frequencies of its own, interleaved pairs, odd counts
        dict(name="rope_image_own_bf16", op="rope", T=4099, H=13, D=128, axes="8,28,28", order="blocks", freq="own",
             layout="interleaved", dtype="bf16", max_pos=4096, **own10k),
        # one token per sequence of a batch of 64 (a few of them padding), q turned along: latency
        dict(name="append_axes_decode_64", op="append", T=64, Hq=32, Hkv=8, D=128, axes="24,20,20", order="cycled",
             freq="shared", layout="half", dtype="fp16", max_pos=131072, pad=7, **plain),
        # a 16K-token video prompt's keys and values into pages, q turned along: memory bandwidth
        dict(name="append_axes_prompt_16k", op="append", T=16384, Hq=32, Hkv=8, D=128, axes="16,24,24", order="blocks",
             freq="shared", layout="half", dtype="bf16", max_pos=16384, pad=0, **parts),
        # 64 new tokens (a turn of a conversation) over a 4K-token cache: latency
        dict(name="prefill_turn_64", op="prefill", B=1, chunk=64, max_len=4096, ragged=False, Hq=32, Hkv=8, D=128,
             causal=True, window=0, dtype="fp16"),
        # a whole prompt of 8K tokens: tensor cores, causal
        dict(name="prefill_prompt_8k", op="prefill", B=1, chunk=8192, max_len=8192, ragged=False, Hq=32, Hkv=8, D=128,
             causal=True, window=0, dtype="bf16"),
        # the last 2K tokens of a 32K prompt that is processed in chunks: tensor cores, long cache
        dict(name="prefill_chunk_2k_32k", op="prefill", B=1, chunk=2048, max_len=32768, ragged=False, Hq=32, Hkv=8, D=128,
             causal=True, window=0, dtype="bf16"),
        # a serving batch of unequal chunks (empty ones and single tokens among them) over unequal caches,
        # sliding-window layers of small heads, eight query heads to a KV head
        dict(name="prefill_ragged_d64", op="prefill", B=12, chunk=1021, max_len=9001, ragged=True, Hq=24, Hkv=3, D=64,
             causal=True, window=4096, dtype="bf16"),
        # weights accumulated at every decoding step of 64 sequences from empty to 16K tokens
        dict(name="weights_decode_64", op="weights", B=64, Q=1, Hq=32, Hkv=8, D=128, max_len=16384, ragged=True, window=0,
             decay=0.95, dtype="bf16"),
        # the last 32 tokens of a 128K prompt say what the cache keeps of it: arithmetic
        dict(name="weights_window_128k", op="weights", B=1, Q=32, Hq=32, Hkv=8, D=128, max_len=131072, ragged=False,
             window=0, decay=0.0, dtype="fp16"),
        # caches of four sequences back to 1000 tokens during decoding: latency
        dict(name="evict_step_4", op="evict", B=4, Hkv=8, D=128, max_len=1100, ragged=False, keep=1000, first=4, recent=128,
             dtype="fp16"),
        # a 128K prompt cut to its 16K heaviest tokens per KV head: selection over long rows, then bandwidth
        dict(name="evict_prompt_128k", op="evict", B=1, Hkv=8, D=128, max_len=131072, ragged=False, keep=16384, first=16,
             recent=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _draw_axes(rng, D):
    n = rng.choice([2, 3, 3, 4])
    pairs = rng.choice([D // 2, D // 2, rng.randint(2 * n, D // 2)])
    cuts = sorted(rng.sample(range(2, pairs - 1), n - 1)) if pairs > 3 * n else []
    axes = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
    if min(axes) < 2 or len(axes) != n:
        axes = [pairs // n] * (n - 1) + [pairs - pairs // n * (n - 1)]
    return dict(axes=",".join(map(str, axes)), order=rng.choice(["blocks", "cycled"]), freq=rng.choice(["shared", "shared", "own"]),
                layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["fp16", "bf16"]),
                base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=rng.choice(["none", "linear", "ntk", "parts", "yarn"]),
                factor=rng.choice([2.0, 4.0, 8.0]), original_ctx=rng.choice([4096, 8192]), low=1.0, high=32.0)


def draw(rng: random.Random):
    op = rng.choice(["rope", "append", "prefill", "prefill", "weights", "evict"])
    D = rng.choice([64, 128, 128])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        H = rng.choice([1, 2, 5, 8, 13, 32, 40])
        return dict(op="rope", T=_log(rng, 1, min(65536, 32768 * 40 * 128 // (H * D))), H=H, D=D, max_pos=_log(rng, 1, 200000),
                    **_draw_axes(rng, D))
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    n_rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if op == "append":
        n_rep = rng.choice([0, n_rep])
        most = 16384 * 48 * 128 // ((n_rep + 2) * Hkv * D)
        return dict(op="append", T=_log(rng, 1, min(32768, most)), Hq=Hkv * n_rep, Hkv=Hkv, D=D, max_pos=_log(rng, 64, 200000),
                    pad=rng.choice([0, 5]), **_draw_axes(rng, D))
    if op == "prefill":
        B, chunk = _log(rng, 1, 16), _log(rng, 1, 8192)
        # (pairs of rows and tokens, padded as the plain form computes them)
        most = 8192 * 8192 * 16 // (B * chunk * Hkv * n_rep)
        n = max(chunk, min(32768, _log(rng, chunk, max(chunk, min(32768, most)))))
        B = max(1, min(B, 8192 * 8192 * 16 // (n * chunk * Hkv * n_rep)))
        chunk = max(1, min(chunk, 8192 * 8192 * 16 // (n * B * Hkv * n_rep)))
        causal = rng.choice([True, True, False])
        return dict(op="prefill", B=B, chunk=chunk, max_len=n, ragged=rng.choice([True, False]), Hq=Hkv * n_rep, Hkv=Hkv, D=D,
                    causal=causal, window=rng.choice([0, 0, 100, 1024]) if causal else 0, dtype=rng.choice(["fp16", "bf16"]))
    if op == "weights":
        B, Q = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 8, 16, 32])
        most = 131072 * 8 * 32 // (B * Hkv * max(Q, 8)) * 4 // max(4, n_rep)
        return dict(op="weights", B=B, Q=Q, Hq=Hkv * n_rep, Hkv=Hkv, D=D, max_len=_log(rng, 1, max(1, min(131072, most))),
                    ragged=rng.choice([True, False]), window=rng.choice([0, 0, 0, 1000]), decay=rng.choice([0.0, 0.9, 1.0]),
                    dtype=rng.choice(["fp16", "bf16"]))
    B = _log(rng, 1, 32)
    n = _log(rng, 2, max(2, min(131072, 131072 * 8 // (B * Hkv))))
    keep = max(1, min(_log(rng, 1, n), 131072 // (B * Hkv)))
    first = rng.choice([0, min(4, keep // 4)])
    return dict(op="evict", B=B, Hkv=Hkv, D=D, max_len=n, ragged=rng.choice([True, False]), keep=keep, first=first,
                recent=rng.choice([0, (keep - first) // 2, min(64, keep - first)]), dtype=rng.choice(["fp16", "bf16"]))


# --------------------------------------------------------------------------------------
# the page layout (64 tokens of one KV head), as index tables
# --------------------------------------------------------------------------------------

def _page_bytes(D):
    return 64 * D + 64 * (D // GROUP) * 8


def _sections(D):
    """Byte offsets of the key codes, value codes, key scales, key offsets, value scales
    and value offsets, and the page's end."""
    c, s = 64 * D // 2, 64 * (D // GROUP) * 2
    return [0, c, 2 * c, 2 * c + s, 2 * c + 2 * s, 2 * c + 3 * s, 2 * c + 4 * s]


def _key_place(D, dev):
    """[64, D] byte (within the key codes) and bit shift of every key code."""
    t = torch.arange(64, device=dev)[:, None]
    c = torch.arange(D, device=dev)[None, :]
    g, a, j = c // 32, (c % 32) // 8, c % 8
    return t * (D // 2) + a * (4 * (D // 32)) + 4 * g + j // 2, (4 * (j % 2)).expand(64, D)


def _value_place(D, dev):
    """[64, D] byte (within the value codes) and bit shift of every value code."""
    t = torch.arange(64, device=dev)[:, None]
    c = torch.arange(D, device=dev)[None, :]
    g, a, j = c // 32, (c % 32) // 4, c % 4
    byte = a * (2 * (D // 32)) + 2 * g + j // 2
    if D == 128:
        row, byte = t ^ ((t >> 1) & 1), byte ^ (32 * ((t >> 2) & 1))
    else:
        row = t ^ ((t >> 2) & 1)
    return row * (D // 2) + byte, (4 * (j % 2)).expand(64, D)


def _value_scale_place(D, dev):
    """[64, D / 32] element (within the value scales or offsets) of every (token, group)."""
    t = torch.arange(64, device=dev)[:, None]
    g = torch.arange(D // 32, device=dev)[None, :]
    return g * 64 + ((t >> 1) & 3) * 16 + (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (t & 1)


def _quantize(x, down):
    """Codes, scale and offset of [..., D] fp32 values in groups of 32 (``down``: counted
    down from the maximum)."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP).clamp(-65504.0, 65504.0)
    lo, hi = g.amin(-1), g.amax(-1)
    off = torch.where(down, hi, lo).half()
    # 64 bits: a scale that binary16 holds exactly must not be pushed up one step
    span = torch.where(down, off.double() - lo.double(), hi.double() - off.double()).clamp_min(0.0) / 15.0
    s = span.half()
    s = torch.where(s.double() < span, (s.view(torch.int16) + 1).view(torch.float16), s)   # rounded up
    d = torch.where(down[..., None], off.float()[..., None] - g, g - off.float()[..., None])
    sf = s.float()[..., None]
    code = torch.where(sf > 0, torch.round(d / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(d))
    return code.clamp(0, 15).to(torch.uint8).reshape(x.shape), torch.where(down, -s, s), off


def _pack(codes, place, shift, n_bytes):
    """[n, 64, D] codes -> [n, n_bytes] bytes."""
    n = codes.shape[0]
    flat, sh = place.reshape(-1), shift.reshape(-1)
    out = torch.zeros(n, n_bytes, dtype=torch.uint8, device=codes.device)
    c = codes.reshape(n, -1)
    low, high = (sh == 0).nonzero()[:, 0], (sh == 4).nonzero()[:, 0]
    out[:, flat[low]] = c[:, low]
    out[:, flat[high]] |= c[:, high] << 4
    return out


def _make_pages(k, v):
    """Pages of [n, 64, D] fp32 keys and values: [n, page bytes] uint8."""
    n, _, D = k.shape
    sec, dev = _sections(D), k.device
    out = torch.empty(n, _page_bytes(D), dtype=torch.uint8, device=dev)
    odd = (torch.arange(64, device=dev) % 2 == 1)[:, None].expand(64, D // GROUP)
    code, s, o = _quantize(k, torch.zeros_like(odd))
    out[:, sec[0]:sec[1]] = _pack(code, *_key_place(D, dev), sec[1])
    out[:, sec[2]:sec[3]] = s.reshape(n, -1).view(torch.uint8)
    out[:, sec[3]:sec[4]] = o.reshape(n, -1).view(torch.uint8)
    code, s, o = _quantize(v, odd)
    at = torch.argsort(_value_scale_place(D, dev).reshape(-1))
    out[:, sec[1]:sec[2]] = _pack(code, *_value_place(D, dev), sec[1])
    out[:, sec[4]:sec[5]] = s.reshape(n, -1)[:, at].contiguous().view(torch.uint8)
    out[:, sec[5]:sec[6]] = o.reshape(n, -1)[:, at].contiguous().view(torch.uint8)
    return out


def _codes(part, place, lead, D):
    at, sh = place
    return ((part[..., at.reshape(-1)] >> sh.reshape(-1).to(torch.uint8)) & 15).reshape(*lead, 64, D // GROUP, GROUP)


def _halves16(raw, a, b):
    return raw[..., a:b].contiguous().view(torch.float16).float()


def _unpack_keys(raw, D):
    """[..., page bytes] -> keys [..., 64, D] in fp32."""
    sec, lead, dev = _sections(D), raw.shape[:-1], raw.device
    ks, ko = (_halves16(raw, sec[i], sec[i + 1]).reshape(*lead, 64, D // GROUP, 1) for i in (2, 3))
    return (_codes(raw[..., sec[0]:sec[1]], _key_place(D, dev), lead, D).float() * ks + ko).reshape(*lead, 64, D)


def _unpack_values(raw, D):
    """[..., page bytes] -> values [..., 64, D] in fp32."""
    sec, lead, dev = _sections(D), raw.shape[:-1], raw.device
    at = _value_scale_place(D, dev).reshape(-1)
    vs, vo = (_halves16(raw, sec[i], sec[i + 1])[..., at].reshape(*lead, 64, D // GROUP, 1) for i in (4, 5))
    return (_codes(raw[..., sec[1]:sec[2]], _value_place(D, dev), lead, D).float() * vs + vo).reshape(*lead, 64, D)


# --------------------------------------------------------------------------------------
# rotary positions with several axes
# --------------------------------------------------------------------------------------

def _axes(case):
    """Pairs of each axis."""
    return [int(n) for n in case["axes"].split(",")]


def _axis_of(case):
    """Axis of every pair: its axis' block, or dealt in turn to the axes that have pairs left."""
    left = _axes(case)
    if case["order"] == "blocks":
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _scaled(i, rd, case):
    """Angle per position (64 bits) of pairs numbered i of rd elements, and the factor on cosine
    and sine."""
    base, f, kind = case["base"], case["factor"], case["scaling"]
    if kind == "ntk":
        base = base * f ** (rd / (rd - 2))
    inv = base ** (-2.0 * i / rd)
    if kind == "linear":
        return inv / f, 1.0
    if kind == "parts":
        turns = case["original_ctx"] * inv / (2 * math.pi)
        keep = ((turns - case["low"]) / (case["high"] - case["low"])).clamp(0, 1)
        return inv * keep + inv / f * (1 - keep), 1.0
    if kind == "yarn":
        def pair(turns):
            return rd * math.log(case["original_ctx"] / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(case["high"])), 0), min(math.ceil(pair(case["low"])), rd - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return inv * (1 - ramp) + inv / f * ramp, 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _frequencies(case):
    """Angle per position of each pair (64 bits), each pair's axis, and the factor."""
    axis = torch.tensor(_axis_of(case), device=_DEV)
    n = len(axis)
    if case["freq"] == "shared":
        inv, factor = _scaled(torch.arange(n, dtype=torch.float64, device=_DEV), 2 * n, case)
        return inv, axis, factor
    inv = torch.empty(n, dtype=torch.float64, device=_DEV)
    factor = 1.0
    for a, size in enumerate(_axes(case)):
        inv[axis == a], factor = _scaled(torch.arange(size, dtype=torch.float64, device=_DEV), 2 * size, case)
    return inv, axis, factor


def _rotate(x, positions, case, inv, axis, factor):
    """[T, H, D] in its own precision -> the rotated values; positions [n_axes, T]."""
    rd = 2 * len(axis)
    angle = (positions.double().t()[:, axis] * inv)[:, None, :]
    cos, sin = (angle.cos() * factor).to(x.dtype), (angle.sin() * factor).to(x.dtype)
    r = x[..., :rd]
    if case["layout"] == "half":
        a, b = r[..., : rd // 2], r[..., rd // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, x[..., rd:]], -1)


def _plan(case):
    import certified_quantized_kv_gb300 as kvq
    return kvq.RopePlan(case["D"], rotary_dim=2 * sum(_axes(case)), layout=case["layout"], base=case["base"],
                        scaling=case["scaling"], factor=case["factor"], original_ctx=case["original_ctx"], low=case["low"],
                        high=case["high"], axes=tuple(_axes(case)), axis_order=case["order"], axis_frequencies=case["freq"])


# --------------------------------------------------------------------------------------
# states
# --------------------------------------------------------------------------------------

def _lengths(case):
    """Tokens of each sequence in the cache (the case's own, whatever the seed)."""
    B, n = case["B"], case["max_len"]
    if not case["ragged"]:
        return [n] * B
    r = random.Random(B * 1000003 + n)
    out = [int(n * r.random() ** 2) for _ in range(B)]
    out[0] = n
    if B > 3:
        out[1], out[2] = 0, min(n, 1)
    return out


def _chunks(case):
    """New tokens of each sequence."""
    lens = _lengths(case)
    if not case["ragged"]:
        return [min(case["chunk"], n) for n in lens]
    r = random.Random(case["chunk"] * 7919 + case["B"])
    out = [min(n, int(case["chunk"] * r.random()) + 1) for n in lens]
    out[0] = min(case["chunk"], lens[0])
    if case["B"] > 4:
        out[3], out[4] = 0, min(1, lens[4])
    return out


def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _positions(T, case, g):
    """[n_axes, T]: a grid of patches (frames, rows, columns ...) somewhere in the context."""
    t = torch.arange(T, device=_DEV)
    n, out = len(_axes(case)), []
    side = max(2, int(round(T ** (1.0 / n))))
    for a in range(n):
        out.append(t if n == 1 else (t // side ** (n - 1 - a)) % side if a else t // side ** (n - 1))
    first = torch.randint(0, case["max_pos"], (1,), generator=g, device=_DEV)
    return (torch.stack(out) + first).to(torch.int32)


def _cache(case, lens, g):
    """A pool of pages with the sequences' tokens, and the page table."""
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    per = max(1, -(-case["max_len"] // PAGE))
    need = [-(-n // PAGE) for n in lens]
    n_pages = max(1, sum(need))
    # keys with a few strong channels per head, as in the benchmark's workloads; the pages of a
    # sequence lie anywhere in the pool
    k = torch.randn(n_pages, Hkv, PAGE, D, generator=g, device=_DEV)
    k[..., torch.randperm(D, generator=g, device=_DEV)[:4]] *= 4.0
    v = torch.randn(n_pages * Hkv, PAGE, D, generator=g, device=_DEV)
    pages = _make_pages(k.reshape(-1, PAGE, D), v).reshape(n_pages, Hkv, -1)
    order = torch.randperm(n_pages, generator=g, device=_DEV).to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(B)], device=_DEV)[:, None]
    page = torch.arange(per, device=_DEV)[None, :]
    table = order[(first + page).clamp(max=n_pages - 1)]
    table = torch.where(page < torch.tensor(need, device=_DEV)[:, None], table, torch.full_like(table, -1))
    return pages, table.contiguous()


def prepare(case, seed):
    g, dt, op = _gen(seed), _DT[case["dtype"]], case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=_DEV)

    if op == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        st = dict(case=case, x=randn(T, H, D).to(dt), pos=_positions(T, case, g))
        st["out"] = torch.empty_like(st["x"])
        return st
    if op == "append":
        T, Hq, Hkv, D = (case[n] for n in ("T", "Hq", "Hkv", "D"))
        n_pages = -(-T // PAGE) + 3
        # the tokens of a prompt follow one another in pages that lie anywhere in the pool;
        # padding tokens of the batch have slot -1
        table = torch.randperm(n_pages, generator=g, device=_DEV)
        t = torch.arange(T, device=_DEV) + 17
        slots = table[t // PAGE] * PAGE + t % PAGE
        if case["pad"]:
            slots = torch.where(t % case["pad"] == 3, torch.full_like(slots, -1), slots)
        st = dict(case=case, k=randn(T, Hkv, D).to(dt), v=randn(T, Hkv, D).to(dt), slots=slots.to(torch.int32),
                  pos=_positions(T, case, g),
                  pages=torch.zeros(n_pages, Hkv, _page_bytes(D), dtype=torch.uint8, device=_DEV))
        st["q"] = randn(T, Hq, D).to(dt) if Hq else None
        st["q_out"] = torch.empty_like(st["q"]) if Hq else None
        st["k_back"], st["v_back"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        return st
    lens = _lengths(case)
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    pages, table = _cache(case, lens, g)
    st = dict(case=case, pages=pages, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=_DEV))
    if op == "prefill":
        new = _chunks(case)
        starts = [sum(new[:b]) for b in range(B + 1)]
        st["q"] = randn(max(1, starts[-1]), case["Hq"], D).to(dt)
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device=_DEV)
        st["out"] = torch.zeros_like(st["q"])
    elif op == "weights":
        N = table.shape[1] * PAGE
        st["q"] = randn(B, case["Q"], case["Hq"], D).to(dt)
        s, seen = _scores(st)
        s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m > -math.inf, m, torch.zeros_like(m))
        lse = (m + torch.log(torch.exp(s - m).sum(-1, keepdim=True)))[..., 0]      # [B, Hkv, Q, n_rep]
        st["lse"] = lse.permute(0, 2, 1, 3).reshape(B, case["Q"], case["Hq"]).contiguous()
        st["weights"] = torch.rand(B, Hkv, N, generator=g, device=_DEV)
        st["weights"] *= torch.arange(N, device=_DEV) < st["lens"][:, None, None]
    else:
        N, keep = table.shape[1] * PAGE, case["keep"]
        # a few tokens carry most of the weight, some none at all
        w = torch.exp(2 * randn(B, Hkv, N))
        st["weights"] = torch.where(torch.rand(B, Hkv, N, generator=g, device=_DEV) < 0.1, torch.zeros_like(w), w)
        per = -(-keep // PAGE)
        st["to"] = torch.randperm(B * per, generator=g, device=_DEV).to(torch.int32).reshape(B, per)
        st["new_pages"] = torch.zeros(B * per, Hkv, _page_bytes(D), dtype=torch.uint8, device=_DEV)
        st["new_lens"] = torch.zeros(B, dtype=torch.int32, device=_DEV)
        st["origin"] = torch.zeros(B, Hkv, keep, dtype=torch.int32, device=_DEV)
        st["new_weights"] = torch.zeros(B, Hkv, keep, device=_DEV)
        j = torch.arange(keep, device=_DEV)
        st["slots"] = (st["to"][:, j // PAGE] * PAGE + j % PAGE).reshape(-1).to(torch.int32).contiguous()
        st["k_back"] = torch.empty(B * keep, Hkv, D, dtype=dt, device=_DEV)
        st["v_back"] = torch.empty_like(st["k_back"])
    return st


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def _run_own(st):
    import certified_quantized_kv_gb300 as kvq
    case = st["case"]
    op = case["op"]
    if op == "prefill":
        st["workspace"] = kvq.paged_prefill(st["q"], st["starts"], st["pages"], st["table"], st["lens"], st["out"],
                                            causal=case["causal"], window=case["window"], workspace=st.get("workspace"))
        return dict(out=st["out"])
    if op == "weights":
        kvq.paged_weights(st["q"], st["lse"], st["pages"], st["table"], st["lens"], st["weights"], decay=case["decay"],
                          window=case["window"])
        return dict(weights=st["weights"])
    if op == "evict":
        # both pools are parts of one in a user's program; here the kept tokens go to a pool of their own
        kvq.paged_evict(st["pages"], st["table"], st["lens"], st["weights"], st["to"], st["new_lens"], keep=case["keep"],
                        first=case["first"], recent=case["recent"], origin=st["origin"], new_weights=st["new_weights"],
                        new_pages=st["new_pages"])
        # what the new pages hold in 4 bits, as the values it stands for
        kvq.paged_gather(st["new_pages"], st["slots"], st["k_back"], st["v_back"])
        return dict(k=st["k_back"], v=st["v_back"], origin=st["origin"], lens=st["new_lens"], weights=st["new_weights"])
    if "plan" not in st:
        st["plan"] = _plan(case)
    if op == "rope":
        kvq.rope(st["x"], st["pos"], st["plan"], out=st["out"])
        return dict(out=st["out"])
    kvq.paged_append(st["pages"], st["k"], st["v"], st["slots"], positions=st["pos"], plan=st["plan"], q=st["q"],
                     q_out=st["q_out"])
    # what the pages now hold in 4 bits, as the values it stands for
    kvq.paged_gather(st["pages"], st["slots"], st["k_back"], st["v_back"])
    return dict(k=st["k_back"], v=st["v_back"], **({"q": st["q_out"]} if case["Hq"] else {}))


def _run_append(st):
    case = st["case"]
    D, pages, slots, dt = case["D"], st["pages"], st["slots"].long(), st["k"].dtype
    turn = _frequencies(case)
    kept = slots >= 0
    at, page = slots.clamp(min=0) % PAGE, slots.clamp(min=0) // PAGE
    odd = (at % 2 == 1)[:, None, None]
    sec, dev, Hkv = _sections(D), pages.device, case["Hkv"]
    heads = torch.arange(Hkv, device=dev)
    # tokens without a slot write their bytes behind the pool's last page
    spill = pages.numel()
    flat = torch.empty(spill + _page_bytes(D), dtype=torch.uint8, device=dev)
    flat[:spill] = pages.reshape(-1)
    start = torch.where(kept[:, None], (page[:, None] * Hkv + heads) * _page_bytes(D), torch.full_like(page[:, None], spill))

    def put(section, byte, data):
        flat[(start[..., None] + sec[section] + byte[:, None, :]).reshape(-1)] = data.reshape(-1)

    def two(element):
        return torch.stack([2 * element, 2 * element + 1], -1).flatten(-2)

    k = _rotate(st["k"].float(), st["pos"], case, *turn)
    token_group = torch.arange(64, device=dev)[:, None] * (D // GROUP) + torch.arange(D // GROUP, device=dev)
    for x, down, section, place, scale_place in (
            (k, torch.zeros_like(odd), (0, 2, 3), _key_place(D, dev), token_group),
            (st["v"].float(), odd, (1, 4, 5), _value_place(D, dev), _value_scale_place(D, dev))):
        code, s, o = _quantize(x, down.expand(*x.shape[:2], D // GROUP))
        put(section[0], place[0][at][:, 0::2], code[..., 0::2] | (code[..., 1::2] << 4))
        put(section[1], two(scale_place[at]), s.contiguous().view(torch.uint8))
        put(section[2], two(scale_place[at]), o.contiguous().view(torch.uint8))
    pages.copy_(flat[:spill].reshape(pages.shape))
    # read back
    raw = pages.reshape(-1, pages.shape[-1])
    zero = torch.zeros((), device=dev)
    back = [torch.where(kept[:, None, None], part(raw, D).reshape(*pages.shape[:2], PAGE, D)[page, :, at], zero).to(dt)
            for part in (_unpack_keys, _unpack_values)]
    out = dict(k=back[0], v=back[1])
    if case["Hq"]:
        out["q"] = _rotate(st["q"].float(), st["pos"], case, *turn).to(dt)
    return out


def _rows_of_pages(x):
    """[B, pages, Hkv, 64, D] -> [B, Hkv, tokens, D]."""
    B, P, H, n, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, P * n, D)


def _scores(st):
    """Scaled scores [B, Hkv, Q, n_rep, tokens] of the last Q tokens of every sequence, and which are seen."""
    case = st["case"]
    B, Q, Hq, Hkv, D = (case[n] for n in ("B", "Q", "Hq", "Hkv", "D"))
    k = _rows_of_pages(_unpack_keys(st["pages"][st["table"].long().clamp(min=0)], D))
    L = k.shape[2]
    q = st["q"].float().reshape(B, Q, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = ((q @ k.transpose(-1, -2)) / math.sqrt(D)).reshape(B, Hkv, Q, Hq // Hkv, L)
    t = torch.arange(L, device=s.device)
    end = (st["lens"].long()[:, None] - Q + 1 + torch.arange(Q, device=s.device))[:, :, None]
    seen = t < end
    if case["window"]:
        seen &= t >= end - case["window"]
    return s, seen[:, None, :, None, :]


def _run_weights(st):
    case = st["case"]
    B, Q, Hkv = case["B"], case["Q"], case["Hkv"]
    s, seen = _scores(st)
    lse = st["lse"].reshape(B, Q, Hkv, -1).permute(0, 2, 1, 3)[..., None]
    p = torch.where(seen & (lse > -math.inf), torch.exp(s - lse), torch.zeros((), device=s.device))
    new = p.sum((2, 3))
    w = st["weights"]
    live = torch.arange(w.shape[-1], device=w.device) < st["lens"][:, None, None]
    st["weights"].copy_(torch.where(live, w * case["decay"] + new, w))
    return dict(weights=st["weights"])


def _run_prefill(st):
    case = st["case"]
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    dev, starts, lens = st["q"].device, st["starts"].long(), st["lens"].long()
    n = starts[1:] - starts[:-1]
    Q = min(case["chunk"], case["max_len"])
    # the chunks side by side, padded to the longest
    i = torch.arange(Q, device=dev)
    here = i < n[:, None]
    rows = torch.where(here, starts[:-1, None] + i, torch.zeros_like(i))
    q = st["q"][rows].float().reshape(B, Q, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    raw = st["pages"][st["table"].long().clamp(min=0)]
    k, v = _rows_of_pages(_unpack_keys(raw, D)), _rows_of_pages(_unpack_values(raw, D))
    L = k.shape[2]
    s = ((q @ k.transpose(-1, -2)) / math.sqrt(D)).reshape(B, Hkv, Q, Hq // Hkv, L)
    t = torch.arange(L, device=dev)
    end = (lens[:, None] - n[:, None] + 1 + i if case["causal"] else lens[:, None].expand(B, Q))[:, :, None]
    seen = (t < end) & (t < lens[:, None, None]) & here[:, :, None]
    if case["window"]:
        seen &= t >= end - case["window"]
    seen = seen[:, None, :, None, :]
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, L) @ v).reshape(B, Hkv, Q, Hq // Hkv, D) / torch.where(l > 0, l, torch.ones_like(l))
    out = torch.zeros_like(st["q"])
    out[rows[here]] = o.permute(0, 2, 1, 3, 4).reshape(B, Q, Hq, D)[here].to(out.dtype)
    return dict(out=out)


def _run_evict(st):
    case = st["case"]
    B, Hkv, D, keep = (case[n] for n in ("B", "Hkv", "D", "keep"))
    w, lens = st["weights"], st["lens"].long()[:, None, None]
    dev, N = w.device, w.shape[-1]
    t = torch.arange(N, device=dev)
    key = torch.where((t < case["first"]) | (t >= lens - case["recent"]), torch.full_like(w, math.inf), w)
    key = torch.where(t < lens, key, torch.full_like(w, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    if N < keep:
        order = torch.cat([order, torch.arange(N, keep, device=dev).expand(B, Hkv, -1)], -1)
    j = torch.arange(keep, device=dev)
    got = torch.where(lens > keep, order[..., :keep], j.expand(B, Hkv, keep)).sort(-1).values
    there = j < lens
    origin = torch.where(there, got, torch.full_like(got, -1))
    at = got.clamp(max=N - 1)
    # the tokens' own bytes: codes, scales and offsets
    page = torch.gather(st["table"].long()[:, None, :].expand(B, Hkv, -1), 2, at // PAGE).clamp(min=0)
    raw = st["pages"].reshape(-1)
    start = (page * Hkv + torch.arange(Hkv, device=dev)[:, None]) * _page_bytes(D)
    i, sec, G = at % PAGE, _sections(D), D // GROUP

    def halves(byte):
        return torch.stack([raw[byte], raw[byte + 1]], -1).view(torch.float16).float()

    token_group = torch.arange(64, device=dev)[:, None] * G + torch.arange(G, device=dev)
    back = []
    for section, place, scale_place in (((0, 2, 3), _key_place(D, dev), token_group),
                                        ((1, 4, 5), _value_place(D, dev), _value_scale_place(D, dev))):
        code = (raw[start[..., None] + sec[section[0]] + place[0][i]] >> place[1][i].to(torch.uint8)) & 15
        s, o = (halves(start[..., None] + sec[x] + 2 * scale_place[i]) for x in section[1:])
        x = (code.reshape(B, Hkv, keep, G, GROUP).float() * s + o).reshape(B, Hkv, keep, D)
        x = torch.where(there[..., None], x, torch.zeros((), device=dev))
        back.append(x.permute(0, 2, 1, 3).reshape(B * keep, Hkv, D).to(_DT[case["dtype"]]))
    weights = torch.where(there, torch.gather(w, 2, at), torch.zeros((), device=dev))
    return dict(k=back[0], v=back[1], origin=origin.to(torch.int32), lens=st["lens"].clamp(max=keep), weights=weights)


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] == "rope":
        return dict(out=_rotate(st["x"].float(), st["pos"], case, *_frequencies(case)).to(st["x"].dtype))
    return {"append": _run_append, "prefill": _run_prefill, "weights": _run_weights, "evict": _run_evict}[case["op"]](st)


# --------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------

def _turn(x, positions, case):
    """Rotation of [T, H, D] in 64 bits, one pair after another as complex numbers."""
    sizes, n = _axes(case), sum(_axes(case))
    # (axis, number within the axis) of every pair
    if case["order"] == "blocks":
        pairs = [(a, k) for a in range(len(sizes)) for k in range(sizes[a])]
    else:
        pairs = [(a, k) for k in range(max(sizes)) for a in range(len(sizes)) if k < sizes[a]]
    f, kind, size = case["factor"], case["scaling"], 1.0
    freq = []
    for at, (a, k) in enumerate(pairs):
        i, rd = (at, 2 * n) if case["freq"] == "shared" else (k, 2 * sizes[a])
        base = case["base"] * (f ** (rd / (rd - 2)) if kind == "ntk" else 1.0)
        w = base ** (-2.0 * i / rd)
        if kind == "linear":
            w /= f
        elif kind == "parts":
            u = (case["original_ctx"] * w / (2 * math.pi) - case["low"]) / (case["high"] - case["low"])
            u = min(1.0, max(0.0, u))
            w = u * w + (1 - u) * w / f
        elif kind == "yarn":
            size = 1.0 + 0.1 * math.log(f)
            edge = [rd * math.log(case["original_ctx"] / (2 * math.pi * r)) / (2 * math.log(base)) for r in (case["high"], case["low"])]
            edge = [max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rd - 1)]
            u = min(1.0, max(0.0, (i - edge[0]) / max(edge[1] - edge[0], 1e-3)))
            w = w * (1 - u) + w / f * u
        freq.append(w)
    angle = torch.stack([positions[a].double() * w for (a, _), w in zip(pairs, freq)], -1)
    turn = torch.polar(torch.full_like(angle, size), angle)[:, None, :]
    y = x.double().clone()
    part = y[..., : 2 * n]
    if case["layout"] == "half":
        z = torch.complex(part[..., :n].contiguous(), part[..., n:].contiguous()) * turn
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    else:
        z = torch.view_as_complex(part.reshape(*part.shape[:-1], n, 2).contiguous()) * turn
        y[..., :2 * n] = torch.view_as_real(z).flatten(-2)
    return y


def _four_bits(x, down):
    """What [T, H, D] in 64 bits stands for once held in 4 bits."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[-1], GROUP):
        w = x[..., c:c + GROUP].clamp(-65504, 65504)
        lo, hi = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
        off = torch.where(down, hi, lo).to(torch.float16).double()
        span = (torch.where(down, off - lo, hi - off) / 15).clamp(min=0)
        s = span.to(torch.float16)
        s = torch.where(s.double() < span, (s.view(torch.int16) + 1).view(torch.float16), s).double()
        steps = torch.round((w - off).abs() * torch.where(torch.where(down, w < off, w > off), 1.0, 0.0) / s.clamp(min=2.0 ** -30))
        out[..., c:c + GROUP] = off + torch.where(down, -s, s) * steps.clamp(0, 15)
    return out


def _halves(raw, at):
    lo, hi = raw[..., at].to(torch.int32), raw[..., at + 1].to(torch.int32)
    return (lo + 256 * hi).to(torch.int16).view(torch.float16).double()


def _read_page(raw, D):
    """Keys and values [n, 64, D] in 64 bits of [n, page bytes]."""
    n, G, dev = raw.shape[0], D // GROUP, raw.device
    row = D // 2
    t, g = torch.arange(64, device=dev)[:, None], torch.arange(G, device=dev)[None, :]
    # keys: rows of tokens, four pieces of eight channels of every group
    b = raw[:, : 64 * row].reshape(n, 64, 4, G, 4).permute(0, 1, 3, 2, 4)
    code = torch.stack([b & 15, b >> 4], -1).reshape(n, 64, G, GROUP).double()
    at = 128 * row + 2 * (t * G + g)
    k = code * _halves(raw, at)[..., None] + _halves(raw, at + 128 * G)[..., None]
    # values: rows exchanged within each eight tokens, eight pieces of four channels of every group
    rows = [(x ^ ((x >> 1) & 1)) if D == 128 else (x ^ ((x >> 2) & 1)) for x in range(64)]
    b = raw[:, 64 * row: 128 * row].reshape(n, 64, 8, G, 2)[:, rows]
    if D == 128:
        far = [x for x in range(64) if x & 4]
        b[:, far] = b[:, far][:, :, [4, 5, 6, 7, 0, 1, 2, 3]]
    b = b.permute(0, 1, 3, 2, 4)
    code = torch.stack([b & 15, b >> 4], -1).reshape(n, 64, G, GROUP).double()
    spot = [16 * ((x // 2) % 4) + 4 * (x // 16) + 2 * ((x // 8) % 2) + x % 2 for x in range(64)]
    at = 128 * row + 256 * G + 2 * (64 * g + torch.tensor(spot, device=dev)[:, None])
    v = code * _halves(raw, at)[..., None] + _halves(raw, at + 128 * G)[..., None]
    return k.reshape(n, 64, D), v.reshape(n, 64, D)


def _read_rows(st, b, h, n, D):
    """Keys and values [n, D] in 64 bits of the first n tokens of sequence b, KV head h."""
    ids = st["table"][b, : -(-n // PAGE)].long()
    return tuple(x.reshape(-1, D)[:n] for x in _read_page(st["pages"][ids, h], D))


def _exact_prefill(st, case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    first = 0
    for b, (n, new) in enumerate(zip(_lengths(case), _chunks(case))):
        b_rows = slice(first, first + new)
        first += new
        if new == 0:
            continue
        t = torch.arange(n, device=_DEV)
        for h in range(Hkv):
            k, v = _read_rows(st, b, h, n, D)
            for r in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                # (a thousand rows at a time)
                for i in range(0, new, 1024):
                    last = torch.arange(n - new + i, n - new + min(new, i + 1024), device=_DEV)[:, None]
                    s = st["q"][b_rows][i:i + 1024, r].double() @ k.T / math.sqrt(D)
                    if case["causal"]:
                        s.masked_fill_(t > last, -math.inf)
                    if case["window"]:
                        s.masked_fill_(t <= last - case["window"], -math.inf)
                    out[b_rows][i:i + 1024, r] = torch.softmax(s, -1) @ v
    return dict(out=out)


def _exact_weights(st, case):
    Q, Hq, Hkv, D = (case[n] for n in ("Q", "Hq", "Hkv", "D"))
    out = st["weights"].double()
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        t = torch.arange(n, device=_DEV)
        for h in range(Hkv):
            k, _ = _read_rows(st, b, h, n, D)
            out[b, h, :n] *= case["decay"]
            for i in range(Q):
                last = n - Q + i
                if last < 0:
                    continue
                rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                p = torch.exp(st["q"][b, i, rows].double() @ k.T / math.sqrt(D) - st["lse"][b, i, rows].double()[:, None])
                p[:, t > last] = 0
                if case["window"]:
                    p[:, t <= last - case["window"]] = 0
                out[b, h, :n] += p.sum(0)
    return dict(weights=out)


def _exact_evict(st, case):
    import numpy as np
    B, Hkv, D, keep = (case[n] for n in ("B", "Hkv", "D", "keep"))
    k_out, v_out = (torch.zeros(B, keep, Hkv, D, dtype=torch.float64, device=_DEV) for _ in range(2))
    origin = np.full((B, Hkv, keep), -1, np.int32)
    new_w = np.zeros((B, Hkv, keep))
    lens, w = _lengths(case), st["weights"].cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(Hkv):
            ids = np.arange(n)
            if n > keep:
                sure = np.r_[ids[: case["first"]], ids[n - case["recent"]:]]
                rest = ids[case["first"]: n - case["recent"]]
                heavy = rest[np.lexsort((rest, -w[b, h, rest].astype(np.float64)))][: keep - len(sure)]
                ids = np.sort(np.r_[sure, heavy])
            m = len(ids)
            if m == 0:
                continue
            origin[b, h, :m], new_w[b, h, :m] = ids, w[b, h, ids]
            k, v = _read_rows(st, b, h, n, D)
            at = torch.from_numpy(ids).to(_DEV)
            k_out[b, :m, h], v_out[b, :m, h] = k[at], v[at]
    return dict(k=k_out.reshape(-1, Hkv, D), v=v_out.reshape(-1, Hkv, D), origin=torch.from_numpy(origin),
                lens=torch.tensor([min(n, keep) for n in lens], dtype=torch.int32), weights=torch.from_numpy(new_w))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return dict(out=_turn(st["x"], st["pos"], case))
    if case["op"] == "append":
        odd, kept = ((st["slots"] % 2 == 1)[:, None, None], (st["slots"] >= 0)[:, None, None])
        zero = torch.zeros((), dtype=torch.float64, device=st["k"].device)
        out = dict(k=torch.where(kept, _four_bits(_turn(st["k"], st["pos"], case), torch.zeros_like(odd)), zero),
                   v=torch.where(kept, _four_bits(st["v"].double(), odd), zero))
        if case["Hq"]:
            out["q"] = _turn(st["q"], st["pos"], case)
        return out
    return {"prefill": _exact_prefill, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](st, case)


def _seen_pairs(n, new, causal, window):
    """(query, token) pairs that are seen, and the tokens that any query sees."""
    w = window or 1 << 40
    if not causal:
        return new * n, n if new else 0
    return sum(max(0, min(n - new + 1 + i, w)) for i in range(new)), min(n, w + new - 1) if new else 0


def work(case):
    if case["op"] == "rope":
        n, rd = case["T"] * case["H"], 2 * sum(_axes(case))
        return {"bytes": 4 * n * case["D"] + 4 * len(_axes(case)) * case["T"], "flops": 3 * n * rd}
    Hkv, D = case["Hkv"], case["D"]
    token = D + 8 * (D // GROUP)                            # bytes of a token's keys and values in a page
    if case["op"] == "append":
        T, Hq, rd = case["T"], case["Hq"], 2 * sum(_axes(case))
        kept = T - (sum((t + 17) % case["pad"] == 3 for t in range(T)) if case["pad"] else 0)
        held = kept * Hkv * token
        moved = 4 * kept * Hkv * D + held + 4 * T * Hq * D + 4 * (1 + len(_axes(case))) * T      # append
        moved += held + 4 * T * Hkv * D + 4 * T                                                  # read back
        return {"bytes": moved, "flops": 3 * T * (Hq + Hkv) * rd + 8 * kept * Hkv * D}
    lens = _lengths(case)
    if case["op"] == "prefill":
        new, Hq = _chunks(case), case["Hq"]
        both = [_seen_pairs(n, m, case["causal"], case["window"]) for n, m in zip(lens, new)]
        return {"bytes": sum(t for _, t in both) * Hkv * token + 4 * sum(new) * Hq * D, "flops": 4 * sum(p for p, _ in both) * Hq * D}
    if case["op"] == "weights":
        Q, Hq = case["Q"], case["Hq"]
        both = [_seen_pairs(n, min(n, Q), True, case["window"]) for n in lens]
        touched = sum(lens) * Hkv * (8 if case["decay"] else 4)
        return {"bytes": sum(t for _, t in both) * Hkv * token // 2 + touched + case["B"] * Q * Hq * (2 * D + 4),
                "flops": 2 * sum(p for p, _ in both) * Hq * D}
    kept = sum(min(n, case["keep"]) for n in lens)
    back = kept * Hkv * (token + 4 * D)
    return {"bytes": sum(lens) * Hkv * 4 + kept * Hkv * (2 * token + 8) + back, "flops": 4 * kept * Hkv * D}

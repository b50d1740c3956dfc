"""Cases for the paged 4-bit cache's operators: rotary positions, the append that rotates
and quantises into pages (with the read-back of what the pages hold), and attention over
the pages.

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
    llama = dict(base=500000.0, scaling="parts", factor=8.0, original_ctx=8192, low=1.0, high=4.0)
    plain = dict(base=10000.0, scaling="none", factor=1.0, original_ctx=0, low=1.0, high=32.0)
    yarn = dict(base=10000.0, scaling="yarn", factor=16.0, original_ctx=4096, low=1.0, high=32.0)
    return [
        # q and k heads of 64 sequences' next tokens, side by side in one buffer: latency
        dict(name="rope_decode_64", op="rope", T=64, H=40, D=128, rd=128, layout="half", dtype="fp16",
             max_pos=131072, **llama),
        # the same heads for a 32K-token prompt: memory bandwidth
        dict(name="rope_prompt_32k", op="rope", T=32768, H=40, D=128, rd=128, layout="half", dtype="fp16",
             max_pos=131072, **llama),
        # interleaved pairs on part of the head, an odd token count, positions far out
        dict(name="rope_partial_bf16", op="rope", T=4099, H=13, D=128, rd=96, layout="interleaved", dtype="bf16",
             max_pos=2000000, **yarn),
        # one token per sequence of a batch of 64 (a few of them padding), q rotated along: latency
        dict(name="append_decode_64", op="append", T=64, Hq=32, Hkv=8, D=128, rd=128, layout="half", dtype="fp16",
             max_pos=131072, pad=7, **llama),
        # a 32K-token prompt's keys and values into pages, q rotated along: memory bandwidth
        dict(name="append_prompt_32k", op="append", T=32768, Hq=32, Hkv=8, D=128, rd=128, layout="half",
             dtype="fp16", max_pos=32768, pad=0, **llama),
        # several prompts in one padded batch, small heads, interleaved pairs
        dict(name="append_ragged_d64", op="append", T=5003, Hq=0, Hkv=5, D=64, rd=64, layout="interleaved",
             dtype="bf16", max_pos=16384, pad=9, **plain),
        # the 4K-token layer of the benchmark's smallest workload, one sequence: latency
        dict(name="attend_4k", op="attend", B=1, Q=1, Hq=32, Hkv=8, D=128, max_len=4096, ragged=False, window=0,
             dtype="fp16"),
        # the benchmark's headline layer: 128K tokens, one sequence, split over the GPU
        dict(name="attend_128k", op="attend", B=1, Q=1, Hq=32, Hkv=8, D=128, max_len=131072, ragged=False,
             window=0, dtype="fp16"),
        # the benchmark's largest batch: eight sequences of 64K tokens
        dict(name="attend_64k_8", op="attend", B=8, Q=1, Hq=32, Hkv=8, D=128, max_len=65536, ragged=False,
             window=0, dtype="fp16"),
        # a serving batch of 64 sequences from empty to 16K tokens
        dict(name="attend_ragged_64", op="attend", B=64, Q=1, Hq=32, Hkv=8, D=128, max_len=16384, ragged=True,
             window=0, dtype="bf16"),
        # four drafted tokens per sequence verified at once, causal among themselves
        dict(name="attend_verify_4", op="attend", B=8, Q=4, Hq=32, Hkv=8, D=128, max_len=16384, ragged=True,
             window=0, dtype="fp16"),
        # sliding-window layers of small heads, eight query heads to a KV head
        dict(name="attend_window_d64", op="attend", B=48, Q=1, Hq=24, Hkv=3, D=64, max_len=40000, ragged=True,
             window=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    rot = dict(base=rng.choice([10000.0, 500000.0, 1000000.0]),
               scaling=rng.choice(["none", "linear", "ntk", "parts", "yarn"]),
               factor=rng.choice([2.0, 4.0, 8.0, 16.0]), original_ctx=rng.choice([4096, 8192]), low=1.0, high=32.0)
    op = rng.choice(["rope", "append", "attend", "attend"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        H = rng.choice([1, 2, 5, 8, 13, 32, 40])
        return dict(op="rope", T=_log(rng, 1, min(65536, 32768 * 40 * 128 // (H * D))), H=H, D=D,
                    rd=rng.choice([D, D, 2 * rng.randint(2, D // 2)]), layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["fp16", "bf16"]), max_pos=_log(rng, 1, 2000000), **rot)
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    n_rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if op == "append":
        n_rep = rng.choice([0, n_rep])
        most = 32768 * 48 * 128 // ((n_rep + 2) * Hkv * D)
        return dict(op="append", T=_log(rng, 1, min(65536, most)), Hq=Hkv * n_rep, Hkv=Hkv, D=D,
                    rd=rng.choice([D, D, 2 * rng.randint(2, D // 2)]), layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["fp16", "bf16"]), max_pos=_log(rng, 64, 2000000), pad=rng.choice([0, 5]), **rot)
    B = _log(rng, 1, 64)
    most = 8 * 65536 * 8 * 128 // (B * Hkv * D * (4 if n_rep > 4 else 1))
    return dict(op="attend", B=B, Q=rng.choice([1, 1, 1, 2, 3, 5, 8]), Hq=Hkv * n_rep, Hkv=Hkv, D=D,
                max_len=_log(rng, 1, min(131072, most)), ragged=rng.choice([True, False]),
                window=rng.choice([0, 0, 0, 100, 1024]), dtype=rng.choice(["fp16", "bf16"]))


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


def _unpack(raw, D):
    """[..., page bytes] -> keys and values [..., 64, D] in fp32."""
    sec, lead, dev = _sections(D), raw.shape[:-1], raw.device

    def codes(part, place):
        at, sh = place
        return ((part[..., at.reshape(-1)] >> sh.reshape(-1).to(torch.uint8)) & 15).reshape(*lead, 64, D // GROUP, GROUP)

    def halves(a, b):
        return raw[..., a:b].contiguous().view(torch.float16).float()

    ks, ko = (halves(sec[i], sec[i + 1]).reshape(*lead, 64, D // GROUP, 1) for i in (2, 3))
    at = _value_scale_place(D, dev).reshape(-1)
    vs, vo = (halves(sec[i], sec[i + 1])[..., at].reshape(*lead, 64, D // GROUP, 1) for i in (4, 5))
    k = codes(raw[..., sec[0]:sec[1]], _key_place(D, dev)).float() * ks + ko
    v = codes(raw[..., sec[1]:sec[2]], _value_place(D, dev)).float() * vs + vo
    return k.reshape(*lead, 64, D), v.reshape(*lead, 64, D)


# --------------------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------------------

def _frequencies(case):
    """Angle per position of each pair (64 bits) and the factor on cosine and sine."""
    rd, base, f = case["rd"], case["base"], case["factor"]
    i = torch.arange(rd // 2, dtype=torch.float64, device=_DEV)
    kind = case["scaling"]
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


def _rotate(x, positions, case, inv, factor):
    """[T, H, D] in its own precision -> the rotated values."""
    rd = case["rd"]
    angle = positions.double()[:, None, None] * inv
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
    return kvq.RopePlan(case["D"], rotary_dim=case["rd"], layout=case["layout"], base=case["base"],
                        scaling=case["scaling"], factor=case["factor"], original_ctx=case["original_ctx"],
                        low=case["low"], high=case["high"])


# --------------------------------------------------------------------------------------
# states
# --------------------------------------------------------------------------------------

def _lengths(case):
    """Tokens of each sequence (the cases' own, whatever the seed)."""
    B, n = case["B"], case["max_len"]
    if not case["ragged"]:
        return [n] * B
    r = random.Random(B * 1000003 + n)
    out = [int(n * r.random() ** 2) for _ in range(B)]
    out[0] = n
    if B > 3:
        out[1], out[2] = 0, min(n, 1)
    return out


def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=_DEV)

    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        pos = torch.randint(0, case["max_pos"], (T,), generator=g, device=_DEV, dtype=torch.int32)
        st = dict(case=case, x=randn(T, H, D).to(dt), pos=pos)
        st["out"] = torch.empty_like(st["x"])
    elif case["op"] == "append":
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
                  pos=torch.randint(0, case["max_pos"], (T,), generator=g, device=_DEV, dtype=torch.int32),
                  pages=torch.zeros(n_pages, Hkv, _page_bytes(D), dtype=torch.uint8, device=_DEV))
        st["q"] = randn(T, Hq, D).to(dt) if Hq else None
        st["q_out"] = torch.empty_like(st["q"]) if Hq else None
        st["k_back"], st["v_back"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    else:
        B, Q, Hq, Hkv, D = (case[n] for n in ("B", "Q", "Hq", "Hkv", "D"))
        lens = _lengths(case)
        per = max(1, -(-case["max_len"] // PAGE))
        need = [-(-n // PAGE) for n in lens]
        n_pages = max(1, sum(need))
        # keys with a few strong channels per head, as in the benchmark's workloads; the
        # pages of a sequence lie anywhere in the pool
        k = randn(n_pages, Hkv, PAGE, D)
        k[..., torch.randperm(D, generator=g, device=_DEV)[:4]] *= 4.0
        pages = _make_pages(k.reshape(-1, PAGE, D), randn(n_pages * Hkv, PAGE, D)).reshape(n_pages, Hkv, -1)
        order = torch.randperm(n_pages, generator=g, device=_DEV).to(torch.int32)
        first = torch.tensor([sum(need[:b]) for b in range(B)], device=_DEV)[:, None]
        page = torch.arange(per, device=_DEV)[None, :]
        table = order[(first + page).clamp(max=n_pages - 1)]
        table = torch.where(page < torch.tensor(need, device=_DEV)[:, None], table, torch.full_like(table, -1))
        st = dict(case=case, q=randn(B, Q, Hq, D).to(dt), pages=pages, table=table.contiguous(),
                  lens=torch.tensor(lens, dtype=torch.int32, device=_DEV))
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(B, Q, Hq, device=_DEV)
    return st


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def _run_own(st):
    import certified_quantized_kv_gb300 as kvq
    case = st["case"]
    if case["op"] == "attend":
        st["workspace"] = kvq.paged_attention(st["q"], st["pages"], st["table"], st["lens"], st["out"], lse=st["lse"],
                                              window=case["window"], workspace=st.get("workspace"))
        return dict(out=st["out"], lse=st["lse"])
    if "plan" not in st:
        st["plan"] = _plan(case)
    if case["op"] == "rope":
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
    inv, factor = _frequencies(case)
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

    k = _rotate(st["k"].float(), st["pos"], case, inv, factor)
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
    kd, vd = (part.reshape(*pages.shape[:2], PAGE, D) for part in _unpack(pages.reshape(-1, pages.shape[-1]), D))
    zero = kept[:, None, None]
    back = [torch.where(zero, part[page, :, at], torch.zeros((), device=dev)).to(dt) for part in (kd, vd)]
    out = dict(k=back[0], v=back[1])
    if case["Hq"]:
        out["q"] = _rotate(st["q"].float(), st["pos"], case, inv, factor).to(dt)
    return out


def _run_attend(st):
    case = st["case"]
    B, Q, Hq, Hkv, D = (case[n] for n in ("B", "Q", "Hq", "Hkv", "D"))
    table, lens, q = st["table"].long(), st["lens"].long(), st["q"]
    raw = st["pages"][table.clamp(min=0)]                                # [B, pages, Hkv, bytes]
    k, v = _unpack(raw, D)
    L = table.shape[1] * PAGE
    k = k.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
    v = v.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
    qf = q.float().reshape(B, Q, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = (qf @ k.transpose(-1, -2)) / math.sqrt(D)
    s = s.reshape(B, Hkv, Q, Hq // Hkv, L)
    t = torch.arange(L, device=q.device)
    end = (lens[:, None] - Q + 1 + torch.arange(Q, device=q.device))[:, :, None]      # tokens that a row sees
    seen = t < end
    if case["window"]:
        seen &= t >= end - case["window"]
    seen = seen[:, None, :, None, :]
    m = s.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m))), torch.zeros_like(s))
    l = p.sum(-1, keepdim=True)
    o = p.reshape(B, Hkv, -1, L) @ torch.where(seen.any(2).any(2)[..., None], v, torch.zeros((), device=v.device))
    o = o.reshape(B, Hkv, Q, Hq // Hkv, D) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    return dict(out=o.permute(0, 2, 1, 3, 4).reshape(B, Q, Hq, D).to(q.dtype),
                lse=lse.permute(0, 2, 1, 3, 4).reshape(B, Q, Hq))


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] == "rope":
        return dict(out=_rotate(st["x"].float(), st["pos"], case, *_frequencies(case)).to(st["x"].dtype))
    return _run_append(st) if case["op"] == "append" else _run_attend(st)


# --------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------

def _turn(x, positions, case):
    """Rotation of [T, H, D] in 64 bits, one pair after another as complex numbers."""
    rd, n = case["rd"], case["rd"] // 2
    base, f, kind = case["base"], case["factor"], case["scaling"]
    if kind == "ntk":
        base *= f ** (rd / (rd - 2))
    freq, size = [], 1.0
    if kind == "yarn":
        size = 1.0 + 0.1 * math.log(f)
        edge = [rd * math.log(case["original_ctx"] / (2 * math.pi * r)) / (2 * math.log(base)) for r in (case["high"], case["low"])]
        edge = [max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rd - 1)]
    for i in range(n):
        w = base ** (-2.0 * i / rd)
        if kind == "linear":
            w /= f
        elif kind == "parts":
            u = (case["original_ctx"] * w / (2 * math.pi) - case["low"]) / (case["high"] - case["low"])
            u = min(1.0, max(0.0, u))
            w = u * w + (1 - u) * w / f
        elif kind == "yarn":
            u = min(1.0, max(0.0, (i - edge[0]) / max(edge[1] - edge[0], 1e-3)))
            w = w * (1 - u) + w / f * u
        freq.append(w)
    angle = positions.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(angle, size), angle)[:, None, :]
    y = x.double().clone()
    pairs = y[..., :rd]
    if case["layout"] == "half":
        z = torch.complex(pairs[..., :n].contiguous(), pairs[..., n:].contiguous()) * turn
        y[..., :n], y[..., n:rd] = z.real, z.imag
    else:
        z = torch.view_as_complex(pairs.reshape(*pairs.shape[:-1], n, 2).contiguous()) * turn
        y[..., :rd] = torch.view_as_real(z).flatten(-2)
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
    B, Q, Hq, Hkv, D = (case[n] for n in ("B", "Q", "Hq", "Hkv", "D"))
    out = torch.zeros(B, Q, Hq, D, dtype=torch.float64, device=_DEV)
    lse = torch.full((B, Q, Hq), -math.inf, dtype=torch.float64, device=_DEV)
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        ids = st["table"][b, : -(-n // PAGE)].long()
        for h in range(Hkv):
            k, v = (x.reshape(-1, D)[:n] for x in _read_page(st["pages"][ids, h], D))
            for i in range(Q):
                end = n - Q + 1 + i
                start = max(0, end - case["window"]) if case["window"] else 0
                if end <= start:
                    continue
                rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                s = st["q"][b, i, rows].double() @ k[start:end].T / math.sqrt(D)
                lse[b, i, rows] = torch.logsumexp(s, -1)
                out[b, i, rows] = torch.softmax(s, -1) @ v[start:end]
    return dict(out=out, lse=lse)


def work(case):
    if case["op"] == "rope":
        n = case["T"] * case["H"]
        return {"bytes": 4 * n * case["D"] + 4 * case["T"], "flops": 3 * n * case["rd"]}
    if case["op"] == "append":
        T, Hq, Hkv, D = (case[n] for n in ("T", "Hq", "Hkv", "D"))
        kept = T - (sum((t + 17) % case["pad"] == 3 for t in range(T)) if case["pad"] else 0)
        held = kept * Hkv * (D + 8 * (D // GROUP))          # codes, scales and offsets of keys and values
        moved = 4 * kept * Hkv * D + held + 4 * T * Hq * D + 8 * T       # append
        moved += held + 4 * T * Hkv * D + 4 * T                          # read back
        return {"bytes": moved, "flops": 3 * T * (Hq + Hkv) * case["rd"] + 8 * kept * Hkv * D}
    Q, Hq, Hkv, D = (case[n] for n in ("Q", "Hq", "Hkv", "D"))
    w = case["window"] or 1 << 40
    lens = _lengths(case)
    tokens = sum(min(n, w + Q - 1) for n in lens)
    pairs = sum(max(0, min(n - Q + 1 + i, w)) for n in lens for i in range(Q))
    io = case["B"] * Q * Hq * (4 * D + 4) + 4 * case["B"] + 4 * (tokens // PAGE)
    return {"bytes": tokens * Hkv * (D + 8 * (D // GROUP)) + io, "flops": 4 * pairs * Hq * D}

"""The block-scaled E4M3 cache: writing it, reading it back, and decode attention over it.

The cache holds E4M3 codes with one fp32 scale for every ``block`` consecutive
tokens of a KV head, K and V apart, contiguous (``[B, S_max, H_kv, d]``) or in
pages (``[num_pages, page_size, H_kv, d]`` behind a block table).  Each case
names one operator:

* ``append``: the last tokens of every sequence, bf16, are quantised into the
  cache; outputs are the codes (as the E4M3 values they are) and the scales.
* ``read``: tokens of the cache as bf16, for attention over a prompt.
* ``decode``: the last ``T_q`` queries of every sequence attend to the cache.

With ``own`` false the operators run in elementary torch operations, in 32 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
MIN_EXP = -100  # the smallest scale is 2**-100


# ------------------------------------------------------------------- cases --
def _case(name, op, B, H_kv, d, lo, hi, block, page, T=1, G=1, fused=0):
    """lo..hi: the range of the sequence lengths; page 0: a contiguous cache;
    T: new tokens (append, at most), queries (decode); G: query heads per KV
    head; fused: the new rows are slices of a fused Q/K/V projection."""
    return dict(name=name, op=op, B=B, H_kv=H_kv, d=d, lo=lo, hi=hi, block=block, page=page, T=T,
                G=G, fused=fused)


def listed():
    return [
        # one sequence gets its next token: nothing but latency
        _case("append_token_b1", "append", 1, 8, 128, 4097, 4097, 64, 64, 1, 8, 1),
        # one step of a served batch, every sequence at its own length
        _case("append_token_b128", "append", 128, 8, 128, 33, 8191, 16, 16, 1, 8, 1),
        # a padded batch of prompts of different lengths, d = 64
        _case("append_prompts_b8", "append", 8, 5, 64, 203, 1531, 32, 0, 1531, 1, 0),
        # a whole 32K prompt of the Llama3-70B heads
        _case("append_prompt_32k", "append", 1, 8, 128, 32768, 32768, 64, 64, 32768, 8, 1),
        # a short cached prefix taken out for the next chunk of its prompt
        _case("read_prefix_b3", "read", 3, 2, 64, 77, 1000, 16, 0),
        # the whole 32K cache of the Llama3-70B heads, out of pages
        _case("read_32k_paged", "read", 1, 8, 128, 32768, 32768, 64, 64),
        # the tiny decode: 8 heads on 2, d = 32, 1024 tokens
        _case("decode_tiny", "decode", 1, 2, 32, 1024, 1024, 16, 0, 1, 4),
        # the Llama3-70B decode at 32K
        _case("decode_32k", "decode", 1, 8, 128, 32768, 32768, 64, 0, 1, 8),
        # verification of eight drafted tokens at 32K, in pages
        _case("decode_32k_8tokens", "decode", 1, 8, 128, 32768, 32768, 64, 128, 8, 8),
        # a served batch of short sequences in small pages
        _case("decode_b64_pages16", "decode", 64, 4, 64, 65, 4001, 16, 16, 1, 6),
        # odd everything: three queries of five heads, lengths off every tile
        _case("decode_odd_3tokens", "decode", 5, 3, 64, 3, 5003, 32, 0, 3, 5),
        # the ragged batch of eight sequences of 1K to 128K tokens
        _case("decode_ragged_128k", "decode", 8, 8, 128, 1024, 131072, 64, 64, 1, 8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode"])
    d = rng.choice([32, 64, 128, 128])
    H_kv = rng.randint(1, 10)
    block = rng.choice([16, 32, 64, 128])
    page = rng.choice([0, block, 2 * block, 256])
    B = _log_int(rng, 1, 96)
    # at most 2^27 elements of K in the padded batch
    hi = _log_int(rng, 2, max(2, min(131072, (1 << 27) // (B * H_kv * d))))
    lo = rng.randint(max(1, hi // 8), hi)
    T, G, fused = 1, rng.randint(1, 16), 0
    if op == "append":
        T = rng.choice([1, min(hi, rng.randint(2, 9)), hi])
        fused = rng.randint(0, 1)
    elif op == "decode":
        T = min(lo, rng.choice([1, 1, rng.randint(1, 64 // G)]))
    return {k: v for k, v in _case("", op, B, H_kv, d, lo, hi, block, page, T, G, fused).items()
            if k != "name"}


def _lengths(case):
    """Sequence lengths, the longest first; a function of the case alone."""
    r = random.Random("%(op)s %(B)d %(H_kv)d %(d)d %(lo)d %(hi)d %(T)d" % case)
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]


def _new_counts(case):
    """New tokens of each sequence in an append: T, or the whole sequence if it is shorter."""
    return [min(case["T"], n) for n in _lengths(case)]


def work(case):
    lens, H, d, blk = _lengths(case), case["H_kv"], case["d"], case["block"]
    if case["op"] == "append":
        new = _new_counts(case)
        blocks = sum((L - 1) // blk - (L - n) // blk + 1 for L, n in zip(lens, new))
        n = sum(new) * H * d * 2
        return {"bytes": 3 * n + blocks * H * 8, "flops": 4 * n}
    tok = sum(lens) * H * d * 2
    scales = sum(-(-L // blk) for L in lens) * H * 8
    if case["op"] == "read":
        return {"bytes": 3 * tok + scales, "flops": tok}
    rows = case["B"] * case["T"] * H * case["G"]
    flops = 4 * d * H * case["G"] * sum(L * case["T"] for L in lens)
    return {"bytes": tok + scales + rows * (4 * d + 4), "flops": flops}


# ------------------------------------------------------------------ inputs --
def _tokens(n, H, d, g, value):
    """Rows of a K (or V) projection: channels of unequal size with a few large
    ones, tokens of unequal norm."""
    gain = torch.exp(0.4 * torch.randn((H, d), generator=g, device=DEV))
    if not value:
        gain[:, :: 29] *= 4.0
    x = torch.randn((n, H, d), generator=g, device=DEV) * gain
    x *= torch.exp(0.3 * torch.randn((n, 1, 1), generator=g, device=DEV))
    return x


def _fill(x, block):
    """Codes and power-of-two scales of rows x [n, H, d] in whole blocks."""
    n, H, d = x.shape
    x = x.view(n // block, block, H, d)
    s = _scale_for(x.abs().amax(dim=(1, 3)))
    c = (x / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).view(n, H, d), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, H, d, blk, page = (case[k] for k in ("B", "H_kv", "d", "block", "page"))
    T, lens, s = case["T"], _lengths(case), dict(case)
    S = max(lens)
    if page:
        used = [-(-L // page) for L in lens]
        pages = sum(used)
        order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
        table = torch.zeros((B, max(used)), dtype=torch.int32, device=DEV)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u]
            at += u
        rows, per, shape = pages * page, page, (pages, page)
        s["table"], s["max_tokens"] = table, max(used) * page
    else:
        rows, per, shape = B * S, S, (B, S)
        s["table"], s["max_tokens"] = None, S
    per_blk = -(-per // blk)
    # one block more than the cache: a place for what the plain form discards
    units = rows // per
    for name, value in (("k", False), ("v", True)):
        x = _tokens(units * per_blk * blk, H, d, g, value)
        codes, scale = _fill(x, blk)
        del x
        codes = codes.view(units, per_blk * blk, H, d)[:, :per].reshape(rows, H, d)
        s[name + "_all"] = torch.cat([codes, codes[:1]])
        s[name + "_scale_all"] = torch.cat([scale, scale[:1]])
        s[name + "_cache"] = s[name + "_all"][:rows].view(*shape, H, d)
        s[name + "_scale"] = s[name + "_scale_all"][:units * per_blk].view(units, per_blk, H)
        del codes, scale
    s.update(per=per, per_blk=per_blk, rows=rows, scale_rows=units * per_blk, S=S)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if case["op"] == "append":
        s["n_new"] = torch.tensor(_new_counts(case), dtype=torch.int32, device=DEV)
        width = (case["G"] + 2 if case["fused"] else 2) * H * d
        rows_new = torch.empty((B, T, width), dtype=torch.bfloat16, device=DEV)
        for name, end in (("k", width - H * d), ("v", width)):
            x = _tokens(B * T, H, d, g, name == "v").view(B, T, H * d)
            rows_new[:, :, end - H * d:end] = x.to(torch.bfloat16)
            s[name + "_new"] = rows_new[:, :, end - H * d:end].view(B, T, H, d)
    elif case["op"] == "read":
        for name in ("k", "v"):
            s[name + "_out"] = torch.zeros((B, S, H, d), dtype=torch.bfloat16, device=DEV)
    else:
        q = torch.randn((B, T, H * case["G"], d), generator=g, device=DEV)
        s["q"] = q.to(torch.bfloat16)
        s["tau"] = 1.0 / math.sqrt(d)
    return s


# -------------------------------------------------------------- plain forms --
def _scale_for(amax):
    """The smallest power of two s >= 2**MIN_EXP with amax / s <= 448 = 0.875 * 2**9."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e + 127) << 23).view(torch.float32)  # 2**e by its bits: pow is not exact on the GPU


def _rows_of(s, pos):
    """Row of the codes and row of the scales for positions pos [B, n] of each sequence."""
    if s["table"] is None:
        b = torch.arange(pos.shape[0], device=DEV)[:, None]
        return b * s["per"] + pos, b * s["per_blk"] + pos // s["block"]
    unit = s["table"].long().gather(1, (pos // s["page"]).clamp(max=s["table"].shape[1] - 1))
    at = pos % s["page"]
    return unit * s["per"] + at, unit * s["per_blk"] + at // s["block"]


def _values(s, name, rows, srows):
    """fp32 values of the cache rows [B, n, H, d]."""
    c = s[name + "_all"][rows].view(torch.float8_e4m3fn).float()
    return c * s[name + "_scale_all"][srows][..., None]


def _append(s):
    B, blk, T, H, d = s["B"], s["block"], s["T"], s["H_kv"], s["d"]
    L, n = s["lens"].long()[:, None], s["n_new"].long()[:, None]
    nb = (T + blk - 2) // blk + 1  # blocks that T tokens can touch
    first = (L - n) // blk
    pos = first * blk + torch.arange(nb * blk, device=DEV)
    new, old = (pos >= L - n) & (pos < L), pos < L - n
    rows, srows = _rows_of(s, pos.clamp(max=s["max_tokens"] - 1))
    rows = torch.where(new | old, rows, s["rows"])
    sblk = torch.where(new.view(B, nb, blk).any(2), srows.view(B, nb, blk)[:, :, 0], s["scale_rows"])
    has_old = old.view(B, nb, blk).any(2)[..., None]
    take = (pos - (L - n)).clamp(0, T - 1)
    out = []
    for name in ("k", "v"):
        codes, scales = s[name + "_all"], s[name + "_scale_all"]
        x = s[name + "_new"][torch.arange(B, device=DEV)[:, None], take].float()
        x = torch.where(torch.isfinite(x), x, math.nan)
        mag = torch.where(new[..., None, None], x.abs().nan_to_num(nan=0.0), 0.0)
        fresh = _scale_for(mag.view(B, nb, blk, H, d).amax(dim=(2, 4)))
        before = scales[sblk]
        scale = torch.where(has_old, torch.maximum(before, fresh), fresh)
        ratio = torch.where(has_old, before / scale, 1.0).repeat_interleave(blk, 1)[..., None]
        was = codes[rows].view(torch.float8_e4m3fn).float() * ratio
        val = torch.where(new[..., None, None], x / scale.repeat_interleave(blk, 1)[..., None], was)
        codes[rows] = val.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[sblk] = scale
        out += [s[name + "_cache"].view(torch.float8_e4m3fn), s[name + "_scale"]]
    return out


def _read(s):
    pos = torch.arange(s["S"], device=DEV).expand(s["B"], -1)
    rows, srows = _rows_of(s, pos)
    live = (pos < s["lens"][:, None])[..., None, None]
    for name in ("k", "v"):
        val = _values(s, name, rows, srows).to(torch.bfloat16)
        s[name + "_out"].copy_(torch.where(live, val, s[name + "_out"]))
    return [s["k_out"], s["v_out"]]


def _decode(s):
    B, T, H, G, d = s["B"], s["T"], s["H_kv"], s["G"], s["d"]
    pos = torch.arange(s["S"], device=DEV).expand(B, -1)
    rows, srows = _rows_of(s, pos)
    live = (pos < s["lens"][:, None])[..., None, None]
    k = torch.where(live, _values(s, "k", rows, srows), 0.0)
    q = s["q"].float().view(B, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["tau"]  # [B, H, T G, S]
    del k
    # query t of sequence b is at L - T + t and sees every position up to its own
    last = s["lens"][:, None] - T + torch.arange(T, device=DEV)
    seen = pos[:, None, :] <= last[:, :, None]
    x = x.view(B, H, T, G, -1).masked_fill(~seen[:, None, :, None], -math.inf).view(B, H, T * G, -1)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    v = torch.where(live, _values(s, "v", rows, srows), 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total
    o = o.view(B, H, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, H * G, d)
    lse = (m + torch.log(total)).view(B, H, T, G).permute(0, 2, 1, 3).reshape(B, T, H * G)
    return [o.to(torch.bfloat16), lse]


# --------------------------------------------------------------------- run --
def _run_own(s):
    import gqa_attention_gb300 as gqa

    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if s["op"] == "append":
        gqa.kv_append_fp8_block(s["k_new"], s["v_new"], *cache, s["lens"], s["block"],
                                n_new=s["n_new"], block_table=s["table"])
        return [s["k_cache"].view(torch.float8_e4m3fn), s["k_scale"],
                s["v_cache"].view(torch.float8_e4m3fn), s["v_scale"]]
    if s["op"] == "read":
        return list(gqa.kv_read_fp8_block(*cache, s["lens"], s["block"], k_out=s["k_out"],
                                          v_out=s["v_out"], block_table=s["table"]))
    return list(gqa.decode_fp8_block(s["q"], *cache, s["lens"], s["block"], scale=s["tau"],
                                     block_table=s["table"]))


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "read": _read, "decode": _decode}[state["op"]](state)


# ------------------------------------------------------------------- exact --
def _f64_pow2(e):
    """2**e in 64 bits, by its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _f64_e4m3(x):
    """The E4M3 value nearest to each x (ties to the even mantissa), in 64 bits."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = torch.where(a < _f64_pow2(e), e - 1, torch.where(a >= _f64_pow2(e + 1), e + 1, e))
    step = _f64_pow2(e.clamp(min=-6) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _f64_codes(codes):
    """Values of E4M3 codes by their fields: sign, four exponent bits (bias 7), three mantissa bits."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _f64_pow2(e - 10))
    return torch.where(c >= 128, -v, v)


def _f64_sequence(s, name, b, L):
    """K (or V) of the first L tokens of sequence b, and where they lie."""
    H, d, blk, per = s["H_kv"], s["d"], s["block"], s["per"]
    t = torch.arange(L, device=DEV)
    unit = torch.full_like(t, b) if s["table"] is None else s["table"][b].long()[t // per]
    at = t if s["table"] is None else t % per
    codes = s[name + "_cache"].view(-1, per, H, d)
    scale = s[name + "_scale"]
    return _f64_codes(codes[unit, at]), scale[unit, at // blk].double(), unit, at


def exact(case, seed):
    s = prepare(case, seed)
    lens, H, d, blk, T, G = _lengths(case), s["H_kv"], s["d"], s["block"], s["T"], s["G"]
    if case["op"] == "read":
        out = []
        for name in ("k", "v"):
            o = torch.zeros((s["B"], s["S"], H, d), dtype=torch.float64, device=DEV)
            for b, L in enumerate(lens):
                c, sc, _, _ = _f64_sequence(s, name, b, L)
                o[b, :L] = c * sc[..., None]
            out.append(o)
        return out
    if case["op"] == "append":
        out = []
        for name in ("k", "v"):
            per = s["per"]
            val = _f64_codes(s[name + "_cache"]).view(-1, per, H, d)
            scales = s[name + "_scale"].double()
            for b, (L, n) in enumerate(zip(lens, _new_counts(case))):
                t0 = (L - n) // blk * blk  # from the first block that changes
                c, sc, unit, at = (v[t0:] for v in _f64_sequence(s, name, b, L))
                x = c * 1.0
                x[L - n - t0:] = s[name + "_new"][b, :n].double()
                held = L - n - t0
                pad = -(L - t0) % blk
                mag = x.abs()
                mag[:held] = 0
                mag = torch.cat([mag, mag.new_zeros((pad, H, d))]).view(-1, blk, H, d).amax((1, 3))
                e = torch.ceil(torch.log2((mag / 448.0).clamp(min=2.0 ** -100)))
                e = torch.where(mag / _f64_pow2(e) > 448.0, e + 1, e)
                e = torch.where(mag / _f64_pow2(e - 1) <= 448.0, e - 1, e).clamp(min=-100)
                new = _f64_pow2(e)
                if held:
                    new[0] = torch.maximum(new[0], sc[0])
                each = new.repeat_interleave(blk, 0)[: L - t0][..., None]
                held_scale = torch.where((torch.arange(L - t0, device=DEV) < held)[:, None, None],
                                         sc[..., None], 1.0)
                val[unit, at] = _f64_e4m3(x * held_scale / each)
                scales[unit, at // blk] = each[..., 0]
            out += [val.view(s[name + "_cache"].shape), scales]
        return out
    o = torch.zeros((s["B"], T, H * G, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["B"], T, H * G), dtype=torch.float64, device=DEV)
    for b, L in enumerate(lens):
        kc, ks, _, _ = _f64_sequence(s, "k", b, L)
        vc, vs, _, _ = _f64_sequence(s, "v", b, L)
        for h in range(H):
            k, v = kc[:, h] * ks[:, h, None], vc[:, h] * vs[:, h, None]
            heads = slice(h * G, h * G + G)
            x = torch.einsum("tgd,sd->tgs", s["q"][b, :, heads].double(), k) * s["tau"]
            past = torch.arange(L, device=DEV) > (L - T + torch.arange(T, device=DEV))[:, None]
            x = x.masked_fill(past[:, None, :], -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, :, heads] = z
            o[b, :, heads] = torch.einsum("tgs,sd->tgd", torch.exp(x - z[..., None]), v)
    return [o, lse]

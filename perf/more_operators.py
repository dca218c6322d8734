"""Rotated append to the caches, and differential attention over them.

Each case names one operator:

* ``append``: new tokens of every sequence go into a key/value cache, keys and
  the step's queries turned by their positions on the way; the cache is bf16 or
  E4M3 with one scale per token, contiguous (``[B, S_max, H_kv, d]``) or in
  pages (``[num_pages, page_size, H_kv, d]`` behind a block table).
* ``decode``: differential attention of the last ``T`` queries of every
  sequence over a bf16 cache.
* ``prefill``: differential attention of a whole prompt, or of a chunk that ends
  each cached sequence, optionally within a sliding window.

Differential attention of a head: O = softmax(tau q1 K1^T) V - lam softmax(tau
q2 K2^T) V.  Shared keys: q1, q2 are two query heads of one KV head, K1 = K2.
Split keys: q1, q2 and K1, K2 are the halves of a query and a key row.  With
``norm``, O is divided by its root mean square over the head, and scaled.

With ``own`` false the operators run in elementary torch operations, in 32 bits
(the angles in 64).
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5
MIN_EXP = -100  # the smallest scale of an E4M3 token is 2**-100


# ------------------------------------------------------------------- cases --
def _case(name, op, B, H, H_kv, d, lo, hi, T=1, page=0, **more):
    """H: query heads (append) or output heads; lo..hi: the range of the lengths; page 0: a
    contiguous cache; T: new tokens (at most), or queries of a sequence."""
    c = dict(name=name, op=op, B=B, H=H, H_kv=H_kv, d=d, lo=lo, hi=hi, T=T, page=page)
    if op == "append":
        c.update(rot=d, inter=0, fp8=0, fused=0)
    else:
        c.update(split=0, norm=0, window=-1)
    c.update(more)
    return c


def listed():
    return [
        # one sequence gets its next token: nothing but latency
        _case("append_token_b1", "append", 1, 64, 8, 128, 4097, 4097, 1, 64, fused=1),
        # one step of a served batch in small pages, every sequence at its own length, E4M3
        _case("append_tokens_b128_e4m3", "append", 128, 64, 8, 128, 33, 1023, 1, 16, fp8=1, fused=1),
        # a padded batch of prompts, half of each head turned, neighbouring channels paired
        _case("append_prompts_b8", "append", 8, 20, 5, 64, 203, 1531, 1531, 0, rot=32, inter=1),
        # a whole 32K prompt of the Llama3-70B heads
        _case("append_prompt_32k", "append", 1, 64, 8, 128, 32768, 32768, 32768, 64, fused=1),
        # the tiny decode: 8 maps on 2 KV heads, d = 32, 1024 tokens
        _case("decode_tiny", "decode", 1, 4, 2, 32, 1024, 1024),
        # 64 maps on 8 KV heads over the 32K cache
        _case("decode_32k", "decode", 1, 32, 8, 128, 32768, 32768),
        # odd everything: three queries, split keys, normed heads, pages of 16
        _case("decode_odd_3tokens", "decode", 5, 15, 3, 64, 3, 5003, 3, 16, split=1, norm=1),
        # verification of four drafted tokens over a batch in pages
        _case("decode_b4_4tokens", "decode", 4, 32, 8, 128, 2048, 16384, 4, 64, norm=1),
        # a ragged batch of long sequences in pages
        _case("decode_ragged_64k", "decode", 8, 32, 8, 128, 1024, 65536, 1, 64, norm=1),
        # a short chunk of a prompt over its cached start, odd lengths, within a window
        _case("prefill_chunk_window", "prefill", 3, 8, 2, 64, 701, 2903, 333, window=1000),
        # prompts with split keys and normed heads, d = 128
        _case("prefill_split_b2", "prefill", 2, 16, 4, 128, 4001, 4001, 4001, split=1, norm=1),
        # the Llama3-70B prompt of 8K tokens: 64 maps
        _case("prefill_8k", "prefill", 1, 32, 8, 128, 8192, 8192, 8192),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill"])
    d = rng.choice([32, 64, 128, 128])
    H_kv = rng.randint(1, 8)
    page = rng.choice([0, 16, 64, 256])
    if op == "append":
        G = rng.randint(1, 8)
        B = _log_int(rng, 1, 96)
        hi = _log_int(rng, 2, max(2, min(32768, (1 << 25) // (B * H_kv * d))))
        lo = rng.randint(max(1, hi // 8), hi)
        T = rng.choice([1, min(hi, rng.randint(2, 9)), hi])
        c = _case("", op, B, G * H_kv, H_kv, d, lo, hi, T, page, rot=16 * rng.randint(1, d // 16),
                  inter=rng.randint(0, 1), fp8=rng.choice([0, 0, 1]), fused=rng.randint(0, 1))
    elif op == "decode":
        G = rng.randint(1, 8)  # output heads of a KV head
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 2, max(2, min(65536, (1 << 27) // (B * H_kv * d))))
        lo = rng.randint(max(1, hi // 8), hi)
        T = min(lo, rng.choice([1, 1, rng.randint(1, 32 // G)]))
        c = _case("", op, B, G * H_kv, H_kv, d, lo, hi, T, page, split=rng.randint(0, 1),
                  norm=rng.randint(0, 1))
    else:
        G = rng.randint(1, 8)
        B = _log_int(rng, 1, 4)
        hi = _log_int(rng, 2, max(2, min(8192, math.isqrt((1 << 29) // (B * 2 * G * H_kv)))))
        lo = rng.randint(max(1, hi // 2), hi)
        T = rng.choice([lo, rng.randint(1, lo)])
        c = _case("", op, B, G * H_kv, H_kv, d, lo, hi, T, 0, split=rng.randint(0, 1),
                  norm=rng.randint(0, 1), window=rng.choice([-1, -1, rng.randint(0, hi)]))
    del c["name"]
    return c


def _lengths(case):
    """Sequence lengths, the longest first; a function of the case alone."""
    r = random.Random("%(op)s %(B)d %(H)d %(H_kv)d %(d)d %(lo)d %(hi)d %(T)d" % case)
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]


def _new_counts(case):
    """New tokens of each sequence in an append: T, or the whole sequence if it is shorter."""
    return [min(case["T"], n) for n in _lengths(case)]


def _visible(case):
    """(query, key) pairs of one map that the mask keeps, over all sequences."""
    T, W = case["T"], case["window"]
    n = 0
    for L in _lengths(case):
        first, last = L - T + 1, L  # keys that the first and the last query would see
        n += (first + last) * T // 2
        if W >= 0:
            over = [max(0, first - (W + 1)), max(0, last - (W + 1))]
            rows = over[1] - over[0] + 1 if over[0] else over[1] + 1
            n -= (over[0] + over[1]) * rows // 2
    return n


def work(case):
    lens, H, Hk, d = _lengths(case), case["H"], case["H_kv"], case["d"]
    if case["op"] == "append":
        n = sum(_new_counts(case))
        rows = (H + 2 * Hk) * d * 2
        kept = Hk * d * (2 if case["fp8"] else 4) + (8 if case["fp8"] else 0)
        return {"bytes": n * (rows + H * d * 2 + kept), "flops": 3 * n * (H + Hk) * case["rot"]}
    q = case["B"] * case["T"] * H
    seen = lens if case["window"] < 0 else [min(L, case["T"] + case["window"]) for L in lens]
    io = q * d * (2 if case["split"] else 4) + q * (d * 2 + 8 + 4)
    per = 3 * d if case["split"] else 4 * d
    return {"bytes": sum(seen) * Hk * d * 4 + io, "flops": per * 2 * H * _visible(case)}


# ------------------------------------------------------------------ inputs --
def _tokens(n, H, d, g, value):
    """Rows of a K (or V, Q) projection: channels of unequal size with a few large ones, tokens
    of unequal norm."""
    gain = torch.exp(0.4 * torch.randn((H, d), generator=g, device=DEV))
    if not value:
        gain[:, :: 29] *= 2.0
    x = torch.randn((n, H, d), generator=g, device=DEV) * gain
    x *= torch.exp(0.3 * torch.randn((n, 1, 1), generator=g, device=DEV))
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, H, Hk, d, page, T = (case[k] for k in ("B", "H", "H_kv", "d", "page", "T"))
    lens, s = _lengths(case), dict(case)
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
        rows, shape = pages * page, (pages, page)
        s["table"], s["max_tokens"] = table, max(used) * page
    else:
        S = -(-S // 4) * 4
        rows, shape = B * S, (B, S)
        s["table"], s["max_tokens"] = None, S
    s["per"], s["rows"] = shape[1], rows
    # one row more than the cache: a place for what the plain form discards
    fp8 = case["op"] == "append" and case["fp8"]
    for name, value in (("k", False), ("v", True)):
        x = _tokens(rows + 1, Hk, d, g, value)
        if fp8:
            scale = _scale_for(x.abs().amax(dim=(1, 2)))
            codes = (x / scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[name + "_all"], s[name + "_scale_all"] = codes.view(torch.uint8), scale
            s[name + "_scale"] = scale[:rows].view(shape)
        else:
            s[name + "_all"] = x.to(torch.bfloat16)
        s[name] = s[name + "_all"][:rows].view(*shape, Hk, d)
        del x
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if case["op"] == "append":
        s["n_new"] = torch.tensor(_new_counts(case), dtype=torch.int32, device=DEV)
        # the frequencies of a rotation with base 500000
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
        s["freqs"] = torch.exp(-math.log(500000.0) * 2 * i / case["rot"]).float()
        x = [_tokens(B * T, n, d, g, v).view(B, T, n, d) for n, v in ((H, 0), (Hk, 0), (Hk, 1))]
        if case["fused"]:
            wide = torch.cat(x, dim=2).to(torch.bfloat16)
            s["q_new"], s["k_new"], s["v_new"] = wide.split([H, Hk, Hk], dim=2)
        else:
            s["q_new"], s["k_new"], s["v_new"] = (t.to(torch.bfloat16) for t in x)
        s["q_out"] = torch.zeros((B, T, H, d), dtype=torch.bfloat16, device=DEV)
        return s
    s["q"] = torch.randn((B, T, H if case["split"] else 2 * H, d), generator=g,
                         device=DEV).to(torch.bfloat16)
    # a weight per token and head, or one for the layer (the normed form)
    raw = torch.randn((1,) if case["norm"] else (B, T, H), generator=g, device=DEV)
    s["lam"] = torch.sigmoid(raw)
    s["weight"] = torch.exp(0.1 * torch.randn((d,), generator=g, device=DEV)) if case["norm"] else None
    s["out_scale"] = 0.2 if case["norm"] else 1.0
    s["tau"] = 1.0 / math.sqrt(d // 2 if case["split"] else d)
    return s


# -------------------------------------------------------------- plain forms --
def _scale_for(amax):
    """The smallest power of two s >= 2**MIN_EXP with amax / s <= 448 = 0.875 * 2**9."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e + 127) << 23).view(torch.float32)  # 2**e by its bits: pow is not exact on the GPU


def _rows_of(s, pos):
    """Cache rows of the positions pos [B, n] of each sequence."""
    if s["table"] is None:
        return torch.arange(pos.shape[0], device=DEV)[:, None] * s["per"] + pos
    unit = s["table"].long().gather(1, (pos // s["page"]).clamp(max=s["table"].shape[1] - 1))
    return unit * s["per"] + pos % s["page"]


def _turn(x, cos, sin, rot, inter):
    """Rows x [B, T, H, d] with their first `rot` channels turned; cos, sin [B, T, rot / 2]."""
    cos, sin = cos[:, :, None], sin[:, :, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _append(s):
    B, T = s["B"], s["T"]
    L, n = s["lens"].long()[:, None], s["n_new"].long()[:, None]
    i = torch.arange(T, device=DEV)
    pos, live = L - n + i, i < n
    angle = pos.double()[..., None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _turn(s["q_new"].float(), cos, sin, s["rot"], s["inter"]).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(live[..., None, None], q, s["q_out"]))
    rows = torch.where(live, _rows_of(s, pos.clamp(max=s["max_tokens"] - 1)), s["rows"])
    k = _turn(s["k_new"].float(), cos, sin, s["rot"], s["inter"])
    v = s["v_new"].float()
    if not s["fp8"]:
        s["k_all"][rows] = k.to(torch.bfloat16)
        s["v_all"][rows] = v.to(torch.bfloat16)
        return [s["k"], s["v"], s["q_out"]]
    ks, vs = _scale_for(k.abs().amax(dim=(2, 3))), _scale_for(v.abs().amax(dim=(2, 3)))
    s["k_all"][rows] = (k / ks[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(
        torch.uint8)
    s["v_all"][rows] = (v / vs[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(
        torch.uint8)
    s["k_scale_all"][rows] = ks
    s["v_scale_all"][rows] = vs
    return [s["k"].view(torch.float8_e4m3fn), s["k_scale"], s["v"].view(torch.float8_e4m3fn),
            s["v_scale"], s["q_out"]]


def _attend(s):
    """Both maps of every head in one product per KV head."""
    B, T, H, Hk, d, W = (s[k] for k in ("B", "T", "H", "H_kv", "d", "window"))
    G = H // Hk
    n = int(s["max_tokens"])
    pos = torch.arange(n, device=DEV).expand(B, -1)
    live = (pos < s["lens"][:, None])[..., None, None]
    rows = _rows_of(s, pos)
    k = torch.where(live, s["k_all"][rows].float(), 0.0).permute(0, 2, 3, 1)  # [B, Hk, d, n]
    v = torch.where(live, s["v_all"][rows].float(), 0.0).permute(0, 2, 1, 3)  # [B, Hk, n, d]
    q = s["q"].float() * s["tau"]
    if s["split"]:  # [B, Hk, 2, G T, d / 2]
        q = q.view(B, T, Hk, G, 2, d // 2).permute(0, 2, 4, 3, 1, 5).reshape(B, Hk, 2, G * T, d // 2)
        x = torch.matmul(q, k.reshape(B, Hk, 2, d // 2, n))
    else:
        q = q.view(B, T, Hk, G, 2, d).permute(0, 2, 4, 3, 1, 5).reshape(B, Hk, 2 * G * T, d)
        x = torch.matmul(q, k)
    del k, q
    x = x.view(B, Hk, 2 * G, T, n)
    # query t of sequence b is at L - T + t and sees every position up to its own, W back at most
    at = s["lens"][:, None] - T + torch.arange(T, device=DEV)
    hidden = pos[:, None, :] > at[:, :, None]
    if W >= 0:
        hidden = hidden | (pos[:, None, :] < at[:, :, None] - W)
    x.masked_fill_(hidden[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp_(x.sub_(m))
    total = x.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).view(B, Hk, 2, G, T)
    o = torch.matmul(x.view(B, Hk, 2 * G * T, n), v).view(B, Hk, 2, G, T, d)
    o = o / total.view(B, Hk, 2, G, T, 1)
    lam = s["lam"].expand(B, T, H).reshape(B, T, Hk, G).permute(0, 2, 3, 1)[..., None]
    o = o[:, :, 0] - lam * o[:, :, 1]  # [B, Hk, G, T, d]
    if s["norm"]:
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    o = (o * s["out_scale"]).permute(0, 3, 1, 2, 4).reshape(B, T, H, d).to(torch.bfloat16)
    if s["op"] == "prefill":  # [B, 2 H, T]
        return [o, lse.transpose(2, 3).reshape(B, 2 * H, T)]
    return [o, lse.permute(0, 4, 1, 3, 2).reshape(B, T, 2 * H)]


# --------------------------------------------------------------------- run --
def _run_own(s):
    import gqa_attention_gb300 as gqa

    if s["op"] == "append":
        more = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if s["fp8"] else {}
        gqa.kv_append(s["k_new"], s["v_new"], s["k"], s["v"], s["lens"], freqs=s["freqs"],
                      interleaved=bool(s["inter"]), n_new=s["n_new"], q=s["q_new"],
                      q_out=s["q_out"], block_table=s["table"], **more)
        if s["fp8"]:
            return [s["k"].view(torch.float8_e4m3fn), s["k_scale"],
                    s["v"].view(torch.float8_e4m3fn), s["v_scale"], s["q_out"]]
        return [s["k"], s["v"], s["q_out"]]
    form = dict(split_keys=bool(s["split"]), norm_eps=EPS if s["norm"] else None,
                norm_weight=s["weight"], out_scale=s["out_scale"], scale=s["tau"])
    if s["op"] == "prefill":
        return list(gqa.prefill_diff(s["q"], s["k"], s["v"], s["lam"], seq_lens=s["lens"],
                                     window=s["window"], **form))
    return list(gqa.decode_diff(s["q"], s["k"], s["v"], s["lens"], s["lam"],
                                block_table=s["table"], **form))


def run(state):
    if own:
        return _run_own(state)
    return _append(state) if state["op"] == "append" else _attend(state)


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


def _f64_scale(a):
    """The smallest power of two s >= 2**-100 with a / s <= 448."""
    e = torch.ceil(torch.log2((a / 448.0).clamp(min=2.0 ** -100)))
    e = torch.where(a / _f64_pow2(e) > 448.0, e + 1, e)
    return _f64_pow2(torch.where(a / _f64_pow2(e - 1) <= 448.0, e - 1, e).clamp(min=-100))


def _f64_place(s, b, pos):
    """Where the positions pos of sequence b lie in the cache."""
    if s["table"] is None:
        return torch.full_like(pos, b), pos
    return s["table"][b].long()[pos // s["page"]], pos % s["page"]


def _f64_turn(x, pos, s):
    """Each pair of channels of x [n, H, d] as a complex number times exp(i pos f)."""
    r = s["rot"]
    pairs = torch.arange(r, device=DEV)
    pairs = pairs.view(r // 2, 2) if s["inter"] else pairs.view(2, r // 2).T
    phase = pos.double()[:, None] * s["freqs"].double()
    spin = torch.polar(torch.ones_like(phase), phase)[:, None]
    y = x.clone()
    z = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]]) * spin
    y[..., pairs[:, 0]], y[..., pairs[:, 1]] = z.real, z.imag
    return y


def _f64_append(s, case):
    k, v, q = ((s[n].view(torch.float8_e4m3fn) if case["fp8"] and n != "q_out" else s[n]).double()
               for n in ("k", "v", "q_out"))
    ks, vs = (s[n].double() if case["fp8"] else None for n in ("k_scale", "v_scale")) \
        if case["fp8"] else (None, None)
    for b, (L, n) in enumerate(zip(_lengths(case), _new_counts(case))):
        pos = torch.arange(L - n, L, device=DEV)
        at = _f64_place(s, b, pos)
        q[b, :n] = _f64_turn(s["q_new"][b, :n].double(), pos, s)
        x, y = _f64_turn(s["k_new"][b, :n].double(), pos, s), s["v_new"][b, :n].double()
        if case["fp8"]:
            a, c = _f64_scale(x.abs().amax((1, 2))), _f64_scale(y.abs().amax((1, 2)))
            ks[at], vs[at] = a, c
            x, y = _f64_e4m3(x / a[:, None, None]), _f64_e4m3(y / c[:, None, None])
        k[at], v[at] = x, y
    return [k, ks, v, vs, q] if case["fp8"] else [k, v, q]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _f64_append(s, case)
    B, T, H, Hk, d, W = (case[k] for k in ("B", "T", "H", "H_kv", "d", "window"))
    o = torch.zeros((B, T, H, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, T, 2 * H), dtype=torch.float64, device=DEV)
    lam = s["lam"].double().expand(B, T, H)
    for b, L in enumerate(_lengths(case)):
        unit, at = _f64_place(s, b, torch.arange(L, device=DEV))
        for h in range(H):
            kv = h // (H // Hk)
            k, v = s["k"][unit, at, kv].double(), s["v"][unit, at, kv].double()
            for t0 in range(0, T, 2048):  # blocks of queries, each over the keys that it can see
                t1 = min(T, t0 + 2048)
                n = L - T + t1
                i = torch.arange(L - T + t0, n, device=DEV)[:, None]
                j = torch.arange(n, device=DEV)
                hidden = (j > i) if W < 0 else (j > i) | (j < i - W)
                maps = []
                for u in (0, 1):
                    if case["split"]:
                        half = slice(u * (d // 2), (u + 1) * (d // 2))
                        x = s["q"][b, t0:t1, h, half].double() @ k[:n, half].T
                    else:
                        x = s["q"][b, t0:t1, 2 * h + u].double() @ k[:n].T
                    x = (x * s["tau"]).masked_fill_(hidden, -math.inf)
                    z = torch.logsumexp(x, -1)
                    lse[b, t0:t1, 2 * h + u] = z
                    maps.append(torch.exp(x - z[:, None]) @ v[:n])
                o[b, t0:t1, h] = maps[0] - lam[b, t0:t1, h, None] * maps[1]
    if case["norm"]:
        o = o / (o.square().mean(-1, keepdim=True) + EPS).sqrt() * s["weight"].double()
    o = o * s["out_scale"]
    return [o, lse.transpose(1, 2) if case["op"] == "prefill" else lse]

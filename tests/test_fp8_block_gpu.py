"""The block-scaled E4M3 cache on the GPU: append, read back, decode and their
sequence, contiguous and paged, against the 64-bit forms of fp8_block_ref."""
import math

import numpy as np
import pytest
import torch

import fp8_block_ref as ref
import gqa_attention_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_gb300 import build

    build.build()
    g.load()
    yield
    assert g.gqa_last_device_error() == g.GQA_OK


class Cache:
    """A cache of sequences of up to S tokens, contiguous (page = 0) or paged, whose unused
    space holds NaN codes and NaN scales, with its 64-bit copy in sequence order."""

    def __init__(self, B, S, H, d, block, page=0, seed=0):
        self.B, self.S, self.H, self.d, self.block, self.page = B, S, H, d, block, page
        self.gen = torch.Generator().manual_seed(seed)
        per, units = (page, B * -(-S // page) + 2) if page else (S, B)
        self.k8, self.v8, self.ks, self.vs = g.kv_cache_fp8_block(units, per, H, d, block, DEV)
        for c in (self.k8, self.v8):
            c.fill_(0x7F)
        for s in (self.ks, self.vs):
            s.fill_(float("nan"))
        self.table = None
        if page:
            nb = -(-S // page)
            perm = torch.randperm(units, generator=self.gen)[: B * nb].view(B, nb)
            self.table = perm.to(torch.int32).to(DEV)
        nblk = -(-S // block)
        self.val = {n: np.zeros((B, S, H, d)) for n in "kv"}
        self.scale = {n: np.full((B, nblk, H), np.nan) for n in "kv"}
        self.len = [0] * B

    def args(self):
        return self.k8, self.v8, self.ks, self.vs

    def lens(self):
        return torch.tensor(self.len, dtype=torch.int32, device=DEV)

    def rows(self, T, gain=1.0):
        return [(torch.randn(self.B, T, self.H, self.d, generator=self.gen) * gain).to(torch.bfloat16)
                for _ in range(2)]

    def append(self, k, v, counts, pad=0):
        """Append counts[b] of the rows k, v; pad: extra elements after each row."""
        T, w = k.shape[1], self.H * self.d
        wide = torch.full((self.B, T, 2 * w + pad), float("nan"), dtype=torch.bfloat16)
        wide[..., :w], wide[..., w:2 * w] = k.flatten(2), v.flatten(2)
        wide = wide.to(DEV)
        shape = (self.B, T, self.H, self.d)
        self.len = [a + n for a, n in zip(self.len, counts)]
        n_new = None
        if any(n != T for n in counts):
            n_new = torch.tensor(counts, dtype=torch.int32, device=DEV)
        g.kv_append_fp8_block(wide[..., :w].view(shape), wide[..., w:2 * w].view(shape),
                              *self.args(), self.lens(), self.block, n_new=n_new,
                              block_table=self.table)
        for b, n in enumerate(counts):
            if n:
                for name, x in (("k", k), ("v", v)):
                    ref.append(x[b, :n].double().numpy(), self.val[name][b], self.scale[name][b],
                               self.len[b] - n, self.block)

    def gather(self):
        """The GPU's codes (as values) and scales in sequence order."""
        out = {}
        for name, c, s in (("k", self.k8, self.ks), ("v", self.v8, self.vs)):
            c, s = c.cpu(), s.cpu()
            if self.page:
                t = self.table.cpu().long()
                c, s = c[t].flatten(1, 2)[:, :self.S], s[t].flatten(1, 2)[:, :-(-self.S // self.block)]
            out[name] = ref.E4M3[c.numpy()], s.double().numpy()
        return out

    def check(self, what=""):
        got = self.gather()
        for name in "kv":
            val, scale = got[name]
            for b, L in enumerate(self.len):
                nb = -(-L // self.block)
                assert np.array_equal(val[b, :L], self.val[name][b, :L], equal_nan=True), (what, name, b)
                assert np.array_equal(scale[b, :nb], self.scale[name][b, :nb]), (what, name, b)
                # nothing past the end was written
                assert np.isnan(val[b, L:]).all() and np.isnan(scale[b, nb:]).all(), (what, name, b)

    def expect(self, q, tau):
        outs = [ref.attention(q[b].double().numpy(), self.val["k"][b], self.scale["k"][b],
                              self.val["v"][b], self.scale["v"][b], self.len[b], self.block, tau)
                for b in range(self.B)]
        return [np.stack(x) for x in zip(*outs)]


def check_decode(c, T_q, G, n_split, q=None, what=""):
    if q is None:
        q = torch.randn(c.B, T_q, c.H * G, c.d, generator=c.gen).to(torch.bfloat16)
    tau = 1 / math.sqrt(c.d)
    o, lse, tol_o, tol_l = c.expect(q, tau)
    qd = q.to(DEV) if T_q > 1 else q[:, 0].contiguous().to(DEV)
    out, l = g.decode_fp8_block(qd, *c.args(), c.lens(), c.block, n_split=n_split,
                                block_table=c.table)
    torch.cuda.synchronize()
    assert g.gqa_last_device_error() == g.GQA_OK
    do = np.abs(out.double().cpu().numpy().reshape(o.shape) - o)
    dl = np.abs(l.double().cpu().numpy().reshape(lse.shape) - lse)
    assert (dl <= tol_l).all(), (what, n_split, "lse", float((dl / tol_l).max()), float(dl.max()))
    assert (do <= tol_o).all(), (what, n_split, "out", float((do / tol_o).max()), float(do.max()))
    return out, l


# ---------------------------------------------------------------- append -----
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [0, 1, 2])  # times the block
def test_append_prompts_then_tokens(d, block, page):
    """Ragged prompts, then single tokens across a block border with growing magnitudes
    (so that present blocks are rounded again), then several at once."""
    c = Cache(4, 3 * block + 37, 3, d, block, page * block, seed=d + block)
    k, v = c.rows(2 * block + 5)
    c.append(k, v, [2 * block + 5, 1, 0, block - 1], pad=8)
    c.check("prompt")
    for i in range(3):
        k, v = c.rows(1, gain=4.0 ** i)
        c.append(k, v, [1, 1, 1, 1], pad=8 * (i % 2))
        c.check(f"token {i}")
    k, v = c.rows(block // 2 + 3, gain=0.1)
    c.append(k, v, [3, block // 2 + 3, 0, 1])
    c.check("several")


def test_append_all_rows_count_none():
    c = Cache(2, 50, 2, 64, 16, 0, seed=3)
    k, v = c.rows(33)
    c.append(k, v, [33, 33])
    c.check()


def test_append_extremes():
    """Zeros, the type's largest and smallest values, amax at 1.75 * 2^k and next to it."""
    c = Cache(1, 16 * 6, 1, 32, 16, 0, seed=5)
    k, v = c.rows(16 * 6)
    k[0, :16] = 0
    k[0, 16:32] = torch.finfo(torch.bfloat16).max
    k[0, 32:48] = 2.0 ** -130
    k[0, 48:64].clamp_(-1.75, 1.75)[0, 0, 0] = 1.75
    k[0, 64:80].clamp_(-1.75, 1.75)[0, 0, 1] = -1.7578125
    k[0, 80:, :, ::2] *= 2.0 ** -20
    c.append(k, v, [16 * 6])
    c.check()
    assert c.scale["k"][0, 0, 0] == 2.0 ** -100


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_append_non_finite(bad):
    """A non-finite element becomes NaN, alone, and leaves the scale as it would be without it."""
    c = Cache(2, 80, 2, 64, 32, 16 * 2, seed=7)
    k, v = c.rows(40)
    k[0, 3, 0, 5] = bad
    v[1, 39, 1, 63] = bad
    k[1, 32:, 0] = bad  # a block with nothing finite
    c.append(k, v, [40, 40])
    c.check()
    got = c.gather()["k"][0]
    assert np.isnan(got[0, 3, 0, 5]) and np.isfinite(got[0, 3, 0, :5]).all()
    k, v = c.rows(2, gain=30.0)  # the NaN stays through a re-encoding
    c.append(k, v, [2, 2])
    c.check()


def test_append_is_the_same_in_one_call_or_token_by_token():
    """Equal where no scale grew inside a block; otherwise codes rounded twice differ by the
    subnormal step only: half a step (2^-10) for each of the two roundings, times s."""
    a, b = (Cache(1, 64, 2, 128, 16, 0, seed=9) for _ in range(2))
    k, v = a.rows(64)
    a.append(k, v, [64])
    for i in range(64):
        b.append(k[:, i:i + 1], v[:, i:i + 1], [1])
    b.check()
    va, vb = a.gather(), b.gather()
    for n in "kv":
        assert np.array_equal(va[n][1], vb[n][1])
        assert np.abs(va[n][0] - vb[n][0]).max() <= 2 * 2.0 ** -10


def test_append_rejects_bad_lengths_and_pages():
    c = Cache(3, 64, 2, 64, 16, 16, seed=11)
    k, v = c.rows(8)
    c.append(k, v, [8, 8, 8])
    before = [x.clone() for x in c.args()]
    kd = k.to(DEV)

    def same(lens, n, table=None):
        g.kv_append_fp8_block(kd, kd, *c.args(), torch.tensor(lens, dtype=torch.int32, device=DEV),
                              16, n_new=torch.tensor(n, dtype=torch.int32, device=DEV),
                              block_table=c.table if table is None else table)
        assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
        for x, y in zip(c.args(), before):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))

    same([65, 0, 0], [1, 0, 0])     # past the cache
    same([3, 0, 0], [4, 0, 0])      # more new tokens than the sequence has
    same([20, 0, 0], [9, 0, 0])     # more than T
    same([20, 0, 0], [-1, 0, 0])
    same([-5, 0, 0], [0, 0, 0])
    wrong = c.table.clone()
    wrong[1] = wrong.new_tensor([2 ** 30, -1, 10 ** 6, -7])
    same([0, 16, 0], [0, 8, 0], wrong)


# ------------------------------------------------------------------ read -----
@pytest.mark.parametrize("d,block,page", [(32, 16, 0), (64, 32, 64), (128, 64, 64), (128, 16, 32),
                                          (64, 128, 0)])
def test_read_back(d, block, page):
    c = Cache(3, 300, 3, d, block, page, seed=d)
    k, v = c.rows(300)
    c.append(k, v, [300, 1, 129])
    for start, S_out in [(0, 300), (7, 100), (128, 172), (299, 1)]:
        ko, vo = (torch.full((3, S_out, 3, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        g.kv_read_fp8_block(*c.args(), c.lens(), block, start, ko, vo, c.table)
        for name, out in (("k", ko), ("v", vo)):
            want = np.full((3, S_out, 3, d), 7.0)
            for b, L in enumerate(c.len):
                n = max(0, min(S_out, L - start))
                at = np.arange(start, start + n)
                want[b, :n] = c.val[name][b, at] * c.scale[name][b, at // block][..., None]
            # power-of-two scales: exact in bf16
            assert np.array_equal(out.double().cpu().numpy(), want), (start, S_out, name)


def test_read_back_any_scale():
    """Scales that are no powers of two round once, to nearest: half a step of bf16."""
    c = Cache(1, 100, 2, 64, 32, 0, seed=2)
    k, v = c.rows(100)
    c.append(k, v, [100])
    c.ks.copy_(torch.rand(c.ks.shape, generator=c.gen) + 0.1)
    ko, _ = g.kv_read_fp8_block(*c.args(), c.lens(), 32)
    s = c.ks.cpu().double().numpy()[0][np.arange(100) // 32][..., None]
    want = (c.val["k"][0] * s).astype(np.float32)  # the product's own rounding: 2^-24
    got = ko[0].float().cpu().numpy()
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()


def test_read_rejects_bad_lengths_and_pages():
    c = Cache(2, 64, 2, 64, 16, 16, seed=4)
    k, v = c.rows(64)
    c.append(k, v, [64, 64])
    lens = torch.tensor([65, 64], dtype=torch.int32, device=DEV)
    ko, vo = g.kv_read_fp8_block(*c.args(), lens, 16, block_table=c.table)
    assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
    assert bool(ko[0].isnan().all()) and bool(vo[0].isnan().all()) and bool(ko[1].isfinite().all())
    wrong = c.table.clone()
    wrong[1, 2] = -3
    ko, _ = g.kv_read_fp8_block(*c.args(), c.lens(), 16, block_table=wrong)
    assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
    assert bool(ko[1, 32:48].isnan().all()) and bool(ko[1, :32].isfinite().all())
    assert bool(ko[1, 48:].isfinite().all()) and bool(ko[0].isfinite().all())


# ---------------------------------------------------------------- decode -----
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
@pytest.mark.parametrize("ctx", [1, 127, 128, 129, 700])
def test_decode_small(d, G, ctx):
    c = Cache(1, ctx + 3, 2, d, 16, 0, seed=ctx + G + d)
    k, v = c.rows(ctx)
    c.append(k, v, [ctx])
    for n_split in (1, 3, None):
        check_decode(c, 1, G, n_split, what=f"d={d} G={G} ctx={ctx}")


@pytest.mark.parametrize("T_q,G", [(2, 4), (3, 5), (2, 16), (8, 8), (64, 1), (13, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_several_tokens(T_q, G, d):
    c = Cache(2, 600, 2, d, 32, 0, seed=T_q + G)
    k, v = c.rows(600)
    c.append(k, v, [600, T_q])  # the second sequence: the queries' own tokens and no more
    for n_split in (1, 5):
        check_decode(c, T_q, G, n_split, what=f"T_q={T_q} G={G}")


@pytest.mark.parametrize("block,page", [(16, 16), (16, 64), (64, 64), (32, 128), (128, 256)])
@pytest.mark.parametrize("T_q,G", [(1, 8), (4, 7)])
def test_decode_paged_ragged(block, page, T_q, G):
    c = Cache(4, 1000, 2, 128, block, page, seed=block + page)
    k, v = c.rows(1000)
    c.append(k, v, [1000, T_q, 385, 128 + T_q])
    for n_split in (1, 2, 7):
        check_decode(c, T_q, G, n_split, what=f"block={block} page={page}")


def test_decode_scales_of_every_size():
    """Neighbouring blocks whose scales differ by 2^24 either way, for K and for V: the large
    V block must not drown where the softmax puts it at zero, nor the small one vanish."""
    c = Cache(1, 400, 1, 128, 16, 0, seed=21)
    k, v = c.rows(400)
    c.append(k, v, [400])
    q = torch.randn(1, 1, 8, 128, generator=c.gen).to(torch.bfloat16)
    e = torch.randint(-12, 13, c.vs.shape, generator=c.gen)
    for name, t, by in (("v", c.vs, 2.0 ** e.float()), ("k", c.ks, 2.0 ** (e.float() / 6))):
        t.mul_(by.to(DEV))
        c.scale[name] = t.double().cpu().numpy()
        for n_split in (1, 3):
            check_decode(c, 1, 8, n_split, q=q, what=name)


def test_decode_zero_and_tiny_value_scales():
    c = Cache(1, 64, 1, 64, 16, 0, seed=22)
    k, v = c.rows(64)
    c.append(k, v, [64])
    c.vs[0, 1] = 0.0
    c.vs[0, 2] = 2.0 ** -101  # counts as zero
    c.scale["v"] = c.vs.double().cpu().numpy()
    c.scale["v"][0, 2] = 0.0
    check_decode(c, 1, 4, 1)
    c.vs.zero_()
    q = torch.ones(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = g.decode_fp8_block(q, *c.args(), c.lens(), 16)
    assert bool((out == 0).all()) and bool(lse.isfinite().all())


def test_decode_one_key_far_above_the_others():
    """A first token that takes nearly all the weight and has a value near zero."""
    c = Cache(1, 3000, 1, 128, 16, 0, seed=23)
    k, v = c.rows(3000)
    q = torch.randn(1, 1, 8, 128, generator=c.gen).to(torch.bfloat16)
    k[0, 0, 0] = q[0, 0, 0] * 1.5
    v[0, :16] *= 2.0 ** -7
    c.append(k, v, [3000])
    for n_split in (1, 4):
        check_decode(c, 1, 8, n_split, q=q)


def test_decode_non_finite():
    """A NaN in the cache reaches the rows that see it; a non-finite query its own row."""
    c = Cache(1, 300, 2, 64, 16, 0, seed=24)
    k, v = c.rows(300)
    k[0, 299, 0, 3] = float("nan")
    c.append(k, v, [300])
    q = torch.randn(1, 2, 8, 64, generator=c.gen).to(torch.bfloat16)
    q[0, 0, 6, 1] = float("inf")
    out, lse = g.decode_fp8_block(q.to(DEV), *c.args(), c.lens(), 16, n_split=2)
    nan = out[0].isnan().all(-1).cpu()
    fin = out[0].isfinite().all(-1).cpu()
    # query 0 does not see token 299; heads 0-3 read KV head 0
    assert nan.tolist() == [[False] * 6 + [True, False], [True] * 4 + [False] * 4]
    assert torch.equal(fin, ~nan) and torch.equal(lse[0].isnan().cpu(), nan)


def test_decode_rejects_bad_lengths_and_pages():
    c = Cache(3, 256, 2, 64, 16, 16, seed=25)
    k, v = c.rows(256)
    c.append(k, v, [256, 200, 100])
    q = torch.randn(3, 2, 4, 64, generator=c.gen).to(torch.bfloat16).to(DEV)
    good, _ = g.decode_fp8_block(q, *c.args(), c.lens(), 16, n_split=1, block_table=c.table)
    wrong = c.table.clone()
    wrong[2, 1] = c.k8.shape[0]
    for n_split in (1, 2):
        for lens in ([257, 200, 100], [1, 200, 100]):
            out, lse = g.decode_fp8_block(q, *c.args(),
                                          torch.tensor(lens, dtype=torch.int32, device=DEV), 16,
                                          n_split=n_split, block_table=c.table)
            assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
            assert bool(out[0].isnan().all()) and bool(lse[0].isnan().all())
            assert bool(out[1:].isfinite().all())
        out, lse = g.decode_fp8_block(q, *c.args(), c.lens(), 16, n_split=n_split,
                                      block_table=wrong)
        assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
        assert bool(out[2].isnan().all()) and bool(out[:2].isfinite().all())
        if n_split == 1:
            assert torch.equal(out[:2], good[:2])


def test_decode_does_not_read_past_the_table():
    """Entries of the block table for tokens past the end may be anything."""
    c = Cache(2, 512, 1, 128, 16, 16, seed=26)
    k, v = c.rows(512)
    c.append(k, v, [512, 33])
    c.table[1, 3:] = -(10 ** 6)
    for n_split in (1, 4):
        check_decode(c, 1, 8, n_split)


def test_decode_is_deterministic():
    c = Cache(2, 5000, 8, 128, 64, 64, seed=27)
    k, v = c.rows(5000)
    c.append(k, v, [5000, 1234])
    q = torch.randn(2, 64, 128, generator=c.gen).to(torch.bfloat16).to(DEV)
    runs = [g.decode_fp8_block(q, *c.args(), c.lens(), 64, block_table=c.table) for _ in range(3)]
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])


# ----------------------------------------------------- as they are used -----
@pytest.mark.parametrize("page", [0, 64])
def test_prompt_chunk_then_tokens(page):
    """A prompt is appended, its second chunk attends through the read-back, then tokens are
    appended and decoded one and three at a time."""
    c = Cache(2, 500, 2, 128, 64, page, seed=31)
    k, v = c.rows(400)
    c.append(k, v, [400, 301])
    T, G, tau = 150, 4, 1 / math.sqrt(128)
    q = torch.randn(2, T, 2 * G, 128, generator=c.gen).to(torch.bfloat16)
    out, lse = g.prefill_chunk_fp8_block(q.to(DEV), *c.args(), c.lens(), 64, block_table=c.table)
    o, l, _, _ = c.expect(q, tau)
    # the parity bar of the bf16 kernels
    assert np.abs(out.double().cpu().numpy() - o).max() <= 2e-2
    assert np.abs(lse.double().cpu().numpy().transpose(0, 2, 1) - l).max() <= 1e-3
    for T in (1, 3, 1):
        k, v = c.rows(T)
        c.append(k, v, [T, T], pad=16)
        check_decode(c, T, G, None)
        check_decode(c, T, G, 3)
    c.check()


def test_captured_step_replays():
    """Append + decode + combine captured once and replayed for the next tokens, lengths and
    rows changing in place, on a stream of its own."""
    B, H, G, d, block = 3, 2, 8, 128, 16
    a, b = (Cache(B, 300, H, d, block, 16, seed=33) for _ in range(2))
    k, v = a.rows(200)
    for c in (a, b):
        c.append(k, v, [200, 31, 100])
    kn = torch.zeros(B, 1, H, d, dtype=torch.bfloat16, device=DEV)
    vn, q = torch.zeros_like(kn), torch.zeros(B, H * G, d, dtype=torch.bfloat16, device=DEV)
    lens = a.lens()
    out = torch.empty_like(q)
    lse = torch.empty(B, H * G, dtype=torch.float32, device=DEV)
    ws = g.decode_workspace(B, H * G, d, 3)

    def step():
        lens.add_(1)
        g.kv_append_fp8_block(kn, vn, *a.args(), lens, block, block_table=a.table)
        g.decode_fp8_block(q, *a.args(), lens, block, n_split=3, workspace=ws, out=out, lse=lse,
                           block_table=a.table)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    lens.copy_(a.lens())
    for i in range(20):
        k, v = b.rows(1, gain=1.0 + i)
        qi = torch.randn(B, H * G, d, generator=b.gen).to(torch.bfloat16)
        kn.copy_(k), vn.copy_(v), q.copy_(qi)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.append(k, v, [1] * B)
        want, wl = g.decode_fp8_block(qi.to(DEV), *b.args(), b.lens(), block, n_split=3,
                                      block_table=b.table)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for x, y in zip(a.args(), b.args()))


def test_two_streams_at_once():
    caches = [Cache(2, 2000, 4, 128, 64, 0, seed=41 + i) for i in range(2)]
    qs, want = [], []
    for c in caches:
        k, v = c.rows(2000)
        c.append(k, v, [2000, 777])
        q = torch.randn(2, 32, 128, generator=c.gen).to(torch.bfloat16).to(DEV)
        qs.append(q)
        want.append(g.decode_fp8_block(q, *c.args(), c.lens(), 64))
    lens = [c.lens() for c in caches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = [[], []]
    for _ in range(8):
        for i, c in enumerate(caches):
            got[i].append(g.decode_fp8_block(qs[i], *c.args(), lens[i], 64, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_helpers_refuse():
    c = Cache(2, 64, 2, 64, 16, 0, seed=51)
    k, v = (x.to(DEV) for x in c.rows(4))
    lens = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    args = (*c.args(), lens, 16)
    for bad in (k.float(), k.transpose(1, 2), k[:, :, :1], k[:1], k.permute(0, 1, 3, 2)):
        with pytest.raises(g.GQAError):
            g.kv_append_fp8_block(bad, bad, *args)
    with pytest.raises(g.GQAError):  # rows of K and V at different strides
        g.kv_append_fp8_block(k, torch.cat([v, v], -1)[..., :64], *args)
    with pytest.raises(g.GQAError):
        g.kv_append_fp8_block(k, v, *c.args(), lens.long(), 16)
    with pytest.raises(g.GQAError):
        g.decode_fp8_block(k[:, 0], *c.args(), lens, 32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(g.GQAError):
        g.decode_fp8_block(q, *args, n_split=2, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(g.GQAError):
        g.decode_fp8_block(q, *args, out=torch.empty(2, 4, 64, device=DEV))
    with pytest.raises(g.GQAError):
        g.kv_read_fp8_block(*args, k_out=torch.empty(2, 4, 2, 64, device=DEV))
    g.kv_append_fp8_block(k[:, :0], v[:, :0], *args)  # no rows: nothing to do


# ------------------------------------------------- heads that share a tile ---
@pytest.mark.parametrize("d,H", [(64, 2), (64, 5), (32, 3), (32, 4), (32, 6)])
@pytest.mark.parametrize("T_q,G", [(1, 1), (1, 6), (3, 5), (1, 16), (2, 16)])
@pytest.mark.parametrize("page", [0, 32])
def test_decode_grids_that_fill_the_gpu(d, H, T_q, G, page):
    """With d = 32, a multiple of four heads and a grid larger than the GPU holds at once, a CTA
    takes four heads (unless their rows do not fit)."""
    c = Cache(2, 900, H, d, 16, page, seed=d + H + T_q + G)
    k, v = c.rows(900)
    c.append(k, v, [900, 130 + T_q])
    check_decode(c, T_q, G, 90, what=f"d={d} H={H} T_q={T_q} G={G}")


def test_decode_heads_that_share_a_tile_stay_apart():
    """NaN in one head's keys and values leaves the neighbours in the tile finite."""
    c = Cache(1, 400, 4, 32, 16, 0, seed=61)
    k, v = c.rows(400)
    k[0, 7, 1, 3] = float("nan")
    v[0, 300, 2, 5] = float("inf")
    c.append(k, v, [400])
    q = torch.randn(1, 1, 12, 32, generator=c.gen).to(torch.bfloat16)
    out, lse = g.decode_fp8_block(q.to(DEV), *c.args(), c.lens(), 16, n_split=200)
    nan = out[0, 0].isnan().cpu()
    want = torch.zeros(12, 32, dtype=torch.bool)
    want[3:6] = True
    want[6:9, 5] = True
    assert torch.equal(nan, want)
    assert lse[0, 0].isnan().cpu().tolist() == [False] * 3 + [True] * 3 + [False] * 6

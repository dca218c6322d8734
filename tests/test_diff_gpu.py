"""Differential attention on the GPU, decode and prefill, against the 64-bit form of diff_ref,
and the append, prefill and decode of a sequence run together."""
import numpy as np
import pytest
import torch

import diff_ref as ref
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


class Case:
    """A cache of sequences whose unused rows and pages hold NaN, and queries."""

    def __init__(self, lens, T, H, Hk, d, split=False, page=0, S=None, norm=False, lam="token", seed=0):
        gen = self.gen = torch.Generator().manual_seed(seed)
        self.lens, self.T, self.H, self.Hk, self.d, self.split = lens, T, H, Hk, d, split
        B, S = len(lens), S or max(lens)
        self.B, self.S, self.page = B, S, page
        rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.seq = [[rnd(L, Hk, d).to(torch.bfloat16) for _ in "kv"] for L in lens]
        per, units = (page, B * -(-S // page) + 2) if page else (S, B)
        self.k, self.v = (torch.full((units, per, Hk, d), float("nan"), dtype=torch.bfloat16)
                          for _ in "kv")
        self.table = None
        if page:
            self.table = torch.randperm(units, generator=gen)[: B * -(-S // page)].view(B, -1)
        for b, (kv, L) in enumerate(zip(self.seq, lens)):
            for c, x in zip((self.k, self.v), kv):
                if page:
                    t = torch.arange(L)
                    c[self.table[b, t // page], t % page] = x
                else:
                    c[b, :L] = x
        self.k, self.v = self.k.to(DEV), self.v.to(DEV)
        if page:
            self.table = self.table.to(torch.int32).to(DEV)
        self.q = rnd(B, T, H if split else 2 * H, d).to(torch.bfloat16)
        shape = {"token": (B, T, H), "layer": (1,), "head": (H,), "row": (B, T, 1)}[lam]
        self.lam = torch.sigmoid(rnd(*shape))
        self.form = dict(split_keys=split)
        self.weight = None
        if norm:
            self.weight = torch.exp(0.2 * rnd(d))
            self.form.update(norm_eps=1e-3, norm_weight=self.weight.to(DEV), out_scale=0.3)

    def dev_lens(self):
        return torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def expect(self, window=-1):
        lam = self.lam.expand(self.B, self.T, self.H).double().numpy()
        more = {} if self.weight is None else dict(norm_eps=1e-3, weight=self.weight.double().numpy(),
                                                   out_scale=0.3)
        outs = [ref.attention(self.q[b].double().numpy(), self.seq[b][0].double().numpy(),
                              self.seq[b][1].double().numpy(), lam[b],
                              ref.default_scale(self.d, self.split), self.split, window=window,
                              **more) for b in range(self.B)]
        return [np.stack(x) for x in zip(*outs)]

    def compare(self, out, lse, want, what=""):
        torch.cuda.synchronize()
        assert g.gqa_last_device_error() == g.GQA_OK
        o, l, tol, tol_l = want
        do = np.abs(out.double().cpu().numpy().reshape(o.shape) - o)
        dl = np.abs(lse.double().cpu().numpy().reshape(l.shape) - l)
        assert (do <= tol).all(), (what, (do / tol).max())
        assert (dl <= tol_l).all(), (what, (dl / tol_l).max())

    def decode(self, **kw):
        q, lam = self.q.to(DEV), self.lam.to(DEV)
        if self.T == 1 and not kw.pop("four", False):
            q = q[:, 0].contiguous()
            lam = lam[:, 0] if lam.dim() == 3 else lam
        return g.decode_diff(q, self.k, self.v, self.dev_lens(), lam, block_table=self.table,
                             **self.form, **kw)

    def prefill(self, **kw):
        return g.prefill_diff(self.q.to(DEV), self.k, self.v, self.lam.to(DEV),
                              **{"seq_lens": self.dev_lens(), **self.form, **kw})


# --------------------------------------------------------------------- decode --
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("T,H,Hk,norm", [
    (1, 3, 3, False),    # two rows of a KV head
    (1, 8, 2, True),     # eight
    (1, 16, 2, False),   # sixteen
    (3, 5, 1, True),     # 30: two groups of a CTA
    (8, 8, 2, False),    # 64: two CTAs
    (7, 3, 1, True),     # 42, off every group
])
def test_decode(d, split, page, T, H, Hk, norm):
    c = Case([T, 77, 300], T, H, Hk, d, split, page, norm=norm, lam="token", seed=T + d)
    want = c.expect()
    for n_split in (1, 3, None):
        out, lse = c.decode(n_split=n_split)
        c.compare(out, lse, want, n_split)


@pytest.mark.parametrize("d,split", [(32, False), (64, True), (64, False)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("T", [3, 8])
def test_decode_of_more_heads_and_sequences_than_sms(d, split, page, T):
    lens = [700, T] + [T + 37 * i % 211 for i in range(38)]
    c = Case(lens, T, 20, 5, d, split, page, norm=T == 3, lam="token", seed=d + T)
    want = c.expect()
    for n_split in (1, 2, 5, None):
        c.compare(*c.decode(n_split=n_split), want, n_split)


@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("page", [0, 16])
def test_decode_of_clusters_on_nearly_every_sm(d, page):
    c = Case([900, 3, 500, 65], 3, 16, 4, d, False, page, norm=True, lam="token", seed=d)
    want = c.expect()
    a, b = c.decode(n_split=1), c.decode(n_split=1)
    c.compare(*a, want)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,split", [(32, False), (64, True), (128, False)])
def test_many_prompts_of_one_tile(d, split):
    # (a CTA takes one item of one tile after another: ten rounds)
    c = Case([100 - b % 7 for b in range(80)], 40, 32, 8, d, split, norm=True, lam="token", seed=d)
    a = c.prefill()
    o, l, tol, tol_l = c.expect()
    c.compare(*a, (o, l.transpose(0, 2, 1), tol, tol_l.transpose(0, 2, 1)))
    for _ in range(20):
        b = c.prefill()
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,split,S,window", [(64, False, 1030, -1), (128, True, 900, -1),
                                              (32, False, 1500, 900)])
def test_prompts_of_few_heads_in_the_default_parts(d, split, S, window):
    c = Case([S], S, 2, 1, d, split, norm=True, lam="token", seed=S)
    assert g.gqa_attn_prefill_diff_default_parts(1, S, S, 2, 1, window) > 1
    want = c.expect(window)
    o, l, tol, tol_l = want
    want = (o, l.transpose(0, 2, 1), tol, tol_l.transpose(0, 2, 1))
    c.compare(*c.prefill(window=window), want)
    if window < 0:
        c.compare(*c.prefill(seq_lens=None), want)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("page,T,H,Hk", [(0, 2, 16, 2), (64, 4, 8, 1), (16, 5, 4, 1), (0, 3, 8, 1)])
def test_decode_of_a_batch_cut_by_its_lengths(split, page, T, H, Hk):
    # (enough tiles of one or two KV heads that the cut is taken: 16 to an SM)
    S = 90000 if Hk == 2 else 180000
    lens = [9000, T, 2000, 300, 129]
    c = Case(lens, T, H, Hk, 128, split, page, norm=page != 64, S=None, lam="head")
    want = c.expect()
    if page:  # a table much wider than the sequences
        wide = torch.zeros(c.B, S // page, dtype=torch.int32, device=DEV)
        wide[:, :c.table.shape[1]] = c.table
        c.table = wide
        for n in (None, 2, 7, 64):
            c.compare(*c.decode(n_split=n), want, n)
        a, b = c.decode(), c.decode()
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
        lens = c.dev_lens()
        lens[2] = T - 1
        out, lse = g.decode_diff(c.q.to(DEV), c.k, c.v, lens, c.lam.to(DEV), block_table=c.table, **c.form)
        torch.cuda.synchronize()
        assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
        assert out[2].isnan().all() and lse[2].isnan().all()
        ok = [0, 1, 3, 4]
        assert (np.abs(out.double().cpu().numpy() - want[0])[ok] <= want[2][ok]).all()
    else:
        k, v = (torch.full((c.B, S, Hk, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
                for _ in "kv")
        k[:, :c.S], v[:, :c.S] = c.k, c.v
        c.k, c.v = k, v
        for n in (None, 3, 16):
            c.compare(*c.decode(n_split=n), want, n)


@pytest.mark.parametrize("d,T,H,Hk,page", [(128, 1, 8, 1, 64), (64, 3, 6, 1, 16), (32, 1, 2, 1, 128),
                                           (64, 16, 2, 1, 32)])
def test_smaller_rows_of_a_batch_cut_by_its_lengths(d, T, H, Hk, page):
    # a table much wider than the sequences: enough tiles of one KV head that the cut is taken
    lens = [9000, T, 64, 129]
    c = Case(lens, T, H, Hk, d, d == 64, page, norm=True, lam="head")
    want = c.expect()
    wide = torch.zeros(c.B, 200000 // page, dtype=torch.int32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    for n in (None, 2, 7, 64):
        c.compare(*c.decode(n_split=n), want, n)
    a, b = c.decode(), c.decode()
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
    for wrong in (0, 200001):
        bad = c.dev_lens()
        bad[1] = wrong
        q, lam = c.q.to(DEV), c.lam.to(DEV)
        out, lse = g.decode_diff(q, c.k, c.v, bad, lam, block_table=c.table, **c.form)
        torch.cuda.synchronize()
        assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
        assert out[1].isnan().all() and lse[1].isnan().all()
        ok = [0, 2, 3]
        assert (np.abs(out.double().cpu().numpy() - want[0])[ok] <= want[2][ok]).all()


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 1000, 5003])
def test_decode_lengths(L):
    for page, n in ((0, 1), (16, None), (64, 7), (0, 40)):
        c = Case([L, max(1, L // 3)], 1, 8, 2, 64, page=page, norm=True, lam="layer", seed=L)
        c.compare(*c.decode(n_split=n), c.expect(), (page, n))


@pytest.mark.parametrize("lam", ["token", "layer", "head", "row"])
def test_lam_broadcasts(lam):
    c = Case([40, 90], 2, 4, 2, 64, lam=lam)
    want = c.expect()
    c.compare(*c.decode(), want)
    c.compare(*c.prefill(), [want[0], want[1].transpose(0, 2, 1), want[2], want[3].transpose(0, 2, 1)])
    c = Case([40, 90], 1, 4, 2, 64, lam=lam)
    want = c.expect()
    c.compare(*c.decode(), want)
    c.compare(*c.decode(four=True), want)
    base = torch.rand(2, 1, 4, 3)  # a strided view
    c = Case([40, 90], 1, 4, 2, 64)
    c.lam = base[..., 1]
    lam = base.to(DEV)[:, 0, :, 1]
    out = g.decode_diff(c.q[:, 0].contiguous().to(DEV), c.k, c.v, c.dev_lens(), lam)
    c.compare(*out, c.expect())


def test_lam_of_any_sign_and_equal_maps():
    c = Case([70], 1, 4, 2, 32)
    c.lam = torch.tensor([-3.0, 0.0, 2.5, 1.0]).view(1, 1, 4)
    c.compare(*c.decode(n_split=1), c.expect())
    # equal maps and lam = 1: exactly nothing is left
    c.q = c.q.view(1, 1, 4, 2, 32)[:, :, :, :1].expand(1, 1, 4, 2, 32).reshape(1, 1, 8, 32).contiguous()
    c.lam = torch.ones(1)
    for n in (1, 2):
        out, _ = c.decode(n_split=n)
        assert (out == 0).all()
        out, _ = c.prefill(n_part=n)
        assert (out == 0).all()


def test_decode_of_one_map_is_the_plain_decode():
    c = Case([2000, 500], 1, 16, 4, 128)
    c.lam = torch.zeros(1)
    out, lse = c.decode()
    ro, rl = g.decode(c.q[:, 0].contiguous().to(DEV), c.k, c.v, c.dev_lens())
    assert (lse - rl).abs().max() <= 2.0 ** -16
    assert (out.float() - ro.float()[:, ::2]).abs().max() <= 2.0 ** -7 * ro.float().abs().max()


def test_decode_is_deterministic():
    c = Case([3000, 100, 1], 1, 16, 2, 128, page=16, norm=True, lam="layer")
    a = c.decode()
    for _ in range(3):
        b = c.decode()
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_values_that_a_query_does_not_see_do_not_reach_it():
    for bad in (float("nan"), float("inf")):
        for d, T, n_split, H in ((64, 6, 1, 4), (128, 4, 2, 4), (32, 4, 1, 4), (128, 6, 1, 4),
                                 (128, 12, 2, 4), (128, 9, 1, 6)):
            c = Case([70 + T, 123 + T // 2], T, H, 2, d, split=T == 9, seed=d + T)
            want = c.expect()
            first = c.decode(n_split=n_split)
            c.compare(*first, want)
            for b, L in enumerate(c.lens):
                c.v[b, L - 2] = bad  # seen by the last two queries
                c.k[b, L - 1] = bad  # seen by the last one
            out, lse = c.decode(n_split=n_split)
            # the others' rows are as before: bit for bit
            assert torch.equal(out[:, :-2].view(torch.int16), first[0][:, :-2].view(torch.int16))
            assert torch.equal(lse[:, :-1], first[1][:, :-1])
            assert not torch.isfinite(out[:, -2:].float()).any()


def test_rows_of_the_cache_past_the_end_may_hold_anything():
    for fill in (float("nan"), float("inf"), 3e38):
        c = Case([5, 66], 1, 4, 2, 64, S=130)
        for b, L in enumerate(c.lens):
            c.k[b, L:] = fill
            c.v[b, L:] = fill
        want = c.expect()
        for n in (1, 2, 5):
            c.compare(*c.decode(n_split=n), want)


def test_large_scores():
    c = Case([200], 1, 4, 2, 64)
    c.q = (c.q.float() * 60).to(torch.bfloat16)
    want = c.expect()
    for n in (1, 3):
        c.compare(*c.decode(n_split=n), want)


def test_bad_lengths_and_pages():
    c = Case([50, 60, 70], 2, 4, 2, 64, page=16, S=80)
    want = c.expect()
    for wrong in (0, 1, 81, -7):
        lens = c.dev_lens()
        lens[1] = wrong
        for n in (1, 4):
            out, lse = g.decode_diff(c.q.to(DEV), c.k, c.v, lens, c.lam.to(DEV), n_split=n,
                                     block_table=c.table)
            torch.cuda.synchronize()
            assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
            assert out[1].isnan().all() and lse[1].isnan().all()
            ok = [0, 2]
            assert (np.abs(out.double().cpu().numpy() - want[0])[ok] <= want[2][ok]).all()
    for wrong in (-1, c.k.shape[0], 2 ** 31 - 1):
        table = c.table.clone()
        table[2, 1] = wrong
        for n in (1, 2):
            out, _ = g.decode_diff(c.q.to(DEV), c.k, c.v, c.dev_lens(), c.lam.to(DEV), n_split=n,
                                   block_table=table)
            torch.cuda.synchronize()
            assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
            assert out[2].isnan().all() and not out[:2].isnan().any()
    # entries past a sequence's end are not looked at
    table = c.table.clone()
    table[0, 4:] = -9
    c.compare(*g.decode_diff(c.q.to(DEV), c.k, c.v, c.dev_lens(), c.lam.to(DEV), block_table=table),
              want)


def test_a_long_split_of_small_pages():
    # 2100 pages in one split
    c = Case([33600], 1, 2, 1, 32, page=16, lam="layer")
    c.compare(*c.decode(n_split=1), c.expect())


def test_pages_that_sequences_share_and_repeat():
    c = Case([64, 64], 1, 4, 2, 64, page=16)
    table = c.table.clone()
    table[1, :2] = table[0, :2]  # a shared prefix
    table[0, 3] = table[0, 2]    # the same page twice in a sequence
    seq = [[torch.cat([x[:48], x[32:48]]) for x in c.seq[0]],
           [torch.cat([x[:32], y[32:]]) for x, y in zip(c.seq[0], c.seq[1])]]
    c.seq, c.table = seq, table
    for n in (1, 2):
        c.compare(*c.decode(n_split=n), c.expect(), n)


def test_cache_rows_past_2_31_elements():
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    B, S, Hk, d = 3, 700032, 8, 128  # sequence 2 starts past 2^30 elements, ends past 2^31
    k, v = (torch.full((B, S, Hk, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    c = Case([130], 1, 8, 8, 128)
    far = torch.tensor([1, 1, S], dtype=torch.int32, device=DEV)
    k[:2, :1], v[:2, :1] = 0, 0
    # all of sequence 2 but its last 130 tokens has keys that no query likes
    k[2], v[2] = 0, 0
    k[2, :, :, 0] = -30000.0
    k[2, -130:], v[2, -130:] = c.k[0], c.v[0]
    q = c.q.clone()
    q[..., 0] = q[..., 0].abs() + 1
    c.q = q
    out, lse = g.decode_diff(q[:, 0].expand(3, -1, -1).contiguous().to(DEV), k, v, far,
                             c.lam[0, 0].to(DEV))
    c.compare(out[2], lse[2], c.expect())


# -------------------------------------------------------------------- prefill --
def check_prefill(c, want=None, window=-1, **kw):
    o, l, tol, tol_l = want or c.expect(window)
    out, lse = c.prefill(window=window, **kw)
    c.compare(out, lse, [o, l.transpose(0, 2, 1), tol, tol_l.transpose(0, 2, 1)], (window, kw))


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("S,B,H,Hk,norm", [(1, 2, 2, 1, True), (17, 1, 6, 2, False), (128, 2, 3, 3, True),
                                           (129, 1, 8, 2, False), (300, 1, 4, 2, True)])
def test_prefill_causal(d, split, S, B, H, Hk, norm):
    c = Case([S] * B, S, H, Hk, d, split, norm=norm, seed=S + d)
    want = c.expect()
    check_prefill(c, want, seq_lens=None)
    check_prefill(c, want)  # the same through lengths


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("window", [-1, 0, 5, 100, 1 << 30])
def test_prefill_chunk(d, split, window):
    c = Case([33, 290, 150], 33, 4, 2, d, split, S=300, norm=d != 64, lam="token", seed=d)
    check_prefill(c, window=window)
    if d == 128 and split:
        c = Case([700, 513], 200, 2, 1, d, split, lam="head", seed=9)
        want = c.expect(window)
        for n_part in (1, 2, 3, 8):
            check_prefill(c, want, window, n_part=n_part)


def test_prefill_parts_with_norm():
    c = Case([900, 131], 130, 3, 1, 64, norm=True, lam="layer", S=1000)
    want = c.expect()
    for n_part in (2, 5, 8):
        check_prefill(c, want, n_part=n_part)


def test_prefill_many_items_and_deterministic():
    # more work items than CTAs, so that each CTA runs several and hands its buffers on
    c = Case([257] * 4, 257, 48, 8, 64, norm=True, lam="row")
    a = c.prefill(seq_lens=None)
    rows = c.expect()
    c.compare(*a, [rows[0], rows[1].transpose(0, 2, 1), rows[2], rows[3].transpose(0, 2, 1)])
    for _ in range(3):
        b = c.prefill(seq_lens=None)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_prefill_bad_length():
    c = Case([50, 60], 20, 4, 2, 64, norm=True, S=64)
    o, _, tol, _ = c.expect()
    for wrong in (0, 19, 65, -1):
        lens = c.dev_lens()
        lens[0] = wrong
        for n_part in (1, 2):
            out, lse = c.prefill(seq_lens=lens, n_part=n_part)
            torch.cuda.synchronize()
            assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
            assert out[0].isnan().all() and lse[0].isnan().all()
            assert (np.abs(out[1].double().cpu().numpy() - o[1]) <= tol[1]).all()


def test_maps_of_the_prefill_are_the_plain_prefill():
    c = Case([513], 513, 4, 2, 128)
    c.lam = torch.zeros(1)
    out, lse = c.prefill(seq_lens=None)
    ro, rl = g.prefill_causal(c.q.to(DEV), c.k, c.v)
    assert torch.equal(out, ro[:, :, ::2]) and torch.equal(lse, rl)


# ------------------------------------------------------------------- together --
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("page", [0, 64])
def test_a_sequence_from_its_prompt_on(split, page):
    """A padded batch of prompts is appended, the first chunk attended to by prefill_diff over the
    contiguous cache, then single tokens and a draft of three go through append and decode."""
    B, H, Hk, d, S = 3, 4, 2, 64, 300
    gen = torch.Generator().manual_seed(5)
    rows = H if split else 2 * H
    heads, dd = (2, d // 2) if split else (1, d)  # what the append calls a head
    freqs = torch.exp(-np.log(1e4) * 2 * torch.arange(dd // 2, dtype=torch.float64) / dd).float()
    x = [torch.randn(B, S, h, d, generator=gen).to(torch.bfloat16) for h in (rows, Hk, Hk)]
    lam = torch.sigmoid(torch.randn(B, S, H, generator=gen))
    tau = ref.default_scale(d, split)
    # in 64 bits: the turned rows and how far the GPU's may be from them
    held = []
    for b in range(B):
        kq = []
        for t in x[:2]:
            n = t.shape[2]
            y, tol = ref.turn(t[b].double().reshape(S, n * heads, dd).numpy(), np.arange(S),
                              freqs.double().numpy(), False)
            kq.append((y.reshape(S, n, d), ref.bf16_tol(y, tol).reshape(S, n, d)))
        held.append(kq)
    dev = [t.to(DEV) for t in x]
    per, units = (page, B * -(-S // page)) if page else (S, B)
    k, v = (torch.zeros(units, per, Hk, d, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    table = torch.randperm(units, generator=gen).view(B, -1).to(torch.int32).to(DEV) if page else None
    view = lambda t: t.view(*t.shape[:2], t.shape[2] * heads, dd)  # noqa: E731

    def append(start, n):  # n[b] tokens from start[b] on
        T = max(n)
        part = [torch.zeros(B, T, *t.shape[2:], dtype=torch.bfloat16, device=DEV) for t in dev]
        for b in range(B):
            for p, t in zip(part, dev):
                p[b, :n[b]] = t[b, start[b]:start[b] + n[b]]
        lens = torch.tensor([s + m for s, m in zip(start, n)], dtype=torch.int32, device=DEV)
        q = g.kv_append(view(part[1]), view(part[2]), view(k), view(v), lens, freqs=freqs.to(DEV),
                        n_new=torch.tensor(n, dtype=torch.int32, device=DEV), q=view(part[0]),
                        block_table=table)
        return q.view(part[0].shape), lens

    def check(q, out, lse, lens, T, prefill):
        for b in range(B):
            L = int(lens[b])
            t = torch.arange(L, device=DEV)
            at = (table[b].long()[t // page], t % page) if page else (b, t)
            kk, vv, qq = (z.double().cpu().numpy() for z in (k[at], v[at], q[b]))
            for got, (want, tol) in ((qq, (z[L - T:L] for z in held[b][0])),
                                     (kk, (z[:L] for z in held[b][1]))):
                assert (np.abs(got - want) <= tol).all()
            assert np.array_equal(vv, x[2][b, :L].double().numpy())
            o, l, tol, tol_l = ref.attention(qq, kk, vv, lam[b, L - T:L].double().numpy(), tau, split,
                                             norm_eps=1e-3)
            assert (np.abs(out[b].double().cpu().numpy().reshape(o.shape) - o) <= tol).all()
            got = lse[b].double().cpu().numpy()
            got = got.T if prefill else got.reshape(l.shape)
            assert (np.abs(got - l) <= tol_l).all()

    n = [40, 256, 129]
    q, lens = append([0] * B, n)
    if not page:
        T = min(n)  # the last 40 of each prompt
        qe = torch.stack([q[b, n[b] - T:n[b]] for b in range(B)])
        le = torch.stack([lam[b, n[b] - T:n[b]] for b in range(B)]).to(DEV)
        out, lse = g.prefill_diff(qe, k, v, le, lens, split_keys=split, norm_eps=1e-3)
        check(qe, out, lse, lens, T, True)
    for step in (1, 1, 3):
        q, lens = append(lens.tolist(), [step] * B)
        le = torch.stack([lam[b, int(lens[b]) - step:int(lens[b])] for b in range(B)]).to(DEV)
        out, lse = g.decode_diff(q, k, v, lens, le, split_keys=split, norm_eps=1e-3,
                                 block_table=table)
        check(q, out, lse, lens, step, False)


@pytest.mark.parametrize("d,T,S,n_split", [(64, 1, 128, 2), (64, 1, 900, None), (128, 4, 600, None),
                                           (32, 1, 5000, None), (128, 1, 200, 1)])
def test_captured_step_replays_over_new_lengths(d, T, S, n_split):
    c = Case([100, S - 20], T, 8, 2, d, norm=True, lam="layer", S=S)
    q, lam, lens = c.q.to(DEV), c.lam.to(DEV), c.dev_lens()
    if T == 1:
        q = q[:, 0].contiguous()
    args = (q, c.k, c.v, lens, lam)
    want = [x.clone() for x in g.decode_diff(*args, n_split=n_split, **c.form)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = g.decode_diff(*args, n_split=n_split, **c.form)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    lens -= 7
    graph.replay()
    fresh = g.decode_diff(*args, n_split=n_split, **c.form)
    torch.cuda.synchronize()
    assert torch.equal(got[0], fresh[0]) and torch.equal(got[1], fresh[1])


def test_captured_prefill_in_parts():
    c = Case([700, 300], 100, 4, 2, 64, norm=True, lam="layer", S=800)
    q, lam, lens = c.q.to(DEV), c.lam.to(DEV), c.dev_lens()
    graph = torch.cuda.CUDAGraph()
    run = lambda: g.prefill_diff(q, c.k, c.v, lam, lens, n_part=3, **c.form)  # noqa: E731
    want = [x.clone() for x in run()]
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_streams_at_once():
    cases = [Case([3000], 1, 8, 2, 64, seed=i) for i in range(4)]
    want = [[x.clone() for x in c.decode()] for c in cases]
    qs = [(c.q[:, 0].contiguous().to(DEV), c.k, c.v, c.dev_lens(), c.lam[:, 0].to(DEV)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [g.decode_diff(*a, stream=s) for a, s in zip(qs, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_what_the_helpers_refuse():
    c = Case([40, 90], 2, 4, 2, 64)
    q, lam, lens = c.q.to(DEV), c.lam.to(DEV), c.dev_lens()
    good = dict(q=q, k=c.k, v=c.v, seq_lens=lens, lam=lam)
    w = torch.ones(64, device=DEV)
    for kw in (dict(q=q[:, :, :7]), dict(q=q.float()), dict(q=q[..., ::2]), dict(lam=lam.double()),
               dict(lam=lam[:, :1, :3]), dict(lam=lam.cpu()), dict(lam=lam[None]), dict(norm_weight=w),
               dict(norm_eps=1e-5, norm_weight=w[:32].contiguous()), dict(norm_eps=-1.0),
               dict(norm_eps=float("nan")), dict(scale=0.0), dict(scale=float("inf")),
               dict(out_scale=float("nan")), dict(seq_lens=lens.long()), dict(k=c.k[:1])):
        with pytest.raises(g.GQAError):
            g.decode_diff(**{**good, **kw})
        with pytest.raises(g.GQAError):
            g.prefill_diff(**{**good, **kw})
    for kw in (dict(n_split=0), dict(n_split=70000), dict(n_split=2, workspace=w),
               dict(out=torch.empty(2, 2, 8, 64, dtype=torch.bfloat16, device=DEV)),
               dict(lse=torch.empty(2, 2, 4, device=DEV))):
        with pytest.raises(g.GQAError):
            g.decode_diff(**good, **kw)
    for kw in (dict(n_part=0), dict(n_part=9), dict(n_part=2, workspace=w),
               dict(lse=torch.empty(2, 2, 8, device=DEV))):
        with pytest.raises(g.GQAError):
            g.prefill_diff(**good, **kw)
    with pytest.raises(g.GQAError):  # 18 rows of a KV head
        g.decode_diff(torch.zeros(2, 18, 64, dtype=torch.bfloat16, device=DEV), c.k[:, :, :1].contiguous(),
                      c.v[:, :, :1].contiguous(), lens, lam[:, 0, :1])

"""The rotated append to bf16 and per-token E4M3 caches on the GPU, against the 64-bit forms of
diff_ref: every layout, odd sizes, padded batches, far positions, refusals on the device,
streams and graphs."""
import numpy as np
import pytest
import torch

import diff_ref as ref
import gqa_attention_gb300 as g
from fp8_block_ref import E4M3

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


def frequencies(rot, base=500000.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return torch.exp(-np.log(base) * 2 * i / rot).float()


class Step:
    """Inputs of one append, its cache full of canaries, and the check of what came out."""

    def __init__(self, B, T, Hq, Hk, d, rot, inter=False, page=0, fp8=False, S=None, fused=False,
                 counts=None, lens=None, positions=None, seed=0, gain=1.0):
        self.gen = torch.Generator().manual_seed(seed)
        self.B, self.T, self.Hq, self.Hk, self.d, self.inter = B, T, Hq, Hk, d, inter
        self.page, self.fp8 = page, fp8
        self.counts = counts if counts is not None else [T] * B
        self.lens = lens if lens is not None else [n + 3 * b for b, n in enumerate(self.counts)]
        S = S if S is not None else max(max(self.lens), 1) + 5
        per, units = (page, B * -(-S // page) + 2) if page else (-(-S // 4) * 4, B)
        self.shape = (units, per, Hk, d)
        self.table = None
        if page:
            perm = torch.randperm(units, generator=self.gen)[: B * -(-S // page)]
            self.table = perm.view(B, -1).to(torch.int32)
        self.freqs = frequencies(rot) if rot else None
        self.pos = positions
        rows = [(torch.randn(B, T, h, d, generator=self.gen) * gain).to(torch.bfloat16)
                for h in (Hq, Hk, Hk)]
        self.q, self.k, self.v = rows
        if fused:
            wide = torch.cat(rows, 2).to(DEV)
            self.dev_rows = wide.split([Hq, Hk, Hk], 2)
        else:
            self.dev_rows = [x.to(DEV) for x in rows]
        if fp8:
            self.kc, self.vc = (torch.full(self.shape, 0x7F, dtype=torch.uint8, device=DEV)
                                for _ in "kv")
            self.ks, self.vs = (torch.full(self.shape[:2], float("nan"), device=DEV) for _ in "kv")
        else:
            self.kc, self.vc = (torch.full(self.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
                                for _ in "kv")
            self.ks = self.vs = None
        self.q_out = torch.full((B, T, Hq, d), float("inf"), dtype=torch.bfloat16, device=DEV)

    def args(self):
        dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        return dict(freqs=dev(self.freqs), interleaved=self.inter, k_scale=self.ks,
                    v_scale=self.vs, block_table=dev(self.table), positions=dev(self.pos),
                    n_new=torch.tensor(self.counts, dtype=torch.int32, device=DEV))

    def run(self, **more):
        q, k, v = self.dev_rows
        a = {**self.args(), "q": q, "q_out": self.q_out, **more}
        out = g.kv_append(k, v, self.kc, self.vc,
                          torch.tensor(self.lens, dtype=torch.int32, device=DEV), **a)
        torch.cuda.synchronize()
        return out

    def place(self, b, t):
        if self.page:
            return int(self.table[b, t // self.page]), t % self.page
        return b, t

    def check(self, skip=(), no_rows=()):
        """skip: sequences that must be untouched; no_rows: (b, i) whose cache rows must be."""
        kc, vc = self.kc.cpu(), self.vc.cpu()
        ks, vs = (None if x is None else x.cpu().numpy() for x in (self.ks, self.vs))
        q_out = self.q_out.double().cpu().numpy()
        written = set()
        for b, (n, L) in enumerate(zip(self.counts, self.lens)):
            if b in skip:
                continue
            n_ = range(n)
            pos = np.array([L - n + i if self.pos is None else int(self.pos[b, i]) for i in n_],
                           dtype=np.int64)
            fr = [] if self.freqs is None else self.freqs.double().numpy()
            k, tk = ref.turn(self.k[b, :n].double().numpy(), pos, fr, self.inter)
            q, tq = ref.turn(self.q[b, :n].double().numpy(), pos, fr, self.inter)
            v = self.v[b, :n].double().numpy()
            assert (np.abs(q_out[b, :n] - q) <= ref.bf16_tol(q, tq)).all()
            assert np.isinf(q_out[b, n:]).all()  # (the canary)
            for i in n_:
                if (b, i) in no_rows:
                    continue
                at = self.place(b, L - n + i)
                written.add(at)
                if self.fp8:
                    ref.check_codes(E4M3[kc[at].numpy()], ks[at], k[i], tk[i])
                    ref.check_codes(E4M3[vc[at].numpy()], vs[at], v[i], 0 * v[i])
                else:
                    got = kc[at].double().numpy()
                    assert (np.abs(got - k[i]) <= ref.bf16_tol(k[i], tk[i])).all()
                    assert np.array_equal(vc[at].double().numpy(), v[i])
        rest = torch.ones(self.shape[:2], dtype=torch.bool)
        for at in written:
            rest[at] = False
        for c in (kc, vc):
            assert (c[rest] == 0x7F).all() if self.fp8 else c[rest].isnan().all()
        if self.fp8:
            assert np.isnan(ks[rest.numpy()]).all() and np.isnan(vs[rest.numpy()]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (32, 16), (32, 32), (64, 48), (64, 64), (128, 16),
                                   (128, 112), (128, 128), (64, 0)])
@pytest.mark.parametrize("page", [0, 16])
def test_every_head_size_and_rotation(d, rot, inter, page, fp8):
    s = Step(3, 5, 6, 2, d, rot, inter, page, fp8, counts=[5, 1, 3], seed=d + rot)
    s.run()
    s.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,d", [
    (1, 1, 64, 8, 128), (130, 1, 8, 8, 32), (2, 700, 5, 1, 64), (1, 1, 1, 1, 128), (3, 257, 7, 7, 32),
    (2, 3, 40, 20, 128),   # more values in a token than a warp holds at once
    (1, 3, 3, 37, 64), (1, 5000, 2, 1, 16),
])
def test_sizes(B, T, Hq, Hk, d, fp8):
    counts = [max(0, T - 2 * b) for b in range(B)]
    s = Step(B, T, Hq, Hk, d, d, B % 2 == 0, 64 if T % 2 else 0, fp8, fused=True, counts=counts,
             seed=T)
    s.run()
    s.check()


@pytest.mark.parametrize("Hq,Hk,d,T", [
    (4, 1, 128, 1203),   # four tokens to a warp
    (3, 3, 16, 1203), (2, 5, 32, 1203), (4, 2, 128, 331),
    (5, 5, 128, 1203),   # two slots to a lane
    (1, 37, 128, 651),   # several warps to a token, two slots to a lane
    (1, 70, 128, 651),   # more than they hold at once
])
def test_many_e4m3_tokens_and_one_that_is_not_finite(Hq, Hk, d, T):
    s = Step(1, T, Hq, Hk, d, d, fp8=True, counts=[T - 2], lens=[T + 1], page=16, seed=Hk)
    s.run()
    s.check()
    was = [x.clone() for x in (s.kc, s.vc, s.ks, s.vs)]
    hit = torch.zeros(T - 2, Hk, d, dtype=torch.bool)
    at = [0, 1, 6, 17, 600, T - 3] if T > 603 else [0, 1, 6, 17, T - 3]
    for n, i in enumerate(at):
        s.dev_rows[2][0, i, i % Hk, i % d] = [float("inf"), float("nan"), -float("inf")][n % 3]
        hit[i, i % Hk, i % d] = True
    s.run()
    where = [s.place(0, s.lens[0] - (T - 2) + i) for i in range(T - 2)]
    unit, row = (torch.tensor(x, device=DEV) for x in zip(*where))
    assert torch.equal(s.kc, was[0])
    assert torch.equal(s.ks.view(torch.int32), was[2].view(torch.int32))
    got = torch.from_numpy(E4M3[s.vc[unit, row].cpu().numpy()])
    assert torch.equal(~torch.isfinite(got), hit)
    clean = torch.ones(T - 2, dtype=torch.bool, device=DEV)
    clean[at] = False
    assert torch.equal(s.vc[unit, row][clean], was[1][unit, row][clean])
    assert torch.equal(s.vs[unit, row][clean], was[3][unit, row][clean])
    for i in at:  # its scale is that of what is finite
        rest = s.v[0, i].double().abs()[~hit[i]].max().item()
        assert s.vs[where[i]].item() == ref.block_scale(rest)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hk,d", [(64, 8, 128), (120, 6, 64), (6, 2, 64)])
def test_padding_in_front_of_a_sequence_in_a_large_batch(Hq, Hk, d, fp8):
    # (enough tokens that a CTA takes several: padding, then the next sequence's first)
    s = Step(8, 1300, Hq, Hk, d, d, fp8=fp8, counts=[3, 40, 0, 17, 1300, 1, 1299, 20], S=1400,
             lens=[5, 40, 9, 1000, 1300, 1, 1299, 33])
    s.run()
    s.check()


def test_far_and_negative_positions():
    pos = torch.tensor([[0, 131071, 131072, 1 << 20, (1 << 24) + 1, (1 << 28) - 1, -1, -70000]],
                       dtype=torch.int32)
    for inter in (False, True):
        s = Step(1, 8, 2, 1, 128, 128, inter, positions=pos, lens=[8])
        s.run()
        s.check()


def test_frequencies_of_many_turns_at_far_positions():
    # (|p f| up to 2.6e8, below 2^28)
    pos = torch.tensor([[1, 1000, 131071, 2600000, 2599999, -2600000, -1, 0]], dtype=torch.int32)
    for inter in (False, True):
        s = Step(1, 8, 2, 1, 128, 128, inter, positions=pos, lens=[8], seed=3)
        s.freqs = 6.5 + 93.5 * torch.rand(64, generator=s.gen)
        s.freqs[0], s.freqs[1], s.freqs[2] = 100.0, -100.0, 6.2831855
        s.run()
        s.check()


@pytest.mark.parametrize("inter", [False, True])
def test_small_negative_frequencies_at_the_farthest_position(inter):
    # p f is next to odd quarters of a turn, so that a cosine of 1e-6 shows the angle's error
    pos = torch.tensor([[2 ** 31 - 1, -(2 ** 31), 0, 1]], dtype=torch.int32)
    s = Step(1, 4, 1, 1, 16, 16, inter, positions=pos, lens=[4])
    f = [float.fromhex("-0x1.858eb8p-26"), float.fromhex("-0x1.3a28cap-26")]
    s.freqs = torch.tensor([*f, *(-x for x in f), *f, *f])
    x = torch.zeros(1, 4, 1, 16, dtype=torch.bfloat16)
    x[..., slice(0, 16, 2) if inter else slice(0, 8)] = 1.0
    s.q, s.k, s.v = x, x, x
    s.dev_rows = [t.to(DEV) for t in (x, x, x)]
    s.run()
    s.check()


def test_far_place_in_a_long_sequence():
    # the position is the token's place: 2M tokens into a paged sequence, a small pool behind it
    nb, page = 1 << 15, 64
    L = nb * page
    s = Step(1, 2, 2, 1, 64, 64, lens=[L], page=page, S=256)
    table = torch.full((1, nb), -5, dtype=torch.int32)
    table[0, -1] = 3
    s.table = table
    s.run()
    s.check()


def test_empty_calls_and_no_queries():
    s = Step(2, 4, 4, 2, 64, 64, counts=[0, 0], lens=[0, 7])
    s.run()
    s.check()  # (nothing written at all)
    s = Step(2, 4, 4, 2, 64, 64)
    assert s.run(q=None, q_out=None) is None
    s.q_out.copy_(s.q_out)
    kc = s.kc.clone()
    s.run()
    assert torch.equal(kc.view(torch.int16), s.kc.view(torch.int16))
    s.check()
    # T = 0 rows: nothing happens
    k0 = torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16, device=DEV)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert g.kv_append(k0, k0, s.kc, s.vc, lens) is None


def test_queries_in_place_and_fresh():
    s = Step(2, 9, 6, 3, 128, 128, counts=[9, 9])
    s.run()
    q = s.dev_rows[0].contiguous().clone()
    assert s.run(q=q, q_out=q) is q
    assert torch.equal(q, s.q_out)
    fresh = s.run(q_out=None)
    assert torch.equal(fresh, s.q_out)
    s.counts = [9, 4]  # with counts, rows past them come back as zeros
    fresh = s.run(q_out=None)
    assert (fresh[1, 4:] == 0).all()


def test_infinities_and_nan_in_bf16_and_e4m3():
    for fp8 in (False, True):
        s = Step(1, 3, 2, 2, 32, 32, fp8=fp8)
        k, v = s.dev_rows[1], s.dev_rows[2]
        k[0, 1, 0, 3], k[0, 1, 1, 5] = float("inf"), float("nan")
        v[0, 2, 0, 1], v[0, 2, 1, 7] = -float("inf"), float("nan")
        s.run()
        val = (lambda c: torch.from_numpy(E4M3[c.cpu().numpy()])) if fp8 else (lambda c: c.cpu())
        kk, vv = val(s.kc[0]), val(s.vc[0])
        hit = torch.zeros(2, 32, dtype=torch.bool)
        hit[0, 3] = hit[0, 19] = hit[1, 5] = hit[1, 21] = True  # both channels of the pair
        assert torch.equal(~torch.isfinite(kk[1]), hit)
        assert torch.isfinite(kk[[0, 2]]).all()
        hit = torch.zeros(2, 32, dtype=torch.bool)
        hit[0, 1] = hit[1, 7] = True
        assert torch.equal(~torch.isfinite(vv[2]), hit)
        if fp8:  # the others keep a scale of their own size
            assert torch.isfinite(s.ks[0, :3]).all() and torch.isfinite(s.vs[0, :3]).all()
            assert s.vs[0, 2].item() == ref.block_scale(
                s.v[0, 2].double().abs().flatten()[~hit.flatten()].max().item())


@pytest.mark.parametrize("gain", [2.0 ** -120, 2.0 ** -110, 1.0, 2.0 ** 100, 2.0 ** 119])
def test_e4m3_scales_of_every_size(gain):
    s = Step(2, 3, 1, 2, 64, 64, fp8=True, gain=gain)
    s.run()
    s.check()
    z = Step(1, 2, 1, 1, 32, 32, fp8=True, gain=0.0)  # all zero: the smallest scale, codes 0
    z.run()
    z.check()
    assert (z.ks[0, :2] == 2.0 ** -100).all() and ((z.kc[0, :2] & 127) == 0).all()  # (zeros keep their signs)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_and_pages_are_reported(fp8):
    # (every access is checked by the kernel before it is made)
    for counts, lens, bad in [([2, 5, 2], [9, 9, 9], 1), ([2, -1, 2], [9, 9, 9], 1),
                              ([2, 2, 3], [9, 1, 9], 1), ([2, 2, 2], [9, 9, 99], 2),
                              ([2, 0, 2], [9, -1, 9], 1)]:
        s = Step(3, 4, 4, 2, 64, 64, fp8=fp8, counts=counts, lens=lens, S=20)
        s.run()
        assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
        s.check(skip=(bad,))
        assert s.q_out[bad].isnan().all()
    s = Step(2, 4, 4, 2, 64, 64, fp8=fp8, page=16, lens=[18, 18], S=30)
    good = int(s.table[1, 1])
    for wrong in (-1, s.shape[0], 2 ** 31 - 1):
        s.table[1, 1] = wrong
        s.run()
        assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
        s.table[1, 1] = good
        # tokens 14, 15 lie on page 0, 16 and 17 on the bad one
        s.check(no_rows={(1, 2), (1, 3)})


def test_more_than_2_31_elements():
    rows = (1 << 21) + 64  # times 1024 elements
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    c = [torch.zeros(1, rows, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    x = [torch.randn(1, 2, 8, 128, device=DEV).to(torch.bfloat16) for _ in "kv"]
    lens = torch.tensor([rows], dtype=torch.int32, device=DEV)
    g.kv_append(*x, *c, lens)
    for a, b in zip(x, c):
        assert torch.equal(b[0, -2:], a[0]) and not b[0, :-2].any()


def test_another_stream_and_a_replayed_graph():
    s = Step(2, 3, 4, 2, 64, 64)
    s.run()
    want = [x.clone() for x in (s.kc, s.vc, s.q_out)]
    q, k, v = s.dev_rows
    a, lens = s.args(), torch.tensor(s.lens, dtype=torch.int32, device=DEV)
    for t in (s.kc, s.vc, s.q_out):
        t.fill_(1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g.kv_append(k, v, s.kc, s.vc, lens, q=q, q_out=s.q_out, stream=side, **a)
    side.synchronize()
    for b, (n, L) in enumerate(zip(s.counts, s.lens)):
        assert torch.equal(s.kc[b, L - n:L], want[0][b, L - n:L])
        assert torch.equal(s.vc[b, L - n:L], want[1][b, L - n:L])
    assert torch.equal(s.q_out, want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.kv_append(k, v, s.kc, s.vc, lens, q=q, q_out=s.q_out, **a)
    for t in (s.kc, s.vc, s.q_out):
        t.fill_(1.0)
    lens += 1  # a replay takes what the tensors then hold
    graph.replay()
    torch.cuda.synchronize()
    ang = Step(2, 3, 4, 2, 64, 64)
    ang.lens = [n + 1 for n in s.lens]
    ang.run()
    assert torch.equal(ang.q_out, s.q_out)
    for b, (n, L) in enumerate(zip(ang.counts, ang.lens)):
        assert torch.equal(s.kc[b, L - n:L], ang.kc[b, L - n:L])
        assert (s.kc[b, : L - n] == 1).all()


def test_what_the_helper_refuses():
    s = Step(2, 3, 4, 2, 64, 64)
    q, k, v = s.dev_rows
    lens, a = torch.tensor(s.lens, dtype=torch.int32, device=DEV), s.args()
    for more in (dict(q_out=s.q_out[:1], q=q), dict(q=q.float()), dict(freqs=a["freqs"].double()),
                 dict(n_new=a["n_new"].long()), dict(k_scale=s.kc.new_zeros(2, 4).float()),
                 dict(positions=torch.zeros(2, 4, dtype=torch.int32, device=DEV)),
                 dict(freqs=torch.ones(5, device=DEV)), dict(freqs=torch.ones(40, device=DEV)),
                 dict(q=q[:, :, :, :32]), dict(q_out=s.q_out)):
        with pytest.raises(g.GQAError):
            g.kv_append(k, v, s.kc, s.vc, lens, **{**a, **more})
    with pytest.raises(g.GQAError):  # tokens that are not dense
        g.kv_append(k[..., ::2], v[..., ::2], s.kc[..., ::2], s.vc[..., ::2], lens)
    with pytest.raises(g.GQAError):
        g.kv_append(k.transpose(0, 1).contiguous().transpose(0, 1), v, s.kc, s.vc, lens)
    with pytest.raises(g.GQAError):
        g.kv_append(k, v, s.kc, s.vc, lens[:1])


# ------------------------------------------------- with the attention over it --
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [0, 16])
def test_appended_tokens_are_what_decode_attends_to(page, fp8):
    """Prompts of a padded batch, then single tokens, through the append and the library's decode:
    the output against attention in 64 bits over what the cache then holds, and what it holds
    against the turned rows."""
    B, S, Hq, Hk, d = 3, 96, 8, 2, 64
    s = Step(B, 40, Hq, Hk, d, d, page=page, fp8=fp8, counts=[40, 7, 23], lens=[40, 7, 23], S=S)
    s.run()
    s.check()
    for step in range(3):
        rows = [torch.randn(B, 1, h, d, generator=s.gen).to(torch.bfloat16) for h in (Hq, Hk, Hk)]
        s.lens = [n + 1 for n in s.lens]
        lens = torch.tensor(s.lens, dtype=torch.int32, device=DEV)
        q, k, v = (x.to(DEV) for x in rows)
        a = {**s.args(), "n_new": None}
        q = g.kv_append(k, v, s.kc, s.vc, lens, q=q, **a)[:, 0].contiguous()
        if fp8:
            out, lse = g.decode_fp8(q, s.kc, s.vc, s.ks, s.vs, lens, block_table=a["block_table"])
        elif page:
            out, lse = g.decode_paged(q, s.kc, s.vc, a["block_table"], lens)
        else:
            out, lse = g.decode(q, s.kc, s.vc, lens)
        torch.cuda.synchronize()
        assert g.gqa_last_device_error() == g.GQA_OK
        for b, L in enumerate(s.lens):
            at = [s.place(b, t) for t in range(L)]
            unit, row = torch.tensor([x[0] for x in at]), torch.tensor([x[1] for x in at])

            def held(c, sc):
                c = c.cpu()[unit, row]
                if not fp8:
                    return c.double().numpy()
                return E4M3[c.numpy()] * sc.cpu().double()[unit, row].numpy()[:, None, None]

            kk, vv = held(s.kc, s.ks), held(s.vc, s.vs)
            # the new key, turned by its place
            y, tol = ref.turn(rows[1][b].double().numpy(), [L - 1], s.freqs.double().numpy(), False)
            near = ref.bf16_tol(y[0], tol[0])
            if fp8:
                near = 2.0 ** -4 * np.abs(y[0]) + s.ks.cpu()[at[-1]].item() * 2.0 ** -10 + 2 * tol[0]
            assert (np.abs(kk[-1] - y[0]) <= near).all()
            for h in range(Hq):
                x = kk[:, h // (Hq // Hk)] @ q[b, h].double().cpu().numpy() / np.sqrt(d)
                z = np.log(np.exp(x - x.max()).sum()) + x.max()
                o = np.exp(x - z) @ vv[:, h // (Hq // Hk)]
                # the parity bar of the decodes
                assert abs(lse[b, h].item() - z) <= 1e-3
                assert np.abs(out[b, h].double().cpu().numpy() - o).max() <= 2e-2

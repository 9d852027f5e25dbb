"""Shared-prefix attention, attention mass and cache eviction on the GPU, against their definitions in 64 bits."""
import math
import random

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAGE = 64
NAN = float("nan")


@pytest.fixture(scope="module")
def abi():
    from ar_lm_decoding_b200 import abi
    return abi


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pad(n):
    return (n + PAGE - 1) // PAGE * PAGE


def _scatter(rows, table, pool):
    """Contiguous rows [.., Hkv, n, D] of one sequence into its pages of a pool."""
    for i in range(0, rows.shape[-2], PAGE):
        part = rows[..., i:i + PAGE, :]
        pool[int(table[i // PAGE]), :, :part.shape[-2]] = part


class Shared:
    """Inputs of one shared-prefix attention call; contiguous tensors are kept beside a paged copy of them."""

    def __init__(self, abi, seed, B, Hq, Hkv, D, k, R, S, lens, paged=False, S_extra=5, P_extra=3):
        g = _gen(seed)
        self.abi, self.B, self.Hq, self.Hkv, self.D, self.k, self.R, self.S, self.lens = abi, B, Hq, Hkv, D, k, R, S, lens
        self.mode, self.scale, self.paged = (0 if k else 1), 1.0 / math.sqrt(D), paged
        self.q = _normal(g, B, R, Hq, D, scale=1.5)
        self.kn, self.vn = _normal(g, B, R, Hkv, D), _normal(g, B, R, Hkv, D)
        self.S_max, self.P_max = (_pad(S + S_extra), _pad(max(lens) + P_extra)) if paged else (S + S_extra, max(lens) + P_extra)
        self.ks, self.vs = _normal(g, Hkv, self.S_max, D), _normal(g, Hkv, self.S_max, D)
        self.kc, self.vc = _normal(g, B, Hkv, self.P_max, D), _normal(g, B, Hkv, self.P_max, D)
        for t in (self.ks, self.vs):
            t[:, S:] = NAN
        for t in (self.kc, self.vc):
            for b in range(B):
                t[b, :, lens[b]:] = NAN
        self.shared_len, self.prefix_len = _i32([S]), _i32(lens)
        self.out = torch.full((B, R, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((B, R, Hq), NAN, dtype=torch.float32, device=DEV)
        self.status = _i32([0])
        self.ws = torch.full((max(256, abi.tidar_attn_shared_workspace_size(B, Hq, Hkv, D, R, self.S_max, self.P_max)),),
                             255, dtype=torch.uint8, device=DEV)
        if paged:
            ns, no = self.S_max // PAGE, self.P_max // PAGE
            ids = torch.randperm(ns + B * no + 3, generator=g, device=DEV).to(torch.int32)
            self.num_pages, self.shared_table = ids.numel(), ids[:ns].contiguous()
            self.table = ids[ns:ns + B * no].reshape(B, no).contiguous()
            self.kp = torch.full((self.num_pages, Hkv, PAGE, D), NAN, dtype=torch.bfloat16, device=DEV)
            self.vp = self.kp.clone()
            for pool, s, c in ((self.kp, self.ks, self.kc), (self.vp, self.vs, self.vc)):
                _scatter(s[:, :S], self.shared_table, pool)
                for b in range(B):
                    _scatter(c[b, :, :lens[b]], self.table[b], pool)

    def call(self, stream=None, lse=True):
        s = self
        tail = (s.out, s.lse if lse else None, s.ws, s.ws.numel(), s.status)
        if s.paged:
            s.abi.tidar_attn_step_shared_paged(
                s.q, s.kn, s.vn, s.kp, s.vp, s.shared_table, s.shared_table.numel(), s.shared_len, s.table,
                s.table.shape[1], s.num_pages, s.prefix_len, s.B, s.Hq, s.Hkv, s.D, s.k, s.R, s.scale, s.mode, *tail,
                stream=stream)
        else:
            s.abi.tidar_attn_step_shared(
                s.q, s.kn, s.vn, s.ks, s.vs, s.shared_len, s.S_max, s.kc, s.vc, s.prefix_len, s.B, s.Hq, s.Hkv, s.D,
                s.k, s.R, s.P_max, s.scale, s.mode, *tail, stream=stream)

    def reference(self):
        return ref.attn_shared(self.q, self.kn, self.vn, self.ks, self.vs, self.S, self.kc, self.vc, self.lens,
                               self.mode, self.k, self.scale)

    def check(self, rows=None):
        out, lse, absum, vmax = self.reference()
        err, tol = (self.out.double() - out).abs(), ref.attn_tolerance(out, absum, vmax)
        off = (self.lse.double() - lse).abs()
        if rows is not None:
            err, tol, off = err[:, rows], tol[:, rows], off[:, rows]
        assert bool((err <= tol).all()), (err / tol).max().item()
        assert bool((off <= 1e-4).all()), off.max().item()


SHARED = [  # B, Hq, Hkv, D, k, R, S, lens
    (1, 1, 1, 64, 0, 1, 1, [0]),
    (1, 2, 1, 128, 0, 1, 0, [0]),
    (1, 2, 1, 64, 1, 3, 0, [1]),
    (2, 2, 1, 64, 4, 24, 128, [128, 5]),
    (3, 6, 2, 128, 2, 8, 127, [0, 129, 64]),
    (2, 5, 1, 64, 3, 15, 129, [200, 1]),
    (5, 7, 1, 128, 0, 1, 1000, [0, 3, 127, 128, 300]),
    (16, 32, 8, 128, 0, 1, 700, [37 * i % 260 for i in range(16)]),
    (70, 8, 2, 64, 0, 1, 257, [11 * i % 90 for i in range(70)]),
    (4, 24, 2, 128, 4, 24, 1001, [64, 0, 513, 400]),
    (2, 32, 8, 128, 8, 80, 515, [256, 31]),
    (2, 16, 2, 128, 16, 288, 640, [100, 383]),
    (2, 12, 1, 64, 5, 35, 2000, [0, 0]),
    (1, 128, 1, 64, 1, 3, 300, [40]),
    (2, 4, 4, 128, 0, 77, 333, [5, 150]),
    (3, 8, 2, 64, 0, 300, 90, [0, 70, 200]),
    (1, 2, 1, 128, 0, 1000, 130, [33]),
    (1000, 2, 1, 64, 0, 1, 140, [i % 3 for i in range(1000)]),
    (3, 10, 2, 128, 7, 63, 64, [64, 65, 192]),
]


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("case", SHARED, ids=lambda c: "B%d-H%d.%d-D%d-k%d-R%d-S%d" % c[:7])
def test_shared_attention(abi, case, paged):
    s = Shared(abi, 11, *case, paged=paged)
    s.call()
    assert s.status.item() == 0
    s.check()


@pytest.mark.parametrize("seed", range(12))
def test_shared_attention_random_shapes(abi, seed):
    r = random.Random(900 + seed)
    Hkv, G, D = r.choice([1, 2, 4]), r.randint(1, 9), r.choice([64, 128])
    k = r.choice([0, 0, 1, 2, 3, 6, 8])
    R = k * (k + 2) if k else r.randint(1, 40)
    B = r.randint(1, 12)
    s = Shared(abi, seed, B, Hkv * G, Hkv, D, k, R, r.choice([0, r.randint(1, 300), r.randint(300, 3000)]),
               [r.choice([0, r.randint(1, 400)]) for _ in range(B)], paged=r.random() < 0.5, S_extra=r.randint(0, 200),
               P_extra=r.randint(0, 200))
    s.call()
    assert s.status.item() == 0
    s.check()


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_shared_attention_does_not_depend_on_timing_or_neighbours(abi, paged):
    """The same bits twice, also with a workspace that held something else, without an LSE, and on another stream."""
    s = Shared(abi, 5, 6, 8, 2, 128, 4, 24, 900, [0, 10, 130, 200, 64, 500], paged=paged)
    s.call()
    first, lse = s.out.clone(), s.lse.clone()
    s.ws.fill_(0x3c)
    s.out.fill_(NAN)
    s.lse.fill_(7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(stream=side, lse=False)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s.out, first) and bool((s.lse == 7.0).all())
    s.call()
    assert torch.equal(s.out, first) and torch.equal(s.lse, lse)


def test_shared_attention_without_caches(abi):
    """No shared rows, no own rows, neither: the parts that are empty need no memory."""
    for S, n in ((200, 0), (0, 90), (0, 0)):
        s = Shared(abi, 13, 3, 6, 2, 64, 3, 15, S, [n] * 3, S_extra=0, P_extra=0)
        abi.tidar_attn_step_shared(
            s.q, s.kn, s.vn, s.ks if S else None, s.vs if S else None, s.shared_len, S, s.kc if n else None,
            s.vc if n else None, s.prefix_len, s.B, s.Hq, s.Hkv, s.D, s.k, s.R, n, s.scale, s.mode, s.out, s.lse, s.ws,
            s.ws.numel(), s.status)
        assert s.status.item() == 0
        s.check()


def test_shared_attention_two_calls_at_once(abi):
    """Two graphs with a workspace each, replayed on two streams at the same time, give what each gives alone."""
    calls = [Shared(abi, 20 + i, 4, 8, 2, 128, 4, 24, 700 + 300 * i, [0, 100, 300, 64], paged=i == 1) for i in (0, 1)]
    want, graphs = [], []
    for s in calls:
        s.call()
        want.append((s.out.clone(), s.lse.clone()))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                s.call(stream=torch.cuda.current_stream())
        graphs.append(g)
        s.out.fill_(NAN)
        s.lse.fill_(NAN)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, (o, z) in zip(calls, want):
        assert s.status.item() == 0
        assert torch.equal(s.out, o) and torch.equal(s.lse, z)


def test_shared_attention_wait_that_runs_out(abi):
    """A wait that expires is reported, and the context and the same buffers stay usable."""
    s = Shared(abi, 14, 2, 8, 2, 128, 2, 8, 900, [100, 300])
    s.ws.fill_(0)
    abi.tidar_testing_attn_step_shared_stalled(
        s.q, s.kn, s.vn, s.ks, s.vs, s.shared_len, s.S_max, s.kc, s.vc, s.prefix_len, s.B, s.Hq, s.Hkv, s.D, s.k, s.R,
        s.P_max, s.scale, s.mode, s.out, s.lse, s.ws, s.ws.numel(), s.status, 200000)
    assert s.status.item() == abi.TIDAR_DEV_TIMEOUT
    s.status.zero_()
    s.call()
    assert s.status.item() == 0
    s.check()


def test_shared_attention_large_scores(abi):
    """Scores beyond the range of exp, with the maximum growing along the keys."""
    s = Shared(abi, 6, 2, 4, 2, 64, 2, 8, 700, [300, 0])
    s.q.mul_(30.0)
    s.ks[:, :s.S].mul_(torch.linspace(0.1, 3.0, s.S, device=DEV)[None, :, None].to(torch.bfloat16))
    s.call()
    out, lse, absum, vmax = s.reference()
    # a score is off by up to D 2^-24 times the sum of |q_i k_i| (fp32 sums); that many times its weight
    mag = (s.q.double().abs().amax() * 64**0.5) * s.scale * 64 * 2.0**-24 * 10
    err = (s.out.double() - out).abs()
    assert bool((err <= ref.attn_tolerance(out, absum, vmax) + 2 * mag * (absum + out.abs())).all())
    assert bool(((s.lse.double() - lse).abs() <= 1e-4 + mag).all())


def test_shared_attention_masked_keys_may_hold_anything(abi):
    s = Shared(abi, 7, 2, 4, 2, 128, 3, 15, 200, [10, 140])
    s.kn[:, 6:9] = NAN                # the keys of pre-draft group 1: only its own rows see them
    s.kn[:, 9:12] = float("inf")      # and of group 2
    s.call()
    torch.cuda.synchronize()
    clean = [r for r in range(15) if not 6 <= r < 12]
    out, lse, absum, vmax = s.reference()
    err = (s.out.double() - out).abs()[:, clean]
    assert bool((err <= ref.attn_tolerance(out, absum, vmax)[:, clean]).all())
    assert bool(torch.isnan(s.out[:, 6:9].float()).all())


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_shared_attention_infinity_in_one_column_of_v(abi, paged):
    """An infinity in V reaches its own column of the rows that see it, as an infinity, and no other column."""
    for D, G in ((64, 2), (128, 3)):
        s = Shared(abi, 57, 3, 2 * G, 2, D, 0, 5, 700, [300, 0, 40], paged=paged)
        v, p = (s.vp, s.shared_table) if paged else (s.vs, None)
        for col, x in ((3, math.inf), (D - 1, -math.inf)):  # shared row 70 of KV head 0
            s.vs[0, 70, col] = x
            if paged:
                v[int(p[1]), 0, 6, col] = x
        s.vc[0, 1, 17, 9] = math.inf  # own row 17 of sequence 0, KV head 1
        if paged:
            s.vp[int(s.table[0, 0]), 1, 17, 9] = math.inf
        s.call()
        assert s.status.item() == 0
        want = torch.zeros_like(s.out, dtype=torch.float32)
        want[:, :, :G, 3], want[:, :, :G, D - 1], want[0, :, G:, 9] = math.inf, -math.inf, math.inf
        assert torch.equal(torch.where(want != 0, s.out.float(), 0.0), want)
        for t in (s.vs, s.vc):
            t[t.isinf()] = 0.0
        out, lse, absum, vmax = s.reference()
        off = (s.out.double() - out).abs() > ref.attn_tolerance(out, absum, vmax)
        assert not bool((off & (want == 0)).any())
        assert bool(((s.lse.double() - lse).abs() <= 1e-4).all())


@pytest.mark.parametrize("v", [0.0, 2.0**-133, 2.0**-130, 2.0**-126, 2.0**-112, 9e37])
def test_shared_attention_values_of_any_size(abi, v):
    """Shared rows of V that are zero but for one element of size v, down to the smallest subnormal; then all of size v."""
    s = Shared(abi, 50, 2, 4, 2, 64, 2, 8, 700, [300, 0])
    s.vs[:, :s.S] = 0.0
    s.vs[:, 3, 5] = v
    if v < 1.0:
        s.call()
        assert s.status.item() == 0
        s.check()
    s = Shared(abi, 52, 1, 2, 1, 128, 0, 1, 2, [0])
    s.q.zero_()  # (equal weights: the shared keys' partial row sums to 2 v)
    s.vs[:], s.vn[:] = v, v
    s.call()
    out, lse, absum, vmax = s.reference()
    err = (s.out.double() - out).abs()
    # (sums below 2^-126 lose up to 2^-126 each: subnormal weights and products may count as zero)
    assert bool((err <= ref.attn_tolerance(out, absum, vmax) + 2.0**-125).all())


def test_shared_attention_weights_of_large_values(abi):
    """V of 1e33 behind scores that grow by 2^9.5 after the first keys: the output stays within V's range."""
    s = Shared(abi, 53, 4, 4, 4, 64, 0, 1, 0, [20000] * 4)
    for x in (s.q, s.kn, s.kc):
        x.zero_()
    s.scale = 1.0
    s.q[..., 0] = 8.0
    s.kc[:, :, 64:20000, 0] = s.kn[..., 0] = 9.5 * math.log(2) / 8
    s.vc[:, :, :20000] = 1e33 * torch.where(torch.arange(64, device=DEV) % 3 == 0, -1.0, 1.0)
    s.vn.copy_(s.vc[:, :, 0][:, None])
    s.call()
    assert s.status.item() == 0
    s.check()


@pytest.mark.parametrize("D,Hq,Hkv,k,B,S", [(128, 14, 2, 8, 4, 8000), (64, 12, 2, 4, 8, 4000), (128, 3, 1, 16, 2, 16000)])
def test_shared_attention_time_does_not_depend_on_the_call_before(abi, D, Hq, Hkv, k, B, S):
    """Groups that do not divide 128 leave rows of a row tile without a query: what a call before left in shared memory
    there (NaN or zeros) changes neither the result nor the time (a second look at every score cost 14 to 23 % more
    after NaN than after zeros; event times come in steps of 1 us, so medians of 25 us and more agree within 10 %)."""
    s = Shared(abi, 55, B, Hq, Hkv, D, k, k * (k + 2), S, [500] * B)
    before = Shared(abi, 56, 1, 4, 1, D, 0, 64, 148 * 128, [0])
    took, outs = {0.0: [], NAN: []}, []
    for _ in range(40):
        for fill in took:
            before.q.fill_(fill)
            before.call()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            s.call()
            b.record()
            b.synchronize()
            took[fill].append(a.elapsed_time(b))
            outs = (outs + [s.out.clone()])[-2:]
    assert torch.equal(*outs)
    zeros, nans = (sorted(x)[len(x) // 2] for x in took.values())
    assert nans <= 1.1 * zeros, (zeros, nans)


@pytest.mark.parametrize("Hq,k,B", [(32, 8, 8), (64, 16, 2)])
def test_shared_attention_padded_sequence_of_nan(abi, Hq, k, B):
    """A padding sequence whose queries are NaN changes neither the others' bits nor the call's time (it took 2.2 to 2.4
    times as long when its rows asked for a maximum again and again)."""
    s = Shared(abi, 58, B, Hq, 8, 128, k, k * (k + 2), 4000, [500] * (B - 1) + [0])
    took, outs = {0.0: [], NAN: []}, []
    for _ in range(15):
        for fill in took:
            s.q[B - 1].fill_(fill)
            s.call()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            s.call()
            b.record()
            b.synchronize()
            took[fill].append(a.elapsed_time(b))
            if len(outs) < 2:
                outs.append((s.out.clone(), s.lse.clone()))
    assert s.status.item() == 0
    (o0, z0), (o1, z1) = outs
    assert torch.equal(o0[:B - 1], o1[:B - 1]) and torch.equal(z0[:B - 1], z1[:B - 1])
    assert bool(o1[B - 1].isnan().all()) and bool(z1[B - 1].isnan().all())
    zeros, nans = (sorted(x)[len(x) // 2] for x in took.values())
    assert nans <= 1.15 * zeros, (zeros, nans)


def test_shared_attention_bad_lengths_and_pages(abi):
    s = Shared(abi, 8, 3, 4, 2, 64, 2, 8, 100, [50, 60, 70])
    for bad in (-1, s.P_max + 1):
        s.out.fill_(7.0)
        s.prefix_len[1] = bad
        s.status.zero_()
        s.call()
        assert s.status.item() == abi.TIDAR_DEV_BAD_PREFIX
        assert bool((s.out[1] == 7.0).all())
        out, _, absum, vmax = Shared.reference(s)
        err = (s.out.double() - out).abs()
        assert bool((err <= ref.attn_tolerance(out, absum, vmax))[[0, 2]].all())
    s.prefix_len[1] = 60
    for bad in (-1, s.S_max + 1):
        s.out.fill_(7.0)
        s.status.zero_()
        s.shared_len[0] = bad
        s.call()
        assert s.status.item() == abi.TIDAR_DEV_BAD_PREFIX
        assert bool((s.out == 7.0).all())
    s = Shared(abi, 9, 3, 4, 2, 64, 2, 8, 100, [50, 60, 170], paged=True)
    keep = s.table[2, 1].item()
    for bad in (-1, s.num_pages):
        s.out.fill_(7.0)
        s.status.zero_()
        s.table[2, 1] = bad
        s.call()
        assert s.status.item() == abi.TIDAR_DEV_BAD_PAGE
        assert bool((s.out[2] == 7.0).all()) and not bool((s.out[:2] == 7.0).all())
    s.table[2, 1] = keep
    s.table[0, 1:] = -5  # pages past a sequence's rows are not read
    s.status.zero_()
    s.call()
    assert s.status.item() == 0
    s.check()
    s.shared_table[1] = s.num_pages
    s.out.fill_(7.0)
    s.call()
    assert s.status.item() == abi.TIDAR_DEV_BAD_PAGE
    assert bool((s.out == 7.0).all())


def test_shared_attention_equals_attention_over_a_copied_prefix(abi):
    """tidar_attn_step on caches that hold the shared rows first gives the same rows, within both calls' rounding."""
    s = Shared(abi, 10, 3, 16, 4, 128, 4, 24, 300, [0, 130, 77], P_extra=0)
    s.call()
    P = s.S + s.P_max
    kc, vc = (torch.cat([x[None, :, :s.S].expand(3, -1, -1, -1), y], 2).contiguous()
              for x, y in ((s.ks, s.kc), (s.vs, s.vc)))
    out, lse = torch.empty_like(s.out), torch.empty_like(s.lse)
    abi.tidar_attn_step(s.q, s.kn, s.vn, kc, vc, s.prefix_len + s.S, 3, 16, 4, 128, 4, P, s.scale, 0, out, lse, None, 0,
                        s.status)
    assert s.status.item() == 0
    _, _, absum, vmax = s.reference()
    tol = 2 * ref.attn_tolerance(out.double(), absum, vmax)
    assert bool(((out.double() - s.out.double()).abs() <= tol).all())
    assert (lse - s.lse).abs().max().item() <= 2e-4


def test_shared_attention_offsets_past_32_bits(abi):
    """A cache of 2^32 elements and more: the last sequence's rows lie behind 4 Gi elements."""
    B, Hkv, D, P_max = 3, 4, 128, 3 << 20
    g = _gen(12)
    kc = torch.zeros((B, Hkv, P_max, D), dtype=torch.bfloat16, device=DEV)
    n = 200
    kc[:, :, :n] = _normal(g, B, Hkv, n, D)
    q, kn, vn = _normal(g, B, 3, Hkv, D), _normal(g, B, 3, Hkv, D), _normal(g, B, 3, Hkv, D)
    out = torch.empty((B, 3, Hkv, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((B, 3, Hkv), dtype=torch.float32, device=DEV)
    st, lens = _i32([0]), [n, 1, n]
    size = abi.tidar_attn_shared_workspace_size(B, Hkv, Hkv, D, 3, 0, P_max)
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    abi.tidar_attn_step_shared(q, kn, vn, None, None, _i32([0]), 0, kc, kc, _i32(lens), B, Hkv, Hkv, D, 1, 3, P_max,
                               D**-0.5, 0, out, lse, ws, ws.numel(), st)
    assert st.item() == 0
    none = kc[0, :, :0]
    want, zl, absum, vmax = ref.attn_shared(q, kn, vn, none, none, 0, kc, kc, lens, 0, 1, D**-0.5)
    assert bool(((out.double() - want).abs() <= ref.attn_tolerance(want, absum, vmax)).all())
    assert (lse.double() - zl).abs().max().item() <= 1e-4
    # the mass and the eviction reach the same places
    mass = torch.zeros((B, Hkv, P_max), device=DEV)
    ptr = abi.pointer_array
    abi.tidar_attn_mass(ptr([q], DEV), ptr([lse], DEV), ptr([kc], DEV), ptr([mass], DEV), None, 0, 0, _i32(lens),
                        _i32([3, 1, 2]), 1, B, Hkv, Hkv, D, 3, P_max, D**-0.5, 1.0, st)
    assert st.item() == 0
    want = ref.mass_update(torch.zeros((Hkv, n), device=DEV), q[2], lse[2], kc[2], n, 2, D**-0.5, 1.0)
    assert bool(((mass[2, :, :n].double() - want).abs() <= ref.MASS_RTOL * want).all())


class Caches:
    """L layers of caches with masses; paged ones keep contiguous copies as the reference's view."""

    def __init__(self, seed, L, B, Hkv, D, lens, paged=False, extra=3, nan=True):
        g = _gen(seed)
        self.g, self.L, self.B, self.Hkv, self.D, self.lens, self.paged = g, L, B, Hkv, D, lens, paged
        self.P_max = _pad(max(lens) + extra) if paged else max(lens) + extra
        self.kc = [_normal(g, B, Hkv, self.P_max, D) for _ in range(L)]
        self.vc = [_normal(g, B, Hkv, self.P_max, D) for _ in range(L)]
        if nan:
            for t in self.kc + self.vc:
                for b in range(B):
                    t[b, :, lens[b]:] = NAN
        self.mass = [torch.rand((B, Hkv, self.P_max), generator=g, device=DEV) for _ in range(L)]
        self.prefix_len, self.status = _i32(lens), _i32([0])
        if paged:
            n = self.P_max // PAGE
            ids = torch.randperm(B * n + 2, generator=g, device=DEV).to(torch.int32)
            self.num_pages, self.table = ids.numel(), ids[:B * n].reshape(B, n).contiguous()
            self.kp, self.vp = ([self._to_pool(t) for t in x] for x in (self.kc, self.vc))

    def _to_pool(self, t):
        pool = torch.full((self.num_pages, self.Hkv, PAGE, self.D), NAN, dtype=torch.bfloat16, device=DEV)
        for b in range(self.B):
            _scatter(t[b], self.table[b], pool)
        return pool

    def view(self, which, l):
        """Contiguous [B, Hkv, P_max, D] view of a layer's K (0) or V (1)."""
        if not self.paged:
            return (self.kc, self.vc)[which][l]
        x = (self.kp, self.vp)[which][l][self.table.long()]  # [B, n, Hkv, 64, D]
        return x.transpose(1, 2).reshape(self.B, self.Hkv, self.P_max, self.D)

    def args(self, abi):
        k, v = (self.kp, self.vp) if self.paged else (self.kc, self.vc)
        paging = (self.table, self.table.shape[1], self.num_pages) if self.paged else (None, 0, 0)
        return abi.pointer_array(k, DEV), abi.pointer_array(v, DEV), abi.pointer_array(self.mass, DEV), paging

    def add_mass(self, abi, q, lse, counts, decay, stream=None):
        k, _, m, paging = self.args(abi)
        L, B, R, Hq, D = q.shape
        self.keep = (k, m, abi.pointer_array(list(q), DEV), abi.pointer_array(list(lse), DEV))
        abi.tidar_attn_mass(self.keep[2], self.keep[3], k, m, *paging, self.prefix_len, counts, L, B, Hq, self.Hkv, D, R,
                            self.P_max, D**-0.5, decay, self.status, stream=stream)

    def evict(self, abi, budget, sink, recent, stream=None):
        k, v, m, paging = self.args(abi)
        self.keep = (k, v, m)
        abi.tidar_kv_evict(k, v, m, *paging, self.prefix_len, self.L, self.B, self.Hkv, self.D, self.P_max, budget, sink,
                           recent, self.status, stream=stream)


MASS = [  # L, B, Hq, Hkv, D, R, lens, counts, decay
    (1, 1, 1, 1, 64, 1, [1], [1], 1.0),
    (1, 1, 4, 1, 128, 8, [8], [8], 1.0),
    (2, 3, 8, 2, 128, 8, [300, 0, 129], [5, 0, 8], 0.9),
    (3, 2, 6, 2, 64, 24, [128, 127], [24, 1], 1.0),
    (2, 2, 32, 8, 128, 8, [1000, 517], None, 0.5),
    (1, 2, 7, 1, 128, 50, [260, 64], [50, 33], 0.0),
    (1, 2, 16, 2, 64, 288, [700, 300], [288, 131], 1.0),
    (40, 1, 2, 1, 64, 4, [333], [3], 0.98),
    (1, 5, 128, 1, 64, 3, [200, 3, 2, 1, 64], [3, 3, 2, 1, 0], 1.0),
    (1, 1, 8, 1, 128, 4, [9000], [4], 1.0),
]


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("case", MASS, ids=lambda c: "L%d-B%d-H%d.%d-D%d-R%d" % c[:6])
def test_attention_mass(abi, case, paged):
    L, B, Hq, Hkv, D, R, lens, counts, decay = case
    c = Caches(21, L, B, Hkv, D, lens, paged=paged)
    q = _normal(c.g, L, B, R, Hq, D, scale=1.5)
    lse = math.log(max(lens) + 1) + torch.rand((L, B, R, Hq), generator=c.g, device=DEV)
    rows = counts if counts is not None else [min(R, n) for n in lens]
    for b in range(B):  # rows past the count are not read
        q[:, b, rows[b]:] = NAN
        lse[:, b, rows[b]:] = NAN
    before = [m.clone() for m in c.mass]
    c.add_mass(abi, q, lse, None if counts is None else _i32(counts), decay)
    assert c.status.item() == 0
    for l in range(L):
        for b in range(B):
            n = lens[b]
            want = ref.mass_update(before[l][b], q[l, b], lse[l, b], c.view(0, l)[b], n, rows[b], D**-0.5, decay)
            got = c.mass[l][b].double()
            assert bool(((got - want)[:, :n].abs() <= ref.MASS_RTOL * want[:, :n] + 1e-30).all())
            assert torch.equal(c.mass[l][b, :, n:], before[l][b, :, n:])


def test_attention_mass_sums_to_the_visible_share(abi):
    """With the LSE over exactly the cache, every row's weights sum to one: the mass over all rows is rows * G."""
    L, B, Hq, Hkv, D, n, a = 1, 1, 8, 2, 128, 900, 6
    c = Caches(22, L, B, Hkv, D, [n])
    q = _normal(c.g, L, B, a, Hq, D, scale=1.5)
    lse = torch.zeros((L, B, a, Hq), device=DEV)
    for j in range(a):
        for h in range(Hq):
            x = (c.kc[0][0, h // 4, :n - a + j + 1].double() @ q[0, 0, j, h].double()) * D**-0.5
            lse[0, 0, j, h] = torch.logsumexp(x, 0)
    c.mass[0].zero_()
    c.add_mass(abi, q, lse, None, 1.0)
    total = c.mass[0][0, :, :n].double().sum(1)
    assert bool(((total - a * 4).abs() <= 2e-4 * a * 4).all())


@pytest.mark.parametrize("D,R,Hq,Hkv", [(64, 3, 1, 1), (128, 5, 8, 2), (64, 77, 12, 2)])
def test_attention_mass_of_keys_with_scores_of_minus_infinity(abi, D, R, Hq, Hkv):
    """A cached key that holds an infinity and that every query scores -inf gets no weight, whatever the rows' number."""
    n = 300
    c = Caches(26, 1, 1, Hkv, D, [n])
    q = _normal(c.g, 1, 1, R, Hq, D)
    q[..., 0] = q[..., 0].abs() + 0.5
    keys = [0, 130, n - R - 1, n - 1]  # the last one is new: only the last query sees it
    c.kc[0][0, :, keys, 0] = -float("inf")
    lse = torch.full((1, 1, R, Hq), 6.0, device=DEV)
    before = c.mass[0].clone()
    c.add_mass(abi, q, lse, None, 0.5)
    assert c.status.item() == 0
    want = ref.mass_update(before[0], q[0, 0], lse[0, 0], c.kc[0][0], n, R, D**-0.5, 0.5)
    got = c.mass[0][0].double()
    assert bool((want[:, keys[:3]] == 0.5 * before[0][:, keys[:3]].double()).all()) and bool((want[:, n - 1] == 0).all())
    assert bool(((got - want)[:, :n].abs() <= ref.MASS_RTOL * want[:, :n]).all())


def test_attention_mass_wait_that_runs_out(abi):
    c = Caches(25, 2, 2, 2, 128, [700, 300])
    q, lse = _normal(c.g, 2, 2, 8, 4, 128), torch.full((2, 2, 8, 4), 6.0, device=DEV)
    before = [m.clone() for m in c.mass]
    k, _, m, _ = c.args(abi)
    qs, ls = abi.pointer_array(list(q), DEV), abi.pointer_array(list(lse), DEV)
    abi.tidar_testing_attn_mass_stalled(qs, ls, k, m, None, 0, 0, c.prefix_len, None, 2, 2, 4, 2, 128, 8, c.P_max,
                                        128**-0.5, 1.0, c.status, 200000)
    assert c.status.item() == abi.TIDAR_DEV_TIMEOUT
    c.status.zero_()
    for x, y in zip(c.mass, before):
        x.copy_(y)
    c.add_mass(abi, q, lse, None, 1.0)
    assert c.status.item() == 0
    for l in range(2):
        for b, n in enumerate((700, 300)):
            want = ref.mass_update(before[l][b], q[l, b], lse[l, b], c.kc[l][b], n, 8, 128**-0.5, 1.0)
            assert bool(((c.mass[l][b, :, :n].double() - want[:, :n]).abs() <= ref.MASS_RTOL * want[:, :n]).all())


def test_attention_mass_same_bits_twice(abi):
    """The sums do not depend on timing: the same bits from the same start, also on another stream."""
    c = Caches(26, 3, 4, 2, 64, [900, 77, 0, 512])
    q, lse = _normal(c.g, 3, 4, 40, 12, 64), torch.full((3, 4, 40, 12), 6.5, device=DEV)
    before, got = [m.clone() for m in c.mass], []
    side = torch.cuda.Stream()
    for stream in (None, None, side):
        for x, y in zip(c.mass, before):
            x.copy_(y)
        side.wait_stream(torch.cuda.current_stream())
        c.add_mass(abi, q, lse, _i32([40, 30, 0, 7]), 0.75, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        got.append([m.clone() for m in c.mass])
    assert c.status.item() == 0
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))


def test_attention_mass_bad_inputs(abi):
    c = Caches(23, 2, 3, 2, 64, [100, 200, 150], paged=True)
    q, lse = _normal(c.g, 2, 3, 8, 4, 64), torch.full((2, 3, 8, 4), 5.0, device=DEV)
    before = [m.clone() for m in c.mass]

    def run(counts, want):
        for m, w in zip(c.mass, before):
            m.copy_(w)
        c.status.zero_()
        c.add_mass(abi, q, lse, _i32(counts), 1.0)
        assert c.status.item() == want
        for l in range(2):
            assert torch.equal(c.mass[l][1], before[l][1])
            assert not torch.equal(c.mass[l][0], before[l][0]) and not torch.equal(c.mass[l][2], before[l][2])

    run([8, -1, 8], abi.TIDAR_DEV_BAD_ACCEPT)
    run([8, 9, 8], abi.TIDAR_DEV_BAD_ACCEPT)
    c.prefix_len[1] = 3
    run([8, 4, 8], abi.TIDAR_DEV_BAD_ACCEPT)  # more rows than the cache holds
    c.prefix_len[1] = -1
    run([8, 0, 8], abi.TIDAR_DEV_BAD_PREFIX)
    c.prefix_len[1] = c.P_max + 1
    run([8, 8, 8], abi.TIDAR_DEV_BAD_PREFIX)
    c.prefix_len[1] = 200
    c.table[1, 2] = c.num_pages
    run([8, 8, 8], abi.TIDAR_DEV_BAD_PAGE)


EVICT = [  # L, B, Hkv, D, lens, budget, sink, recent
    (1, 1, 1, 64, [2], 1, 0, 0),
    (1, 1, 1, 64, [5], 0, 0, 0),
    (1, 2, 2, 128, [5, 3], 4, 2, 2),
    (2, 3, 2, 128, [300, 100, 129], 100, 4, 32),
    (2, 2, 2, 64, [1000, 1009], 1000, 1, 77),
    (36, 1, 8, 128, [264], 256, 4, 16),
    (1, 1, 1, 128, [5000], 700, 0, 600),
    (1, 1, 2, 64, [9000], 8000, 16, 4000),
    (1, 1, 1, 64, [30000], 20000, 3, 500),
    (1, 1, 9, 64, [29000], 28000, 3, 500),
    (1, 2, 1, 64, [60000, 8300], 30000, 2, 100),
    (1, 2, 80, 64, [26500, 130], 120, 4, 16),
    (1, 2, 1, 128, [700, 650], 600, 0, 600),
    (1, 2, 1, 128, [700, 650], 600, 600, 0),
    (3, 7, 3, 64, [64 * i + i for i in range(7)], 130, 3, 60),
]


def _check_evict(c, kept_k, kept_v, kept_m, lens, budget, sink, recent):
    assert c.prefix_len.tolist() == [min(n, budget) for n in lens]
    for l in range(c.L):
        k, v = c.view(0, l), c.view(1, l)
        for b, n in enumerate(lens):
            for h in range(c.Hkv):
                to, of = ref.evict_moves(kept_m[l][b, h].tolist(), n, budget, sink, recent)
                for got, had in ((k, kept_k[l]), (v, kept_v[l]), (c.mass[l], kept_m[l])):
                    want = had[b, h].clone()
                    want[to] = had[b, h][of]
                    assert torch.equal(got[b, h].nan_to_num(9.0), want.nan_to_num(9.0))


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("masses", ["spread", "ties", "odd"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "L%d-B%d-H%d-D%d-n%d-to%d" % (*c[:4], max(c[4]), c[5]))
def test_evict(abi, case, masses, paged):
    L, B, Hkv, D, lens, budget, sink, recent = case
    c = Caches(31, L, B, Hkv, D, lens, paged=paged, extra=1, nan=not paged)
    for m in c.mass:
        if masses == "spread":
            m.copy_(torch.exp(4 * torch.randn(m.shape, generator=c.g, device=DEV)))
        elif masses == "ties":  # few values, many equal, most of them zero
            m.copy_(torch.randint(0, 4, m.shape, generator=c.g, device=DEV).clamp_min(1) - 1)
        else:  # negative values, both zeros, infinities and NaN, and neighbouring floats
            pick = torch.randint(0, 8, m.shape, generator=c.g, device=DEV)
            vals = torch.tensor([0.0, -0.0, 1.0, 1.0000001, float("inf"), NAN, -2.5, 1e-40], device=DEV)
            m.copy_(vals[pick])
    had = [[c.view(x, l).clone() for l in range(L)] for x in (0, 1)] + [[m.clone() for m in c.mass]]
    c.evict(abi, budget, sink, recent)
    assert c.status.item() == 0
    _check_evict(c, *had, lens, budget, sink, recent)


def test_evict_twice_and_below_the_budget(abi):
    c = Caches(32, 2, 2, 2, 64, [400, 90])
    c.evict(abi, 128, 4, 16)
    state = [t.clone() for t in c.kc + c.vc + c.mass]
    assert c.prefix_len.tolist() == [128, 90]
    c.evict(abi, 128, 4, 16)
    c.evict(abi, 10**6, 4, 16)  # a budget no cache reaches
    assert c.prefix_len.tolist() == [128, 90] and c.status.item() == 0
    for t, w in zip(c.kc + c.vc + c.mass, state):
        assert torch.equal(t.nan_to_num(9.0), w.nan_to_num(9.0))


def test_evict_longest_cache(abi):
    n, budget = 65536, 32768 + 100
    c = Caches(33, 1, 1, 1, 64, [n], extra=0)
    had = [[c.kc[0].clone()], [c.vc[0].clone()], [c.mass[0].clone()]]
    c.evict(abi, budget, 0, 100)
    assert c.status.item() == 0
    _check_evict(c, *had, [n], budget, 0, 100)


def test_evict_bad_inputs_leave_the_sequence(abi):
    c = Caches(34, 2, 3, 2, 64, [300, 300, 300], paged=True, nan=False)
    page = c.table[1, 3].item()
    for what in ("negative", "long", "page"):
        if what == "page":
            c.table[1, 3] = -1
        c.prefix_len.copy_(_i32([300, {"negative": -4, "long": c.P_max + 1, "page": 300}[what], 300]))
        c.status.zero_()
        had = [[t[page].clone() for t in c.kp + c.vp], [m[1].clone() for m in c.mass]]
        c.evict(abi, 128, 4, 16)
        assert c.status.item() == (abi.TIDAR_DEV_BAD_PAGE if what == "page" else abi.TIDAR_DEV_BAD_PREFIX)
        assert c.prefix_len.tolist()[0] == 128 and c.prefix_len.tolist()[2] == 128
        assert c.prefix_len.tolist()[1] == {"negative": -4, "long": c.P_max + 1, "page": 300}[what]
        for t, w in zip([t[page] for t in c.kp + c.vp] + [m[1] for m in c.mass], had[0] + had[1]):
            assert torch.equal(t, w)


def test_evict_offsets_past_32_bits(abi):
    B, Hkv, D, P_max, n = 72, 8, 128, 65536, 500
    g = _gen(35)
    kc = torch.zeros((B, Hkv, P_max, D), dtype=torch.bfloat16, device=DEV)
    kc[B - 1, :, :n] = _normal(g, Hkv, n, D)
    vc = torch.zeros((B, Hkv, P_max, D), dtype=torch.bfloat16, device=DEV)
    vc[B - 1, :, :n] = _normal(g, Hkv, n, D)
    mass = torch.rand((B, Hkv, P_max), generator=g, device=DEV)
    lens, st = _i32([0] * (B - 1) + [n]), _i32([0])
    k0, v0, m0 = kc[B - 1, :, :n].clone(), vc[B - 1, :, :n].clone(), mass[B - 1, :, :n].clone()
    ptr = abi.pointer_array
    abi.tidar_kv_evict(ptr([kc], DEV), ptr([vc], DEV), ptr([mass], DEV), None, 0, 0, lens, 1, B, Hkv, D, P_max, 200, 4,
                       50, st)
    assert st.item() == 0 and lens.tolist() == [0] * (B - 1) + [200]
    for h in range(Hkv):
        to, of = ref.evict_moves(m0[h].tolist(), n, 200, 4, 50)
        want = k0[h].clone()
        want[to] = k0[h][of]
        assert torch.equal(kc[B - 1, h, :200], want[:200])
    assert bool((kc[0] == 0).all())
    assert torch.equal(vc[B - 1, :, 150:200], v0[:, n - 50:])


@pytest.mark.parametrize("budget,sink,recent", [(200, 4, 50), (450, 0, 7)])
def test_evict_keys_values_and_masses_past_32_bits(abi, budget, sink, recent):
    """The last sequence's rows lie behind 4 Gi elements: its keys, its values and its masses all move, and nothing else."""
    B, Hkv, D, P_max, n = 66, 8, 128, 65536, 500
    g = _gen(36)
    k, v = (torch.zeros((B, Hkv, P_max, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[B - 1, :, :n], v[B - 1, :, :n] = _normal(g, Hkv, n, D), _normal(g, Hkv, n, D)
    mass = torch.rand((B, Hkv, P_max), generator=g, device=DEV)
    lens, st = _i32([0] * (B - 1) + [n]), _i32([0])
    had = [t[B - 1, :, :n].clone() for t in (k, v, mass)]
    others = mass[:B - 1].clone()
    ptr = abi.pointer_array
    abi.tidar_kv_evict(ptr([k], DEV), ptr([v], DEV), ptr([mass], DEV), None, 0, 0, lens, 1, B, Hkv, D, P_max, budget, sink,
                       recent, st)
    assert st.item() == 0 and lens.tolist() == [0] * (B - 1) + [budget]
    for h in range(Hkv):
        to, of = ref.evict_moves(had[2][h].tolist(), n, budget, sink, recent)
        for got, was in zip((k, v, mass), had):
            want = was[h].clone()
            want[to] = was[h][of]
            assert torch.equal(got[B - 1, h, :n], want)
    for t in (k, v):
        assert not bool(t[0].any()) and not bool(t[B - 2].any()) and not bool(t[B - 1, :, n:].any())
    assert torch.equal(mass[:B - 1], others)


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_decode_with_shared_prefix_and_bounded_caches(abi, paged):
    """The operators as a serving loop uses them: attention over [shared | own | new] in every layer, verify + commit,
    the accepted drafts' mass, then the eviction; every step against 64-bit references, captured into a graph and
    replayed for the odd steps."""
    L, B, Hq, Hkv, D, k, V, S = 2, 3, 8, 2, 64, 4, 128, 150
    R, G, budget, sink, recent = k * (k + 2), 4, 96, 2, 16
    scale = D**-0.5
    c = Caches(41, L, B, Hkv, D, [90, 12, 140], paged=paged, extra=60, nan=False)
    g = c.g
    ks, vs = [_normal(g, Hkv, S, D) for _ in range(L)], [_normal(g, Hkv, S, D) for _ in range(L)]
    if paged:  # the shared rows in pages of their own behind the sequences' pages
        ns = _pad(S) // PAGE
        shared_table = _i32(list(range(c.num_pages, c.num_pages + ns)))
        for pools, s in ((c.kp, ks), (c.vp, vs)):
            for l in range(L):
                pools[l] = torch.cat([pools[l], torch.full((ns, Hkv, PAGE, D), NAN, dtype=torch.bfloat16, device=DEV)])
                _scatter(s[l], shared_table, pools[l])
        c.num_pages += ns
    for m in c.mass:
        m.zero_()
    q, kn, vn = (torch.empty((L, B, R, h, D), dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    out = torch.empty((L, B, R, Hq, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((L, B, R, Hq), device=DEV)
    p_log, q_log = torch.empty((B, k, V), device=DEV), torch.empty((B, k, V), device=DEV)
    g_log, u = torch.empty((B, k + 1, k, V), device=DEV), torch.empty((3, B, k), device=DEV)
    drafts, pre = torch.zeros((B, k), dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.uint8, device=DEV)
    u_res = torch.empty(B, device=DEV)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    acc, res, tok, nem, nd, nqg = i32(B), i32(B), i32(B, k), i32(B), i32(B, k), i32(B)
    npre = torch.empty(B, dtype=torch.uint8, device=DEV)
    shared_len = _i32([S])
    wsa = torch.empty(max(256, abi.tidar_attn_shared_workspace_size(B, Hq, Hkv, D, R, _pad(S), c.P_max)),
                      dtype=torch.uint8, device=DEV)
    wsv = torch.empty(abi.tidar_verify_commit_workspace_size(B, k, V), dtype=torch.uint8, device=DEV)
    kp_, vp_, mp_, paging = c.args(abi)
    ptrs = [abi.pointer_array(list(t), DEV) for t in (kn, vn, q, lse)]

    def step():
        st = torch.cuda.current_stream()
        for l in range(L):
            tail = (out[l], lse[l], wsa, wsa.numel(), c.status)
            if paged:
                abi.tidar_attn_step_shared_paged(q[l], kn[l], vn[l], c.kp[l], c.vp[l], shared_table,
                                                 shared_table.numel(), shared_len, *paging, c.prefix_len, B, Hq, Hkv, D,
                                                 k, R, scale, 0, *tail, stream=st)
            else:
                abi.tidar_attn_step_shared(q[l], kn[l], vn[l], ks[l], vs[l], shared_len, S, c.kc[l], c.vc[l],
                                           c.prefix_len, B, Hq, Hkv, D, k, R, c.P_max, scale, 0, *tail, stream=st)
        abi.tidar_verify_commit(p_log, q_log, 1, drafts, pre, u[0], u_res, 1.0, kp_, vp_, ptrs[0], ptrs[1], *paging, L, B,
                                Hkv, D, k, c.P_max, V, c.prefix_len, g_log, u[1], acc, res, tok, nem, None, None, nd, npre,
                                nqg, wsv, wsv.numel(), c.status, stream=st)
        abi.tidar_attn_mass(ptrs[2], ptrs[3], kp_, mp_, *paging, c.prefix_len, acc, L, B, Hq, Hkv, D, R, c.P_max, scale,
                            0.95, c.status, stream=st)
        abi.tidar_kv_evict(kp_, vp_, mp_, *paging, c.prefix_len, L, B, Hkv, D, c.P_max, budget, sink, recent, c.status,
                           stream=st)

    graph = torch.cuda.CUDAGraph()
    lens, accepted = [90, 12, 140], 0
    for t in range(8):
        for x in (kn, vn):
            x.copy_(_normal(g, L, B, R, Hkv, D))
        q.copy_(_normal(g, L, B, R, Hq, D, scale=1.5))
        for x in (q_log, g_log):
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        p_log.copy_(q_log + 0.3 * torch.randn(q_log.shape, generator=g, device=DEV))
        drafts.copy_(torch.randint(0, V, (B, k), generator=g, device=DEV))
        u.copy_(torch.rand(u.shape, generator=g, device=DEV))
        u_res.copy_(torch.rand(B, generator=g, device=DEV))
        old = [[c.view(x, l).clone() for l in range(L)] for x in (0, 1)] + [[m.clone() for m in c.mass]]
        if t == 1:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        if t % 2:
            graph.replay()
        else:
            step()
        assert c.status.item() == 0
        a = acc.tolist()
        accepted += sum(a)
        for l in range(L):
            o, z, absum, vmax = ref.attn_shared(q[l], kn[l], vn[l], ks[l], vs[l], S, old[0][l], old[1][l], lens, 0, k, scale)
            assert bool(((out[l].double() - o).abs() <= ref.attn_tolerance(o, absum, vmax)).all())
            assert bool(((lse[l].double() - z).abs() <= 1e-4).all())
            for b in range(B):
                n = lens[b] + a[b]
                had = []
                for x, new in ((0, kn), (1, vn)):
                    full = old[x][l][b].clone()
                    full[:, lens[b]:n] = new[l, b, :a[b]].transpose(0, 1)
                    had.append(full)
                want = ref.mass_update(old[2][l][b], q[l, b], lse[l, b], had[0], n, a[b], scale, 0.95)
                for h in range(Hkv):
                    # (the reference decides by its own masses: at these seeds no two candidates are that close)
                    got = c.mass[l][b, h].double()
                    to, of = ref.evict_moves(want[h].tolist(), n, budget, sink, recent)
                    w = want[h].clone()
                    w[to] = want[h][of]
                    m = min(n, budget)
                    assert bool(((got - w)[:m].abs() <= 2 * ref.MASS_RTOL * w[:m] + 1e-30).all())
                    for x in (0, 1):
                        rows = had[x][h].clone()
                        rows[to] = had[x][h][of]
                        assert torch.equal(c.view(x, l)[b, h, :m], rows[:m])
        lens = [min(n + x, budget) for n, x in zip(lens, a)]
        assert c.prefix_len.tolist() == lens
    assert accepted > 0

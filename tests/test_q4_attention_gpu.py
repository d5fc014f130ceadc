"""GPU: decode attention over the 4-bit cache against the oracle (64 bits, over
the values that the pools stand for).

The tolerance is an error bound, computed for each output element from the
oracle's own numbers; `reference` derives it."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import q4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
RAGGED = [0, 1, 7, 15, 16, 17, 33, 100, 129, 300, 513]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


class Case:
    """A batch over pools whose unreached slots hold 0xFF: NaN scales and
    minima, codes of 15."""

    def __init__(self, dtype, Hq, Hkv, D, B, lens, seed=0, k=None, v=None, q=None, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.B, self.Hkv, self.D = dtype, B, Hkv, D
        self.lens = torch.tensor(lens, dtype=torch.int32)
        need = [-(-n // B) for n in lens]
        nb, width = sum(need) + extra, max(1, max(need))
        order = torch.randperm(nb, generator=g).tolist()
        self.tables = torch.full((len(lens), width), -1, dtype=torch.int32)
        slots, at = [], 0
        for s, n in enumerate(lens):
            ids = order[at:at + need[s]]
            at += need[s]
            self.tables[s, :need[s]] = torch.tensor(ids, dtype=torch.int32)
            slots += [ids[p // B] * B + p % B for p in range(n)]
        T = len(slots)
        key = torch.randn(T, Hkv, D, generator=g) + torch.randn(1, Hkv, D, generator=g)
        value = torch.randn(T, Hkv, D, generator=g)
        key, value = (key if k is None else k(key)).to(dtype), (value if v is None else v(value)).to(dtype)
        self.k = torch.full(pkv.q4_cache_shape(nb, Hkv, B, D), 0xFF, dtype=torch.uint8)
        self.v = self.k.clone()
        q4.kv_write(self.k, self.v, key, value, torch.tensor(slots, dtype=torch.int64))
        self.q = torch.randn(len(lens), Hq, D, generator=g)
        self.q = (self.q if q is None else q(self.q)).to(dtype)
        self.scale = 1 / math.sqrt(D)

    def run(self, P=0, plan=False, out_dtype=torch.float32, tables=None, lens=None, pin=False):
        S, Hq, D = self.q.shape
        tables = self.tables if tables is None else tables
        lens = self.lens if lens is None else lens
        out = torch.full((S, Hq, D), float("nan"), dtype=out_dtype)
        out, q = (out.pin_memory(), self.q.pin_memory()) if pin else (out.to(DEV), self.q.to(DEV))
        ws = None
        if P or plan:
            n = pkv.decode_workspace_bytes(S, Hq, D, tables.shape[1] * self.B, P)
            ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
        pkv.paged_decode_attention_q4(out, q, self.k.to(DEV), self.v.to(DEV), tables.to(DEV),
                                      lens.to(DEV), self.scale, self.B, self.Hkv,
                                      partition_size=P, workspace=ws)
        torch.cuda.synchronize()
        return out.cpu()


def codes_of(pool, D, dtype, is_v):
    """Codes, scales and minima of every slot, float64 [NB, Hkv, B, D]."""
    nb, hkv, B, _ = pool.shape
    tiles = pool.reshape(nb, hkv, -1)
    c, s, m = (np.empty((nb, hkv, B, D)) for _ in range(3))
    for i in range(B):
        at, shift = q4.code_place(i, np.arange(D), B, D, is_v)
        c[:, :, i] = (tiles.numpy()[:, :, at] >> shift) & 15
        pair = tiles[:, :, q4.pair_place(i, B, D)].contiguous().view(dtype).double().numpy()
        pair = pair.reshape(nb, hkv, D // 64, 2).repeat(64, 2)
        s[:, :, i], m[:, :, i] = pair[..., 0], pair[..., 1]
    return c, s, m


def reference(case, out_dtype=torch.float32, tables=None, lens=None, gone=None):
    """The oracle's output and a bound on what the kernel's fp32 sums and its one
    fp16 rounding may leave, element by element.

    Scores: 64 exact products a run summed in fp32 by the MMA (at most a step,
    2^-23, of the sum of sizes for each of its 4 steps and each of 16 terms in
    one: 80 are allowed), then a handful of fp32 operations (8 half steps of
    the sizes of s A and m sum q; sum q itself 64 half steps).  An error dx of
    a score (natural log) moves out by at most 2 dx sum p |v - out|.
    Weights: w = p s' kappa rounded to fp16 (half a step, 2^-11), which weighs
    on s' |c' - 7.5|; exponentials to 2^-21.  Sums over n tokens in a warp:
    one step of 2^-23 of the sum of sizes (7.5 s' and c' s') for each MMA, n / 16
    of them at most, and as many for its 16 terms.
    Output: half a step of its type, 2^-20 for the merges.
    Tokens marked in `gone` are left out."""
    tables = case.tables if tables is None else tables
    lens = case.lens if lens is None else lens
    q = case.q.double().numpy()
    S, Hq, D = q.shape
    nb, B, G = case.k.shape[0], case.B, Hq // case.Hkv
    kc, ks, km = codes_of(case.k, D, case.dtype, False)
    vc, vs, vm = codes_of(case.v, D, case.dtype, True)
    out, tol = np.zeros((S, Hq, D)), np.zeros((S, Hq, D))
    for s in range(S):
        n = int(lens[s])
        ids = tables[s, :-(-n // B)].numpy()
        fine = (ids >= 0) & (ids < nb)
        seen, ids = np.repeat(fine, B)[:n], np.where(fine, ids, 0)
        if gone is not None:
            seen = seen & ~gone.numpy()
        if not seen.any():
            continue
        for h in range(Hq):
            g = h // G
            row = lambda x: x[ids, g].reshape(-1, D)[:n][seen]  # noqa: E731
            kcr, ksr, kmr, vcr, vsr, vmr = (row(x) for x in (kc, ks, km, vc, vs, vm))
            x = (kmr + kcr * ksr) @ q[s, h] * case.scale
            a = np.abs(q[s, h])
            dx = case.scale * (80 * 2.0 ** -23 * (ksr * kcr) @ a +
                               (8 * (ksr * kcr) @ a + 72 * np.abs(kmr) @ a) * 2.0 ** -24)
            dx = float(dx.max()) + 2.0 ** -21
            p = np.exp(x - x.max())
            p /= p.sum()
            v = vmr + vcr * vsr
            o = p @ v
            out[s, h] = o
            steps = (n / 16 + 16) * 2.0 ** -23
            tol[s, h] = 2.0 ** -11 * (p @ (vsr * np.abs(vcr - 7.5))) + \
                2 * dx * (p @ np.abs(v - o)) + steps * (p @ (vsr * (vcr + 7.5))) + \
                2.0 ** -20 * (p @ (np.abs(vmr) + 15 * vsr))
            tol[s, h] += np.abs(o) * torch.finfo(out_dtype).eps / 2 + \
                float(torch.finfo(out_dtype).smallest_normal) * torch.finfo(out_dtype).eps
    return out, tol


def check(case, out, out_dtype=torch.float32, status=0, **kw):
    want, tol = reference(case, out_dtype, **kw)
    got = out.double().numpy()
    assert np.isfinite(got).all()
    worst = np.abs(got - want) - tol
    assert (worst <= 0).all(), "off by %g where %g is allowed, at %s" % (
        np.abs(got - want).flat[worst.argmax()], tol.flat[worst.argmax()],
        np.unravel_index(worst.argmax(), worst.shape))
    assert pkv.device_status() == status


SMALL = [("bf16", 8, 1, 128, 16), ("bf16", 32, 4, 128, 16), ("bf16", 4, 4, 128, 32),
         ("f16", 8, 4, 128, 8), ("bf16", 4, 2, 64, 32), ("f16", 16, 4, 64, 16),
         ("f16", 6, 2, 128, 32), ("f16", 3, 3, 64, 8), ("bf16", 16, 1, 64, 8),
         ("f16", 12, 1, 128, 16), ("bf16", 34, 2, 128, 8), ("f16", 64, 1, 64, 16),
         ("bf16", 100, 1, 128, 32)]


@pytest.mark.parametrize("dt,Hq,Hkv,D,B", SMALL)
def test_ragged_contexts(dt, Hq, Hkv, D, B):
    case = Case(DT[dt], Hq, Hkv, D, B, RAGGED)
    check(case, case.run())
    check(case, case.run(plan=True))
    check(case, case.run(P=B))
    check(case, case.run(P=96))


@pytest.mark.parametrize("dt,Hq,Hkv,D,B,P", [("bf16", 8, 2, 128, 16, 256), ("f16", 16, 1, 64, 8, 64),
                                             ("bf16", 5, 1, 128, 32, 1024)])
def test_long_and_near_equal_contexts(dt, Hq, Hkv, D, B, P):
    """Pieces of near-equal contexts, up to 64 of them, and one long one."""
    check_all = [Case(DT[dt], Hq, Hkv, D, B, [2000, 2048, 1999, 2017], seed=1),
                 Case(DT[dt], Hq, Hkv, D, B, [9001], seed=2)]
    for case in check_all:
        check(case, case.run(P=P))
        check(case, case.run(plan=True))


@pytest.mark.parametrize("dt,Hq,Hkv,D,B,lens,P", [
    ("bf16", 8, 8, 128, 16, [2000, 2048, 1999, 2017], 32),  # near-equal: pieces
    ("f16", 16, 4, 64, 8, [2000, 2048, 1999, 2017], 32),
    ("bf16", 32, 2, 128, 32, [9001], 32),
    ("bf16", 8, 4, 128, 16, [3, 0, 700, 2040, 64, 1], 16),  # ragged: runs of their own number
    ("f16", 64, 8, 64, 8, [700, 5, 0, 300, 40] * 10, 16),  # and rows enough for a warp each
    ("bf16", 64, 8, 128, 16, [40, 900, 1, 0, 520] * 8, 32),
    ("f16", 16, 8, 64, 8, [1, 0, 60, 17] * 25, 0)])  # not split: the order alone
def test_work_plans(dt, Hq, Hkv, D, B, lens, P):
    """Launches of more CTAs than the GPU holds at once run by the plan's list."""
    case = Case(DT[dt], Hq, Hkv, D, B, lens, seed=4)
    check(case, case.run(P=P, plan=True))


def lengths_of(kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "ragged":
        return (torch.randn(300, generator=g).exp() * 150).int().clamp(0, 3000)
    if kind == "few long":
        return torch.cat([torch.tensor([3000, 2999, 1500]), torch.randint(0, 30, (60,), generator=g)])
    if kind == "equal and none":
        return torch.cat([torch.full((9,), 1800), torch.tensor([1700, 0, 0])])
    return torch.randint(200, 900, (20,), generator=g)  # "fewer than a warp"


@pytest.mark.parametrize("kind", ["ragged", "few long", "equal and none", "fewer than a warp"])
@pytest.mark.parametrize("P", [16, 64, 512])
def test_every_piece_of_a_plan_is_attended(kind, P):
    """Split calls against the call that is not split.  Values lie in [-4, 4], so
    scales are at most 8 / 15, and each of the two rounds its weights (2^-11) on at
    most 7.5 scales: 2e-3 each, and 1e-4 for the fp32 sums.  A piece left out moves
    the mean of a few thousand random values by more."""
    Hq, Hkv, D, B = 16, 8, 64, 8
    lens = lengths_of(kind, P).to(torch.int32)
    need = (lens + B - 1) // B
    S, nb, width = len(lens), int(need.sum()), int(need.max())
    g = torch.Generator().manual_seed(5)
    order = torch.randperm(nb, generator=g).int()
    tables = torch.full((S, width), -1, dtype=torch.int32)
    tables[torch.arange(width)[None] < need[:, None]] = order
    k = torch.zeros(pkv.q4_cache_shape(nb, Hkv, B, D), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    rows = [torch.randn(nb * B, Hkv, D, generator=g).clamp(-4, 4).half().to(DEV) for _ in range(2)]
    pkv.kv_write_q4(k, v, *rows, torch.arange(nb * B, device=DEV))
    q = torch.randn(S, Hq, D, generator=g).half().to(DEV)
    tables, lens, outs = tables.to(DEV), lens.to(DEV), []
    for split in (0, P):
        ws = torch.full((pkv.decode_workspace_bytes(S, Hq, D, width * B, split),), 0xFF,
                        dtype=torch.uint8, device=DEV)
        out = torch.full((S, Hq, D), float("nan"), device=DEV)
        pkv.paged_decode_attention_q4(out, q, k, v, tables, lens, 0.125, B, Hkv,
                                      partition_size=split, workspace=ws if split else None)
        outs.append(out)
    assert pkv.device_status() == 0
    assert float((outs[0] - outs[1]).abs().max()) <= 2 * 7.5 * 8 / 15 * 2 ** -11 + 1e-4


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_output_types_and_host_memory(dt, out):
    od = DT.get(out, torch.float32)
    case = Case(DT[dt], 8, 2, 128, 16, [5, 77, 0, 200])
    check(case, case.run(out_dtype=od), od)
    check(case, case.run(P=32, out_dtype=od), od)
    check(case, case.run(out_dtype=od, pin=True), od)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("rise", [30.0, -30.0])
def test_a_maximum_that_moves(P, rise):
    """Scores that climb (or fall) by tens over the context."""
    def key(k):
        n = k.shape[0]
        return k + torch.linspace(0, rise, n)[:, None, None]

    case = Case(torch.bfloat16, 4, 1, 128, 16, [700], k=key, q=lambda q: q.abs() * 0.3)
    check(case, case.run(P=P))


@pytest.mark.parametrize("dt,span", [("f16", 4), ("bf16", 20)])
@pytest.mark.parametrize("heavy_is", ["small", "large"])
@pytest.mark.parametrize("first", ["heavy", "light"])
def test_value_scales_of_very_different_sizes(dt, span, heavy_is, first):
    """Tokens that the softmax prefers hold values 10^span times smaller (or
    larger) than the others', and come first or last: the weights p s' span far
    more than fp16 does."""
    n, D = 200, 128
    heavy = torch.arange(n) < n // 2 if first == "heavy" else torch.arange(n) >= n // 2
    size = torch.where(heavy == (heavy_is == "large"), 10.0 ** (span / 2), 10.0 ** (-span / 2))
    case = Case(DT[dt], 8, 2, D, 16, [n], v=lambda v: v * size[:, None, None],
                k=lambda k: k * 0.1 + heavy[:, None, None] * 2.0, q=lambda q: 0.2 + q.abs() * 0.1)
    check(case, case.run())
    check(case, case.run(P=48))


def test_values_without_spread_and_without_size():
    """Runs of equal values (scale 0), all zero ones, and one token among them
    with a scale."""
    def value(v):
        v = torch.zeros_like(v) + 2.5
        v[:, :, 64:] = 0
        v[20, 0] = torch.linspace(-1, 1, 128)
        return v

    case = Case(torch.float16, 4, 1, 128, 8, [1, 40, 19], v=value)
    check(case, case.run())


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("P", [0, 32])
def test_values_without_spread_beside_unseen_ones(first, P):
    """The softmax rests on tokens whose values are constant (scale 0), and leaves
    nothing of tokens with scales: their p is 0 in fp32."""
    n, D = 96, 128
    heavy = torch.arange(n) < 20 if first else torch.arange(n) >= n - 20
    case = Case(torch.bfloat16, 8, 2, D, 16, [n], q=lambda q: 1.0 + q.abs(),
                k=lambda k: k * 0.1 + heavy[:, None, None] * 60.0,
                v=lambda v: torch.where(heavy[:, None, None], torch.full_like(v, 1.5), v * 1e4))
    check(case, case.run(P=P))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_queries_of_all_sizes(dt):
    """Zero, tiny and large queries, and single large elements in small ones."""
    def query(q):
        q[0] = 0
        q[1] *= 1e-4
        q[2] *= 100.0
        q[3, :, 5] = 3000.0
        q[4] = q[4] * 1e-3
        q[4, :, 64:] *= 1e3
        return q

    lens = [33, 50, 20, 64, 65]
    # large queries: small keys keep the scores' spread within what a double exp shows
    case = Case(DT[dt], 4, 2, 128, 16, lens, q=query, k=lambda k: k * 0.02)
    check(case, case.run())


@pytest.mark.parametrize("first", [True, False])
def test_scores_below_fp32(first):
    """Tokens whose scores overflow to minus infinity weigh nothing, whichever
    tokens a warp meets first; the rest are as if they were alone."""
    n, low = 300, 130
    gone = torch.arange(n) < low if first else torch.arange(n) >= n - low
    case = Case(torch.bfloat16, 8, 2, 128, 16, [n], q=lambda q: 1.0 + q.abs(),
                k=lambda k: torch.where(gone[:, None, None], torch.full_like(k, -3e37), k * 0.1))
    rest = Case(torch.bfloat16, 8, 2, 128, 16, [n], q=lambda q: 1.0 + q.abs(), k=lambda k: k * 0.1)
    assert torch.equal(rest.v, case.v)
    want, tol = reference(rest, gone=gone)
    for P in (0, 32):
        got = case.run(P=P).double().numpy()
        assert (np.abs(got - want) <= tol).all()


def test_bad_block_ids_hide_their_tokens():
    case = Case(torch.bfloat16, 8, 2, 64, 8, [64, 40, 24, 9])
    tables = case.tables.clone()
    tables[0, 3] = -7
    tables[1, 0] = 1 << 30
    tables[2, :3] = case.k.shape[0]  # all of it
    tables[3, 1] = -1
    for kw in (dict(), dict(P=16), dict(plan=True)):
        check(case, case.run(tables=tables, **kw), status=1, tables=tables)


def test_bad_lengths_count_as_empty():
    case = Case(torch.float16, 4, 1, 128, 16, [30, 16, 48])
    lens = torch.tensor([-3, 16, 49], dtype=torch.int32)
    for kw in (dict(), dict(P=16), dict(plan=True)):
        check(case, case.run(lens=lens, **kw), status=2,
              lens=torch.tensor([0, 16, 0], dtype=torch.int32))


def test_nan_in_the_context_shows():
    """A NaN scale of a seen key makes its row NaN, one of a value the run's
    64 elements; other rows and elements stay."""
    case = Case(torch.bfloat16, 4, 2, 128, 16, [40, 40])
    nan = torch.full((1, 2, 128), float("nan"), dtype=torch.bfloat16)
    k, v = case.k.clone(), case.v.clone()
    slot = int(case.tables[0, 1]) * 16 + 3
    q4.kv_write(case.k, case.v.clone(), nan, nan, torch.tensor([slot]))
    out = case.run()
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    case.k = k
    half = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    half[:, :, :64] = float("nan")
    q4.kv_write(k.clone(), v, half, half, torch.tensor([slot]))
    case.v = v
    for P in (0, 16):
        out = case.run(P=P)
        assert torch.isnan(out[0, :, :64]).all()
        assert torch.isfinite(out[0, :, 64:]).all() and torch.isfinite(out[1]).all()
    assert pkv.device_status() == 0


def test_repeated_calls_give_the_same_bits():
    case = Case(torch.bfloat16, 32, 4, 128, 16, [900, 30, 1111, 5])
    for kw in (dict(), dict(P=64), dict(plan=True)):
        a = case.run(**kw)
        for _ in range(4):
            assert torch.equal(case.run(**kw), a)


def test_pools_past_2_32_bytes():
    nb, Hkv, B, D = 1 << 16, 32, 32, 128
    small = Case(torch.bfloat16, 32, Hkv, D, B, [100], extra=0)
    k = torch.empty(pkv.q4_cache_shape(nb, Hkv, B, D), dtype=torch.uint8, device=DEV)
    v = torch.empty_like(k)
    tables = small.tables.clone()
    for j, id in enumerate([nb - 1, 3, nb // 2, nb - 2]):
        k[id], v[id] = small.k[tables[0, j]].to(DEV), small.v[tables[0, j]].to(DEV)
        tables[0, j] = id
    out = torch.empty(1, 32, D, device=DEV)
    pkv.paged_decode_attention_q4(out, small.q.to(DEV), k, v, tables.to(DEV), small.lens.to(DEV),
                                  small.scale, B, Hkv)
    check(small, out.cpu())


def test_batches_beyond_the_plan():
    """More sequences than the work plan holds: grid order, with and without a
    split."""
    S = 4100
    g = torch.Generator().manual_seed(9)
    case = Case(torch.float16, 2, 1, 64, 8, torch.randint(0, 20, (S,), generator=g).tolist())
    check(case, case.run(plan=True))
    check(case, case.run(P=8))


@pytest.mark.parametrize("P", [0, 32])
def test_a_serving_loop_in_one_graph(P):
    """extend, write and attend as one captured step, replayed: the tables, the
    slots and the cache follow from the previous replay alone."""
    dtype, S, Hq, Hkv, D, B, width, nb = torch.bfloat16, 6, 8, 2, 128, 16, 6, 40
    g = torch.Generator().manual_seed(3)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    tables = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
    lens, count, stack = i32([0] * S), i32([nb]), torch.randperm(nb, generator=g).int().to(DEV)
    k = torch.full(pkv.q4_cache_shape(nb, Hkv, B, D), 0xFF, dtype=torch.uint8, device=DEV)
    v = k.clone()
    tws = torch.empty(pkv.tables_workspace_bytes(S), dtype=torch.uint8, device=DEV)
    ws = torch.empty(pkv.decode_workspace_bytes(S, Hq, D, width * B, P), dtype=torch.uint8,
                     device=DEV)
    qs = torch.zeros(S + 1, dtype=torch.int32, device=DEV)

    def rows(T):
        return [torch.randn(T, Hkv, D, generator=g).to(dtype) for _ in range(2)]

    # the prompts, eagerly
    first = [0, 1, 15, 16, 17, 40]
    T = sum(first)
    slots = torch.zeros(T, dtype=torch.int64, device=DEV)
    pkv.tables_extend(tables, lens, i32(first), stack, count, B, qs, slots, None, tws)
    kv = rows(T)
    pkv.kv_write_q4(k, v, kv[0].to(DEV), kv[1].to(DEV), slots)
    hk, hv = torch.full(k.shape, 0xFF, dtype=torch.uint8), torch.full(k.shape, 0xFF, dtype=torch.uint8)
    q4.kv_write(hk, hv, *kv, slots.cpu())
    # one decode step, captured
    new, step_slots = i32([1] * S), torch.zeros(S + 2, dtype=torch.int64, device=DEV)
    nk, nv = (torch.zeros(S + 2, Hkv, D, dtype=dtype, device=DEV) for _ in range(2))
    q, out = torch.zeros(S, Hq, D, dtype=dtype, device=DEV), torch.zeros(S, Hq, D, device=DEV)

    def step():
        pkv.tables_extend(tables, lens, new, stack, count, B, qs, step_slots, None, tws)
        pkv.kv_write_q4(k, v, nk, nv, step_slots)
        pkv.paged_decode_attention_q4(out, q, k, v, tables, lens, 1 / math.sqrt(D), B, Hkv,
                                      partition_size=P, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(20):
        a, b = rows(S + 2)
        query = torch.randn(S, Hq, D, generator=g).to(dtype)
        nk.copy_(a), nv.copy_(b), q.copy_(query)
        if n % 3:
            graph.replay()
        else:
            step()
        assert lens.tolist() == [x + n + 1 for x in first]
        assert step_slots[S:].tolist() == [-1, -1]
        q4.kv_write(hk, hv, a[:S], b[:S], step_slots[:S].cpu())
        assert torch.equal(k.cpu(), hk) and torch.equal(v.cpu(), hv)
        case = Case(dtype, Hq, Hkv, D, B, [1])
        case.q, case.k, case.v, case.tables, case.lens = query, hk, hv, tables.cpu(), lens.cpu()
        check(case, out.cpu())


def test_other_streams():
    case = Case(torch.float16, 8, 2, 128, 16, [300, 20])
    want = case.run(P=32)
    side = torch.cuda.Stream()
    S, Hq, D = case.q.shape
    ws = torch.empty(pkv.decode_workspace_bytes(S, Hq, D, case.tables.shape[1] * 16, 32),
                     dtype=torch.uint8, device=DEV)
    args = [t.to(DEV) for t in (case.q, case.k, case.v, case.tables, case.lens)]
    out = torch.zeros(S, Hq, D, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pkv.paged_decode_attention_q4(out, *args, case.scale, 16, 2, partition_size=32, workspace=ws)
    side.synchronize()
    assert torch.equal(out.cpu(), want)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, beside each other."""
    cases = [Case(torch.bfloat16, 8, 2, 128, 16, [3000, 20], seed=1),
             Case(torch.bfloat16, 8, 2, 128, 16, [500, 2000, 1], seed=2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = [case.run(P=64) for case in cases]
    args, outs, work = [], [], []
    for case in cases:
        S, Hq, D = case.q.shape
        args.append([t.to(DEV) for t in (case.q, case.k, case.v, case.tables, case.lens)])
        outs.append([torch.zeros(S, Hq, D, device=DEV) for _ in range(20)])
        n = pkv.decode_workspace_bytes(S, Hq, D, case.tables.shape[1] * 16, 64)
        work.append(torch.empty(n, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    for i in range(20):
        for c in range(2):
            with torch.cuda.stream(streams[c]):
                pkv.paged_decode_attention_q4(outs[c][i], *args[c], cases[c].scale, 16, 2,
                                              partition_size=64, workspace=work[c])
    torch.cuda.synchronize()
    for c in range(2):
        assert all(torch.equal(o.cpu(), want[c]) for o in outs[c])


def test_an_empty_batch():
    k = torch.zeros(pkv.q4_cache_shape(4, 2, 16, 128), dtype=torch.uint8, device=DEV)
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    pkv.paged_decode_attention_q4(q.clone(), q, k, k.clone(),
                                  torch.zeros(0, 3, dtype=torch.int32, device=DEV),
                                  torch.zeros(0, dtype=torch.int32, device=DEV), 0.1, 16, 2)
    torch.cuda.synchronize()
    assert pkv.device_status() == 0

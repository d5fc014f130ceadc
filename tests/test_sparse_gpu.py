"""GPU: bounds of blocks, the selection by them and the attention over what is selected, against
the oracle.  Bounds, scores and selections must be equal; attention is within 2e-3 (16 bits) or
1e-5 (fp32), over a 4-bit cache as near as the dense call over the same tiles."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import sparse as oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


def tables(lens, block, spare=3, seed=0):
    """Tables over a shuffled pool, -1 behind the last block; (table, blocks of the pool)."""
    need = [-(-n // block) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), max(1, max(need)) + 2), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table, sum(need) + spare


def keys(nb, hkv, block, d, dtype, seed=1):
    """Keys with channels and blocks of very different sizes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(nb, hkv, block, d, generator=g)
    x = x * (2 * torch.randn(nb, hkv, 1, 1, generator=g)).exp() + torch.randn(hkv, 1, d, generator=g)
    return x.to(dtype)


def oracle_bounds(b, sc, kc, table, lens, new, most):
    b, sc = b.numpy().copy(), sc.double().numpy().copy()
    status = oracle.block_bounds(b, sc, kc.double().numpy(), table.tolist(), lens, new, most)
    return b, sc, status


# ---- bounds ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block,d,hkv", [(8, 64, 1), (16, 128, 3), (32, 128, 2), (32, 64, 5),
                                         (8, 128, 2), (16, 64, 4)])
def test_bounds_match_the_oracle(dtype, block, d, hkv):
    lens = [1, block, block + 1, 0, 5 * block - 1, 3 * block + 2, 77]
    new = [1, block, 2, 0, 5 * block - 1, 1, block + 3]
    table, nb = tables(lens, block)
    kc = keys(nb, hkv, block, d, dtype)
    for s, n in enumerate(lens):  # behind the context: never read
        if n % block:
            kc[table[s, n // block], :, n % block:] = math.nan
    g = torch.Generator().manual_seed(4)
    b = torch.randint(-128, 128, (nb, hkv, 2, d), generator=g).to(torch.int8)
    sc = torch.rand(nb, hkv, generator=g)
    want_b, want_sc, _ = oracle_bounds(b, sc, kc, table, lens, new, max(new))
    db, dsc = b.to(DEV), sc.to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pkv.block_bounds(db, dsc, kc.to(DEV), table.to(DEV), i32(lens), i32(new), max(new))
    assert pkv.device_status() == 0
    assert (db.cpu().numpy() == want_b).all() and (dsc.cpu().double().numpy() == want_sc).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_bounds_of_extreme_keys(dtype):
    """Zeros, whole powers (127 * 2^e is the last that fits a scale), subnormals, the type's ends,
    keys past 127 * 2^50, NaN and infinities of both signs, at a place that only one lane reads."""
    d, block, hkv = 64, 8, 1
    fin = torch.finfo(dtype)
    zero = torch.zeros(block, d, dtype=torch.float64)
    tiles = [zero]
    for value in (127.0, 127.5, 128.0, -127.0, 3.96875, 4.0, fin.max, -fin.max, fin.tiny,
                  -fin.tiny, fin.tiny / 4, 127 * 2.0 ** 50, 127.5 * 2.0 ** 50, -127 * 2.0 ** -50,
                  2.0 ** -51, math.nan, math.inf, -math.inf):
        for at in ((0, 0), (block - 1, d - 1)):
            tile = zero.clone()
            tile[at] = value
            tiles += [tile, tile + torch.where(tile == 0, 1.0, 0.0) * 2.0 ** -60]
    kc = torch.stack(tiles).to(dtype)[:, None]
    nb = len(tiles)
    table = torch.arange(nb, dtype=torch.int32)[None]
    b, sc = torch.full((nb, hkv, 2, d), 7, dtype=torch.int8), torch.zeros(nb, hkv)
    lens = [nb * block]
    want_b, want_sc, _ = oracle_bounds(b, sc, kc, table, lens, lens, lens[0])
    db, dsc = b.to(DEV), sc.to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pkv.block_bounds(db, dsc, kc.to(DEV), table.to(DEV), n, n, lens[0])
    assert (dsc.cpu().double().numpy() == want_sc).all()
    assert (db.cpu().numpy() == want_b).all()


def test_bounds_of_bad_lengths_and_blocks():
    block, d, hkv = 8, 64, 2
    lens = [20, 9, 17, 100000, 30, -4, 24]
    new = [3, 10, 17, 4, 9, 1, 24]  # 1: more than there are; 4: more than the most; 5: no length
    table, nb = tables([n if 0 <= n < 999 else 8 for n in lens], block)
    table[0, 2], table[6, 1], table[6, 2] = nb, -7, 2 ** 31 - 1
    kc = keys(nb, hkv, block, d, torch.float16)
    b, sc = torch.full((nb, hkv, 2, d), 7, dtype=torch.int8), torch.full((nb, hkv), 0.3)
    for most in (8, 24):
        want_b, want_sc, status = oracle_bounds(b, sc, kc, table, lens, new, most)
        db, dsc = b.to(DEV), sc.to(DEV)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        pkv.block_bounds(db, dsc, kc.to(DEV), table.to(DEV), i32(lens), i32(new), most)
        assert pkv.device_status() == status and status & 2
        assert (db.cpu().numpy() == want_b).all() and (dsc.cpu().numpy() == want_sc.astype(
            np.float32)).all()


@pytest.mark.parametrize("count,hkv,dtype,block,d", [
    (255, 8, torch.bfloat16, 8, 64), (256, 8, torch.float16, 16, 128), (1000, 3, torch.float32, 32, 64),
    (2500, 2, torch.bfloat16, 16, 64), (9000, 1, torch.float16, 8, 128)])
def test_bounds_of_prompts_among_decoding_sequences(count, hkv, dtype, block, d):
    """Calls of many possible tiles, of which most sequences have one: a few long prompts, bad
    lengths and sequences without new tokens among sequences of one new token, at odd places."""
    lens = [1 + s % 20 for s in range(count)]
    new = [1] * count
    for s, (n, fresh) in {0: (1000, 1000), 1: (17, 17), 9: (800, 790), 100: (900, 5),
                          101: (0, 0), 102: (5, 9), 103: (-3, 1), 104: (30, -1),
                          count - 2: (12, 0), count - 1: (1111, 1111)}.items():
        lens[s], new[s] = n, fresh
    table, nb = tables([max(n, 1) for n in lens], block)
    table[9, 800 // block - 1] = nb
    kc = keys(nb, hkv, block, d, dtype)
    b, sc = torch.full((nb, hkv, 2, d), 7, dtype=torch.int8), torch.full((nb, hkv), 0.25)
    want_b, want_sc, status = oracle_bounds(b, sc, kc, table, lens, new, max(new))
    db, dsc = b.to(DEV), sc.to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pkv.block_bounds(db, dsc, kc.to(DEV), table.to(DEV), i32(lens), i32(new), max(new))
    assert pkv.device_status() == status and status
    assert (db.cpu().numpy() == want_b).all() and (dsc.cpu().double().numpy() == want_sc).all()


def test_bounds_in_a_graph_whose_lengths_change():
    """One captured call of a step's largest size: replays with a prompt, with decoding steps and
    with nothing to do, each over what the replay before it left."""
    block, d, hkv, most = 16, 64, 4, 640
    table, nb = tables([most] * 100, block)
    kc = keys(nb, hkv, block, d, torch.bfloat16)
    b, sc = torch.full((nb, hkv, 2, d), 7, dtype=torch.int8), torch.full((nb, hkv), 0.25)
    db, dsc, dkc, dtable = b.to(DEV), sc.to(DEV), kc.to(DEV), table.to(DEV)
    dl = torch.zeros(100, dtype=torch.int32, device=DEV)
    dn = torch.zeros(100, dtype=torch.int32, device=DEV)
    pkv.block_bounds(db, dsc, dkc, dtable, dl, dn, most)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.block_bounds(db, dsc, dkc, dtable, dl, dn, most)
    for lens, new in (([0] * 100, [0] * 100),
                      ([s + 1 for s in range(100)], [1] * 100),
                      ([640] + [200 + s for s in range(99)], [640] + [1, 0, 33] * 33),
                      ([640] * 100, [640 - 6 * s for s in range(100)])):
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        dn.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        b, sc, _ = oracle_bounds(b, sc, kc, table, lens, new, most)
        b, sc = torch.from_numpy(b), torch.from_numpy(sc).float()
        assert torch.equal(db.cpu(), b) and torch.equal(dsc.cpu(), sc)
    assert pkv.device_status() == 0


# ---- selection -------------------------------------------------------------------------------

def run_select(q, b, sc, table, lens, block, k, first=1, recent=1, stream=None):
    S, hkv, width = q.shape[0], b.shape[1], table.shape[1]
    sel = torch.full((S, hkv, k), 99, dtype=torch.int32, device=DEV)
    slens = torch.full((S, hkv), 99, dtype=torch.int32, device=DEV)
    scores = torch.full((S, hkv, width), 0.5, device=DEV)
    pkv.select_blocks(sel, slens, scores, q.to(DEV), b.to(DEV), sc.to(DEV), table.to(DEV),
                      torch.as_tensor(lens, dtype=torch.int32).to(DEV), block, first, recent,
                      stream=stream)
    return sel, slens, scores


def check_select(q, b, sc, table, lens, block, k, first=1, recent=1):
    """Against the oracle; a narrow table, as one kernel takes it, and the same in wide tables,
    which go to others."""
    sel, slens, scores = run_select(q, b, sc, table, lens, block, k, first, recent)
    want = oracle.select(q.double().numpy(), b.numpy(), sc.double().numpy(), table.tolist(), lens,
                         block, k, first, recent, np.full(scores.shape, 0.5))
    assert (scores.cpu().double().numpy() == want[2]).all()
    assert (slens.cpu().numpy() == want[1]).all()
    assert (sel.cpu().numpy() == want[0]).all()
    assert pkv.device_status() == want[3]
    columns = table.shape[1]
    for width in (520, 9000) if columns <= 512 and max(lens) <= columns * block else ():
        wide = torch.nn.functional.pad(table, (0, width - columns), value=-1)
        again = run_select(q, b, sc, wide, lens, block, k, first, recent)
        assert pkv.device_status() == want[3]
        assert torch.equal(again[0], sel) and torch.equal(again[1], slens)
        assert torch.equal(again[2][:, :, :columns], scores)
        assert bool((again[2][:, :, columns:] == 0.5).all())
    return sel, slens


def bound_set(nb, hkv, d, seed=0, spread=2):
    g = torch.Generator().manual_seed(seed)
    hi = torch.randint(-40, 128, (nb, hkv, d), generator=g)
    lo = hi - torch.randint(0, 90, (nb, hkv, d), generator=g)
    b = torch.stack([hi, lo.clamp(min=-127)], 2).to(torch.int8)
    sc = 2.0 ** torch.randint(-5 - spread, -4 + spread, (nb, hkv), generator=g).float()
    return b, sc


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d,block,k,first,recent", [
    (1, 1, 64, 8, 1, 0, 1), (8, 2, 128, 16, 5, 1, 1), (3, 3, 64, 32, 2, 1, 1),
    (16, 1, 128, 8, 40, 2, 3), (14, 2, 64, 16, 33, 0, 32), (128, 1, 128, 32, 17, 1, 2),
    (20, 4, 128, 16, 300, 4, 4), (12, 4, 64, 8, 64, 63, 1)])
def test_selection_matches_the_oracle(dtype, hq, hkv, d, block, k, first, recent):
    lens = [0, 1, block * k, block * k + 1, block * (k + 7) - 3, block * 350, 299 * block + 1]
    table, nb = tables(lens, block)
    b, sc = bound_set(nb, hkv, d)
    q = torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(k)).to(dtype)
    check_select(q, b, sc, table, lens, block, k, first, recent)


@pytest.mark.parametrize("n,k", [(5000, 64), (5000, 4999), (70000, 1000), (257, 256), (2, 1)])
def test_selection_over_long_contexts(n, k):
    block, d = 8, 64
    lens = [n * block - 5]
    table, nb = tables(lens, block)
    b, sc = bound_set(nb, 1, d, spread=0 if n == 70000 else 2)
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(n)).bfloat16()
    check_select(q, b, sc, table, lens, block, k, 0, 1)


@pytest.mark.parametrize("width", [512, 513, 1024, 1025, 2048, 2049, 8191, 8192, 8193])
def test_selection_at_the_widths_where_the_kernel_changes(width):
    """As many blocks as the table is wide, one fewer, and about half."""
    block, d, hkv = 8, 64, 2
    lens = [width * block, (width - 1) * block, width * 4 + 3]
    g = torch.Generator().manual_seed(width)
    nb = 700
    table = torch.randint(0, nb, (3, width), generator=g, dtype=torch.int32)  # blocks repeat
    b, sc = bound_set(nb, hkv, d)
    q = torch.randn(3, 6, d, generator=g).bfloat16()
    for k in (40, width - 1, width):
        check_select(q, b, sc, table, lens, block, k)


@pytest.mark.parametrize("rows,width", [(20, 2100), (160, 2100), (160, 9000)])
def test_selection_of_many_rows_of_wide_tables(rows, width):
    """Few rows and many (two KV heads each), contexts short and long in wide tables: what a CTA
    holds, and what it reads again."""
    block, d, hkv, k = 8, 64, 2, 50
    g = torch.Generator().manual_seed(rows)
    lens = [int(x) for x in torch.randint(0, 120 * block, (rows,), generator=g)]
    lens[1], lens[rows // 2], lens[-1] = width * block, 2049 * block, 2048 * block - 3
    table = torch.randint(0, 900, (rows, width), generator=g, dtype=torch.int32)
    b, sc = bound_set(900, hkv, d)
    q = torch.randn(rows, 4, d, generator=g).half()
    check_select(q, b, sc, table, lens, block, k)


@pytest.mark.parametrize("kinds", [1, 2, 3, 40])
def test_equal_scores_take_the_lowest_blocks(kinds):
    """A context whose blocks have a handful of different bounds: almost all scores are equal."""
    block, d, hkv = 16, 64, 2
    lens = [400 * block, 401 * block - 1, 37 * block]
    table, nb = tables(lens, block)
    few, fsc = bound_set(kinds, hkv, d, 5)
    pick = torch.randint(0, kinds, (nb,), generator=torch.Generator().manual_seed(2))
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(3)).half()
    for k in (3, 32, 200, 399):
        check_select(q, few[pick], fsc[pick], table, lens, block, k)


@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_sums_are_exact(d):
    """Bounds and query elements at their ends, +-127 and their neighbours: sums of up to
    128 * 255 * 127 on the way, whose last digits tell blocks apart."""
    block, hkv = 8, 2
    lens = [120 * block, 77 * block]
    table, nb = tables(lens, block)
    g = torch.Generator().manual_seed(d)
    ends = lambda *n: (torch.randint(0, 2, n, generator=g) * 2 - 1) * (  # noqa: E731
        127 - (torch.rand(*n, generator=g) < 0.02).long())
    b, sc = ends(nb, hkv, 2, d).to(torch.int8), torch.ones(nb, hkv)
    b[::3] = 127 - (torch.rand(b[::3].shape, generator=g) < 0.02).to(torch.int8)
    q = torch.where(torch.rand(2, 8, 1, generator=g) < 0.5, 127.0, ends(2, 8, d).float())
    check_select(q, b, sc, table, lens, block, 9)
    check_select(q.half(), b, sc, table, lens, block, 40)


def test_queries_and_bounds_of_extreme_values():
    """Query rows of zeros, halves (rounded up), one large element, NaN, infinities, the type's
    ends; bounds of all scales, infinite ones among them and more of those than are picked."""
    block, d, hkv = 8, 64, 1
    g = torch.Generator().manual_seed(7)
    q = torch.randn(12, 2, d, generator=g)
    q[0] = 0
    q[1] = (torch.arange(128).view(2, d) % 19 - 9) / 2 + 0.0
    q[1, :, 0] = 127
    q[2, :, 5] = 1e30
    q[3, 0, 7] = math.nan
    q[4, 0, 9] = math.inf
    q[5, 1, 9] = -math.inf
    q[6] *= 1e-38
    q[7] *= 1e-20
    q[8] = torch.finfo(torch.float32).max * q[8].sign()
    q[9, 0] = math.nan
    q[10, :, 1:] = 2.0 ** -26 - 0.5
    q[10, :, 0] = 127
    q[11, :, 1:] = 0.5 - 2.0 ** -25
    q[11, :, 0] = -127
    lens = [60 * block] * 12
    table, nb = tables(lens, block)
    b, sc = bound_set(nb, hkv, d, 3, 45)
    sc[::9] = math.inf
    b[::9] = 0
    check_select(q, b, sc, table, lens, block, 10)
    check_select(q, b, sc, table, lens, block, 4, 2, 2)
    check_select(q.bfloat16(), b, sc, table, lens, block, 10)


def test_scales_that_are_none_count_as_infinite():
    """Bounds that were never written: any bits as scales.  Every row stays in its place."""
    block, d, hkv = 8, 64, 1
    lens = [50 * block] * 2
    table, nb = tables(lens, block)
    b, sc = bound_set(nb, hkv, d)
    odd = torch.tensor([math.nan, -math.nan, -1.0, -math.inf, math.inf, -1e-40])
    sc[::4, 0] = odd[torch.arange(len(sc[::4])) % 6]
    q = torch.randn(2, 4, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    q[0] = 0
    fine = torch.where((sc >= 0) & (sc < math.inf), sc, math.inf)
    for k in (5, 20, 49):
        got = run_select(q, b, sc, table, lens, block, k)
        want = run_select(q, b, fine, table, lens, block, k)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    check_select(q, b, fine, table, lens, block, 20)


def test_selection_with_bad_blocks_and_lengths():
    block, d, hkv = 16, 128, 2
    lens = [20 * block, 33 * block, 9 * block, -3, 10 ** 6, 30 * block + 1]
    table, nb = tables([n if 0 <= n < 9999 else 16 for n in lens], block)
    table[0, 3], table[1, 0], table[1, 32], table[2, 4], table[5, 7] = -1, nb, -9, 2 ** 30, nb + 5
    b, sc = bound_set(nb, hkv, d)
    q = torch.randn(6, 4, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    for k in (4, 12, 19, 32):
        check_select(q, b, sc, table, lens, block, k)


# ---- attention -------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d,block,k,partition,plan", [
    (1, 1, 64, 8, 3, 0, False), (8, 2, 128, 16, 9, 0, True), (32, 4, 128, 32, 12, 64, True),
    (6, 6, 64, 16, 40, 160, True), (32, 1, 128, 16, 5, 0, True), (40, 2, 64, 32, 7, 0, False)])
def test_attention_matches_the_oracle(dtype, hq, hkv, d, block, k, partition, plan):
    lens = [0, 1, block * k, block * (k + 9) - 3, block * 60 + 1]
    S = len(lens)
    table, nb = tables(lens, block)
    kc, vc = (torch.randn(nb, hkv, block, d, generator=torch.Generator().manual_seed(i)).to(dtype)
              for i in (1, 2))
    for s, n in enumerate(lens):
        if n % block:
            kc[table[s, n // block], :, n % block:] = math.nan
            vc[table[s, n // block], :, n % block:] = math.nan
    q = torch.randn(S, hq, d, generator=torch.Generator().manual_seed(3)).to(dtype)
    b, sc = torch.zeros(nb, hkv, 2, d, dtype=torch.int8), torch.zeros(nb, hkv)
    b, sc, _ = oracle_bounds(b, sc, kc, table, lens, lens, max(lens))
    sel, slens = check_select(q, torch.from_numpy(b), torch.from_numpy(sc).float(), table, lens,
                              block, k)
    ws = None
    if plan:
        ws = torch.empty(pkv.decode_workspace_bytes(S, hq, d, k * block, partition),
                         dtype=torch.uint8, device=DEV)
    out = torch.full((S, hq, d), 9.0, device=DEV)
    pkv.paged_decode_attention_selected(out, q.to(DEV), kc.to(DEV), vc.to(DEV), sel, slens, 0.11,
                                        block, hkv, partition, ws)
    want = oracle.attention(q.double().numpy(), np.nan_to_num(kc.double().numpy()),
                            np.nan_to_num(vc.double().numpy()), sel.tolist(), slens.tolist(), 0.11)
    off = np.abs(out.cpu().double().numpy() - want).max()
    assert off <= (1e-5 if dtype is torch.float32 else 2e-3), off
    assert (out[0] == 0).all() and pkv.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,d,block,k", [
    (1, 1, 64, 8, 1024), (8, 1, 128, 8, 1025), (7, 7, 128, 16, 100), (32, 4, 64, 32, 50),
    (40, 8, 128, 32, 17), (15, 15, 128, 16, 256), (24, 8, 64, 8, 333), (9, 1, 128, 16, 60),
    (32, 16, 64, 16, 60)])
def test_attention_split_over_few_sequences(dtype, hq, hkv, d, block, k):
    """A split asked for: clusters of eight CTAs, of four, and (nine query heads a KV head, or many
    tokens) the split with a plan.  Lengths from none to all, tiles in any order, some not there;
    what lies behind a context and in the tiles left out is NaN."""
    S, nb = 5, 60
    g = torch.Generator().manual_seed(hq * k)
    kc, vc = (torch.randn(nb, hkv, block, d, generator=g).to(dtype) for _ in range(2))
    kc[nb - 1] = vc[nb - 1] = math.nan
    sel = torch.randint(0, nb - 2, (S, hkv, k), generator=g, dtype=torch.int32) * hkv
    sel = sel + torch.arange(hkv, dtype=torch.int32)[None, :, None]
    lens = torch.randint(1, k * block, (S, hkv), generator=g, dtype=torch.int32)
    lens[0], lens[1, 0], lens[2], lens[3, -1] = 0, 1, k * block, 16 * (k * block // 16)
    for s in range(S):
        for h in range(hkv):
            n = int(lens[s, h])
            if n % block:  # a last tile of its own
                sel[s, h, n // block] = (nb - 2) * hkv + h
            sel[s, h, -(-n // block):] = (nb - 1) * hkv + h
    # the partial last tiles share a block: the least length's end decides what is read
    for h in range(hkv):
        most = max(int(lens[s, h]) % block for s in range(S))
        kc[nb - 2, h, most:] = vc[nb - 2, h, most:] = math.nan
    q = torch.randn(S, hq, d, generator=g).to(dtype)
    ws = torch.empty(pkv.decode_workspace_bytes(S, hq, d, k * block, 64), dtype=torch.uint8,
                     device=DEV)
    outs = []
    for bad in (False, True):
        tiles = sel.clone()
        if bad:  # of sequence 4: its first two, and one past the pool
            tiles[4, :, 0], tiles[4, 0, 1] = -1, nb * hkv
        for _ in range(2):
            out = torch.full((S, hq, d), 9.0, device=DEV)
            pkv.paged_decode_attention_selected(out, q.to(DEV), kc.to(DEV), vc.to(DEV),
                                                tiles.to(DEV), lens.to(DEV), 0.11, block, hkv, 64,
                                                ws)
            outs.append(out.cpu())
        assert torch.equal(outs[-1], outs[-2])
        assert pkv.device_status() == (1 if bad else 0)
        want = oracle.attention(q.double().numpy(), np.nan_to_num(kc.double().numpy()),
                                np.nan_to_num(vc.double().numpy()), tiles.tolist(), lens.tolist(),
                                0.11)
        off = np.abs(outs[-1].double().numpy() - want).max()
        # scores of 128 products: 128 * 2^-23 * 90 * 0.11, weights 2^-18, twice, values below 6
        assert off <= 2e-3, off
    assert (outs[0][0] == 0).all()
    lens[1], lens[3] = -1, k * block + 1  # bad lengths count as none
    out = torch.full((S, hq, d), 9.0, device=DEV, dtype=dtype)
    pkv.paged_decode_attention_selected(out, q.to(DEV), kc.to(DEV), vc.to(DEV), sel.to(DEV),
                                        lens.to(DEV), 0.11, block, hkv, 64, ws)
    assert pkv.device_status() == 2
    assert (out[1] == 0).all() and (out[3] == 0).all()


def test_attention_over_all_blocks_is_the_dense_call():
    """Every block selected: the same kernel on the same tokens, bit for bit where a sequence has
    one KV head."""
    hq, d, block, lens = 8, 128, 16, [700, 33, 1]
    table, nb = tables(lens, block)
    for hkv, exact in ((1, True), (4, False)):
        kc, vc = (torch.randn(nb, hkv, block, d, device=DEV).bfloat16() for _ in range(2))
        q = torch.randn(3, hq, d, device=DEV).bfloat16()
        b, sc = bound_set(nb, hkv, d)
        sel, slens, _ = run_select(q, b, sc, table, lens, block, table.shape[1])
        a, c = torch.empty(3, hq, d, device=DEV), torch.empty(3, hq, d, device=DEV)
        pkv.paged_decode_attention_selected(a, q, kc, vc, sel, slens, 0.1, block, hkv)
        pkv.paged_decode_attention(c, q, kc, vc, table.to(DEV),
                                   torch.tensor(lens, dtype=torch.int32, device=DEV), 0.1, block,
                                   hkv)
        assert float((a - c).abs().max()) <= (0.0 if exact else 2e-6)


def test_attention_with_tiles_that_are_not_there():
    hq, hkv, d, block, nb = 4, 2, 64, 8, 10
    kc, vc = (torch.randn(nb, hkv, block, d, generator=torch.Generator().manual_seed(i)).half()
              for i in (1, 2))
    q = torch.randn(2, hq, d, generator=torch.Generator().manual_seed(3)).half()
    sel = torch.tensor([[[0, 4, -1], [3, 2 ** 30, 7]], [[19, -1, -1], [nb * hkv, 1, -1]]],
                       dtype=torch.int32)
    slens = torch.tensor([[24, 19], [8, 13]], dtype=torch.int32)
    out = torch.empty(2, hq, d, device=DEV)
    pkv.paged_decode_attention_selected(out, q.to(DEV), kc.to(DEV), vc.to(DEV), sel.to(DEV),
                                        slens.to(DEV), 0.2, block, hkv)
    want = oracle.attention(q.double().numpy(), kc.double().numpy(), vc.double().numpy(),
                            sel.tolist(), slens.tolist(), 0.2)
    assert np.abs(out.cpu().numpy() - want).max() <= 2e-3 and pkv.device_status() == 1


def test_attention_with_queries_and_output_in_pinned_host_memory():
    hq, hkv, d, block, k, lens = 16, 2, 128, 16, 5, [200, 40, 16]
    table, nb = tables(lens, block)
    kc, vc = (torch.randn(nb, hkv, block, d, device=DEV).bfloat16() for _ in range(2))
    b, sc = bound_set(nb, hkv, d)
    q = torch.randn(3, hq, d).bfloat16()
    sel, slens, _ = run_select(q, b, sc, table, lens, block, k)
    outs = [torch.zeros(3, hq, d, device=DEV), torch.zeros(3, hq, d).pin_memory()]
    for out, queries in zip(outs, (q.to(DEV), q.pin_memory())):
        pkv.paged_decode_attention_selected(out, queries, kc, vc, sel, slens, 0.1, block, hkv)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].cpu(), outs[1]) and float(outs[1].abs().max()) > 0.1
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_selected(outs[0], q, kc, vc, sel, slens, 0.1, block, hkv)


def test_a_split_over_few_sequences_with_pinned_and_unaligned_rows():
    """Queries and output in pinned host memory, four bytes off 16."""
    hq, hkv, d, block, k, nb = 8, 2, 64, 8, 30, 64
    g = torch.Generator().manual_seed(5)
    kc, vc = (torch.randn(nb, hkv, block, d, generator=g).half() for _ in range(2))
    sel = torch.randint(0, nb, (2, hkv, k), generator=g, dtype=torch.int32) * hkv
    sel += torch.arange(hkv, dtype=torch.int32)[None, :, None]
    lens = torch.tensor([[k * block, 77], [5, 200]], dtype=torch.int32)
    ws = torch.empty(pkv.decode_workspace_bytes(2, hq, d, k * block, 32), dtype=torch.uint8,
                     device=DEV)
    rows = torch.empty(2 * hq * d + 2, dtype=torch.float16).pin_memory()
    out = torch.full((2 * hq * d + 2,), 9.0).pin_memory()
    q = rows[2:].view(2, hq, d)
    q.copy_(torch.randn(2, hq, d, generator=g))
    pkv.paged_decode_attention_selected(out[1:-1].view(2, hq, d), q, kc.to(DEV), vc.to(DEV),
                                        sel.to(DEV), lens.to(DEV), 0.15, block, hkv, 32, ws)
    torch.cuda.synchronize()
    want = oracle.attention(q.double().numpy(), kc.double().numpy(), vc.double().numpy(),
                            sel.tolist(), lens.tolist(), 0.15)
    assert np.abs(out[1:-1].view(2, hq, d).double().numpy() - want).max() <= 2e-3
    assert float(out[0]) == 9.0 and float(out[-1]) == 9.0 and pkv.device_status() == 0


def test_pools_past_2_31_elements():
    """Blocks whose keys start beyond 2^31 elements (4.3 GB), bounds beyond 2^31 bytes (2.3 GB)."""
    nb, hkv, block, d = (1 << 17) + 8, 8, 16, 128
    kc = torch.empty(nb, hkv, block, d, dtype=torch.bfloat16, device=DEV)
    ids = [nb - 1, 3, nb - 2, nb // 2]
    small = torch.randn(4, hkv, block, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    kc[ids] = small.to(DEV)
    b = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device=DEV)
    sc = torch.zeros(nb, hkv, device=DEV)
    n = torch.tensor([4 * block - 3], dtype=torch.int32, device=DEV)
    pkv.block_bounds(b, sc, kc, torch.tensor([ids], dtype=torch.int32, device=DEV), n, n, 64)
    want_b, want_sc, _ = oracle_bounds(torch.zeros(4, hkv, 2, d, dtype=torch.int8),
                                       torch.zeros(4, hkv), small, torch.arange(4)[None],
                                       [4 * block - 3], [4 * block - 3], 64)
    assert (b[ids].cpu().numpy() == want_b).all() and (sc[ids].cpu().numpy() == want_sc).all()
    del kc, b, sc
    nb, block = 1_100_000, 8
    b = torch.empty(nb, hkv, 2, d, dtype=torch.int8, device=DEV)
    sc = torch.empty(nb, hkv, device=DEV)
    few, fsc = bound_set(40, hkv, d)
    ids = torch.randint(nb - 200_000, nb, (40,), generator=torch.Generator().manual_seed(2))
    b[ids], sc[ids] = few.to(DEV), fsc.to(DEV)
    table, lens = ids[None].to(torch.int32), [40 * block - 1]
    q = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    sel, slens, scores = run_select(q, b, sc, table, lens, block, 9)
    order = {int(x): i for i, x in enumerate(ids.tolist())}
    got = [[order[t // hkv] for t in row] for row in sel[0].tolist()]
    want = oracle.select(q.double().numpy(), few.numpy(), fsc.double().numpy(),
                         [list(range(40))], lens, block, 9)
    assert got == [[t // hkv for t in row] for row in want[0][0].tolist()]
    assert (scores.cpu().double().numpy() == want[2]).all()


@pytest.mark.parametrize("dtype,partition", [(torch.bfloat16, 0), (torch.float16, 96)])
def test_attention_over_a_4_bit_cache(dtype, partition):
    """As the 4-bit call over a pool that holds the selected tiles of one (sequence, head)."""
    hq, hkv, d, block, k = 8, 2, 128, 16, 6
    lens = [500, 95, 0, 301]
    table, nb = tables(lens, block)
    g = torch.Generator().manual_seed(5)
    rows = [torch.randn(nb * block, hkv, d, generator=g).to(dtype).to(DEV) for _ in range(2)]
    kp, vp = (torch.zeros(pkv.q4_cache_shape(nb, hkv, block, d), dtype=torch.uint8, device=DEV)
              for _ in range(2))
    pkv.kv_write_q4(kp, vp, *rows, torch.arange(nb * block, device=DEV))
    b, sc = bound_set(nb, hkv, d)
    q = torch.randn(4, hq, d, generator=g).to(dtype)
    sel, slens, _ = run_select(q, b, sc, table, lens, block, k)
    ws = torch.empty(pkv.decode_workspace_bytes(4, hq, d, k * block, partition), dtype=torch.uint8,
                     device=DEV)
    out = torch.empty(4, hq, d, device=DEV)
    pkv.paged_decode_attention_selected(out, q.to(DEV), kp, vp, sel, slens, 0.1, block, hkv,
                                        partition, ws)
    group = hq // hkv
    for s in range(4):
        for h in range(hkv):
            ids = sel[s, h].clamp(min=0).long()
            one = torch.empty(1, group, d, device=DEV)
            pkv.paged_decode_attention_q4(
                one, q[s:s + 1, h * group:(h + 1) * group].contiguous().to(DEV),
                kp.view(nb * hkv, 1, block, -1)[ids].contiguous(),
                vp.view(nb * hkv, 1, block, -1)[ids].contiguous(),
                torch.arange(k, dtype=torch.int32, device=DEV)[None], slens[s, h:h + 1], 0.1,
                block, 1)
            # two ways of cutting the same sums: the weights' fp16 rounding against references
            # that differ by at most 2^8, 2^-11 of values below 8 each
            assert float((out[s, h * group:(h + 1) * group] - one[0]).abs().max()) <= 8 * 2.0 ** -10
    assert pkv.device_status() == 0


# ---- a step, as it is used -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_decode_loop_in_one_graph(dtype):
    """Extend, rotate and write, bounds, selection, attention: captured once, replayed for each
    token, against the oracle on the cache as it stands."""
    S, hq, hkv, d, block, k, width = 5, 8, 2, 64, 8, 6, 20
    nb, steps = 100, 20
    start = [70, 1, 33, 0, 128]
    gen = torch.Generator(DEV).manual_seed(0)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)  # noqa: E731
    table, lens, count = i32(S, width).fill_(-1), i32(S), i32(1).fill_(nb)
    stack = torch.arange(nb, dtype=torch.int32, device=DEV)
    ws = torch.empty(pkv.tables_workspace_bytes(S), dtype=torch.uint8, device=DEV)
    kc, vc = (torch.full((nb, hkv, block, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    b, sc = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device=DEV), torch.zeros(nb, hkv, device=DEV)
    turns = pkv.rope_turns([10000.0 ** (-i / 32) for i in range(32)], DEV)
    sel, slens = i32(S, hkv, k), i32(S, hkv)
    scores, out = torch.zeros(S, hkv, width, device=DEV), torch.zeros(S, hq, d, device=DEV)

    def step(new, rows, most, qs, slots, pos, x, q_rot):
        q, key, value = x.split([hq, hkv, hkv], 1)
        pkv.tables_extend(table, lens, new, stack, count, block, qs, slots, pos, ws)
        pkv.rope_write(q_rot, kc, vc, q, key, value, pos, turns, slots)
        pkv.block_bounds(b, sc, kc, table, lens, new, most)

    def attend(q_rot):
        pkv.select_blocks(sel, slens, scores, q_rot, b, sc, table, lens, block)
        pkv.paged_decode_attention_selected(out, q_rot, kc, vc, sel, slens, 0.125, block, hkv)

    def rows_of(n):
        return (i32(S + 1), torch.zeros(n, dtype=torch.int64, device=DEV), i32(n),
                torch.randn(n, hq + 2 * hkv, d, generator=gen, device=DEV).to(dtype),
                torch.zeros(n, hq, d, dtype=dtype, device=DEV))

    prompt = torch.tensor(start, dtype=torch.int32, device=DEV)
    step(prompt, 0, max(start), *rows_of(sum(start)))
    one, fixed = i32(S).fill_(1), rows_of(S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one, S, 1, *fixed)
        attend(fixed[4])
    for n in range(steps):
        fixed[3].copy_(torch.randn(fixed[3].shape, generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert pkv.device_status() == 0 and lens.tolist() == [x + n + 1 for x in start]
        hk, hv = kc.cpu().double().numpy(), vc.cpu().double().numpy()
        tb, ln = table.tolist(), lens.tolist()
        hb, hsc = np.zeros(b.shape, np.int8), np.zeros(sc.shape)
        assert oracle.block_bounds(hb, hsc, hk, tb, ln, ln, max(ln)) == 0
        used = hsc > 0
        assert (b.cpu().numpy()[used] == hb[used]).all()
        assert (sc.cpu().double().numpy()[used] == hsc[used]).all()
        q = fixed[4].cpu().double().numpy()
        w_sel, w_lens, _, _ = oracle.select(q, hb, hsc, tb, ln, block, k)
        assert (sel.cpu().numpy() == w_sel).all() and (slens.cpu().numpy() == w_lens).all()
        want = oracle.attention(q, np.nan_to_num(hk), np.nan_to_num(hv), w_sel, w_lens, 0.125)
        off = np.abs(out.cpu().double().numpy() - want).max()
        assert off <= (1e-5 if dtype is torch.float32 else 2e-3), off


def test_other_streams_and_repeats_give_the_same():
    block, d, hkv, k = 16, 128, 4, 20
    lens = [3000, 1700, 5, 4096]
    table, nb = tables(lens, block)
    b, sc = bound_set(nb, hkv, d)
    q = torch.randn(4, 32, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    first = run_select(q, b, sc, table, lens, block, k)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    many = []
    for i in range(6):
        with torch.cuda.stream(side[i % 2]):
            many.append(run_select(q, b, sc, table, lens, block, k))
    torch.cuda.synchronize()
    for got in many:
        assert all(torch.equal(x, y) for x, y in zip(first, got))
    with pytest.raises(ValueError):
        other = torch.empty(1, dtype=torch.int32)
        pkv.select_blocks(first[0], first[1], first[2], q.to(DEV), b.to(DEV), sc.to(DEV),
                          table.to(DEV), other.expand(4).contiguous(), block)


def test_no_sequences_and_no_tokens():
    b, sc = torch.zeros(4, 2, 2, 64, dtype=torch.int8, device=DEV), torch.zeros(4, 2, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    table = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    kc = torch.zeros(4, 2, 8, 64, dtype=torch.float16, device=DEV)
    pkv.block_bounds(b, sc, kc, table, none, none, 5)
    q = torch.zeros(0, 4, 64, dtype=torch.float16, device=DEV)
    sel, slens = none.view(0, 2, 0).new_zeros(0, 2, 3), none.new_zeros(0, 2)
    pkv.select_blocks(sel, slens, torch.zeros(0, 2, 3, device=DEV), q, b, sc, table, none, 8)
    pkv.paged_decode_attention_selected(q.clone(), q, kc, kc, sel, slens, 0.1, 8, 2)

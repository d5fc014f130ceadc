"""GPU: attention directly behind an extend or a release of the block tables, with
no other kernel and no wait of the host between them: it sees the lengths and
tables that those wrote.

Each step's output is kept, with a copy of the lengths and tables that the step
ended with; once all is done the same attention over those copies has to give the
same bits.  Lengths and tables are the oracle's, number for number, and a few
outputs are the attention oracle's within 2e-3 (unit normals; weights are rounded
once to 16 bits)."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_312_gb300 as pkv
from oracle import q4
from oracle import tables as table_oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D, B = 64, 8


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Batch:
    """S sequences with blocks of a full cache, all of whose slots hold unit normals."""

    def __init__(self, kind, S, width, seed):
        self.kind, self.S, self.width = kind, S, width
        self.Hkv, self.Hq = 8, 16
        self.nb = S * width
        g = torch.Generator().manual_seed(seed)
        dtype = torch.float16
        self.q = torch.randn(S, self.Hq, D, generator=g).to(dtype).to(DEV)
        if kind.startswith("q4"):
            self.k = torch.zeros(pkv.q4_cache_shape(self.nb, self.Hkv, B, D), dtype=torch.uint8,
                                 device=DEV)
            self.v = torch.zeros_like(self.k)
            # within 4, so that a scale is at most 8 / 15 and the weights' rounding at
            # most 2^-11 of 7.5 scales, 2e-3
            rows = [torch.randn(self.nb * B, self.Hkv, D, generator=g).clamp(-4, 4).to(dtype).to(DEV)
                    for _ in range(2)]
            pkv.kv_write_q4(self.k, self.v, *rows, torch.arange(self.nb * B, device=DEV))
        else:
            self.k, self.v = (torch.randn(self.nb, self.Hkv, B, D, generator=g).to(dtype).to(DEV)
                              for _ in range(2))
        self.stack = torch.randperm(self.nb, generator=g).tolist()
        self.count, self.lens = self.nb, [0] * S
        self.tables = [[-1] * width for _ in range(S)]
        self.d_tables, self.d_lens = i32(self.tables), i32(self.lens)
        self.d_stack, self.d_count = i32(self.stack), i32([self.nb])
        self.tws = torch.empty(pkv.tables_workspace_bytes(S), dtype=torch.uint8, device=DEV)
        self.qs = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
        P = self.P = 64 if kind.endswith("split") else 0
        self.ws = None
        if P or kind.endswith("planned"):
            self.ws = torch.empty(pkv.decode_workspace_bytes(S, self.Hq, D, width * B, P),
                                  dtype=torch.uint8, device=DEV)
        self.groups, self.shared = i32(list(range(S + 1))), i32([0] * S)

    def attend(self, out, tables, lens):
        if self.kind == "16-bit groups":
            pkv.paged_decode_grouped(out, self.q, self.k, self.v, tables, lens, self.groups,
                                     self.shared, 0.125, B, self.Hkv, max_members=1)
            return
        call = pkv.paged_decode_attention_q4 if self.kind.startswith("q4") else \
            pkv.paged_decode_attention
        call(out, self.q, self.k, self.v, tables, lens, 0.125, B, self.Hkv, partition_size=self.P,
             workspace=self.ws)

    def extend(self, new, slots):
        pkv.tables_extend(self.d_tables, self.d_lens, new, self.d_stack, self.d_count, B, self.qs,
                          slots, None, self.tws)

    def release(self, done):
        pkv.tables_release(self.d_tables, self.d_lens, done, self.d_stack, self.d_count, B, self.tws)

    def oracle_step(self, new, done, rows):
        """The oracle's lengths and tables after an extend, and after the release."""
        self.lens, self.count, _, _, _, refused, bad = table_oracle.extend(
            self.tables, self.lens, new, self.stack, self.count, B, self.nb, rows)
        assert not refused and not bad
        after = (list(self.lens), [list(r) for r in self.tables])
        self.count, refused, bad = table_oracle.release(self.tables, self.lens, done, self.stack,
                                                        self.count, B, self.nb)
        assert not refused and not bad
        return after, (list(self.lens), [list(r) for r in self.tables])


KINDS = ["16-bit plain", "16-bit planned", "16-bit split", "16-bit groups",
         "q4 plain", "q4 planned", "q4 split"]


# 100 sequences of 8 KV heads are more CTAs than the GPU holds at once: a plan is
# used; 20 of them go through the plan of few sequences.  Steps of up to 2048 rows
# (and releases of up to 1024 entries) run in one launch, others in two.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S,width,most", [(100, 40, 6), (100, 40, 40), (20, 300, 250), (20, 40, 8)])
@pytest.mark.parametrize("graph", [False, True])
def test_attention_sees_what_the_table_calls_wrote(kind, S, width, most, graph):
    batch = Batch(kind, S, width, seed=S + most)
    g = torch.Generator().manual_seed(most)
    steps, rows = 8, S * most
    lens = torch.zeros(S, dtype=torch.int64)
    plan = []
    for _ in range(steps):
        new = torch.minimum(torch.randint(0, most + 1, (S,), generator=g), width * B - lens)
        done = (torch.rand(S, generator=g) < 0.2).int()
        lens = (lens + new) * (done == 0)
        plan.append((new.tolist(), done.tolist()))
    slots = torch.zeros(rows, dtype=torch.int64, device=DEV)
    inputs = [(i32(new), i32(done)) for new, done in plan]
    outs = [[torch.full(batch.q.shape, float("nan"), device=DEV) for _ in range(2)]
            for _ in range(steps)]
    held = [[(torch.empty_like(batch.d_tables), torch.empty_like(batch.d_lens)) for _ in range(2)]
            for _ in range(steps)]

    def run():
        for n, (new, done) in enumerate(inputs):
            for half in range(2):
                if half == 0:
                    batch.extend(new, slots)
                else:
                    batch.release(done)
                batch.attend(outs[n][half], batch.d_tables, batch.d_lens)
                held[n][half][0].copy_(batch.d_tables)
                held[n][half][1].copy_(batch.d_lens)

    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            run()
        captured.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert pkv.device_status() == 0
    again = torch.empty_like(outs[0][0])
    for n, (new, done) in enumerate(plan):
        for half, (want_lens, want_tables) in enumerate(batch.oracle_step(new, done, rows)):
            tables, lens = held[n][half]
            assert lens.tolist() == want_lens and tables.tolist() == want_tables
            again.fill_(float("nan"))
            torch.cuda.synchronize()
            batch.attend(again, tables, lens)
            torch.cuda.synchronize()
            assert torch.equal(outs[n][half], again), (n, half)
            if n == steps - 2:
                q, k, v = batch.q.cpu(), batch.k.cpu(), batch.v.cpu()
                if kind.startswith("q4"):
                    want = q4.paged_decode_attention(q, k, v, tables.cpu(), want_lens, 0.125)
                else:
                    want = oracle.paged_decode_attention(q, k, v, tables.cpu(), lens.cpu(), 0.125, B,
                                                         batch.Hkv, nthreads=oracle.default_threads())
                assert np.abs(again.cpu().double().numpy() - want).max() <= 2e-3


def test_a_16_bit_cache_served_from_tables_built_on_the_gpu():
    """Prompts and decode steps with kv_write, prefill and decode attention over slots,
    row starts, lengths and tables that never leave the GPU."""
    S, Hq, Hkv, dim, block, width = 5, 8, 2, 128, 16, 20
    dtype, nb = torch.bfloat16, 60
    g = torch.Generator().manual_seed(11)
    stack = torch.randperm(nb, generator=g).tolist()
    tables, lens = i32([[-1] * width for _ in range(S)]), i32([0] * S)
    d_stack, count = i32(stack), i32([nb])
    ws = torch.empty(pkv.tables_workspace_bytes(S), dtype=torch.uint8, device=DEV)
    qs = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    k, v = (torch.full((nb, Hkv, block, dim), float("nan"), dtype=dtype, device=DEV)
            for _ in range(2))
    hk, hv = k.cpu(), v.cpu()
    scale = dim ** -0.5
    state = ([[-1] * width for _ in range(S)], [0] * S, nb)
    for new in ([33, 1, 0, 100, 16], [1] * S, [60, 1, 200, 1, 1], [1] * S):
        rows = sum(new) + 3
        key, value = (torch.randn(rows, Hkv, dim, generator=g).to(dtype) for _ in range(2))
        q = torch.randn(rows, Hq, dim, generator=g).to(dtype)
        slots = torch.zeros(rows, dtype=torch.int64, device=DEV)
        out = torch.full((rows, Hq, dim), float("nan"), device=DEV)
        args = [t.to(DEV) for t in (key, value, q)]
        pkv.tables_extend(tables, lens, i32(new), d_stack, count, block, qs, slots, None, ws)
        pkv.kv_write(k, v, args[0], args[1], slots)
        pkv.paged_prefill_attention(out, args[2], k, v, tables, lens, qs, scale, block, Hkv,
                                    max_query_len=max(new))
        last = torch.full((S, Hq, dim), float("nan"), device=DEV)
        dq = torch.randn(S, Hq, dim, generator=g).to(dtype)
        pkv.paged_decode_attention(last, dq.to(DEV), k, v, tables, lens, scale, block, Hkv)
        host_tables, host_lens, left = state
        host_lens, left, start, want_slots, _, refused, bad = table_oracle.extend(
            host_tables, host_lens, new, stack, left, block, nb, rows)
        state = (host_tables, host_lens, left)
        assert not refused and not bad
        assert slots.tolist() == want_slots and qs.tolist() == start
        assert lens.tolist() == host_lens and tables.tolist() == host_tables
        oracle.kv_write(hk, hv, key, value, torch.tensor(want_slots), block)
        assert torch.equal(k.cpu().view(torch.int16), hk.view(torch.int16))
        ht, hl = tables.cpu(), lens.cpu()
        real = sum(new)
        want = oracle.paged_prefill_attention(q[:real], hk, hv, ht, hl, torch.tensor(start).int(),
                                              scale, block, Hkv, nthreads=oracle.default_threads())
        assert np.abs(out[:real].cpu().double().numpy() - want).max() <= 2e-3
        want = oracle.paged_decode_attention(dq, hk, hv, ht, hl, scale, block, Hkv)
        assert np.abs(last.cpu().double().numpy() - want).max() <= 2e-3
    assert pkv.device_status() == 0

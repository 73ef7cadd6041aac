"""kvc_plan_step against its plain form: every output a whole number, so everything is equal."""
import numpy as np
import pytest
import torch

from sparse_reference import plan

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class State:
    """Tables, lengths and free blocks of a server; a pool of one narrow head, which only lends its shape."""

    def __init__(self, kvc, B, bs, width, lens, seed=0, spare=40, extra=0):
        r = np.random.default_rng(seed)
        self.kvc, self.bs, self.B = kvc, bs, B
        self.lens = np.asarray(lens, np.int32)
        held = sum(-(-int(n) // bs) for n in lens)
        self.N = held + spare
        ids = r.permutation(self.N).astype(np.int32)
        self.table = np.full((B, width), -7, np.int32)
        at = 0
        for b, n in enumerate(lens):
            k = -(-int(n) // bs)
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.stack = np.full(self.N + extra, -9, np.int32)
        self.stack[:spare] = ids[at:]
        self.count = spare
        self.pool = kvc.kvc_pool_create(self.N, bs, 1, 1, 64)

    def run(self, new, rows, place=False, offset=0, maps=(True, True), stream=None):
        """One call; (what the plain form gives, what the call gives)."""
        want = plan(self.table, self.lens, new, self.stack, self.count, rows, self.bs)
        t, lens, stack, count = dev(self.table), dev(self.lens), dev(self.stack), dev([self.count])
        fresh = dev(new)
        lens_out = lens if place else torch.full_like(lens, 99)
        count_out = count if place else torch.full_like(count, 99)
        cu = torch.full((self.B + 1,), 99, dtype=torch.int32, device="cuda")
        s, p, q = (torch.full((rows + offset + 2,), 99, dtype=torch.int32, device="cuda") for _ in range(3))
        cut = slice(offset, offset + rows)
        self.kvc.kvc_plan_step(self.pool, t, lens, fresh, stack, count, lens_out, count_out, cu, s[cut],
                               p[cut] if maps[0] else None, q[cut] if maps[1] else None, stream=stream)
        torch.cuda.synchronize()
        for x in (s, p, q):   # around the map nothing is written
            assert torch.all(x[:offset] == 99) and torch.all(x[offset + rows:] == 99)
        got = [x.cpu().numpy() for x in (t, stack, count_out, lens_out, cu, s[cut], p[cut], q[cut])]
        got[2] = int(got[2][0])
        return want, got

    def check(self, new, rows, **how):
        want, got = self.run(new, rows, **how)
        maps = how.get("maps", (True, True))
        for name, w, g in zip(("table", "stack", "count", "lens", "cu", "slots", "positions", "seqs"), want, got):
            if (name == "positions" and not maps[0]) or (name == "seqs" and not maps[1]):
                assert np.all(g == 99)
                continue
            assert np.array_equal(w, g), f"{name}: {np.flatnonzero(np.ravel(w != g))[:5]}"
        assert self.kvc.kvc_pool_sync_status(self.pool) == self.kvc.KVC_OK
        return want

    def close(self):
        self.pool.close()


def requests(r, B, top, prompts=0.1, finish=0.1, cut=0.1, idle=0.1, long=50):
    lens, new = [], []
    for x in r.random(B):
        n = int(r.integers(0, top + 1))
        if x < prompts:
            lens.append(0), new.append(int(r.integers(0, long)))
        elif x < prompts + finish:
            lens.append(n), new.append(0)
        elif x < prompts + finish + cut:
            lens.append(n), new.append(max(0, n - int(r.integers(0, 6))))
        elif x < prompts + finish + cut + idle:
            lens.append(n), new.append(n)
        else:
            lens.append(n), new.append(n + 1)
    return lens, new


@pytest.mark.parametrize("B,bs,top,long,pad,spare", [
    (1, 16, 0, 40, 0, 3), (1, 16, 100, 40, 3, 10), (5, 1, 9, 8, 0, 60), (7, 3, 40, 90, 5, 200), (64, 16, 300, 700, 2, 900),
    (511, 16, 60, 20, 1, 4000), (512, 16, 60, 9, 0, 4000), (513, 16, 60, 9, 4, 4000), (700, 128, 1000, 3000, 9, 2000),
    (5000, 16, 33, 30, 13, 9000), (32768, 16, 20, 5, 0, 40000)])
def test_random_steps(kvc, B, bs, top, long, pad, spare):
    r = np.random.default_rng(B + bs)
    lens, new = requests(r, B, top, long=long)
    if B == 1:
        lens, new = [top], [top + long]
    width = -(-max(max(lens), max(new), 1) // bs) + 2
    st = State(kvc, B, bs, width, lens, seed=B, spare=spare)
    try:
        st.check(new, sum(max(0, z - a) for a, z in zip(lens, new)) + pad)
    finally:
        st.close()


@pytest.mark.parametrize("B", [3, 600])
@pytest.mark.parametrize("scarce", ["blocks", "rows", "both", "no block at all", "no row at all"])
def test_first_come_first_served(kvc, B, scarce):
    """Growth stops at the first sequence that does not fit, even for a later one that needs no block."""
    r = np.random.default_rng(B)
    lens, new = requests(r, B, 90, finish=0.02, long=120)
    rows = sum(max(0, z - a) for a, z in zip(lens, new))
    need = sum(max(0, -(-z // 16) + (-a // 16)) for a, z in zip(lens, new))
    spare = {"blocks": need // 2, "both": need // 2, "no block at all": 0}.get(scarce, need + 4)
    rows = {"rows": rows // 2, "both": rows // 2 + 3, "no row at all": 0}.get(scarce, rows + 5)
    st = State(kvc, B, 16, -(-max(lens + new) // 16) + 1, lens, seed=1, spare=spare)
    try:
        want = st.check(new, rows)
        assert np.any(want[3] < np.asarray(new)) or B == 3
    finally:
        st.close()


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("maps", [(True, True), (False, True), (True, False), (False, False)])
def test_maps_that_are_left_out_or_stand_anywhere(kvc, offset, maps):
    st = State(kvc, 4, 16, 40, [0, 17, 300, 5], spare=60)
    try:
        st.check([523, 18, 300, 0], 523 + 1 + 6, offset=offset, maps=maps)
    finally:
        st.close()


def test_a_server_runs_in_place_and_in_a_graph(kvc):
    """Steps in place, captured once and replayed: no block is lost or held twice, and every step is the plain form's."""
    B, bs, width = 40, 16, 20
    r = np.random.default_rng(5)
    st = State(kvc, B, bs, width, [0] * B, spare=150)
    t, lens, stack, count = dev(st.table), dev(st.lens), dev(st.stack), dev([st.count])
    new, cu = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    s, p, q = (torch.zeros(700, dtype=torch.int32, device="cuda") for _ in range(3))

    def call():
        kvc.kvc_plan_step(st.pool, t, lens, new, stack, count, lens, count, cu, s, p, q)

    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for step in range(30):
            want_new = [int(n + r.integers(0, 30)) if r.random() < 0.8 else int(n * r.random()) for n in st.lens]
            want_new = [min(n, width * bs) for n in want_new]
            want = plan(st.table, st.lens, want_new, st.stack, st.count, 700, bs)
            new.copy_(dev(want_new))
            graph.replay() if step % 3 else call()
            got = [x.cpu().numpy() for x in (t, stack, count, lens, cu, s, p, q)]
            for name, w, g in zip(("table", "stack", "count", "lens", "cu", "slots", "positions", "seqs"), want, got):
                assert np.array_equal(np.ravel(w), np.ravel(g)), (step, name)
            st.table, st.stack, st.count, st.lens = want[0], want[1], want[2], want[3]
            held = [st.table[b, j] for b in range(B) for j in range(-(-int(st.lens[b]) // bs))]
            assert sorted(held + st.stack[:st.count].tolist()) == list(range(st.N))
        assert kvc.kvc_pool_sync_status(st.pool) == kvc.KVC_OK
    finally:
        st.close()


def test_no_sequences(kvc):
    st = State(kvc, 0, 16, 4, [], spare=5)
    try:
        want, got = st.run([], 9)
        assert got[2] == 5 and got[4].tolist() == [0] and np.all(got[5] == -1) and np.all(got[6] == -1)
    finally:
        st.close()


@pytest.mark.parametrize("bad", [(-1, 5), (5, -1), (1000, 3), (3, 1000), (-2147483648, 2147483647)])
def test_a_sequence_with_bad_lengths_is_left_out(kvc, bad):
    lens, new = [20, 30, 40], [21, 31, 0]
    st = State(kvc, 3, 16, 6, lens, spare=8)
    try:
        st.lens[1], new[1] = bad
        fixed = list(new)
        fixed[1] = st.lens[1]
        want = plan(st.table, np.where(np.arange(3) == 1, 0, st.lens), [21, 0, 0], st.stack, st.count, 6, 16)
        _, got = State.run(st, fixed, 6)
        t, lens_d, stack, count = dev(st.table), dev(st.lens), dev(st.stack), dev([st.count])
        cu, s = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
        out, left = torch.zeros_like(lens_d), torch.zeros_like(count)
        kvc.kvc_plan_step(st.pool, t, lens_d, dev(new), stack, count, out, left, cu, s)
        assert kvc.kvc_pool_sync_status(st.pool) == kvc.KVC_ERR_RANGE
        assert out.tolist() == [21, bad[0], 0] and cu.tolist() == [0, 1, 1, 1]
        assert np.array_equal(s.cpu().numpy(), want[5]) and np.array_equal(stack.cpu().numpy(), want[1])
    finally:
        st.close()


def test_bad_counts_and_entries_are_recorded(kvc):
    st = State(kvc, 2, 16, 6, [20, 30], spare=8)

    def call(count, table, new, rows=40):
        t, stack, cnt = dev(table), dev(st.stack), dev([count])
        left, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        cu, s = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
        kvc.kvc_plan_step(st.pool, t, dev(st.lens), dev(new), stack, cnt, out, left, cu, s)
        return kvc.kvc_pool_sync_status(st.pool), int(left), s.cpu().numpy(), out.tolist()

    try:
        status, left, s, out = call(-5, st.table, [33, 30])
        assert status == kvc.KVC_ERR_RANGE and left == 0 and out == [20, 30] and np.all(s == -1)
        status, left, _, out = call(st.N + 3, st.table, [21, 30])   # the list holds N
        assert status == kvc.KVC_ERR_RANGE and left == st.N and out == [21, 30]
        status, left, _, _ = call(st.N, st.table, [0, 30])          # more returned than it has room for
        assert status == kvc.KVC_ERR_RANGE and left == st.N
        broken = st.table.copy()
        broken[0, 1], broken[1, 1] = -1, st.N
        status, _, s, _ = call(8, broken, [21, 31])                 # the tokens' own blocks
        assert status == kvc.KVC_ERR_BAD_BLOCK and s[:2].tolist() == [-1, -1]
        status, left, _, _ = call(8, broken, [0, 0])                # returned as they stand
        assert status == kvc.KVC_ERR_BAD_BLOCK and left == 12
        assert call(8, st.table, [21, 31])[0] == kvc.KVC_OK
    finally:
        st.close()


def test_on_another_stream(kvc):
    st = State(kvc, 30, 16, 30, [9] * 30, spare=60)
    try:
        side = torch.cuda.Stream()
        st.check([40] * 30, 31 * 30, stream=side)
        with torch.cuda.stream(side):
            st.check([40] * 30, 31 * 30)
    finally:
        st.close()


def test_refusals(kvc):
    st = State(kvc, 2, 16, 6, [20, 30], spare=8)
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    good = dict(block_tables=z(2, 6), seq_lens=z(2), new_lens=z(2), free_list=z(st.N), free_count=z(1), lens_out=z(2),
                count_out=z(1), cu_tokens=z(3), slots=z(4), positions=z(4), seq_ids=z(4))
    try:
        kvc.kvc_plan_step(st.pool, **good)
        for name, bad in [("block_tables", z(3, 6)), ("block_tables", z(12)), ("seq_lens", z(3)), ("new_lens", z(1)),
                          ("free_count", z(2)), ("lens_out", z(5)), ("cu_tokens", z(2)), ("slots", None),
                          ("positions", z(3)), ("seq_ids", z(5)), ("slots", z(4, 2)[:, 0]),
                          ("seq_lens", torch.zeros(2, dtype=torch.int64, device="cuda")),
                          ("new_lens", torch.zeros(2, dtype=torch.int32))]:
            with pytest.raises(ValueError):
                kvc.kvc_plan_step(st.pool, **{**good, name: bad})
        with pytest.raises(kvc.KvcError) as e:
            kvc.kvc_plan_step(st.pool, **{**good, "free_list": z(st.N - 1)})
        assert e.value.status == kvc.KVC_ERR_ARG
        big = 32769
        with pytest.raises(kvc.KvcError) as e:
            kvc.kvc_plan_step(st.pool, **{**good, "block_tables": z(big, 1), "seq_lens": z(big), "new_lens": z(big),
                                          "lens_out": z(big), "cu_tokens": z(big + 1)})
        assert e.value.status == kvc.KVC_ERR_UNSUPPORTED
        assert kvc.kvc_pool_sync_status(st.pool) == kvc.KVC_OK
    finally:
        st.close()

"""The page calls on the GPU against the same rules written out in Python lists: tables,
lengths, counts, pairs and page contents are equal."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


class Pool:
    """The rules of include/gqla.h, one sequence and one page at a time."""

    def __init__(self, batch, width, pages):
        self.table = [[-3] * width for _ in range(batch)]
        self.lens, self.refs, self.width = [0] * batch, [0] * pages, width

    def free_page(self):
        return next((i for i, r in enumerate(self.refs) if r == 0), None)

    def extend(self, grow):
        bad, full = [], False
        for b, n in enumerate(grow):
            if n == 0:
                continue
            if n < 0 or self.lens[b] + n > self.width * 64:
                bad.append(b)
                continue
            have, want = -(-self.lens[b] // 64), -(-(self.lens[b] + n) // 64)
            free = [i for i, r in enumerate(self.refs) if r == 0]
            if want > have and (full or want - have > len(free)):
                full = True
                bad.append(b)
                continue
            for j, p in zip(range(have, want), free):
                self.table[b][j] = p
                self.refs[p] = 1
            self.lens[b] += n
        return bad

    def fork(self, forks):
        kids = [c for _, c in forks]
        lens = list(self.lens)
        pairs, bad = [], []
        for i, (a, c) in enumerate(forks):
            ok = 0 <= a < len(lens) and 0 <= c < len(lens) and a != c and kids.count(c) == 1 and a not in kids and lens[c] == 0
            page = self.free_page() if ok and lens[a] % 64 else None
            if not ok or (lens[a] % 64 and page is None):
                pairs.append((-1, -1))
                bad.append(i)
                continue
            for j in range(lens[a] // 64):
                self.table[c][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            pairs.append((-1, -1))
            if lens[a] % 64:
                pairs[-1] = (self.table[a][lens[a] // 64], page)
                self.table[c][lens[a] // 64] = page
                self.refs[page] = 1
            self.lens[c] = lens[a]
        return pairs, bad

    def free(self, ids):
        bad = []
        for i, b in enumerate(ids):
            if not 0 <= b < len(self.lens):
                bad.append(i)
                continue
            for p in self.table[b][:-(-self.lens[b] // 64)]:
                self.refs[p] -= 1
            self.lens[b] = 0
        return bad

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        moves = list(zip([i for i in range(n, len(self.refs)) if self.refs[i] > 0],
                         [i for i in range(n) if self.refs[i] == 0]))
        to = dict(moves)
        for b, row in enumerate(self.table):
            for j in range(-(-self.lens[b] // 64)):
                row[j] = to.get(row[j], row[j])
        for a, c in moves:
            self.refs[c], self.refs[a] = self.refs[a], 0
        return n, moves


class Gpu:
    def __init__(self, ref, groups=2, seed=0, caches=True):
        from decode_attention_06_b200 import gqla
        self.gqla = gqla
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        self.i32 = i32
        self.table, self.lens, self.refs = i32(ref.table), i32(ref.lens), i32(ref.refs)
        self.pool = gqla.make_page_pool(self.table, self.lens, self.refs)
        self.ws, self.dims = gqla.new_workspace(), gqla.make_dims(16 * groups, groups)
        self.pages = len(ref.refs)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        bf = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
        if caches:
            self.latent, self.kv, self.rope = bf(self.pages, 64, 576), bf(groups, self.pages * 64, 256), bf(self.pages * 64, 64)

    def same(self, ref):
        assert self.lens.tolist() == ref.lens
        assert self.refs.tolist() == ref.refs
        assert self.table.tolist() == ref.table

    def error(self, bad):
        """The recorded error is one of the expected ones (the first to be recorded); clears it."""
        st, info = self.gqla.gqla_read_device_error(self.ws)
        assert (st == -5 and info in bad) if bad else st == 0, (st, info, bad)
        self.gqla.gqla_clear_device_error(self.ws)

    def extend(self, grow):
        self.gqla.gqla_extend_sequences(self.pool, self.i32(grow), self.ws)

    def fork(self, forks):
        pairs = torch.full((len(forks), 2), 99, dtype=torch.int32).cuda()
        self.gqla.gqla_fork_sequences(self.pool, self.i32(forks), pairs, self.ws)
        return pairs

    def free(self, ids):
        self.gqla.gqla_free_sequences(self.pool, self.i32(ids), self.ws)

    def compact(self, inplace=True):
        t, r = (self.table, self.refs) if inplace else (torch.empty_like(self.table), torch.full_like(self.refs, 77))
        pairs = torch.full((max(1, self.pages // 2), 2), 99, dtype=torch.int32).cuda()
        counts = torch.zeros(2, dtype=torch.int32).cuda()
        self.gqla.gqla_compact_pages(self.pool, t, r, pairs, counts, self.ws)
        return t, r, pairs, counts

    def copy(self, pairs, **which):
        which = which or dict(latent_cache=self.latent, kv_expanded=self.kv, k_rope=self.rope)
        self.gqla.gqla_copy_pages(self.dims, pairs, self.pages, self.ws, **which)


def copied(caches, groups, pairs):
    """The page contents after `pairs`, by indexing."""
    latent, kv, rope = (x.clone() for x in caches)
    kv4, rope3 = kv.view(groups, -1, 64, 256), rope.view(-1, 64, 64)
    src = torch.tensor([a for a, _ in pairs], dtype=torch.long).cuda()
    dst = torch.tensor([b for _, b in pairs], dtype=torch.long).cuda()
    if len(pairs):
        latent[dst], kv4[:, dst], rope3[dst] = latent[src], kv4[:, src], rope3[src]
    return latent, kv, rope


@pytest.mark.parametrize("pages,n", [(2, 1), (40, 7), (600, 250), (33, 16)])
@pytest.mark.parametrize("groups", [1, 8])
def test_copy_pages(pages, n, groups):
    g = Gpu(Pool(1, 1, pages), groups)
    order = random.Random(pages).sample(range(pages), 2 * n)
    pairs = [(order[2 * i], order[2 * i + 1]) for i in range(n)]
    if n > 3:
        pairs[1] = (pairs[0][0], pairs[1][1])  # one page to two
    want = copied((g.latent, g.kv, g.rope), groups, pairs)
    listed = [(-1, -1), (5 % pages, 5 % pages)] + pairs + [(-1, 3 % pages)]
    g.copy(torch.tensor(listed, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    g.error([])
    for got, exp in zip((g.latent, g.kv, g.rope), want):
        assert torch.equal(got, exp)


def test_copy_pages_of_one_cache_leaves_the_others():
    g = Gpu(Pool(1, 1, 6), 2)
    before = [x.clone() for x in (g.latent, g.kv, g.rope)]
    pairs = torch.tensor([[0, 4], [1, 5]], dtype=torch.int32).cuda()
    want = copied(before, 2, [(0, 4), (1, 5)])
    g.copy(pairs, kv_expanded=g.kv)
    torch.cuda.synchronize()
    assert torch.equal(g.kv, want[1]) and torch.equal(g.latent, before[0]) and torch.equal(g.rope, before[2])
    g.copy(pairs, latent_cache=g.latent)
    torch.cuda.synchronize()
    assert torch.equal(g.latent, want[0]) and torch.equal(g.rope, before[2])
    g.error([])


def test_copy_pages_leaves_out_clashing_pairs():
    """A target written twice, a source that another pair writes, pages outside the pool."""
    g = Gpu(Pool(1, 1, 12), 2)
    listed = [(0, 8), (1, 8), (2, 9), (9, 10), (3, 12), (13, 4), (5, -2), (6, 11)]
    want = copied((g.latent, g.kv, g.rope), 2, [(2, 9), (6, 11)])
    g.copy(torch.tensor(listed, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    g.error([0, 1, 3, 4, 5, 6])
    for got, exp in zip((g.latent, g.kv, g.rope), want):
        assert torch.equal(got, exp)


@pytest.mark.parametrize("seed", range(6))
def test_random_lifetimes(seed):
    """Extend, fork (with the copies), free and compact in random turns, full pools included."""
    rng = random.Random(seed)
    batch, width = rng.choice([(3, 4), (40, 9), (70, 30)])
    ref = Pool(batch, width, rng.choice([7, 100, 1500]))
    g = Gpu(ref, 2, seed)
    for turn in range(25):
        what = rng.choice(["extend", "fork", "free", "compact"]) if turn else "extend"
        if what == "extend":
            grow = [rng.choice([0, 0, 1, 5, 64, 65, rng.randint(0, 600)]) for _ in range(batch)]
            g.extend(grow)
            bad = ref.extend(grow)
        elif what == "fork":
            forks = [(rng.randrange(batch), rng.randrange(batch)) for _ in range(rng.randint(1, batch))]
            before = (g.latent, g.kv, g.rope)
            pairs = g.fork(forks)
            exp, bad = ref.fork(forks)
            assert pairs.tolist() == [list(p) for p in exp]
            want = copied(before, 2, [p for p in exp if p[0] >= 0])
            g.copy(pairs)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((g.latent, g.kv, g.rope), want))
        elif what == "free":
            ids = [rng.randrange(batch) for _ in range(rng.randint(1, batch))]
            g.free(ids)
            bad = ref.free(ids)
        else:
            t, r, pairs, counts = g.compact(inplace=rng.random() < 0.5)
            n, moves = ref.compact()
            bad = []
            torch.cuda.synchronize()
            assert counts.tolist() == [n, len(moves)]
            assert pairs.tolist() == [list(m) for m in moves] + [[-1, -1]] * (pairs.shape[0] - len(moves))
            want = copied((g.latent, g.kv, g.rope), 2, moves)
            g.copy(pairs)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((g.latent, g.kv, g.rope), want))
            g.table.copy_(t)
            g.refs.copy_(r)
        torch.cuda.synchronize()
        g.same(ref)
        g.error(bad)


def test_large_batch_and_pool():
    """More sequences than a block has threads, more pages than one round of a scan."""
    rng = random.Random(5)
    ref = Pool(2600, 6, 20000)
    g = Gpu(ref, caches=False)
    for turn in range(3):
        grow = [rng.choice([0, 1, 100, 130]) for _ in range(2600)]
        g.extend(grow)
        bad = ref.extend(grow)
        ids = rng.sample(range(2600), 900)
        g.free(ids)
        ref.free(ids)
        empty = [b for b in range(2600) if ref.lens[b] == 0]
        forks = [(rng.choice([b for b in range(50) if b not in empty] or [0]), c) for c in empty[100:]]
        pairs = g.fork(forks)
        exp, bad2 = ref.fork(forks)
        torch.cuda.synchronize()
        assert pairs.tolist() == [list(p) for p in exp]
        g.same(ref)
        g.error(bad + bad2)
    t, r, pairs, counts = g.compact(inplace=False)
    n, moves = ref.compact()
    torch.cuda.synchronize()
    assert counts.tolist() == [n, len(moves)] and len(moves) > 0
    assert pairs.tolist()[:len(moves)] == [list(m) for m in moves]
    assert t.tolist() == ref.table and r.tolist() == ref.refs


def test_forks_beyond_one_block_of_threads():
    ref = Pool(3000, 3, 4000)
    g = Gpu(ref, caches=False)
    grow = [70 if b % 2 else 64 for b in range(100)] + [0] * 2900
    g.extend(grow)
    ref.extend(grow)
    forks = [(i % 100, 100 + i) for i in range(2900)]
    pairs = g.fork(forks)
    exp, bad = ref.fork(forks)
    torch.cuda.synchronize()
    assert pairs.tolist() == [list(p) for p in exp]
    g.same(ref)
    g.error(bad)


def test_pages_outside_the_pool_are_reported():
    ref = Pool(4, 3, 8)
    ref.extend([130, 70, 0, 0])
    g = Gpu(ref)
    g.table[0, 1], g.table[1, 1] = 8, -1
    g.free([0])
    g.error([0])
    g.fork([(1, 2)])  # its partly filled page is not in the pool: refused
    torch.cuda.synchronize()
    assert g.lens.tolist() == [0, 70, 0, 0]
    g.error([0])
    refs = g.refs.clone()
    g.compact(inplace=False)
    g.error([1])
    g.free([3, 9, -1])
    g.error([1, 2])
    assert torch.equal(g.refs, refs)


def test_copy_pages_far_offsets():
    pages = 140_000
    from decode_attention_06_b200 import gqla
    kv = torch.zeros(1, pages * 64, 256, dtype=torch.bfloat16, device="cuda")
    v = kv.view(pages, 64, 256)
    v[3], v[pages - 2] = 3.0, 5.0
    pairs = torch.tensor([[3, pages - 1], [pages - 2, 7]], dtype=torch.int32, device="cuda")
    ws = gqla.new_workspace()
    gqla.gqla_copy_pages(gqla.make_dims(16, 1), pairs, pages, ws, kv_expanded=kv)
    torch.cuda.synchronize()
    assert gqla.gqla_read_device_error(ws)[0] == 0
    assert bool((v[pages - 1] == 3.0).all()) and bool((v[7] == 5.0).all()) and float(v.float().sum()) == 16.0 * 64 * 256


def test_page_calls_in_a_graph():
    """Fork, copy, extend and free captured once and replayed: each replay starts from the pool as it is."""
    ref = Pool(4, 6, 30)
    ref.extend([100, 64, 0, 0])
    g = Gpu(ref)
    forks, grow, gone = g.i32([[0, 2], [1, 3]]), g.i32([0, 0, 70, 1]), g.i32([2, 3])
    pairs = torch.full((2, 2), 9, dtype=torch.int32, device="cuda")
    kept = [x.clone() for x in (g.latent, g.kv, g.rope)]

    def cycle():
        g.gqla.gqla_fork_sequences(g.pool, forks, pairs, g.ws)
        g.copy(pairs)
        g.gqla.gqla_extend_sequences(g.pool, grow, g.ws)
        g.gqla.gqla_free_sequences(g.pool, gone, g.ws)

    cycle()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cycle()
    exp, _ = ref.fork([(0, 2), (1, 3)])
    want = copied(kept, 2, [p for p in exp if p[0] >= 0])
    ref.extend([0, 0, 70, 1])
    ref.free([2, 3])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        g.same(ref)
        assert pairs.tolist() == [list(p) for p in exp]
        assert all(torch.equal(a, b) for a, b in zip((g.latent, g.kv, g.rope), want))
    g.error([])


def test_a_full_pool():
    ref = Pool(4, 8, 5)
    g = Gpu(ref)
    for grow in ([130, 64, 65, 1], [0, 0, 0, 0], [62, 1, 0, 0]):
        g.extend(grow)
        bad = ref.extend(grow)
        torch.cuda.synchronize()
        g.same(ref)
        g.error(bad)
    pairs = g.fork([(0, 3)])
    exp, bad = ref.fork([(0, 3)])
    torch.cuda.synchronize()
    assert pairs.tolist() == [list(p) for p in exp]
    g.same(ref)
    g.error(bad)


def test_empty_calls():
    ref = Pool(3, 4, 8)
    g = Gpu(ref)
    e = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    g.gqla.gqla_fork_sequences(g.pool, e, e.clone(), g.ws)
    g.copy(e)
    g.gqla.gqla_free_sequences(g.pool, torch.empty(0, dtype=torch.int32, device="cuda"), g.ws)
    t, r, pairs, counts = g.compact(inplace=False)
    torch.cuda.synchronize()
    assert counts.tolist() == [0, 0] and pairs.tolist() == [[-1, -1]] * 4 and not bool(r.any())
    g.same(ref)
    g.error([])


def test_one_page_pool():
    ref = Pool(2, 1, 1)
    g = Gpu(ref)
    g.extend([64, 0])
    ref.extend([64, 0])
    g.fork([(0, 1)])
    ref.fork([(0, 1)])
    t, r, pairs, counts = g.compact()
    torch.cuda.synchronize()
    assert counts.tolist() == [1, 0] and pairs.tolist() == [[-1, -1]]
    g.same(ref)
    g.error([])


def test_extend_by_more_pages_than_32_bits_count():
    from decode_attention_06_b200 import gqla
    batch, width, pages = 66, 1 << 25, 8  # every row may hold 2^31 tokens
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    table = torch.empty(batch, width, dtype=torch.int32, device="cuda")
    table[:, :pages] = -7
    lens, refs, ws = i32([0] * batch), i32([0] * pages), gqla.new_workspace()
    pool = gqla.make_page_pool(table, lens, refs)
    most = (1 << 31) - 1
    gqla.gqla_extend_sequences(pool, i32([100] + [most] * (batch - 1)), ws)
    torch.cuda.synchronize()
    assert lens.tolist() == [100] + [0] * (batch - 1)
    assert refs.tolist() == [1, 1] + [0] * (pages - 2)
    assert table[0, :pages].tolist() == [0, 1] + [-7] * (pages - 2) and bool((table[1:, :pages] == -7).all())
    st, info = gqla.gqla_read_device_error(ws)
    assert st == -5 and 1 <= info < batch


@pytest.mark.parametrize("batch,room", [(700, 12000), (1024, 5300), (1500, 14000)])
def test_extend_by_thousands_of_pages_from_a_fragmented_pool(batch, room):
    """More pages for one group of 1024 sequences than the list in shared memory holds: given out in
    several rounds from free pages that lie scattered, until the pool is full in the smaller pools."""
    rng = random.Random(room)
    ref = Pool(batch, 12, room)
    grow = [rng.choice([0, 64, 200, 300]) for _ in range(batch)]
    ref.extend(grow)
    ref.free(rng.sample(range(batch), batch // 2))
    for p in rng.sample([p for p, r in enumerate(ref.refs) if r == 0], 50):
        ref.refs[p] = 1  # held by a table of another kind
    g = Gpu(ref, caches=False)
    for _ in range(2):
        grow = [rng.choice([0, 64, 400, 500, 500]) for _ in range(batch)]
        g.extend(grow)
        bad = ref.extend(grow)
        torch.cuda.synchronize()
        g.same(ref)
        g.error(bad)


def test_lengths_up_to_the_largest():
    """2^31 - 1 tokens: the pages of such a length, its free and its compaction, and no growth past it."""
    from decode_attention_06_b200 import gqla
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    most, width = (1 << 31) - 1, 1 << 25
    table = torch.full((2, width), 3, dtype=torch.int32, device="cuda")
    table[1, 0] = 2
    lens, refs, ws = i32([most, 5]), i32([0, 0, 1, width, 0]), gqla.new_workspace()
    pool = gqla.make_page_pool(table, lens, refs)
    gqla.gqla_extend_sequences(pool, i32([1, 1]), ws)
    torch.cuda.synchronize()
    assert lens.tolist() == [most, 6] and refs.tolist() == [0, 0, 1, width, 0]
    assert gqla.gqla_read_device_error(ws) == (-5, 0)
    gqla.gqla_clear_device_error(ws)
    pairs, counts = i32([[9, 9]] * 2), i32([0, 0])
    gqla.gqla_compact_pages(pool, table, refs, pairs, counts, ws)
    torch.cuda.synchronize()
    assert counts.tolist() == [2, 2] and pairs.tolist() == [[2, 0], [3, 1]]
    assert refs.tolist() == [1, width, 0, 0, 0] and bool((table[0] == 1).all()) and int(table[1, 0]) == 0
    gqla.gqla_free_sequences(pool, i32([0]), ws)
    torch.cuda.synchronize()
    assert lens.tolist() == [0, 6] and refs.tolist() == [1, 0, 0, 0, 0]
    assert gqla.gqla_read_device_error(ws)[0] == 0


def test_copy_pages_in_more_than_one_round():
    """More pieces than the CTAs take in one round of 256 each (about 37900 on 148 SMs), with pairs that
    are skipped or clash strewn among them, so that the rounds hold uneven counts."""
    pages, groups, n = 2400, 8, 1100  # 42 pieces a pair
    g = Gpu(Pool(1, 1, pages), groups)
    rng = random.Random(77)
    order = rng.sample(range(pages), 2 * n + 60)
    good = [(order[2 * i], order[2 * i + 1]) for i in range(n)]
    spare = order[2 * n:]
    clash = [(spare[2 * i], spare[40 + i % 20]) for i in range(20)]  # targets named twice below
    clash += [(spare[2 * i + 1], spare[40 + i % 20]) for i in range(20)]
    listed = good + clash + [(-1, 3)] * 150 + [(7, 7)] * 100
    rng.shuffle(listed)
    want = copied((g.latent, g.kv, g.rope), groups, good)
    for _ in range(2):
        g.copy(torch.tensor(listed, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    g.error([i for i, p in enumerate(listed) if p in clash])
    for got, exp in zip((g.latent, g.kv, g.rope), want):
        assert torch.equal(got, exp)

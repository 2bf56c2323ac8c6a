"""The paged cache on the GPU: its pages against a model on the host, its
attention against plain attention in 64 bits, and a serving run of all of it."""
import itertools
import math
import random

import pytest

from int4_quantized_attention_b200 import api, build
from serve_reference import D, check, paged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return api.lib()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """The page operations by their definition, one page after another."""

    def __init__(self, cache):
        self.cache, p = cache, cache.p
        self.page, self.n = p.page_size, p.n_pages
        self.rows = [[] for _ in range(p.max_seqs)]
        self.lens = [0] * p.max_seqs
        self.refs = [0] * p.n_pages
        self.pool = cache.pool.clone()

    def lowest(self):
        return self.refs.index(0)

    def extend(self, seqs, new):
        for s, m in zip(seqs, new):
            if s < 0:
                continue
            while len(self.rows[s]) * self.page < self.lens[s] + m:
                x = self.lowest()
                self.rows[s].append(x)
                self.refs[x] = 1
            self.lens[s] += m

    def write(self, layer, seqs, counts, k, v):
        at = 0
        for s, m in zip(seqs, counts):
            for t in range(m):
                if s >= 0:
                    pos = self.lens[s] - m + t
                    x = self.rows[s][pos // self.page]
                    self.pool[0, layer, x, :, pos % self.page] = k[at + t]
                    self.pool[1, layer, x, :, pos % self.page] = v[at + t]
            at += m

    def fork(self, parents, children):
        for a, b in zip(parents, children):
            if b < 0:
                continue
            full, rest = divmod(self.lens[a], self.page)
            self.rows[b], self.lens[b] = self.rows[a][:full], self.lens[a]
            if rest:
                x = self.lowest()
                self.rows[b].append(x)
                self.pool[:, :, x, :, :rest] = self.pool[:, :, self.rows[a][full], :, :rest]
            for x in self.rows[b]:
                self.refs[x] += 1

    def free(self, seqs):
        for s in seqs:
            if s < 0:
                continue
            for x in self.rows[s]:
                self.refs[x] -= 1
            self.rows[s], self.lens[s] = [], 0

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        holes = [i for i in range(n) if self.refs[i] == 0]
        movers = [i for i in range(n, self.n) if self.refs[i] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.pool[:, :, b] = self.pool[:, :, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[to.get(x, x) for x in r] for r in self.rows]

    def same(self, pool=True):
        c = self.cache
        c.check()
        assert c.refs.tolist() == self.refs
        assert c.lens.tolist() == self.lens
        table = c.table.tolist()
        for got, want in zip(table, self.rows):
            assert got == want + [-1] * (len(got) - len(want))
        if pool:
            assert torch.equal(c.pool.view(torch.int16), self.pool.view(torch.int16))


def make(layers=1, n_pages=40, page=16, hkv=2, max_seqs=8, max_pages=12, dtype=F16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = torch.randn(2, layers, n_pages, hkv, page, D, generator=g, device="cuda").to(dtype)
    c = api.PagedCache(layers, n_pages, page, hkv, max_seqs, max_pages, dtype=dtype, pool=pool)
    return c, Model(c)


def rand(seed, *shape, dtype=F16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_extend_write_free(page):
    c, m = make(layers=2, page=page, hkv=3)
    m.same()
    seqs, new = [3, -1, 0, 7], [page + 5, 9, 1, 0]
    c.extend(ints(seqs), ints(new))
    m.extend(seqs, new)
    m.same()
    total = sum(new)
    k, v = rand(1, total, 3, D), rand(2, 3, total, D).transpose(0, 1)
    cu = [0] + list(itertools.accumulate(new))
    c.write(1, ints(seqs), k, v, cu_new=ints(cu))
    m.write(1, seqs, new, k, v)
    m.same()
    for step in range(2 * page // 3):
        c.extend(ints([0, 3]), ints([1, 1]))
        m.extend([0, 3], [1, 1])
        k, v = rand(3 + step, 2, 3, D), rand(90 + step, 2, 3, D)
        c.write(0, ints([0, 3]), k, v)
        m.write(0, [0, 3], [1, 1], k, v)
    m.same()
    c.free(ints([3, -1, 7]))
    m.free([3, 7])
    m.same()
    c.extend(ints([5]), ints([2 * page + 1]))          # takes the lowest free pages again
    m.extend([5], [2 * page + 1])
    m.same()


@pytest.mark.parametrize("page,dtype", [(16, F16), (128, BF16)])
def test_fork_and_compact(page, dtype):
    c, m = make(layers=3, n_pages=60, page=page, hkv=2, max_seqs=10, max_pages=9, dtype=dtype)
    lens = [3 * page + 7, page, 1, 0]
    c.extend(ints([0, 1, 2, 3]), ints(lens))
    m.extend([0, 1, 2, 3], lens)
    parents, children = [0, 0, 1, 2, 3, 0], [4, 5, 6, 7, 8, -1]
    c.fork(ints(parents), ints(children))
    m.fork(parents, children)
    m.same()
    c.extend(ints([4, 0, 6]), ints([page, 3, 1]))      # copies and parent part
    m.extend([4, 0, 6], [page, 3, 1])
    m.same()
    c.free(ints([0, 7]))                               # shared pages stay with the children
    m.free([0, 7])
    m.same()
    c.compact()
    m.compact()
    m.same()
    c.compact()                                        # nothing left to move
    m.same()
    c.free(ints(list(range(10))))
    m.free(range(10))
    c.compact()
    m.same()


def test_random_run():
    rng = random.Random(7)
    c, m = make(layers=1, n_pages=300, page=16, hkv=1, max_seqs=40, max_pages=30)
    for step in range(60):
        busy = [i for i in range(40) if m.lens[i]]
        empty = [i for i in range(40) if not m.lens[i]]
        room = 300 - sum(r > 0 for r in m.refs)
        do = rng.choice(["extend", "extend", "fork", "free", "compact"])
        if do == "extend":
            seqs = rng.sample(range(40), rng.randint(1, 8))
            new = [rng.randint(0, min(90, 30 * 16 - m.lens[s])) for s in seqs]
            if sum(n // 16 + 1 for n in new) > room:
                continue
            c.extend(ints(seqs), ints(new))
            m.extend(seqs, new)
        elif do == "fork" and busy and empty:
            kids = rng.sample(empty, min(len(empty), rng.randint(1, 6)))
            if len(kids) > room:
                continue
            dads = [rng.choice(busy) for _ in kids]
            c.fork(ints(dads), ints(kids))
            m.fork(dads, kids)
        elif do == "free" and busy:
            seqs = rng.sample(busy, rng.randint(1, len(busy)))
            c.free(ints(seqs))
            m.free(seqs)
        elif do == "compact":
            c.compact()
            m.compact()
        m.same(pool=step % 10 == 9)
    m.same()


def test_large_state():
    # more pages than the state cluster has threads, long rows, a wide list
    n = 20000
    c, m = make(n_pages=n, page=16, hkv=1, max_seqs=700, max_pages=400)
    seqs = list(range(0, 700, 2))
    new = [(i * 37) % 800 for i in seqs]
    c.extend(ints(seqs), ints(new))
    m.extend(seqs, new)
    kids = list(range(1, 700, 2))
    c.fork(ints(seqs), ints(kids))
    m.fork(seqs, kids)
    gone = list(range(0, 700, 3))
    c.free(ints(gone))
    m.free(gone)
    m.same()
    c.compact()
    m.compact()
    m.same()


def refused(c, m, status, call):
    before = c.state.clone()
    call()
    with pytest.raises(api.RotateAttnError) as e:
        c.check()
    assert e.value.status == status
    assert torch.equal(c.state, before)
    m.same()


def test_refused_calls_change_nothing():
    c, m = make(n_pages=10, page=16, max_seqs=6, max_pages=7)
    c.extend(ints([0, 1]), ints([40, 20]))              # 3 + 2 pages of 10
    m.extend([0, 1], [40, 20])
    bounds, full = api.RA_ERR_DEVICE_BOUNDS, api.RA_ERR_CACHE_FULL
    refused(c, m, bounds, lambda: c.extend(ints([2, 2]), ints([1, 1])))
    refused(c, m, bounds, lambda: c.extend(ints([6]), ints([1])))
    refused(c, m, bounds, lambda: c.extend(ints([-2]), ints([1])))
    refused(c, m, bounds, lambda: c.extend(ints([2, 3]), ints([5, -1])))
    refused(c, m, full, lambda: c.extend(ints([2]), ints([6 * 16])))            # 6 pages, 5 are free
    refused(c, m, full, lambda: c.extend(ints([2, 3]), ints([48, 33])))
    refused(c, m, full, lambda: c.extend(ints([0]), ints([2 ** 31 - 1])))       # a row of 7 pages at most
    refused(c, m, full, lambda: c.extend(ints([0]), ints([7 * 16 - 40 + 1])))
    refused(c, m, bounds, lambda: c.fork(ints([0, 0]), ints([2, 2])))
    refused(c, m, bounds, lambda: c.fork(ints([0]), ints([0])))
    refused(c, m, bounds, lambda: c.fork(ints([0, 2]), ints([2, 3])))           # a child that is a parent
    refused(c, m, bounds, lambda: c.fork(ints([0]), ints([1])))                 # not empty
    refused(c, m, bounds, lambda: c.fork(ints([9]), ints([2])))
    refused(c, m, bounds, lambda: c.fork(ints([-1]), ints([2])))
    refused(c, m, bounds, lambda: c.free(ints([0, 1, 0])))
    refused(c, m, bounds, lambda: c.free(ints([0, 77])))
    c.extend(ints([2]), ints([5 * 16 - 1]))
    m.extend([2], [5 * 16 - 1])
    refused(c, m, full, lambda: c.fork(ints([0]), ints([3])))                   # no page for its last tokens
    c.fork(ints([3]), ints([4]))                                                # an empty sequence needs none
    c.extend(ints([2]), ints([1]))
    m.extend([2], [1])
    m.same()
    k = rand(5, 3, 2, D)
    refused(c, m, bounds, lambda: c.write(0, ints([4]), k[:1], k[:1]))          # a row without the token
    with pytest.raises(api.RotateAttnError):
        c.write(1, ints([0]), k[:1], k[:1])
    with pytest.raises(api.RotateAttnError):
        c.write(0, ints([0]), k[:1, :1], k[:1, :1])
    with pytest.raises(api.RotateAttnError):
        c.extend(torch.tensor([0], device="cuda"), ints([1]))
    with pytest.raises(api.RotateAttnError):
        c.attention(0, k.float(), ints([0]))


@pytest.mark.parametrize("rows,tokens", [(3, 1), (3, 40), (3, 400), (300, 1), (300, 2)])
def test_refused_writes_change_nothing(rows, tokens):
    # short and long lists, few and many tokens: beside a bad entry nothing of the good ones is written
    c, m = make(n_pages=rows * 27, page=16, max_seqs=rows + 2, max_pages=27)
    every = list(range(rows))
    c.extend(ints(every), ints([tokens + 5] * rows))
    m.extend(every, [tokens + 5] * rows)
    k, v = rand(5, rows * tokens, 2, D), rand(6, rows * tokens, 2, D)
    cu = [i * tokens for i in range(rows + 1)]

    def write(seqs, offsets=cu):
        single = tokens == 1 and offsets is cu
        c.write(0, ints(seqs), k, v, cu_new=None if single else ints(offsets))

    def with_entry(values, i, x):
        return values[:i] + [x] + values[i + 1:]

    bounds = api.RA_ERR_DEVICE_BOUNDS
    for i in (0, rows // 2, rows - 1):
        for bad in (every[i - 1], rows + 2, -2, 2 ** 31 - 1, rows):         # twice, outside, a row without tokens
            refused(c, m, bounds, lambda: write(with_entry(every, i, bad)))
        for bad in (-1, -2 ** 31, 2 ** 31 - 1, rows * tokens + 1):
            refused(c, m, bounds, lambda: write(every, with_entry(cu, i, bad)))
    refused(c, m, bounds, lambda: write(every, with_entry(cu, 1, cu[2] + 1)))
    refused(c, m, bounds, lambda: write(every, cu[:-1] + [rows * tokens + 1]))
    refused(c, m, bounds, lambda: write(every, [0] * rows + [tokens + 6]))  # longer than the row
    last = (tokens + 5 - 1) // 16
    keep = int(c.table[rows - 1, last])
    for bad in (-1, c.p.n_pages, 2 ** 31 - 1):
        c.table[rows - 1, last] = bad
        m.rows[rows - 1][last] = bad
        before = c.pool.clone()
        write(every)
        with pytest.raises(api.RotateAttnError) as e:
            c.check()
        assert e.value.status == bounds and torch.equal(c.pool, before)
    c.table[rows - 1, last] = m.rows[rows - 1][last] = keep
    some = with_entry(every, 1, -1)                     # a padded list, whose tokens of the entry are passed over
    write(some)
    m.write(0, some, [tokens] * rows, k, v)
    m.same()
    write(every)
    m.write(0, every, [tokens] * rows, k, v)
    m.same()
    inner = [1] + [min(2 + i * tokens, rows * tokens - 1) for i in range(rows)]   # tokens outside the offsets
    c.write(0, ints(every), k, v, cu_new=ints(inner))
    for r, (a, b) in enumerate(zip(inner, inner[1:])):
        m.write(0, [r], [b - a], k[a:b], v[a:b])
    m.same()
    c.write(0, ints(every), k[:0], v[:0], cu_new=ints([0] * (rows + 1)))
    m.same()
    refused(c, m, bounds, lambda: c.write(0, ints(every), k[:0], v[:0], cu_new=ints([0] * rows + [1])))


@pytest.mark.parametrize("kids,pages", [(1, 2), (2, 90), (300, 2)])
def test_writes_do_not_reach_shared_pages(kids, pages):
    # the last tokens of a row lie in full pages that its forks share: neither side may overwrite them
    page = 16
    c, m = make(n_pages=pages + 3 * kids + 10, page=page, max_seqs=kids + 3, max_pages=pages + 2)
    n = pages * page
    children = list(range(1, kids + 1))
    c.extend(ints([0, kids + 1]), ints([n, 5]))
    m.extend([0, kids + 1], [n, 5])
    c.fork(ints([0] * kids), ints(children))
    m.fork([0] * kids, children)
    bounds = api.RA_ERR_DEVICE_BOUNDS
    k, v = rand(5, 2 * n, 2, D), rand(6, 2 * n, 2, D)
    for row in (0, 1, kids):
        for count in (1, page, page + 1, n):
            refused(c, m, bounds, lambda: c.write(0, ints([kids + 1, row]), k[:2 + count], v[:2 + count],
                                                  cu_new=ints([0, 2, 2 + count])))
        refused(c, m, bounds, lambda: c.write(0, ints([row]), k[:1], v[:1]))
    # what was written behind the fork is each row's own; a token further back is not
    every = [0] + children
    c.extend(ints(every), ints([3] * len(every)))
    m.extend(every, [3] * len(every))
    cu = [3 * i for i in range(len(every) + 1)]
    kk, vv = rand(7, cu[-1] + 1, 2, D), rand(8, cu[-1] + 1, 2, D)
    c.write(0, ints(every), kk[:-1], vv[:-1], cu_new=ints(cu))
    m.write(0, every, [3] * len(every), kk, vv)
    m.same()
    refused(c, m, bounds, lambda: c.write(0, ints(every), kk, vv, cu_new=ints(cu[:-1] + [cu[-1] + 1])))
    # the last row that still names the pages may write them
    c.free(ints(every[:-1]))
    m.free(every[:-1])
    c.write(0, ints([kids]), k[:n + 3], v[:n + 3], cu_new=ints([0, n + 3]))
    m.write(0, [kids], [n + 3], k, v)
    m.same()


def full(c, status=api.RA_ERR_CACHE_FULL):
    with pytest.raises(api.RotateAttnError) as e:
        c.check()
    assert e.value.status == status


@pytest.mark.parametrize("many", [1, 300])
def test_writes_behind_a_refused_extend(many):
    # the tokens had no slots: nothing of the row's own is overwritten, whatever else the stream does
    page, rows = 16, many + 5
    c, m = make(layers=2, n_pages=3 * rows - 1, page=page, max_seqs=rows, max_pages=3 * rows)
    c._work[256:] = 0x77
    every = list(range(rows - 1))                           # the last row stays empty
    c.extend(ints(every), ints([40] * len(every)))
    m.extend(every, [40] * len(every))                      # 3 pages of a row, 2 are left
    for layer in range(2):
        k, v = rand(layer, 40 * len(every), 2, D), rand(9 + layer, 40 * len(every), 2, D)
        c.write(layer, ints(every), k, v, cu_new=ints([40 * i for i in range(rows)]))
        m.write(layer, every, [40] * len(every), k, v)
    m.same()
    a, b = every[:many], every[many:]                       # two lists of a step; the first wants too much
    k, v = rand(20, many * 9, 2, D), rand(21, many * 9, 2, D)
    write = lambda seqs, n=1: c.write(1, ints(seqs), k[:n * len(seqs)], v[:n * len(seqs)], cu_new=None if n == 1 else   # noqa: E731
                                      ints([n * i for i in range(len(seqs) + 1)]))
    c.extend(ints(a), ints([50] * many))                         # 3 more each
    c.extend(ints(b), ints([1] * len(b)))
    m.extend(b, [1] * len(b))
    write(a)
    write(a, 9)
    k2, v2 = rand(22, len(b) + many, 2, D), rand(23, len(b) + many, 2, D)
    c.write(1, ints(a + b), k2, v2)                         # one list with both
    m.write(1, [-1] * many + b, [1] * len(every), k2, v2)
    full(c)
    m.same()
    # once read, the error holds nothing back: the last token may be written again
    write(a)
    m.write(1, a, [1] * many, k, v)
    m.same()
    # a second refusal holds its own rows alone
    c.extend(ints([b[0]]), ints([2 ** 20]))
    write(a)
    write([b[0]])
    m.write(1, a, [1] * many, k, v)
    full(c)
    m.same()
    # so does one for another reason
    c.extend(ints([b[0], b[0]]), ints([1, 1]))
    write([b[0]])
    full(c, api.RA_ERR_DEVICE_BOUNDS)
    m.same()
    # an extend that is carried out gives the row its slots; the error stands until it is read
    c.extend(ints([b[0], b[1], rows - 1]), ints([2 ** 20, 0, 0]))
    c.extend(ints([b[0]]), ints([2]))
    write([b[0]], 2)
    write([b[1]])
    m.extend([b[0]], [2])
    m.write(1, [b[0]], [2], k, v)
    # so do a free and a fork
    c.free(ints([b[1]]))
    m.free([b[1]])
    c.fork(ints([b[0]]), ints([rows - 1]))
    m.fork([b[0]], [rows - 1])
    write([rows - 1])
    m.write(1, [rows - 1], [1], k, v)
    full(c)
    m.same()


@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1, 7 * 16 + 1])
def test_compact_beside_a_row_of_unknown_length(bad):
    # its pages would move and its table row would not follow
    c, m = make(n_pages=20, page=16, max_seqs=4, max_pages=7)
    c.extend(ints([0, 1, 2]), ints([50, 30, 70]))
    m.extend([0, 1, 2], [50, 30, 70])
    c.free(ints([0]))
    m.free([0])
    keep, m.lens[2] = int(c.lens[2]), bad
    c.lens[2] = bad
    refused(c, m, api.RA_ERR_DEVICE_BOUNDS, c.compact)
    c.lens[2] = m.lens[2] = keep
    c.compact()
    m.compact()
    m.same()


def test_a_state_that_counts_no_references():
    # a program that lays out the table itself and leaves refs at 0: attention and writes need none
    c, m = make(n_pages=9, page=16, max_seqs=2, max_pages=4)
    c.table[0, :3] = ints([7, 2, 5])
    c.lens[0] = 41
    m.rows[0], m.lens[0] = [7, 2, 5], 41
    for tokens in (1, 41):
        k, v = rand(1, tokens, 2, D), rand(2, tokens, 2, D)
        c.write(0, ints([0]), k, v, cu_new=ints([0, tokens]))
        m.write(0, [0], [tokens], k, v)
    m.same()
    run_attention(c, m, [0], [1], 4, 0)


def test_captured_step_on_a_full_cache():
    # extend and write in one graph: replays beyond the last page leave the cache as it was
    c, m = make(n_pages=4, page=16, max_seqs=2, max_pages=4)
    c.extend(ints([0, 1]), ints([30, 30]))
    m.extend([0, 1], [30, 30])
    s, one, k, v = ints([0, 1]), ints([1, 1]), rand(1, 2, 2, D), rand(2, 2, 2, D)

    def step():
        c.extend(s, one)
        c.write(0, s, k, v)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(2):
        k.copy_(rand(30 + r, 2, 2, D))
        graph.replay()
        m.extend([0, 1], [1, 1])
        m.write(0, [0, 1], [1, 1], k, v)
        m.same()
    for r in range(3):
        k.copy_(rand(40 + r, 2, 2, D))
        graph.replay()
        if r != 1:                                          # read, or not, before the next replay
            full(c)
            m.same()


# ---------------------------------------------------------------- attention

def filled(lens, shared, page, hkv, dtype, seed, layers=1, nan_tail=True):
    """A cache with len(lens) rows that share their first `shared` tokens; every
    slot that holds no token holds NaN."""
    n = len(lens)
    lead = shared // page
    own = [-(-m // page) for m in lens]
    c, m = make(layers=layers, n_pages=lead + sum(own) + 3, page=page, hkv=hkv, max_seqs=n + 1,
                max_pages=lead + max(own) + 1, dtype=dtype, seed=seed)
    if shared:
        c.extend(ints([n]), ints([shared]))
        m.extend([n], [shared])
        c.fork(ints([n] * n), ints(list(range(n))))
        m.fork([n] * n, list(range(n)))
        c.free(ints([n]))
        m.free([n])
    order = list(range(n))
    random.Random(seed).shuffle(order)
    for i in order:                                     # pages in another order than rows
        c.extend(ints([i]), ints([lens[i]]))
        m.extend([i], [lens[i]])
    if nan_tail:
        held = torch.zeros(c.p.n_pages, page, dtype=torch.bool, device="cuda")
        for r, total in zip(m.rows, m.lens):
            for j, x in enumerate(r):
                held[x, :min(page, total - j * page)] = True
        c.pool.masked_fill_(~held[None, None, :, None, :, None], math.nan)
        m.pool.copy_(c.pool)
    m.same()
    return c, m


def run_attention(c, m, seqs, counts, hq, shared, seed=3, layer=0, scale=None, gain=1.0):
    cu = [0] + list(itertools.accumulate(counts))
    q = gain * rand(seed, cu[-1], hq, D, dtype=c.dtype)
    single = all(x == 1 for x in counts)
    o, lse = c.attention(layer, q, ints(seqs), cu_q=None if single else ints(cu), shared=shared, scale=scale or 0.0,
                         return_lse=True)
    c.check()
    want, wl, tol, tl = paged(c.pool, layer, m.rows, m.lens, q, seqs, cu, scale)
    check(o, want, tol, "o")
    check(lse, wl, tl, "lse")
    return q, cu, o


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (5, 1), (28, 4)])
@pytest.mark.parametrize("shared", [0, 128, 640])
def test_single_tokens(page, dtype, hq, hkv, shared):
    c, m = filled([1, 16, 17, 127, 128, 129, 400, 1000], shared, page, hkv, dtype, seed=page)
    run_attention(c, m, list(range(8)), [1] * 8, hq, shared)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_one_sequence_one_token(dtype):
    c, m = filled([1], 0, 16, 1, dtype, seed=4)
    run_attention(c, m, [0], [1], 1, 0)
    c, m = filled([333], 0, 16, 24, dtype, seed=4)
    run_attention(c, m, [0], [1], 24, 0)


@pytest.mark.parametrize("shared", [0, 256])
def test_several_tokens_each(shared):
    c, m = filled([5, 40, 300, 7], shared, 32, 2, F16, seed=8)
    run_attention(c, m, [2, 0, 3, 1], [3, 5, 0, 33], 6, shared)


def test_prompt_over_the_cache():
    # whole prompts whose keys lie in pages
    c, m = filled([300, 129, 1], 64, 64, 2, BF16, seed=9)
    run_attention(c, m, [0, 1, 2], [300, 129, 1], 8, 64)


def test_same_result_every_time():
    # many full 64-row parts: what one warp still copies or reads must not meet what another lays out
    rng = random.Random(1)
    lens = [rng.randint(1, 3000) for _ in range(90)]
    counts = [rng.choice([0, 1, 1, 2, 5, min(n + 3, 70)]) for n in lens]
    for hq, dtype in ((64, F16), (24, BF16)):
        c, m = filled(lens, 0, 128, 1, dtype, seed=5)
        q, cu, o = run_attention(c, m, list(range(90)), counts, hq, 0)
        for _ in range(30):
            assert torch.equal(c.attention(0, q, ints(list(range(90))), cu_q=ints(cu)), o)


def test_more_query_tokens_than_the_row_holds():
    c, m = filled([3, 70, 2], 0, 16, 2, F16, seed=20)
    q, cu, o = run_attention(c, m, [0, 1, 2], [5, 70, 90], 4, 0)
    assert bool((o[:2] == 0).all()) and bool((o[75:75 + 88] == 0).all())


@pytest.mark.parametrize("shared", [0, 256])
def test_many_heads_per_key_head(shared):
    # more rows per token than the kernel of few rows takes
    c, m = filled([1, 130, 700], shared, 32, 1, BF16, seed=21)
    run_attention(c, m, [0, 1, 2], [1, 1, 1], 128, shared)
    run_attention(c, m, [0, 1, 2], [1, 3, 2], 72, shared)


def test_rows_behind_the_last_sequence_stay():
    for shared in (0, 64):
        c, m = filled([30, 200], shared, 16, 2, F16, seed=22)
        q = rand(3, 40, 4, D)
        out = torch.full((40, 4, D), 3.0, device="cuda", dtype=F16)
        lse = torch.full((40, 4), 5.0, device="cuda")
        c.attention(0, q, ints([0, 1]), cu_q=ints([0, 2, 25]), shared=shared, out=out, lse=lse)
        c.check()
        assert bool((out[25:] == 3).all()) and bool((lse[25:] == 5).all())
        want, wl, tol, tl = paged(c.pool, 0, m.rows, m.lens, q[:25], [0, 1], [0, 2, 25])
        check(out[:25], want, tol, "o")
        check(lse[:25], wl, tl, "lse")


def test_every_row_shorter_than_the_shared_part():
    c, m = filled([30, 60, 9], 128, 16, 1, F16, seed=23, nan_tail=False)
    for i, n in enumerate((40, 100, 0)):
        c.lens[i] = n
        m.lens[i], m.rows[i] = n, m.rows[i][:-(-n // 16)]
    run_attention(c, m, [0, 1, 2], [1, 1, 1], 2, 128)
    run_attention(c, m, [2, 0, 1], [1, 40, 3], 2, 128)


def test_strided_queries_and_outputs():
    c, m = filled([30, 200, 5], 32, 16, 2, BF16, seed=24)
    big = rand(3, 3, 10, D, dtype=BF16)
    q = big[:, 1:9]                                     # heads 1 to 8 of 10
    out = torch.full((3, 16, D), 3.0, device="cuda", dtype=BF16)[:, ::2]
    got = c.attention(0, q, ints([0, 1, 2]), shared=32, out=out)
    c.check()
    want, _, tol, _ = paged(c.pool, 0, m.rows, m.lens, q, [0, 1, 2], [0, 1, 2, 3])
    check(got, want, tol, "o")
    headed = rand(3, 8, 3, D, dtype=BF16).transpose(0, 1)   # head-major
    headed.copy_(q)
    assert torch.equal(c.attention(0, headed, ints([0, 1, 2]), shared=32), out)


def test_workspace_content_does_not_matter():
    c, m = filled([30, 200, 700], 128, 16, 2, F16, seed=25)
    q = rand(3, 8, 8, D)
    cu = ints([0, 1, 7, 8])
    want = c.attention(0, q, ints([0, 1, 2]), cu_q=cu, shared=128)
    c._ws.current()[256:] = 0x77
    c._work[256:] = 0x77
    assert torch.equal(c.attention(0, q, ints([0, 1, 2]), cu_q=cu, shared=128), want)
    c.extend(ints([1]), ints([40]))
    m.extend([1], [40])
    c.fork(ints([1, 0]), ints([3, -1]))
    m.fork([1], [3])
    c.free(ints([0]))
    m.free([0])
    c.compact()
    m.compact()
    m.same()


def test_growing_while_capturing_is_refused():
    c, m = filled([30], 0, 16, 2, F16, seed=26)
    q, row = rand(3, 1, 4, D), ints([0])
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(api.RotateAttnError):
        with torch.cuda.graph(graph):
            c.attention(0, q, row)
    torch.cuda.synchronize()
    run_attention(c, m, [0], [1], 4, 0)


def test_padded_and_repeated_rows():
    c, m = filled([30, 200], 32, 16, 2, F16, seed=10)
    q, cu, o = run_attention(c, m, [-1, 1, 0, 1, -1], [1] * 5, 4, 32)
    assert bool((o[0] == 0).all()) and bool((o[4] == 0).all())
    run_attention(c, m, [-1, -1], [1, 1], 4, 32)
    run_attention(c, m, [2, 0], [1, 1], 4, 32)          # row 2 is empty


def test_row_shorter_than_the_shared_part():
    # a batch may hold a row that ends inside the shared pages
    c, m = filled([30, 60], 64, 16, 1, F16, seed=12, nan_tail=False)
    c.lens[0] = 40
    m.lens[0], m.rows[0] = 40, m.rows[0][:3]
    q = rand(3, 2, 2, D)
    o, lse = c.attention(0, q, ints([0, 1]), shared=64, return_lse=True)
    c.check()
    want, wl, tol, tl = paged(c.pool, 0, m.rows, m.lens, q, [0, 1], [0, 1, 2])
    check(o, want, tol, "o")
    check(lse, wl, tl, "lse")


@pytest.mark.parametrize("hq,hkv", [(16, 1), (64, 8)])
def test_wide_batch_long_prefix(hq, hkv):
    rng = random.Random(3)
    lens = [rng.randint(1, 300) for _ in range(150)]
    c, m = filled(lens, 4096, 128, hkv, BF16, seed=13)
    run_attention(c, m, list(range(150)), [1] * 150, hq, 4096)


def test_time_rises_with_the_shared_part_and_does_not_jump():
    # long own parts behind shared parts of any length: never the few SMs that a shared part would leave, but
    # half of them or all, so at most twice the time that they take after a longer shared part
    rows, own, page, longest = 25, 8000, 64, 8192
    pages = -(-own // page)
    c = api.PagedCache(1, longest // page + rows * pages, page, 8, rows, longest // page + pages, dtype=BF16)
    c.pool.normal_()
    q, s = rand(1, rows, 40, D, dtype=BF16), ints(list(range(rows)))
    at = torch.arange(rows * pages, device="cuda", dtype=torch.int32).view(rows, pages) + longest // page

    def took(shared):
        lead = shared // page
        c.table.fill_(-1)
        c.table[:, :lead] = torch.arange(lead, device="cuda", dtype=torch.int32)
        c.table[:, lead:lead + pages] = at
        c.lens.fill_(shared + own)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                c.attention(0, q, s, shared=shared)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[1:])

    whole = took(longest)                               # about 0.2 ms a call
    for shared in (128, 1024, 1984, 2304, 3008, 3392, 3520, 4096, 5120, 6144, 6912, 7040, 7104):
        assert took(shared) < 2 * whole, shared
    c.check()


@pytest.mark.parametrize("shared", [0, 2048])
def test_nan_queries_and_hidden_values(shared):
    # drafted tokens: a value that only the later ones see; a NaN query beside others
    c, m = filled([700, 40, 5], shared, 16, 2, BF16, seed=18)
    own = [m.rows[i][(shared + n - 1) // 16] for i, n in ((0, 700), (1, 40))]
    c.pool[1, 0, own[0], 1, (shared + 699) % 16, 3] = math.inf       # the last token's value
    c.pool[1, 0, own[1], 0, (shared + 39) % 16, 100] = math.nan
    q = rand(4, 9, 8, D, dtype=BF16)
    q[8, 5, 0] = math.nan
    cu = [0, 4, 8, 9]
    o, lse = c.attention(0, q, ints([0, 1, 2]), cu_q=ints(cu), shared=shared, return_lse=True)
    c.check()
    assert bool(torch.isnan(o[8, 5]).all()) and bool(torch.isnan(lse[8, 5]))
    q[8, 5, 0] = 0.0
    o[8, 5], lse[8, 5] = 0.0, 0.0
    want, wl, tol, tl = paged(c.pool, 0, m.rows, m.lens, q, [0, 1, 2], cu)
    want[8, 5], wl[8, 5] = 0.0, 0.0
    assert int((~torch.isfinite(want)).sum()) == 8                   # one channel of the 4 heads of two tokens
    check(o, want, tol, "o")
    check(lse, wl, tl, "lse")


@pytest.mark.parametrize("first_short", [True, False])
def test_infinities_in_the_shared_part_beside_shorter_rows(first_short):
    # rows that end inside the shared pages beside rows that see a value of infinity there with a weight that
    # vanishes: the same result every time, whichever query tile comes first
    n, shared, page = 64, 512, 16                       # 4 heads per key head: 32 tokens are a query tile
    c, m = filled([5] * n, shared, page, 1, BF16, seed=27, nan_tail=False)
    short = [i for i in range(n) if (i < 32) == first_short]
    for i in short:
        c.lens[i] = 100
        m.lens[i], m.rows[i] = 100, m.rows[i][:7]
    q = rand(4, n, 4, D, dtype=BF16).abs()
    for tile in range(1, 4):                            # in each tile that only the longer rows see
        where = c.table[short[0] ^ 32, (128 * tile + 40) // page].long(), (128 * tile + 40) % page
        c.pool[0, 0, where[0], 0, where[1]] = -30.0     # scores below -1000
        c.pool[1, 0, where[0], 0, where[1], 10 * tile] = math.inf
    cu = list(range(n + 1))
    want, wl, tol, tl = paged(c.pool, 0, m.rows, m.lens, q, list(range(n)), cu)
    assert int((want == math.inf).sum()) == 3 * 32 * 4
    for _ in range(20):
        o, lse = c.attention(0, q, ints(list(range(n))), shared=shared, return_lse=True)
        c.check()
        check(o, want, tol, "o")
        check(lse, wl, tl, "lse")


def test_layers_scale_and_peaked_scores():
    c, m = filled([500, 3], 128, 64, 2, F16, seed=14, layers=3)
    run_attention(c, m, [0, 1], [1, 1], 4, 128, layer=2, scale=0.5, gain=10.0)
    run_attention(c, m, [0, 1], [1, 1], 4, 128, layer=1, gain=0.0)


def test_bad_pages_are_reported():
    c, m = filled([100, 50], 0, 16, 1, F16, seed=15)
    q = rand(3, 2, 1, D)
    good = c.attention(0, q, ints([0, 1]))
    for bad in (-1, c.p.n_pages, 2 ** 30, -2 ** 31):
        keep = int(c.table[0, 2])
        c.table[0, 2] = bad
        o = c.attention(0, q, ints([0, 1]))
        with pytest.raises(api.RotateAttnError) as e:
            c.check()
        assert e.value.status == api.RA_ERR_DEVICE_BOUNDS
        assert torch.equal(o[1], good[1])
        c.table[0, 2] = keep
    for seqs in ([7, 1], [-5, 1]):
        o = c.attention(0, q, ints(seqs))
        with pytest.raises(api.RotateAttnError):
            c.check()
        assert torch.equal(o[1], good[1]) and bool((o[0] == 0).all())
    c.lens[0] = 10 ** 6
    c.attention(0, q, ints([0, 1]))
    with pytest.raises(api.RotateAttnError):
        c.check()
    c.lens[0] = 100
    assert torch.equal(c.attention(0, q, ints([0, 1])), good)
    c.check()


@pytest.mark.parametrize("shared", [0, 128])
@pytest.mark.parametrize("hq", [2, 64])
def test_a_bad_query_offset_is_reported(shared, hq):
    n = 150
    c, m = filled([50 + i % 9 for i in range(n)], shared, 16, 2, F16, seed=28)
    seqs, counts = list(range(n)), [1 + i % 3 for i in range(n)]
    cu = [0] + list(itertools.accumulate(counts))
    q = rand(3, cu[-1], hq, D)
    for at in (1, n // 2, n - 1, n):
        for bad in (-1, -2 ** 31, cu[at - 1] - 1, cu[-1] + 1, 2 ** 31 - 1):
            c.attention(0, q, ints(seqs), cu_q=ints(cu[:at] + [bad] + cu[at + 1:]), shared=shared)
            with pytest.raises(api.RotateAttnError) as e:
                c.check()
            assert e.value.status == api.RA_ERR_DEVICE_BOUNDS
    run_attention(c, m, seqs, counts, hq, shared)


@pytest.mark.parametrize("shared", [0, 32])
def test_lengths_near_the_largest_int_are_reported(shared):
    # a length that no table row holds leaves the sequence out, also where one page more passes 2^31
    c, m = filled([100, 50], shared, 16, 1, F16, seed=15)
    q = rand(3, 2, 1, D)
    want, wl, tol, tl = paged(c.pool, 0, m.rows, m.lens, q, [-1, 1], [0, 1, 2])
    for bad in (2 ** 31 - 1, 2 ** 31 - 14, 2 ** 31 - 16, 2 ** 30, c.p.max_pages * 16 + 1, -1, -2 ** 31):
        c.lens[0] = bad
        for cu in (None, ints([0, 1, 2])):
            o, lse = c.attention(0, q, ints([0, 1]), cu_q=cu, shared=shared, return_lse=True)
            with pytest.raises(api.RotateAttnError) as e:
                c.check()
            assert e.value.status == api.RA_ERR_DEVICE_BOUNDS
            check(o, want, tol, "o")                    # row 0: zeros, -inf
            check(lse, wl, tl, "lse")
        before = c.state.clone()
        c.free(ints([0]))
        with pytest.raises(api.RotateAttnError):
            c.check()
        assert torch.equal(c.state, before)


def test_a_pool_past_32_bit_offsets():
    # the last pages of a 9 GB pool: element offsets pass 2^32
    n = 1 << 16
    c = api.PagedCache(1, n, 128, 2, 2, 8, dtype=F16)
    row = [n - 1, 5, n - 2, n - 3]
    for j, x in enumerate(row):
        c.table[0, j] = x
        c.refs[x] = 1
    c.lens[0] = 3 * 128 + 40
    k, v = rand(1, 424, 2, D), rand(2, 424, 2, D)
    c.write(0, ints([0]), k, v, cu_new=ints([0, 424]))
    q = rand(3, 1, 4, D)
    o, lse = c.attention(0, q, ints([0]), return_lse=True)
    c.check()
    want, wl, tol, tl = paged(c.pool, 0, [row], [424], q, [0], [0, 1])
    check(o, want, tol, "o")
    c.compact()
    c.check()
    assert sorted(c.table[0, :4].tolist()) == [0, 1, 2, 3]
    assert torch.equal(c.attention(0, q, ints([0])), o)


def test_serving_run():
    """A prompt is read, its continuations fork, decode with the shared part
    read once, some end, the cache is compacted and decoding goes on: each
    step's attention against 64 bits, the state against the model."""
    hq, hkv, page, dtype = 8, 2, 16, BF16
    c, m = make(layers=2, n_pages=200, page=page, hkv=hkv, max_seqs=9, max_pages=40, dtype=dtype)
    op = api.PackedAttention()
    n = 16 * page + 5
    c.extend(ints([0]), ints([n]))
    m.extend([0], [n])
    for layer in range(2):
        k, v = rand(layer, n, hkv, D, dtype=dtype), rand(10 + layer, n, hkv, D, dtype=dtype)
        c.write(layer, ints([0]), k, v, cu_new=ints([0, n]))
        m.write(layer, [0], [n], k, v)
        q = rand(20 + layer, n, hq, D, dtype=dtype)
        # the prompt over its own keys, packed, is the prompt over the pages
        o = op.forward(q, k, v, ints([0, n]), ints([0, n]))
        cu = [0, n]
        o2 = c.attention(layer, q, ints([0]), cu_q=ints(cu))
        want, _, tol, _ = paged(c.pool, layer, m.rows, m.lens, q, [0], cu)
        check(o, want, tol, "packed")
        check(o2, want, tol, "paged")
    kids = [1, 2, 3, 4, 5]
    c.fork(ints([0] * 5), ints(kids))
    m.fork([0] * 5, kids)
    alive = [0] + kids
    for step in range(20):
        if step == 8:
            c.free(ints([0, 2]))
            m.free([0, 2])
            alive = [1, 3, 4, 5]
            c.compact()
            m.compact()
        s = ints(alive)
        c.extend(s, ints([1] * len(alive)))
        m.extend(alive, [1] * len(alive))
        for layer in range(2):
            k, v = (rand(100 * step + 10 * layer + x, len(alive), hkv, D, dtype=dtype) for x in (1, 2))
            c.write(layer, s, k, v)
            m.write(layer, alive, [1] * len(alive), k, v)
            run_attention(c, m, alive, [1] * len(alive), hq, 16 * page, seed=step, layer=layer)
        m.same()
    op.check()


def test_captured_decode_step():
    # extend, write, attention in one graph; replays go on from the state they find
    c, m = filled([20, 31, 100], 32, 16, 2, F16, seed=16)
    s, one = ints([0, 1, 2]), ints([1, 1, 1])
    k, v, q = rand(1, 3, 2, D), rand(2, 3, 2, D), rand(3, 3, 4, D)
    out, lse = torch.empty(3, 4, D, device="cuda", dtype=F16), torch.empty(3, 4, device="cuda")

    def step():
        c.extend(s, one)
        c.write(0, s, k, v)
        c.attention(0, q, s, shared=32, out=out, lse=lse)

    def model():
        m.extend([0, 1, 2], [1, 1, 1])
        m.write(0, [0, 1, 2], [1, 1, 1], k, v)

    step()
    model()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        k.copy_(rand(50 + r, 3, 2, D))
        q.copy_(rand(60 + r, 3, 4, D))
        graph.replay()
        model()
        m.same()
        want, wl, tol, tl = paged(c.pool, 0, m.rows, m.lens, q, [0, 1, 2], [0, 1, 2, 3])
        check(out, want, tol, "o")
        check(lse, wl, tl, "lse")

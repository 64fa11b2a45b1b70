"""The paged cache through what a serving loop does between its steps: rows cut
back to less than they were forked with. Every output is compared with the same
attention over contiguous caches that hold each row's own tokens; pages, counts
and tables have to be equal to a sequential model's."""

import numpy as np
import pytest
import torch

from online_kv_cache_quantize_gb300 import binding as B
from test_gpu_pages import Model, _contents, _gpu, _pool, _same, _ws

pytestmark = pytest.mark.gpu

# Both sides read the same codes and add the same fp32 terms, at most a few hundred of unit scale, in another
# order: each is rounded to 2^-24 or split in fp16 halves to 2^-22, which stays far below this.
TOL = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_kv_cache_quantize_gb300 import build
    build.build()


def _rand(r, *shape):
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).cuda().to(torch.bfloat16)


class Histories:
    """Contiguous caches with a row per sequence, whose tokens come and go on their own."""

    def __init__(self, paged, cap):
        self.p, self.cap, self.n = paged, cap, [0] * paged.batch
        self.k = B.Cache("prod", 3, 128, rows=paged.batch * paged.hkv, capacity=cap)
        self.v = B.Cache("mse", 3, 128, rows=paged.batch * paged.hkv, capacity=cap)

    def append(self, k, v, count=None):
        """k, v [batch, hkv, C, 128]; the first count[b] tokens (all) go to row b."""
        c = k.shape[2]
        count = [c] * len(self.n) if count is None else count
        slots = np.full((len(self.n), self.p.hkv, c), -1, dtype=np.int64)
        for b, n in enumerate(self.n):
            for h in range(self.p.hkv):
                slots[b, h, :count[b]] = (b * self.p.hkv + h) * self.cap + n + np.arange(count[b])
            self.n[b] += count[b]
        s = torch.from_numpy(slots.reshape(-1)).cuda()
        B.tq_quantize_kv(self.k, self.p.rot, k.reshape(-1, 128), qjl=self.p.qjl, dst_slot=s)
        B.tq_quantize_kv(self.v, self.p.rot, v.reshape(-1, 128), dst_slot=s)

    def fork(self, parent):
        for p in (self.k.codes, self.k.signs, self.k.norm, self.k.rnorm, self.v.codes, self.v.norm):
            x = p.view(len(self.n), -1)
            x.copy_(x[torch.tensor([max(i, 0) for i in parent], device="cuda")].clone())
        self.n = [self.n[i] if i >= 0 else 0 for i in parent]

    def attend(self, q):
        out = torch.empty(q.shape, device="cuda")
        a = (q, self.k, self.v, torch.tensor(self.n, dtype=torch.int32, device="cuda"), max(max(self.n), 1), self.p.rot,
             self.p.qjl, out)
        view = B.View(self.p.window, self.p.sinks)
        B.tq_attn_decode_view(*a, B.workspace(B.tq_attn_decode_view_workspace(*a, view)), view)
        return out

    def step(self, r, hq):
        """One step of both: the paged cache's output must be this one's."""
        q, k, v = _rand(r, len(self.n), hq, 128), _rand(r, len(self.n), self.p.hkv, 128), _rand(r, len(self.n), self.p.hkv, 128)
        out = self.p.step(q, k, v)
        self.append(k[:, :, None], v[:, :, None])
        err = float((out - self.attend(q)).abs().max())
        assert err <= TOL, err
        assert self.p.lengths.tolist() == self.n


def _counts_match(p):
    t = p.table[p.table >= 0].cpu().numpy()
    assert np.array_equal(np.bincount(t, minlength=p.pool.n_pages), p.pool.refs.cpu().numpy())


# ------------------------------------------- rows that go back below a fork ---
@pytest.mark.parametrize("short", [0, 3, 4])
@pytest.mark.parametrize("page,hkv", [(16, 2), (208, 8)])
def test_reserve_copies_a_shared_last_page(page, hkv, short):
    """Rows whose tokens go on in the middle of a shared page take a copy, in row order with the other requests;
    a full shared page, a page of one holder and rows that add nothing keep theirs. Without a free page the
    entry is empty, and counted."""
    pool = _pool(9 - short, hkv=hkv, page=page, seed=5)
    t = np.array([[3, 4, -1], [3, 4, 1], [3, 4, -1], [0, 4, -1], [3, 2, -1], [3, 4, -1]], dtype=np.int32)
    lengths = np.array([page + 5, page + 9, 2 * page, page - 1, page + 3, 2 * page - 1])
    add = np.array([2, 1, 1, 1, page, 0])
    m = Model(9 - short, page)
    for e in t[t >= 0]:
        m.refs[e] += 1
    pool.refs.copy_(_gpu(m.refs))
    data, refs0, free, lost = _contents(pool), m.refs.copy(), m.free(), 0
    want = t.copy()
    for b in range(len(t)):
        if not add[b]:
            continue
        for j in range(lengths[b] // page, -(-(lengths[b] + add[b]) // page)):
            e = t[b, j]
            own = j == lengths[b] // page and lengths[b] % page and e >= 0 and refs0[e] > 1
            if e >= 0 and not own:
                continue
            got = m.take(free)
            want[b, j] = got
            lost += got < 0
            if got >= 0:
                m.refs[got] = 1
            if own:
                m.refs[e] -= 1
                if got >= 0:
                    data[got] = data[e]
    assert lost == short
    table, word = _gpu(t), torch.full((1,), 9, dtype=torch.int32, device="cuda")
    B.tq_pages_reserve(pool, table, _gpu(lengths), _gpu(add), _ws(pool, len(t)), shortage=word)
    _same(pool, m, ("table", table, want), ("shortage", word, [lost]))
    assert np.array_equal(_contents(pool), data)


@pytest.mark.parametrize("back", [[77, 77, 77], [77, 88, 64], [88, 3, 85], [0, 88, 16]])
@pytest.mark.parametrize("again", [False, True])
def test_rows_go_back_below_a_fork(back, again):
    """A prompt of 80 tokens forked to every row, some tokens each, then rows cut back into pages that they
    share (all of them, some, to a page's start, to nothing), and different tokens from there on; also
    forked again before they go on."""
    r = np.random.default_rng(sum(back))
    hq, hkv = 4, 2
    p = B.PagedKVCache(3, hq, hkv, n_pages=40, max_tokens=160, page=16)
    ref = Histories(p, 160)
    q, k, v = _rand(r, 3, 80, hq, 128), _rand(r, 3, hkv, 80, 128), _rand(r, 3, hkv, 80, 128)
    p.prefill_chunk(q, k, v)
    ref.append(k, v)
    p.fork(_gpu([1, 1, 1]))
    ref.fork([1, 1, 1])
    for _ in range(8):
        ref.step(r, hq)
    p.rollback(_gpu(back))
    ref.n = list(back)
    if again:
        p.fork(_gpu([0, 0, 1]))
        ref.fork([0, 0, 1])
    for _ in range(20):
        ref.step(r, hq)
    assert int(p.shortage) == 0
    _counts_match(p)
    p.rollback(torch.zeros_like(p.lengths))
    assert int(p.pool.refs.abs().sum()) == 0


def test_chunk_below_a_fork():
    """The same for a chunk of tokens."""
    r = np.random.default_rng(1)
    p = B.PagedKVCache(2, 4, 2, n_pages=20, max_tokens=96, page=16)
    ref = Histories(p, 96)
    k, v = _rand(r, 2, 2, 40, 128), _rand(r, 2, 2, 40, 128)
    p.prefill_chunk(_rand(r, 2, 40, 4, 128), k, v)
    ref.append(k, v)
    p.fork(_gpu([0, 0]))
    ref.fork([0, 0])
    p.rollback(_gpu([20, 21]))
    ref.n = [20, 21]
    k, v = _rand(r, 2, 2, 33, 128), _rand(r, 2, 2, 33, 128)
    p.prefill_chunk(_rand(r, 2, 33, 4, 128), k, v)
    ref.append(k, v)
    ref.step(r, 4)
    _counts_match(p)


# --------------------------------------------------- more tokens than pages ---
def _lossy_step(p, ref, r, hq, stored):
    """A step of which row b keeps its token where stored[b] == 1."""
    q, k, v = _rand(r, len(ref.n), hq, 128), _rand(r, len(ref.n), p.hkv, 128), _rand(r, len(ref.n), p.hkv, 128)
    out = p.step(q, k, v)
    ref.append(k[:, :, None], v[:, :, None], stored)
    assert p.lengths.tolist() == ref.n
    err = float((out - ref.attend(q)).abs().max())
    assert err <= TOL, err


@pytest.mark.parametrize("window", [0, 40])
def test_steps_without_a_free_page(window):
    """Tokens that found no page are lost, counted, and never replaced by what a page held before: once there are
    pages again, the rows go on behind the tokens they have."""
    r = np.random.default_rng(3)
    p = B.PagedKVCache(3, 4, 2, n_pages=7, max_tokens=160, page=16, window=window)
    ref = Histories(p, 160)
    k, v = _rand(r, 3, 2, 30, 128), _rand(r, 3, 2, 30, 128)
    p.prefill_chunk(_rand(r, 3, 30, 4, 128), k, v)
    ref.append(k, v)
    for _ in range(2):
        _lossy_step(p, ref, r, 4, [1, 1, 1])
    assert int(p.shortage) == 0
    for i in range(3):  # one page for three rows
        _lossy_step(p, ref, r, 4, [1, 0, 0])
        assert int(p.shortage) == 2 * (i + 1)
    p.rollback(_gpu([0, 500, 500]))  # three pages with another row's tokens
    ref.n[0] = 0
    for _ in range(12):
        _lossy_step(p, ref, r, 4, [1, 1, 1])
    assert int(p.shortage) == 6
    _counts_match(p)


def test_chunk_without_enough_pages():
    """A chunk of which only the first tokens find pages keeps those."""
    r = np.random.default_rng(4)
    p = B.PagedKVCache(3, 4, 2, n_pages=7, max_tokens=160, page=16)
    ref = Histories(p, 160)
    for c, stored in ((10, [10, 10, 10]), (50, [50, 22, 6]), (5, [4, 0, 0])):
        k, v = _rand(r, 3, 2, c, 128), _rand(r, 3, 2, c, 128)
        p.prefill_chunk(_rand(r, 3, c, 4, 128), k, v)
        ref.append(k, v, stored)
        assert p.lengths.tolist() == ref.n
    p.rollback(_gpu([0, 500, 500]))
    ref.n[0] = 0
    for _ in range(9):
        _lossy_step(p, ref, r, 4, [1, 1, 1])
    _counts_match(p)


def test_fork_without_a_free_page():
    """Children whose copy of the half-filled page found no page go on from the page's start."""
    r = np.random.default_rng(5)
    p = B.PagedKVCache(4, 4, 2, n_pages=14, max_tokens=96, page=16)
    ref = Histories(p, 96)
    k, v = _rand(r, 4, 2, 42, 128), _rand(r, 4, 2, 42, 128)
    p.prefill_chunk(_rand(r, 4, 42, 4, 128), k, v)  # 12 of 14 pages
    ref.append(k, v)
    p.fork(_gpu([2, 2, 2, 2]))  # three copies, two pages
    assert int(p.shortage) == 1
    ref.fork([2, 2, 2, 2])
    ref.n = [42, 42, 42, 32]
    assert p.lengths.tolist() == ref.n
    for _ in range(9):
        _lossy_step(p, ref, r, 4, [1, 1, 1, 1])
    assert int(p.shortage) == 1
    _counts_match(p)


def test_a_copy_without_a_free_page():
    """Rows back below their fork that find no page for a copy of their last one lose its tokens, and are cut."""
    r = np.random.default_rng(12)
    p = B.PagedKVCache(3, 4, 2, n_pages=8, max_tokens=96, page=16)
    ref = Histories(p, 96)
    k, v = _rand(r, 3, 2, 32, 128), _rand(r, 3, 2, 32, 128)
    p.prefill_chunk(_rand(r, 3, 32, 4, 128), k, v)
    ref.append(k, v)
    p.fork(_gpu([0, 0, 2]))
    ref.fork([0, 0, 2])
    p.rollback(_gpu([26, 20, 32]))  # both in the shared second page
    ref.n = [26, 20, 32]
    others = p.pool.refs == 0
    p.pool.refs[others] = 1  # somebody else's
    ref.n = [16, 16, 32]
    _lossy_step(p, ref, r, 4, [0, 0, 0])
    assert int(p.shortage) == 3
    p.pool.refs[others] = 0
    for _ in range(16):
        _lossy_step(p, ref, r, 4, [1, 1, 1])
    assert int(p.shortage) == 3
    # 32, 32 and 48 tokens: a shared page, two of their own and three are in use, two are left for three rows
    for _ in range(4):
        _lossy_step(p, ref, r, 4, [1, 1, 0])
    assert int(p.shortage) == 7
    _counts_match(p)


def test_a_page_taken_for_lost_tokens_is_cleared():
    """An entry filled in the middle of its page: the tokens before are zero vectors, not what the page held."""
    for mode in ("prod", "polar"):
        pool = _pool(6, hkv=2, page=32, seed=6, mode=mode)
        table = _gpu([[0, -1], [-1, -1], [-1, 9]])
        pool.refs[0] = 1
        before = _contents(pool)
        granted = _gpu([7] * 3)
        B.tq_pages_reserve(pool, table, _gpu([45, 5, 64]), _gpu([20, 2, 3]), _ws(pool, 3), granted=granted)
        assert table.tolist() == [[0, 1], [2, -1], [-1, 9]]
        assert granted.tolist() == [19, 2, 0]
        planes = [pool.k.norm, pool.k.rnorm, pool.v.norm] if mode == "prod" else [pool.k.norm, pool.v.norm]
        for x in planes:
            x = x.view(6, 2, 32)
            assert torch.all(x[1, :, :13] == 0) and torch.all(x[2, :, :5] == 0)
            x[1, :, :13] = x[2, :, :5] = 1
        want = torch.from_numpy(before)
        got = torch.from_numpy(_contents(pool))
        same = (want == got).all(dim=1)
        assert same.tolist() == [True, False, False, True, True, True]
        # nothing else of the two pages changed
        assert int((want != got).sum()) <= len(planes) * 2 * 2 * (13 + 5)


def test_granted_tokens():
    """granted is the row's tokens that lie in pages it holds, from the first on."""
    pool = _pool(5, hkv=1, page=16)
    table = _gpu([[0, -1, -1], [-1, -1, 1], [2, -1, -1], [-1, -1, -1]])
    pool.refs[:3] = 1
    granted = _gpu([9] * 4)
    add = _gpu([40, 48, 6, 0])
    B.tq_pages_reserve(pool, table, _gpu([10, -3, 16, 5]), add, _ws(pool, 4), granted=granted)
    # free: 3, 4. Row 0 takes both (tokens 10 .. 47 of 10 .. 49); rows 1 and 2 find none
    assert table.tolist() == [[0, 3, 4], [-1, -1, 1], [2, -1, -1], [-1, -1, -1]]
    assert granted.tolist() == [38, 0, 0, 0]
    # no page for the rows' own last tokens: an empty entry, and a shared page that finds no copy
    table = _gpu([[0, -1], [-1, -1], [1, -1], [1, -1]])
    pool.refs.copy_(_gpu([1, 2, 1, 1, 1]))
    B.tq_pages_reserve(pool, table, _gpu([15, 5, 9, 16]), _gpu([3, 20, 1, 2]), _ws(pool, 4), granted=granted)
    assert granted.tolist() == [1, -5, -9, 0] and table.tolist() == [[0, -1], [-1, -1], [-1, -1], [1, -1]]
    assert pool.refs.tolist() == [1, 1, 1, 1, 1]


# -------------------------------------------------- captured calls and others ---
def _captured(p, r, hq):
    """A step captured with inputs of its own, and a function that replays it with new ones on both sides."""
    bufs = [_rand(r, p.batch, hq, 128), _rand(r, p.batch, p.hkv, 128), _rand(r, p.batch, p.hkv, 128)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = p.step(*bufs)

    def replay(ref):
        for b in bufs:
            b.copy_(_rand(r, *b.shape))
        g.replay()
        ref.append(bufs[1][:, :, None], bufs[2][:, :, None])
        err = float((out - ref.attend(bufs[0])).abs().max())
        assert err <= TOL, err
        assert p.lengths.tolist() == ref.n

    return replay


def test_a_fork_between_replays():
    """A captured step goes on from what a fork, a rollback and a compaction made of the rows since."""
    r = np.random.default_rng(6)
    p = B.PagedKVCache(3, 4, 2, n_pages=30, max_tokens=128, page=16)
    ref = Histories(p, 128)
    k, v = _rand(r, 3, 2, 20, 128), _rand(r, 3, 2, 20, 128)
    p.prefill_chunk(_rand(r, 3, 20, 4, 128), k, v)
    ref.append(k, v)
    ref.step(r, 4)
    replay = _captured(p, r, 4)
    replay(ref)
    for parent in ([2, 2, 0], [1, 0, 0], [0, 1, 2]):
        p.fork(_gpu(parent))
        ref.fork(parent)
        for _ in range(9):
            replay(ref)
        p.compact()
    p.rollback(_gpu([30, 40, 8]))
    ref.n = [30, 40, 8]
    for _ in range(5):
        replay(ref)
    _counts_match(p)


def test_calls_on_a_stream_of_their_own():
    """Every call on a side stream that is behind, while the stream of the constructor takes and gives back
    memory: nothing that the queued work still reads may have moved or gone."""
    r = np.random.default_rng(9)
    p = B.PagedKVCache(2, 4, 2, n_pages=24, max_tokens=128, page=16)
    ref = Histories(p, 128)
    at = (p.table.data_ptr(), p.lengths.data_ptr())
    xs = [(_rand(r, 2, 4, 128), _rand(r, 2, 2, 128), _rand(r, 2, 2, 128)) for _ in range(20)]
    k, v = _rand(r, 2, 2, 30, 128), _rand(r, 2, 2, 30, 128)
    q = _rand(r, 2, 30, 4, 128)
    forks = [_gpu([1, 1]), _gpu([1, 0])]
    back = _gpu([33, 20])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    p.prefill_chunk(q, k, v, stream=s)
    for i, x in enumerate(xs):
        outs.append(p.step(*x, stream=s))
        if i in (4, 12):
            p.fork(forks[i == 12], stream=s)
        if i == 8:
            p.rollback(back, stream=s)
        junk = [torch.full((n,), 0x7FFFFFFF, dtype=torch.int32, device="cuda") for n in (2, 2, 16, 16, 512)]
        del junk
    s.synchronize()
    ref.append(k, v)
    for i, x in enumerate(xs):
        ref.append(x[1][:, :, None], x[2][:, :, None])
        assert float((outs[i] - ref.attend(x[0])).abs().max()) <= TOL, i
        if i in (4, 12):
            ref.fork(forks[i == 12].tolist())
        if i == 8:
            ref.n = [33, 20]
    assert p.lengths.tolist() == ref.n and at == (p.table.data_ptr(), p.lengths.data_ptr())


def test_steps_outside_after_replays():
    """rollback's at_most says how long the rows are then; replays make them longer, and a step outside sees it."""
    r = np.random.default_rng(7)
    p = B.PagedKVCache(2, 4, 2, n_pages=20, max_tokens=128, page=16)
    ref = Histories(p, 128)
    ref.step(r, 4)
    replay = _captured(p, r, 4)
    for _ in range(30):
        replay(ref)
    p.rollback(_gpu([25, 11]), at_most=25)
    ref.n = [25, 11]
    ref.step(r, 4)
    for _ in range(40):
        replay(ref)
    ref.step(r, 4)
    k, v = _rand(r, 2, 2, 5, 128), _rand(r, 2, 2, 5, 128)
    p.prefill_chunk(_rand(r, 2, 5, 4, 128), k, v)
    ref.append(k, v)
    ref.step(r, 4)


def test_a_captured_rollback_has_not_run():
    r = np.random.default_rng(8)
    p = B.PagedKVCache(2, 4, 2, n_pages=20, max_tokens=128, page=16)
    ref = Histories(p, 128)
    for _ in range(20):
        ref.step(r, 4)
    to = _gpu([10, 10])
    p.rollback(_gpu([20, 20]))  # outside first
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.rollback(to, at_most=10)
    ref.step(r, 4)  # 21 tokens
    g.replay()
    ref.n = [10, 10]
    ref.step(r, 4)


# -------------------------------------------------------- windowed rollback ---
@pytest.mark.parametrize("window,sinks,keep", [(20, 0, 24), (33, 5, 16), (16, 20, 40), (1, 0, 8)])
def test_windowed_rollback_keeps_what_the_window_reaches(window, sinks, keep):
    """Drafts of up to max_rollback tokens, of which some are dropped: every query sees all tokens of its window."""
    r = np.random.default_rng(window)
    p = B.PagedKVCache(2, 4, 2, n_pages=2 * (5 + (window + keep) // 16), max_tokens=512, page=16, window=window, sinks=sinks,
                       max_rollback=keep)
    ref = Histories(p, 512)
    for _ in range(12):
        c = int(r.integers(1, keep + 1))
        k, v = _rand(r, 2, 2, c, 128), _rand(r, 2, 2, c, 128)
        p.prefill_chunk(_rand(r, 2, c, 4, 128), k, v)
        ref.append(k, v)
        to = [n - int(r.integers(0, c + 1)) for n in ref.n]
        p.rollback(_gpu(to))
        ref.n = to
        ref.step(r, 4)
    assert int(p.shortage) == 0
    _counts_match(p)


def test_windowed_rollback_past_the_margin_is_counted():
    """Pages of the new window that are already gone count as shortage; freeing a row does not."""
    r = np.random.default_rng(2)
    p = B.PagedKVCache(2, 4, 2, n_pages=20, max_tokens=256, page=16, window=32)
    ref = Histories(p, 256)
    k, v = _rand(r, 2, 2, 100, 128), _rand(r, 2, 2, 100, 128)
    p.prefill_chunk(_rand(r, 2, 100, 4, 128), k, v)  # tokens 64 .. stay
    ref.append(k, v)
    p.rollback(_gpu([98, 0]))
    assert int(p.shortage) == 0 and p.lengths.tolist() == [98, 0]
    p.rollback(_gpu([70, 0]))  # sees 38 .. 69: pages 2 and 3 are gone
    assert int(p.shortage) == 2 and p.lengths.tolist() == [70, 0]
    p.rollback(_gpu([41, 0]))  # the page it would go on in is gone: on from its start
    assert p.lengths.tolist() == [32, 0]
    ref.n = [0, 0]
    p.rollback(_gpu([0, 0]))
    ref.step(r, 4)
    _counts_match(p)


def test_a_workspace_that_grows_on_another_stream():
    """The workspace that a larger call replaces is not given to others while a stream still has work that uses it."""
    r = np.random.default_rng(10)
    p = B.PagedKVCache(2, 4, 2, n_pages=40, max_tokens=256, page=16)
    ref = Histories(p, 256)
    ref.step(r, 4)  # the workspace belongs to this stream
    old = p._ws.data_ptr()
    size = p._ws.numel()
    x = [_rand(r, 2, 4, 128), _rand(r, 2, 2, 128), _rand(r, 2, 2, 128)]
    k, v, q = _rand(r, 2, 2, 200, 128), _rand(r, 2, 2, 200, 128), _rand(r, 2, 200, 4, 128)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    out = p.step(*x, stream=s)
    p.prefill_chunk(q, k, v, stream=s)
    assert p._ws.data_ptr() != old
    if not s.query():  # the step has not run yet
        taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
        assert all(t.data_ptr() != old for t in taken)
    s.synchronize()
    ref.append(x[1][:, :, None], x[2][:, :, None])
    assert float((out - ref.attend(x[0])).abs().max()) <= TOL


# ------------------------------------------------------------------ inputs ---
def test_strided_inputs_are_copied():
    """Slices of a packed projection give what contiguous inputs give."""
    r = np.random.default_rng(11)
    a, b = (B.PagedKVCache(2, 4, 2, n_pages=20, max_tokens=64, page=16) for _ in range(2))
    x = _rand(r, 2, 7, 8, 128)  # [batch, tokens, q heads, k heads, v heads]
    q, k, v = x[:, :, :4], x[:, :, 4:6].transpose(1, 2), x[:, :, 6:].transpose(1, 2)
    assert torch.equal(a.prefill_chunk(q, k, v), b.prefill_chunk(q.contiguous(), k.contiguous(), v.contiguous()))
    y = _rand(r, 2, 8, 256)
    q, k, v = y[:, :4, :128], y[:, 4:6, :128], y[:, 6:, 128:]
    assert torch.equal(a.step(q, k, v), b.step(q.contiguous(), k.contiguous(), v.contiguous()))
    y = _rand(r, 2, 128, 8).transpose(1, 2)  # heads inside
    assert torch.equal(a.step(y[:, :4], y[:, 4:6], y[:, 6:]),
                       b.step(*(t.contiguous() for t in (y[:, :4], y[:, 4:6], y[:, 6:]))))


def test_inputs_refused_before_anything_changes():
    p = B.PagedKVCache(2, 4, 2, n_pages=20, max_tokens=64, page=16)
    z = lambda *s, dtype=torch.float32, device="cuda": torch.zeros(s, dtype=dtype, device=device)
    q, k, v = z(2, 4, 128), z(2, 2, 128), z(2, 2, 128)
    bad = [(z(2, 8, 128), k, v), (z(1, 4, 128), k, v), (q, z(2, 4, 128), v), (q, k, z(2, 2, 64)), (q, k, v.bfloat16()),
           (q.half(), k, v), (q, k.half(), v.half()), (q.cpu(), k, v), (q, k.cpu(), v.cpu()), (q, k, v, z(2, 4, 64)),
           (q, k, v, z(2, 4, 128, dtype=torch.float16)), (q, k, v, z(2, 4, 256)[..., :128]), (q, k, v, z(2, 4, 128).cpu())]
    for args in bad:
        with pytest.raises(ValueError):
            p.step(*args)
    q, k, v = z(2, 5, 4, 128), z(2, 2, 5, 128), z(2, 2, 5, 128)
    for args in [(z(2, 5, 8, 128), k, v), (q, z(2, 2, 4, 128), v), (q.half(), k, v), (q, k, v.bfloat16()), (q, k.cpu(), v.cpu()),
                 (q, k, v, z(2, 5, 4, 64))]:
        with pytest.raises(ValueError):
            p.prefill_chunk(*args)
    with pytest.raises(ValueError):
        p.rollback(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        p.fork(torch.zeros(2, dtype=torch.int32))
    assert int(p.pool.refs.sum()) == 0 and p.lengths.tolist() == [0, 0] and p._bound == 0


# --------------------------------------------------------------- many rows ---
@pytest.mark.parametrize("rows", [2048, 2049, 5000])
def test_reserve_and_fork_of_many_rows(rows):
    """Beyond a few thousand rows the requests before a row are added up by blocks: the same pages."""
    r = np.random.default_rng(rows)
    n_pages, mp = 3 * rows, 3
    pool = _pool(n_pages, hkv=1)
    m, t = Model(n_pages, 16), np.full((rows, mp), -1, dtype=np.int32)
    lengths = r.integers(0, 30, rows)
    table, short = _gpu(t), torch.zeros(1, dtype=torch.int32, device="cuda")
    zero = np.zeros(rows, dtype=np.int64)
    ws = _ws(pool, 2 * rows)
    B.tq_pages_reserve(pool, table, _gpu(zero), _gpu(lengths), ws, shortage=short)
    want = m.reserve(t, zero, lengths)
    _same(pool, m, ("table", table, t), ("shortage", short, [want]))
    m.data = _contents(pool)
    for keep, children in ((True, rows // 3), (True, 2 * rows), (False, 2 * rows - 7)):
        parent = r.integers(-1, rows + 1, children)
        child, dl = pool.table(children, mp), torch.zeros(children, dtype=torch.int32, device="cuda")
        B.tq_pages_fork(pool, table, child, _gpu(parent), _gpu(lengths), dl, ws, keep_src=keep, shortage=short)
        got = np.full((children, mp), -1, dtype=np.int32)
        wl, ws_short = m.fork(t, got, parent, lengths, keep)
        _same(pool, m, ("src", table, t), ("dst", child, got), ("lengths", dl, wl), ("shortage", short, [ws_short]))
        if keep:
            B.tq_pages_trim(pool, child, torch.zeros_like(dl))
            m.trim(got, np.zeros(children, dtype=np.int64), 0, 0)
    assert np.array_equal(_contents(pool), m.data)


def test_calls_go_to_the_caches_device(monkeypatch):
    """Work for one GPU is not launched while another one is current (nothing is: the check is the host's)."""
    p = B.PagedKVCache(2, 4, 2, n_pages=20, max_tokens=64, page=16)
    x = torch.zeros(2, 4, 128, device="cuda"), torch.zeros(2, 2, 128, device="cuda"), torch.zeros(2, 2, 128, device="cuda")
    p.step(*x)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        p.step(*x)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        B.prepare(B.tq_pages_trim, p.pool, p.table, p.lengths)
    monkeypatch.undo()
    p.step(*x)
    assert p.lengths.tolist() == [2, 2]


def test_captured_chunks_rollbacks_and_compactions():
    """Everything but a fork in graphs, replayed with other inputs and lengths."""
    r = np.random.default_rng(13)
    p = B.PagedKVCache(2, 4, 2, n_pages=24, max_tokens=96, page=16, window=40, sinks=3, max_rollback=8)
    ref = Histories(p, 96 + 64)
    bufs = [_rand(r, 2, 6, 4, 128), _rand(r, 2, 2, 6, 128), _rand(r, 2, 2, 6, 128)]
    to = _gpu([0, 0])

    def run():
        out = p.prefill_chunk(*bufs)
        p.rollback(to)
        p.compact()
        return out

    run()  # outside first, and back to nothing
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for i in range(12):
        for b in bufs:
            b.copy_(_rand(r, *b.shape))
        n = ref.n
        to.copy_(_gpu([n[0] + 6 - i % 3, n[1] + 6 - (i + 1) % 4]))
        g.replay()
        ref.append(bufs[1], bufs[2])
        # the last query of each row sees all of its window
        err = float((out[:, -1] - ref.attend(bufs[0][:, -1].contiguous())).abs().max())
        assert err <= TOL, (i, err)
        ref.n = to.tolist()
        assert p.lengths.tolist() == ref.n
    assert int(p.shortage) == 0
    _counts_match(p)

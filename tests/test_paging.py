"""PagePool against a plain model: every sequence's rows kept as a list of tokens, the pool
as an array that only the returned moves and the appended rows change."""
import random

import pytest

from linear_attention_serving_02_gb300.paging import PagePool


class Model:
    def __init__(self, pages, size):
        self.pool, self.size = PagePool(pages, size), size
        self.rows = [[None] * size for _ in range(pages)]
        self.seqs = {}

    def move(self, moves):
        for a, b in zip(*moves):
            self.rows[b] = list(self.rows[a])

    def append(self, s, tokens):
        self.move(self.pool.grow(s, len(tokens)))
        for t in tokens:
            i = len(self.seqs[s])
            self.rows[self.pool.pages(s)[i // self.size]][i % self.size] = t
            self.seqs[s].append(t)

    def check(self):
        for s, want in self.seqs.items():
            pages = self.pool.pages(s)
            assert self.pool.length(s) == len(want) and len(pages) == -(-len(want) // self.size)
            assert [self.rows[pages[i // self.size]][i % self.size] for i in range(len(want))] == want
        used = {p for s in self.seqs for p in self.pool.pages(s)}
        assert self.pool.free_pages == self.pool.num_pages - len(used)


@pytest.mark.parametrize("seed", range(6))
def test_random_life_of_a_pool(seed):
    r = random.Random(seed)
    m, made, token = Model(40, r.choice([1, 3, 16])), 0, 0
    for _ in range(400):
        do, live = r.choice(["add", "fork", "append", "append", "append", "truncate", "free", "compact"]), list(m.seqs)
        if do == "add":
            m.pool.add(made)
            m.seqs[made] = []
            made += 1
        elif do == "compact":
            src, dst = m.pool.compact()
            assert not set(src) & set(dst) and len(set(dst)) == len(dst) == len(src)
            m.move((src, dst))
            used = {p for s in m.seqs for p in m.pool.pages(s)}
            assert used == set(range(len(used)))
        elif live:
            s = r.choice(live)
            if do == "fork":
                m.pool.fork(s, made)
                m.seqs[made] = list(m.seqs[s])
                made += 1
            elif do == "append":
                n, before = r.randrange(0, 3 * m.size + 1), (m.pool.pages(s), m.pool.free_pages)
                try:
                    m.append(s, list(range(token, token + n)))
                except MemoryError:
                    assert (m.pool.pages(s), m.pool.free_pages) == before
                token += n
            elif do == "truncate":
                n = r.randrange(0, len(m.seqs[s]) + 1)
                m.pool.truncate(s, n)
                del m.seqs[s][n:]
            else:
                m.pool.free(s)
                del m.seqs[s]
        m.check()


def test_rows_written_after_a_truncation_do_not_reach_a_fork():
    """The parent drops half a page that the child still reads, then appends: the page is copied."""
    m = Model(8, 4)
    m.pool.add(0)
    m.seqs[0] = []
    m.append(0, [1, 2, 3, 4, 5, 6])
    m.pool.fork(0, 1)
    m.seqs[1] = list(m.seqs[0])
    m.pool.truncate(0, 2)
    del m.seqs[0][2:]
    m.append(0, [70, 80])
    m.check()


def test_table_and_refusals():
    p = PagePool(4, 16)
    p.add("a")
    p.add("b")
    assert p.grow("a", 17) == ([], [])
    table, lens = p.table(["b", "a"])
    assert table.tolist() == [[-1, -1], [0, 1]] and lens.tolist() == [0, 17]
    assert p.table(["a"], max_pages=3)[0].tolist() == [[0, 1, -1]]
    with pytest.raises(ValueError):
        p.table(["a"], max_pages=1)
    with pytest.raises(MemoryError):
        p.grow("b", 33)
    with pytest.raises(ValueError):
        p.add("a")
    with pytest.raises(ValueError):
        p.truncate("a", 18)
    with pytest.raises(ValueError):
        p.grow("a", -1)
    with pytest.raises(KeyError):
        p.fork("c", "d")
    with pytest.raises(ValueError):
        PagePool(1, 0)


def test_state_slots_of_a_copied_sequence():
    """A KDA state's slot: one page of length 1, never shared by a copy."""
    pool = PagePool(4, 1)
    pool.add("a")
    assert pool.grow("a", 1) == ([], [])
    pool.add("b")
    assert pool.grow("b", 1) == ([], [])
    move = pool.pages("a") + pool.pages("b")  # the pair for kda_pages_copy
    assert len(set(move)) == 2
    pool.free("a")
    assert pool.compact() == ([move[1]], [move[0]]) and pool.pages("b") == [move[0]]

"""Page planning on the GPU against the sequential reference: integers, equal."""
import numpy as np
import pytest
import torch

import exact_attention_13_gb300 as ea
from oracle import kv

pytestmark = pytest.mark.gpu


def setup(rng, B, page, width, free, head, maxlen=None):
    lens = rng.integers(0, (maxlen or width * page) + 1, B)
    table = rng.permutation(B * width).reshape(B, width)
    cap = B * width
    queue = np.full(cap, -7)
    have = -(-lens // page)
    spare = np.concatenate([table[b, have[b]:] for b in range(B)])[:free]
    queue[(head + np.arange(len(spare))) % cap] = spare
    return lens, table, queue, [head, len(spare)]


def compare(lens, new, table, queue, state, page, T):
    cuda = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    tab, que = cuda(table), cuda(queue)
    plan = ea.page_plan(cuda(lens), cuda(new), tab, que, cuda(state), page, T)
    want = kv.page_plan(lens, new, np.asarray(table).tolist(), np.asarray(queue).tolist(), state, page, T)
    got = [*plan, tab, que]
    for name, g, w in zip(("lens", "q_offsets", "positions", "slots", "state", "table", "queue"), got, want):
        assert g.tolist() == w, name
    return got


@pytest.mark.parametrize("B,page,width,free,chunk", [
    (1, 16, 4, 3, 1), (8, 64, 8, 40, 1), (33, 16, 9, 150, 40), (600, 32, 5, 1000, 30),
    (1025, 128, 2, 700, 100), (3, 16, 300, 20, 500), (16384, 16, 2, 9000, 4),
])
def test_against_the_reference(B, page, width, free, chunk):
    rng = np.random.default_rng(B)
    lens, table, queue, state = setup(rng, B, page, width, free, head=(3 * B) % (B * width))
    new = rng.integers(-1, chunk + 1, B)
    total = int(np.maximum(new, 0).sum())
    compare(lens, new, table, queue, state, page, total + 5)
    if total > 3:  # a packed batch smaller than the tokens: what fits is written
        compare(lens, new, table, queue, state, page, total - 3)


def test_refused_requests_and_no_tokens():
    # 0: too wide; 1: takes 2 of 2 pages; 2: refused; 3: fits in its last page; 4: ended
    lens, new = [60, 0, 16, 17, 33], [10, 32, 1, 3, -1]
    table = np.arange(20).reshape(5, 4)
    queue, state = [18, 19] + [-1] * 18, [0, 2]
    got = compare(lens, new, table, queue, state, 16, 50)
    assert got[0].tolist() == [60, 32, 16, 20, 0]
    assert got[3].tolist()[:10] == [-1] * 10 and got[3].tolist()[42] == -1
    assert got[4].tolist() == [2, 3]
    compare([0, 5], [0, 0], np.zeros((2, 1), int), [0], [0, 0], 16, 0)
    compare([0, 5], [-1, -1], np.array([[3], [4]]), [9, 9], [1, 0], 16, 0)


def test_more_tokens_than_32_bits_hold():
    """Beyond the documented sizes, but device data: places are still ones that the request has."""
    big, page, width = 2 ** 31 - 1, 16, 4
    new = [big, 1, 4, big, big, big, 20, 0, 3]
    table = np.arange(100, 100 + 9 * width).reshape(9, width)
    queue = np.arange(40)
    cuda = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    out = ea.page_plan(cuda([5] * 9), cuda(new), cuda(table), cuda(queue), cuda([0, 40]), page, 3000)
    slots = out.slots.cpu().numpy()
    assert set(np.unique(slots[slots >= 0] // page)) <= set(range(40)) | set(range(100, 136))
    assert out.lens.tolist() == [5, 6, 9, 5, 5, 5, 25, 5, 8]


def test_many_steps_keep_every_page_once():
    rng = np.random.default_rng(5)
    B, page, width = 40, 16, 6
    lens, table, queue, state = setup(rng, B, page, width, 10 ** 6, 0)
    for _ in range(6):
        new = rng.integers(-1, 25, B)
        got = compare(lens, new, table, queue, state, page, 1200)
        lens, state, table, queue = got[0].tolist(), got[4].tolist(), got[5].cpu().numpy(), got[6].cpu().numpy()


def test_captured_into_a_graph_and_given_buffers():
    rng = np.random.default_rng(6)
    B, page, width = 5, 32, 6
    lens, table, queue, state = setup(rng, B, page, width, 20, 4, maxlen=40)
    cuda = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    ins = [cuda(x) for x in (lens, [1] * B, table, queue, state)]
    out = ea.page_plan(*ins, page, B)
    with pytest.raises(ea.AttentionError):  # not in place
        ea.page_plan(*ins, page, B, out=out._replace(lens=ins[0]))
    with pytest.raises(ValueError):
        ea.page_plan(*ins, page, B + 1, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ea.page_plan(*ins, page, B, out=out)
        ins[0].copy_(out.lens)
        ins[4].copy_(out.queue_state)
    for step in range(40):
        want = kv.page_plan(ins[0].tolist(), [1] * B, ins[2].tolist(), ins[3].tolist(), ins[4].tolist(), page, B)
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip([*out, ins[2], ins[3]], want):
            assert g.tolist() == w


@pytest.mark.parametrize("cap", [4, 11, 60])
def test_a_ring_without_room_for_every_page_gives_none_twice(cap):
    """Pages come back to a ring that cannot hold them all: some are lost, no page is both free and a
    request's, or free twice."""
    rng = np.random.default_rng(cap)
    B, page, width = 12, 16, 8
    lens, table = rng.integers(0, width * page + 1, B), rng.permutation(B * width).reshape(B, width)
    queue, state = [1000 + i for i in range(cap)], [cap // 2, cap]
    for _ in range(12):
        new = rng.integers(-1, 40, B)
        got = compare(lens, new, table, queue, state, page, 500)
        lens, state = got[0].cpu().numpy(), got[4].tolist()
        table, queue = got[5].cpu().numpy(), got[6].tolist()
        held = [p for b in range(B) for p in table[b, :-(-lens[b] // page)].tolist()]
        idle = [queue[(state[0] + i) % cap] for i in range(state[1])]
        assert len(set(held + idle)) == len(held + idle)


@pytest.mark.parametrize("page", [16, 128])
def test_page_ids_that_no_cache_has_give_no_slot(page):
    """Ids in the table and in the ring whose slots would pass 31 bits and wrap into other pages."""
    last = 2 ** 31 // page - 1  # the last page that slots can name
    bad = [2 ** 32 // page, 2 ** 31 // page, -1, -2 ** 31, 2 ** 31 - 1, last]
    table = np.array([[b, 3, 3] for b in bad] + [[3, 3, 3]])
    lens, new = [5] * len(bad) + [0], [page] * len(bad) + [2 * page]
    got = compare(lens, new, table, bad + [7] * 14, [0, 20], page, sum(new))
    slots = got[3].cpu().numpy()
    assert (slots[:5 * page] == -1).all() and slots.max() == 2 ** 31 - 1


def test_page_sizes_past_32_bits_are_refused():
    cuda = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    args = cuda([0]), cuda([3]), cuda([[0, 0]]), cuda([3, 1]), cuda([0, 2])
    for page in (2 ** 32 + 16, -16, 0):
        with pytest.raises(ValueError):
            ea.page_plan(*args, page, 3)
    assert ea.page_plan(*args, 16, 3).slots.tolist() == [48, 49, 50]

"""The forms of the whole-cache decode over 4 bits, each of them seen to run: how many groups a CTA serves side by
side (four together by TMA, two, or one) is read from what the call leaves in its workspace."""
import pytest
import torch

from block_sparse_gqa_topk_gb300 import _lib, ops
from test_gpu_decode_e2m1 import Batch4, tables  # noqa: F401
from test_gpu_decode_paged import query

pytestmark = pytest.mark.gpu


def decode(batch, q, workspace=None):
    """msa_decode_paged_dense with a workspace that the caller has: o, lse and the groups side by side, the last
    of the B + 2 numbers at the workspace's end."""
    cache, (B, H_q, d) = batch.cache, q.shape
    pages, _ = ops._pages_arg(cache, batch.table, batch.lens_t)
    size = _lib.msa_decode_paged_workspace_size(cache._c, pages, H_q, 0)
    assert size > 0
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    o, lse = torch.empty_like(q), torch.empty(B, H_q, device="cuda")
    ops._call(cache.index, "msa_decode_paged_dense", _lib.msa_decode_paged_dense, cache._c, pages,
              batch.lens_t.data_ptr(), H_q, d ** -0.5, q.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), size)
    at = size - (4 * (B + 2) + 255) // 256 * 256 + 4 * (B + 1)
    return o, lse, ws[at:at + 4].view(torch.int32)


def check(batch, q, groups):
    o, lse, side = decode(batch, q)
    assert ops.device_status() == 0 and int(side) == groups
    batch.check_dense(q, batch.d ** -0.5, o, lse)
    again = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


# The work of one group side by side with none: a sequence's units of 128 tokens and 2 more, times H; two groups
# begin at 48 a CTA, four at 12, of 608 CTAs (304 for more than 8 heads with d = 128).
TWO = [  # d, G, tokens of one sequence and 6 groups, groups side by side
    (64, 2, 4862 * 128, 2), (64, 2, 4861 * 128, 1), (128, 4, 4862 * 128, 2), (128, 4, 4861 * 128, 1),
    (64, 16, 4861 * 128 + 1, 2), (64, 16, 4861 * 128, 1), (128, 11, 2430 * 128, 2), (128, 11, 2429 * 128, 1),
]


@pytest.mark.parametrize("d,G,n,groups", TWO)
def test_two_groups(d, G, n, groups):
    """Both sides of where two groups go side by side."""
    batch = Batch4([n], 128, 6, d, 0, seed=111)
    check(batch, query(1, 6 * G, d, 112), groups)


@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 16), (128, 11)])
def test_two_groups_of_ragged_sequences(d, G):
    """Parts of two groups that begin and end anywhere, pages of half a unit, empty slots, one token."""
    lens = [300007, 1, 0, 345678, 16, 129]
    batch = Batch4(lens, 16, 6, d, 0, seed=113)
    check(batch, query(len(lens), 6 * G, d, 114), 2)


FOUR = [  # d, G, tokens of one sequence and 8 groups, groups side by side
    (64, 2, 910 * 128, 4), (64, 2, 909 * 128, 1), (128, 4, 909 * 128 + 1, 4), (128, 4, 909 * 128, 1),
    (64, 16, 910 * 128, 4), (64, 16, 909 * 128, 1), (128, 11, 454 * 128, 4), (128, 11, 453 * 128, 1),
]


@pytest.mark.parametrize("d,G,n,groups", FOUR)
def test_four_groups(d, G, n, groups):
    """Both sides of where four groups come together."""
    batch = Batch4([n], 128, 8, d, 0, seed=115)
    check(batch, query(1, 8 * G, d, 116), groups)


@pytest.mark.parametrize("d,G", [(128, 4), (64, 2), (128, 16)])
def test_four_groups_on_two_streams_and_in_two_graphs(d, G):
    """Calls whose groups come together, at the same time on two streams and replayed together."""
    batches = [Batch4([90000 + 31 * i, 60001], 64, 8, d, 0, seed=117 + i) for i in range(2)]
    qs = [query(2, 8 * G, d, 119 + i) for i in range(2)]
    want = [decode(batches[i], qs[i]) for i in range(2)]
    assert all(int(w[2]) == 4 for w in want)
    for i in range(2):
        batches[i].check_dense(qs[i], d ** -0.5, *want[i][:2])

    def call(i):
        return ops.msa_decode_paged_dense(qs[i], batches[i].cache, batches[i].table, batches[i].lens_t)

    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(i))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for out in got[i] for x, y in zip(want[i], out))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(i)
        graphs.append((g, out))
    for _, out in graphs:
        for x in out:
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[i], graphs[i][1]))
    assert ops.device_status() == 0


def test_a_replayed_call_follows_the_lengths():
    """A captured call whose lengths change between replays: the form is chosen on the device, so that one graph
    serves one, four groups together, and one again, over the workspace that the others left."""
    d, G, H = 128, 4, 8
    batch = Batch4([131000, 60001], 64, H, d, 0, seed=121)
    q = query(2, H * G, d, 122)
    pages, _ = ops._pages_arg(batch.cache, batch.table, batch.lens_t)
    ws = torch.full((_lib.msa_decode_paged_workspace_size(batch.cache._c, pages, H * G, 0),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    decode(batch, q, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse, side = decode(batch, q, ws)
    for lens, groups in (([131000, 60001], 4), ([700, 0], 1), ([0, 60001], 1), ([100003, 45000], 4), ([1, 1], 1)):
        batch.lens_t.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        assert int(side) == groups
        batch.lens = lens
        batch.check_dense(q, d ** -0.5, o, lse)
        again = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert ops.device_status() == 0

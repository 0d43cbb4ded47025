"""Attention over a paged cache on the GPU (attn_forward through the C ABI) against the float64 oracle, every row, within the bound
derived in attn_util."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
from attn_util import DEV, Batch, TYPES, ints, put, random_tree

pytestmark = pytest.mark.gpu


def show(*a):
    print("attention", *a, flush=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [2, 31, 32, 33], [127, 128, 129, 500], [1, 700, 64, 5]])
def test_single_tokens(dtype, D, lens):
    show("single", dtype, D, lens)
    Batch([1] * len(lens), lens, 8, 2, D, 16, dtype, seed=len(lens) + D).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (3, 1), (16, 2), (12, 12), (34, 2), (65, 1)])
def test_head_layouts(dtype, nq, nkv):
    show("heads", dtype, nq, nkv)
    Batch([1, 3], [40, 150], nq, nkv, 64, 32, dtype, seed=nq).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 2, 8, 64, 1024])
def test_page_sizes(dtype, page):
    show("pages", dtype, page)
    Batch([2, 1, 5], [70, 33, 5], 4, 2, 64, page, dtype, seed=page).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news,lens", [([5], [5]), ([17, 1, 40], [17, 30, 95]), ([130], [201]), ([33, 0, 66], [40, 12, 66])])
def test_prompts(dtype, D, news, lens):
    show("prompts", dtype, D, news, lens)
    Batch(news, lens, 4, 2, D, 16, dtype, seed=D + len(news)).check()


@pytest.mark.parametrize("dtype,D,each", [("bf16", 64, 2), ("bf16", 128, 4), ("bf16", 256, 8), ("f32", 128, 3)])
def test_longer_prompts(dtype, D, each):
    """More rows than a block takes, keys over many tiles, a last tile that is not whole."""
    show("longer", dtype, D, each)
    Batch([300, 77], [431, 300], each, 1, D, 64, dtype, seed=each).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("news", [[1], [7, 2, 31], [64, 33]])
def test_trees(dtype, news):
    show("trees", dtype, news)
    b = Batch(news, [n + 45 * i for i, n in enumerate(news)], 4, 2, 128, 16, dtype, seed=sum(news))
    b.tree = np.concatenate([random_tree(b.rng, n) for n in news])
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype):
    """A mask without a bit and nothing cached; bits past the sequence's new tokens; a sequence shorter than its new tokens."""
    show("nothing", dtype)
    b = Batch([6, 3], [6, 20], 4, 2, 64, 16, dtype, seed=1)
    b.tree = np.array([0, 1, 1 << 40, 4, 2, 63, 0, 1 << 63, 7], dtype=np.uint64)
    got = b.check()
    assert np.all(got[0] == 0) and np.all(got[2] == 0)
    b = Batch([6, 3, 4], [2, 0, -3], 4, 2, 64, 16, dtype, seed=2)
    got = b.check()
    assert np.all(got[:4] == 0) and np.all(got[6:] == 0) and np.any(got[4] != 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("news,lens,tree", [([40], [60], False), ([20], [50], True), ([1], [50], False), ([150], [160], False)])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_unseen_values_that_are_not_finite(dtype, news, lens, tree, what):
    """Keys and values of later tokens, of other branches and behind the end reach no row that does not see them."""
    show("unseen", dtype, news, tree, what)
    b = Batch(news, lens, 8, 2, 64, 16, dtype, seed=5)
    if tree:
        b.tree = random_tree(b.rng, news[0])
    first = lens[0] - news[0]
    clean = b.forward()
    marked = first + news[0] // 2 if news[0] > 1 else None
    for p in range(b.n_pages):                                  # everything that no sequence holds
        if p not in b.table[0]:
            b.pages[p] = what
    last = b.table[0, (lens[0] - 1) // 16]
    if lens[0] % 16:
        b.pages[last, :, :, lens[0] % 16:] = what
    assert np.array_equal(b.forward(), clean)
    if marked is None:
        return
    b.pages[b.table[0, marked // 16], 1, 1, marked % 16, 5] = what
    got = b.check()
    j = marked - first
    seen = (np.arange(news[0]) >= j) if not tree else np.array([(int(m) >> j) & 1 == 1 for m in b.tree])
    assert np.all(~np.isfinite(got[seen][:, 4:, 5])) and np.all(np.isfinite(got[~seen])) and np.array_equal(got[:, :4], clean[:, :4])
    b.pages[b.table[0, marked // 16], 0, 1, marked % 16, 9] = np.nan
    got = b.check()
    assert np.all(np.isnan(got[seen][:, 4:])) and np.all(np.isfinite(got[~seen]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Scores over hundreds: the running maximum is what keeps the exponentials in range."""
    show("large", dtype)
    b = Batch([3, 40], [400, 300], 4, 2, 64, 16, dtype, seed=9, spread=30.0)
    b.check()
    b.scale = -0.5
    b.check()
    b.scale = 0.0
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_and_bounds(dtype):
    """Rows in front of and behind the sequences stay; pages that are not there hold nothing; bounds cut."""
    show("padding", dtype)
    b = Batch([3, 0, 20, 1], [90, 40, 77, 300], 8, 2, 128, 16, dtype, seed=11, first=4, behind=9)
    b.check()
    b.check(new_max=7)
    b.check(len_max=80)
    b.table[0, 1], b.table[2, 0], b.table[3, 18] = -1, b.n_pages, 1 << 30
    b.check()
    b.table[3, :] = -5
    got = b.check()
    assert np.all(got[27] == 0)
    b.lens[2] = 100000                                          # beyond its table
    b.check(len_max=200000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_pages_twice_and_shared(dtype):
    show("shared", dtype)
    b = Batch([1, 1, 2], [100, 100, 64], 8, 2, 64, 16, dtype, seed=13)
    b.table[1] = b.table[0]
    b.table[2, :4] = b.table[0, 3]
    b.q[1] = b.q[0]
    got = b.check()
    assert np.array_equal(got[0], got[1])


def test_split_or_not_and_workspace_contents():
    """Few rows over many keys: the keys are split; what the workspace held does not matter."""
    show("split")
    b = Batch([1, 2], [5000, 3111], 8, 2, 64, 64, "bf16", seed=17)
    first = b.check()
    d = b.desc()
    need = M.attn_workspace_bytes(d, 2, 3, 2, 5000)
    assert need > 0
    ws = torch.full((need,), 0x7f, dtype=torch.uint8, device=DEV)
    assert np.array_equal(b.forward(ws=ws), first) and np.array_equal(b.forward(ws=ws), first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_beyond_32_bits(dtype):
    """Offsets past 4 GiB and past 2^32 elements: the last pages of a large pool."""
    D, nkv, page = 128, 8, 1024
    elems = 2 * nkv * page * D
    n_pages = (1 << 32) // elems + 3
    show("far", dtype, n_pages)
    pages = torch.zeros((n_pages, 2, nkv, page, D), dtype=TYPES[dtype], device=DEV)
    b = Batch([1, 3], [1500, 40], 16, nkv, D, page, dtype, seed=19)
    far = [n_pages - 1, 0, n_pages - 2, n_pages // 2]
    pages[torch.tensor(far[:b.n_pages], device=DEV)] = put(b.pages[:4], dtype)[:b.n_pages]
    table = np.array([[far[p] if p < 4 else -1 for p in row] for row in b.table])
    d = M.attn_desc(16, nkv, D, page, n_pages, b.cols, dtype=dtype)
    ws = torch.empty(M.attn_workspace_bytes(d, 2, 4, 3, 1500), dtype=torch.uint8, device=DEV)
    out = torch.empty((4, 16, D), dtype=TYPES[dtype], device=DEV)
    M.attn_forward(d, 2, 4, 3, 1500, ints(b.cu), ints(b.lens), ints(table), None, put(b.q, dtype), pages, out, ws)
    near = b.forward()
    assert np.array_equal(out.double().cpu().numpy(), near)


def test_streams_and_graphs():
    """On another stream; captured as its first call, replayed with other lengths between eager work."""
    show("graphs")
    b = Batch([1, 4], [700, 333], 8, 2, 128, 16, "bf16", seed=23)
    want = b.forward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert np.array_equal(b.forward(), want)
    d = b.desc()
    cu, lens, table, q, pages = ints(b.cu), ints(b.lens), ints(b.table), put(b.q, "bf16"), put(b.pages, "bf16")
    out = torch.empty((b.N, 8, 128), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(M.attn_workspace_bytes(d, 2, b.N, 4, 700), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.attn_forward(d, 2, b.N, 4, 700, cu, lens, table, None, q, pages, out, ws)
    for step, change in enumerate(([700, 333], [650, 100], [5, 4], [700, 333])):
        lens.copy_(ints(change))
        out.fill_(3.0)
        ws.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        b.lens = change
        assert np.array_equal(out.double().cpu().numpy(), b.forward(new_max=4, len_max=700)), change


def test_launch_timer_counts_the_kernels():
    b = Batch([1], [3000], 8, 2, 128, 16, "bf16", seed=29)
    timer = M.LaunchTimer()
    timer.arm()
    b.forward()
    torch.cuda.synchronize()
    assert timer.n_recorded == 4 and all(t > 0 for t in timer.kernel_us())

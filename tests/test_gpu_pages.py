"""The page operations against plain Python integers, and the blocks they move."""
import numpy as np
import pytest
import torch

import long_context_quantized_b200 as nf
import sessionref as ref

pytestmark = pytest.mark.gpu

FORMATS = [nf.NF_KV_K8V4, nf.NF_KV_K8V8, nf.NF_KV_F8, nf.NF_KV_K4V4, nf.NF_KV_BF16]


def dev(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda").contiguous()


def state(blocks, rows, width, fill, seed=0, shared=0):
    """A consistent random state: rows hold random prefixes of pages."""
    rng = np.random.default_rng(seed)
    table = np.full((rows, width), -1, np.int32)
    ids = list(rng.permutation(blocks))
    for r in range(rows):
        n = int(rng.integers(0, width + 1) * fill)
        for e in range(n):
            if rng.random() < 0.9 and ids:
                table[r, e] = ids.pop()
    for _ in range(shared):
        a, b = rng.integers(0, rows, 2)
        e, f = rng.integers(0, width, 2)
        if table[a, e] >= 0 and table[b, f] < 0:
            table[b, f] = table[a, e]
    refs = np.zeros(blocks, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    return refs, table


def same(refs, table, want, lens=None):
    torch.cuda.synchronize()
    assert table.cpu().tolist() == want.table
    assert refs.cpu().tolist() == want.refs
    if lens is not None:
        assert lens.cpu().tolist() == want.lens


@pytest.mark.parametrize("blocks, rows, width", [(1, 1, 1), (7, 3, 4), (40, 5, 33), (3000, 64, 50), (20000, 1500, 9), (5000, 1, 4500),
                                                 (9000, 3, 8500)])
@pytest.mark.parametrize("seed", [0, 1])
def test_reserve(blocks, rows, width, seed):
    rng = np.random.default_rng(seed + 10)
    refs, table = state(blocks, rows, width, 0.5, seed)
    frm = rng.integers(0, width * 256 + 1, rows)
    to = np.minimum(frm + rng.integers(-300, 256 * 3 if rows > 100 else width * 256, rows), width * 256)
    want = ref.Pages(refs, table)
    want.reserve(frm.tolist(), to.tolist())
    short = any(e < 0 for row, f, t in zip(want.table, frm, to) if f < t for e in row[f // 256:-(-t // 256)])
    r, t = dev(refs), dev(table)
    nf.nf_kv_reserve(r, t, dev(frm), dev(to))
    same(r, t, want)
    assert nf.nf_get_device_error() == (nf.NF_DEVERR_POOL if short else 0)


def test_reserve_more_than_one_round():
    """Above 8192 fresh pages in one call, and a row that spans two rounds."""
    refs, table = np.zeros(20000, np.int32), np.full((3, 7000), -1, np.int32)
    refs[5::7] = 1
    frm, to = [0, 256, 0], [6000 * 256, 6500 * 256 - 3, 700 * 256 + 1]
    want = ref.Pages(refs, table)
    want.reserve(frm, to)
    r, t = dev(refs), dev(table)
    nf.nf_kv_reserve(r, t, dev(frm), dev(to))
    same(r, t, want)
    assert nf.nf_get_device_error() == 0


def test_reserve_errors():
    refs, table = np.zeros(50, np.int32), np.full((4, 3), -1, np.int32)
    r, t = dev(refs), dev(table)
    frm, to = [0, -5, 500, 600], [100, 300, 3000, 300]
    nf.nf_kv_reserve(r, t, dev(frm), dev(to))
    want = ref.Pages(refs, table)
    want.reserve(frm, to)
    same(r, t, want)
    assert nf.nf_get_device_error() == nf.NF_DEVERR_TABLE
    r, t = dev([1, 0, 1, 0]), dev(table)
    nf.nf_kv_reserve(r, t, dev([0, 0, 0, 0]), dev([256, 257, 1, 1]))
    want = ref.Pages([1, 0, 1, 0], table)
    want.reserve([0, 0, 0, 0], [256, 257, 1, 1])
    same(r, t, want)
    assert nf.nf_get_device_error() == nf.NF_DEVERR_POOL


def test_reserve_counts_more_than_two_to_the_31_pages():
    """256 rows of the largest width ask for 2^31 pages between them: the free blocks go to the first row, and
    the call says that they ran out."""
    rows, width = 256, 1 << 23
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    r = dev([0, 1, 0, 0, 1, 0])
    nf.nf_kv_reserve(r, table, dev([0] * rows), dev([2 ** 31 - 1] * rows))
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == nf.NF_DEVERR_POOL
    assert r.tolist() == [1] * 6
    assert table[0, :4].tolist() == [0, 2, 3, 5]
    table[0, :4] = -1
    assert all(bool((part == -1).all()) for part in table.split(16))


def test_reserve_on_an_unaligned_view():
    refs = torch.zeros(21, dtype=torch.int32, device="cuda")[1:]
    refs[::3] = 1
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    want = ref.Pages(refs.tolist(), table.tolist())
    want.reserve([0, 0], [700, 700])
    nf.nf_kv_reserve(refs, table, dev([0, 0]), dev([700, 700]))
    same(refs, table, want)


@pytest.mark.parametrize("blocks, rows, width", [(1, 1, 1), (30, 4, 9), (4000, 100, 300)])
@pytest.mark.parametrize("seed", [0, 1])
def test_release(blocks, rows, width, seed):
    rng = np.random.default_rng(seed)
    refs, table = state(blocks, rows, width, 1, seed, shared=200)
    frm = rng.integers(0, 400, rows)
    to = rng.integers(0, width * 256 + 500, rows)
    to[0] = 2 ** 31 - 1
    want = ref.Pages(refs, table)
    want.release(frm.tolist(), to.tolist())
    r, t = dev(refs), dev(table)
    nf.nf_kv_release(r, t, dev(frm), dev(to))
    same(r, t, want)
    assert nf.nf_get_device_error() == 0


def test_release_errors():
    refs, table = [1, 0, 2], [[0, 1, 2], [2, 9, -1], [-4, 0, 0]]
    r, t = dev(refs), dev(table)
    nf.nf_kv_release(r, t, dev([0, 0, -1]), dev([768, 768, 768]))
    want = ref.Pages(refs, table)
    want.release([0, 0, -1], [768, 768, 768])
    same(r, t, want)
    assert nf.nf_get_device_error() in (nf.NF_DEVERR_REFS, nf.NF_DEVERR_BLOCK_ID, nf.NF_DEVERR_TABLE)
    r, t = dev([0]), dev([[0]])
    nf.nf_kv_release(r, t, dev([0]), dev([256]))
    torch.cuda.synchronize()
    assert r.item() == 0 and t.item() == -1
    assert nf.nf_get_device_error() == nf.NF_DEVERR_REFS


def test_evicting_behind_a_window_keeps_what_the_window_reads():
    """The next query at L sees (L - window, L] and the sinks."""
    for L, window, n_sink in ((1000, 100, 4), (1024, 256, 256), (1023, 255, 257), (512, 1, 0), (300, 1000, 4)):
        table = np.arange(5, dtype=np.int32)[None]
        r, t = dev(np.ones(5)), dev(table)
        nf.nf_kv_release(r, t, dev([n_sink]), dev([max(0, L + 1 - window)]))
        torch.cuda.synchronize()
        seen = [p for p in range(L + 1) if p > L - window or p < n_sink]
        kept = t.cpu().numpy()[0]
        for e in range(5):
            touched = any(e * 256 <= p < e * 256 + 256 for p in seen)
            behind = (e + 1) * 256 <= L - window + 1  # wholly behind the window
            assert (kept[e] >= 0) == (touched or not behind), (L, window, n_sink, e)


def layers_of(fmt, n, blocks, heads, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    layers = [nf.KVLayer.empty(fmt, blocks, heads) for _ in range(n)]
    for layer in layers:
        for plane in layer.planes():
            b = plane.view(torch.uint8)
            b.copy_(torch.randint(0, 256, b.shape, generator=gen, device="cuda", dtype=torch.uint8))
    return nf.KVLayers(layers)


def bytes_of(layers):
    return [[p.contiguous().view(torch.uint8).clone() for p in layer.planes()] for layer in layers.layers]


def same_bytes(layers, was, moves):
    """Every block as it was, but the moves' destinations, which hold their sources."""
    for layer, planes in zip(layers.layers, was):
        for got, old in zip(layer.planes(), planes):
            want = old.clone()
            for s, d in moves:
                want[d] = old[s]
            assert torch.equal(got.view(torch.uint8), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_layers, heads", [(1, 1), (3, 5), (128, 1)])
def test_copy_blocks(fmt, n_layers, heads):
    layers = layers_of(fmt, n_layers, 12, heads)
    was = bytes_of(layers)
    src, dst = [3, -1, 3, 7, 5, -9], [0, 3, 1, 11, 5, 99]  # one source twice, unused pairs, a pair onto itself
    nf.nf_kv_copy_blocks(layers, dev(src), dev(dst))
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == 0
    same_bytes(layers, was, [(3, 0), (3, 1), (7, 11)])


def test_copy_blocks_conflicts_and_bad_ids():
    layers = layers_of(nf.NF_KV_K8V4, 2, 12, 2)
    was = bytes_of(layers)
    # 1 -> 2 and 2 -> 3: the first would overwrite the second's source; 4 -> 6 and 5 -> 6 meet
    nf.nf_kv_copy_blocks(layers, dev([1, 2, 4, 5, 0]), dev([2, 3, 6, 6, 7]))
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == nf.NF_DEVERR_CONFLICT
    same_bytes(layers, was, [(2, 3), (0, 7)])
    was = bytes_of(layers)
    for src, dst in (([12, 0], [1, 2]), ([1, 0], [12, 2]), ([1, 0], [-1, 2])):
        nf.nf_kv_copy_blocks(layers, dev(src), dev(dst))
        torch.cuda.synchronize()
        assert nf.nf_get_device_error() == nf.NF_DEVERR_BLOCK_ID
        same_bytes(layers, was, [(0, 2)])


def test_copy_many_blocks():
    layers = layers_of(nf.NF_KV_K4V4, 1, 2000, 1)
    was = bytes_of(layers)
    order = np.random.default_rng(0).permutation(2000)
    nf.nf_kv_copy_blocks(layers, dev(order[:900]), dev(order[900:1800]))
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == 0
    same_bytes(layers, was, list(zip(order[:900], order[900:1800])))


def workspace(blocks, n=0):
    return torch.full((nf.nf_kv_pages_workspace_size(blocks, n),), 0x77, dtype=torch.uint8, device="cuda")


def fork_case(refs, table, lens, src, dst, layers, errors=0):
    was = bytes_of(layers)
    r, t, n = dev(refs), dev(table), dev(lens)
    nf.nf_kv_fork(layers, r, t, dev(src), dev(dst), n, workspace(len(refs), len(src)))
    want = ref.Pages(refs, table, lens)
    copies = want.fork(list(src), list(dst))
    same(r, t, want, n)
    same_bytes(layers, was, copies)
    assert nf.nf_get_device_error() == errors
    return want


@pytest.mark.parametrize("fmt", FORMATS)
def test_fork(fmt):
    layers = layers_of(fmt, 3, 40, 2)
    table = np.full((9, 6), -1, np.int32)
    lens = np.zeros(9, np.int32)
    for row, n, first in ((0, 700, 3), (1, 512, 10), (2, 1, 20), (3, 0, 0), (4, 6 * 256, 22)):
        table[row, :-(-n // 256)] = first + np.arange(-(-n // 256))
        lens[row] = n
    table[5, :2] = [30, 31]  # what a destination held is given up
    table[6, 0] = 30         # (shared with another row)
    refs = np.zeros(40, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    fork_case(refs, table, lens, [0, 0, 2, -1, 4], [5, 7, 8, 3, 3], layers)
    fork_case(refs, table, lens, [1, 3], [5, 6], layers)
    table[0, 0] = -1  # released behind a window: stays released
    refs[3] = 0
    fork_case(refs, table, lens, [0, 0], [5, 8], layers)


def test_fork_refusals_leave_the_row():
    layers = layers_of(nf.NF_KV_K8V4, 1, 8, 1)
    table = np.array([[0, 1], [2, -1], [-1, -1], [3, -1]], np.int32)
    refs = np.array([1, 1, 1, 1, 0, 0, 0, 0], np.int32)
    lens = np.array([300, 100, 0, 256], np.int32)
    C, T, S, B, P = nf.NF_DEVERR_CONFLICT, nf.NF_DEVERR_TABLE, nf.NF_DEVERR_SEQLEN, nf.NF_DEVERR_BLOCK_ID, nf.NF_DEVERR_POOL
    fork_case(refs, table, lens, [0, 1], [2, 2], layers, C)   # the same destination twice
    fork_case(refs, table, lens, [0, 3], [3, 2], layers, C)   # a destination that is a source
    fork_case(refs, table, lens, [0, 1], [0, 2], layers, C)   # onto itself
    fork_case(refs, table, lens, [4, 1], [2, 3], layers, T)
    fork_case(refs, table, lens, [0, 1], [-1, 3], layers, T)
    fork_case(refs, table, [513, 100, 0, 256], [0, 1], [2, 3], layers, S)
    fork_case(refs, table, [-1, 100, 0, 256], [0, 1], [2, 3], layers, S)
    fork_case(refs, table, [300, 300, 0, 256], [1, 0], [2, 3], layers, B)  # row 1's second page is missing
    fork_case([1, 1, 1, 1, 0, 1, 1, 1], table, lens, [0, 1], [2, 3], layers, P)


def test_fork_many():
    layers = layers_of(nf.NF_KV_K4V4, 1, 3000, 1)
    rng = np.random.default_rng(1)
    table = np.full((1100, 4), -1, np.int32)
    lens = np.zeros(1100, np.int32)
    ids = rng.permutation(3000)
    for row in range(40):
        lens[row] = int(rng.integers(0, 1025))
        n = -(-lens[row] // 256)
        table[row, :n] = ids[row * 4:row * 4 + n]
    refs = np.zeros(3000, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    src = rng.integers(0, 40, 1024)
    fork_case(refs, table, lens, src.tolist(), (40 + rng.permutation(1060)[:1024]).tolist(), layers)


def compact_case(refs, table, layers, errors=0):
    was = bytes_of(layers)
    r, t = dev(refs), dev(table)
    nf.nf_kv_compact(layers, r, t, workspace(len(refs)))
    want = ref.Pages(refs, table)
    moves = want.compact()
    same(r, t, want)
    same_bytes(layers, was, moves)
    assert nf.nf_get_device_error() == errors
    live = sum(x > 0 for x in want.refs)
    assert all(x > 0 for x in want.refs[:live]) and not any(want.refs[live:])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seed", [0, 1])
def test_compact(fmt, seed):
    layers = layers_of(fmt, 2, 60, 3)
    compact_case(*state(60, 6, 12, 0.6, seed, shared=10), layers)


def test_compact_edges():
    layers = layers_of(nf.NF_KV_K8V4, 1, 5, 1)
    compact_case([0] * 5, [[-1, -1]], layers)
    compact_case([1] * 5, [[0, 1, 2], [3, 4, -1]], layers)
    compact_case([0, 0, 0, 0, 2], [[4, -1], [4, -1]], layers)
    compact_case([1, 1, 0, 0, 0], [[0, 4]], layers, nf.NF_DEVERR_REFS)  # an entry of a free block
    one = layers_of(nf.NF_KV_K8V4, 1, 1, 1)
    compact_case([1], [[0]], one)
    r = dev([0, 1])
    nf.nf_kv_compact(layers_of(nf.NF_KV_K8V4, 1, 2, 1), r, dev(np.zeros((0, 3))), workspace(2))  # no rows
    assert r.tolist() == [1, 0]


def test_compact_large_pool():
    layers = layers_of(nf.NF_KV_K4V4, 1, 9000, 1)
    compact_case(*state(9000, 40, 150, 1, 3), layers)


def test_captured_turn():
    """reserve and release of a decode step in one graph, replayed step by step."""
    window, n_sink, rows = 300, 4, 5
    lens = torch.tensor([10, 255, 256, 700, 1], dtype=torch.int32, device="cuda")
    refs, table = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.full((rows, 8), -1, dtype=torch.int32, device="cuda")
    zero, sinks = torch.zeros_like(lens), torch.full_like(lens, n_sink)
    nf.nf_kv_reserve(refs, table, zero, lens)
    want = ref.Pages(refs.tolist(), table.tolist())
    to, old = torch.empty_like(lens), torch.empty_like(lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        torch.add(lens, 1, out=to)
        torch.sub(lens, window - 1, out=old)
        nf.nf_kv_reserve(refs, table, lens, to)
        nf.nf_kv_release(refs, table, sinks, old)
        lens.add_(1)
    at = lens.tolist()
    for _ in range(600):
        graph.replay()
        want.reserve(at, [n + 1 for n in at])
        want.release([n_sink] * rows, [n - window + 1 for n in at])
        at = [n + 1 for n in at]
    same(refs, table, want)
    assert nf.nf_get_device_error() == 0


def test_captured_fork_and_compact():
    """Fork, release of a source and compaction in one graph, replayed on three states."""
    layers = layers_of(nf.NF_KV_K8V4, 2, 40, 2)
    r, t, n = dev(np.zeros(40)), dev(np.full((6, 5), -1)), dev(np.zeros(6))
    src, dst, ws = dev([0, 0, 1]), dev([3, 4, 5]), workspace(40, 3)
    frm, to = dev([0] * 6), dev([0, 5 * 256, 0, 0, 0, 0])

    def call():
        nf.nf_kv_fork(layers, r, t, src, dst, n, ws)
        nf.nf_kv_release(r, t, frm, to)
        nf.nf_kv_compact(layers, r, t, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(3):
        rng = np.random.default_rng(seed)
        lens = [int(x) for x in rng.integers(0, 5 * 256 + 1, 2)] + [0] * 4
        table, ids = np.full((6, 5), -1, np.int32), rng.permutation(40)
        for row in (0, 1):
            pages = -(-lens[row] // 256)
            table[row, :pages] = ids[5 * row:5 * row + pages]
        refs = np.zeros(40, np.int32)
        np.add.at(refs, table[table >= 0], 1)
        r.copy_(dev(refs)), t.copy_(dev(table)), n.copy_(dev(lens))
        was = bytes_of(layers)
        graph.replay()
        want = ref.Pages(refs, table, lens)
        copies = want.fork([0, 0, 1], [3, 4, 5])
        want.release([0] * 6, [0, 5 * 256, 0, 0, 0, 0])
        moves = want.compact()
        same(r, t, want, n)
        # the copies first, then the moves: what each moved block held after the copies
        held = dict((d, s) for s, d in copies)
        final = {d: held.get(s, s) for s, d in moves}
        still = {d: s for d, s in held.items() if d not in final}
        same_bytes(layers, was, [(s, d) for d, s in {**still, **final}.items()])
        assert nf.nf_get_device_error() == 0


def test_pages_binding_refusals():
    layers = layers_of(nf.NF_KV_K8V4, 1, 4, 1)
    refs, table, rows = dev(np.zeros(4)), dev(np.full((2, 3), -1)), dev([0, 0])
    ws = workspace(4, 2)
    bad = [lambda: nf.nf_kv_reserve(refs.long(), table, rows, rows), lambda: nf.nf_kv_reserve(refs, table, rows[:1], rows),
           lambda: nf.nf_kv_release(refs, table[:, ::2], rows, rows), lambda: nf.nf_kv_release(refs, table, rows, rows.cpu()),
           lambda: nf.nf_kv_copy_blocks(layers, rows, rows[:1]), lambda: nf.nf_kv_copy_blocks(layers, rows.long(), rows),
           lambda: nf.nf_kv_fork(layers, refs[:3].contiguous(), table, rows, rows, rows, ws),
           lambda: nf.nf_kv_fork(layers, refs, table, rows, rows, rows[:1], ws),
           lambda: nf.nf_kv_fork(layers, refs, table, rows, rows, rows, ws[:16]),
           lambda: nf.nf_kv_compact(layers, refs, table, ws[:256].cpu()), lambda: nf.nf_kv_compact(layers, refs[1:], table, ws),
           lambda: nf.KVLayers([layers.layers[0], layers.layers[0]]) and nf.nf_kv_compact(
               nf.KVLayers([layers.layers[0], nf.KVLayer.empty(nf.NF_KV_F8, 4, 1)]), refs, table, ws)]
    for call in bad:
        with pytest.raises(nf.NfError):
            call()
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == 0

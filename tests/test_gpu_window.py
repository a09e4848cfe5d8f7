"""Windowed attention with sinks (decode and prefill forms) against its
definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import long_context_quantized_b200 as nf
import sessionref as ref

pytestmark = pytest.mark.gpu

FORMATS = [nf.NF_KV_K8V4, nf.NF_KV_K8V8, nf.NF_KV_F8, nf.NF_KV_K4V4, nf.NF_KV_BF16]
SCALE = 128 ** -0.5


class Case:
    def __init__(self, fmt, seqlens, n_q=1, hq=8, hkv=2, dtype=torch.bfloat16, width=None, q_seed=5, spare=2):
        self.seqlens, self.n_q = list(seqlens), n_q
        blocks = sum(math.ceil(L / 256) for L in seqlens) + spare
        self.kv = ref.filled_pool(fmt, blocks, hkv)
        self.np_table = ref.make_table(seqlens, blocks, width)
        self.lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
        self.max_len = max(max(seqlens), n_q)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(q_seed)
        self.q = torch.randn((len(seqlens), n_q, hq, 128), generator=gen, device="cuda").to(dtype)
        self.lse = torch.empty(self.q.shape[:3], device="cuda")
        self.ws = torch.zeros(nf.nf_decode_attn_window_workspace_size(len(seqlens), n_q, hq, hkv, self.max_len),
                              dtype=torch.uint8, device="cuda")

    @property
    def table(self):
        return torch.as_tensor(self.np_table, device="cuda")

    def run(self, window, n_sink, out_dtype=torch.float32, prefill=False):
        out = torch.full(self.q.shape, 7.0, dtype=out_dtype, device="cuda")
        self.lse.fill_(7.0)
        if prefill:
            nf.nf_prefill_attn_window(self.kv, self.q, self.table, self.lens, self.max_len, window, n_sink, SCALE, out,
                                      self.lse)
        else:
            nf.nf_decode_attn_window(self.kv, self.q, self.table, self.lens, self.max_len, window, n_sink, SCALE, out,
                                     self.lse, self.ws)
        torch.cuda.synchronize()
        return out

    def check(self, window, n_sink, out_dtype=torch.float32, prefill=False, errors=0):
        out = self.run(window, n_sink, out_dtype, prefill)
        assert nf.nf_get_device_error() == errors
        o, lse, parts = ref.window_attention(self.kv, self.q, self.np_table, self.seqlens, window, n_sink, SCALE)
        ref.check_out(out, o, ref.prefill_tolerance(parts) if prefill else ref.decode_tolerance(parts))
        got = self.lse.double().cpu().numpy()
        assert np.array_equal(np.isfinite(got), np.isfinite(lse))
        fin = np.isfinite(lse)
        # a score moves by at most 2^-16 dq (decode) or 2^-11 dk + 2^-25 dq (prefill)
        d = 2.0 ** -16 * parts["dq"] if not prefill else 2.0 ** -11 * parts["dk"] + 2.0 ** -25 * parts["dq"]
        assert np.all(np.abs(got[fin] - lse[fin]) <= np.broadcast_to(d[..., 0], lse.shape)[fin] + 2.0 ** -14)
        if out_dtype == torch.float32 and np.linalg.norm(o) > 0:  # the library's stated accuracy
            assert np.linalg.norm(out.double().cpu().numpy() - o) <= 1e-3 * np.linalg.norm(o)
        return out


def wipe(kv, page, slot):
    """All bits of one token's codes and scales set: not-a-number scales (and e4m3 and bf16 codes)."""
    for plane in kv.planes():
        plane.view(torch.uint8).reshape(*plane.shape[:2], 256, -1)[page, :, slot] = 0xFF


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window, n_sink", [(1, 0), (33, 4), (256, 0), (300, 300), (100, 31), (4096, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_window_formats(fmt, window, n_sink):
    Case(fmt, [1500, 700, 33]).check(window, n_sink)


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 255, 256, 257, 1021])
@pytest.mark.parametrize("window, n_sink", [(1, 1), (32, 32), (255, 5), (256, 257)])
def test_decode_window_lengths(L, window, n_sink):
    Case(nf.NF_KV_K8V4, [L]).check(window, n_sink, torch.bfloat16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q, hq, hkv", [(4, 8, 8), (4, 8, 1), (3, 10, 2), (2, 40, 8), (8, 8, 1), (5, 12, 1)])
def test_decode_window_many_rows(fmt, n_q, hq, hkv):
    """Each query has its own window; up to 64 rows a kv-head."""
    c = Case(fmt, [900, n_q, 417], n_q=n_q, hq=hq, hkv=hkv)
    for window, n_sink in ((1, 0), (2, 3), (130, 40)):
        c.check(window, n_sink)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_dtype", [torch.float32, torch.bfloat16])
def test_decode_window_types(q_dtype, out_dtype):
    for fmt in FORMATS:
        Case(fmt, [777, 256], dtype=q_dtype).check(200, 7, out_dtype)


def test_decode_window_unused_rows():
    """Length 0: zeros and -inf, no error; lengths between are errors."""
    for fmt in FORMATS:
        c = Case(fmt, [0, 500, 0], n_q=2)
        for dtype in (torch.float32, torch.bfloat16):
            out = c.check(64, 4, dtype)
            assert not out[0].any() and not out[2].any() and torch.isinf(c.lse[0]).all()
    c = Case(nf.NF_KV_K8V4, [1, 500], n_q=2)
    c.check(64, 4, errors=nf.NF_DEVERR_SEQLEN)  # its rows are zeros too
    for fmt in FORMATS:
        Case(fmt, [0, 0]).check(64, 4)
        Case(fmt, [0, 0], hq=24).check(64, 4, torch.bfloat16)  # 12 rows a kv-head
        Case(fmt, [0, 300, 0], hq=24, n_q=2).check(64, 4, torch.bfloat16)


def test_decode_window_large_batch():
    rng = np.random.default_rng(3)
    c = Case(nf.NF_KV_K8V4, [int(n) for n in rng.integers(0, 700, 256)], hq=4, hkv=1)
    c.check(100, 3, torch.bfloat16)


def test_decode_window_long_splits():
    """Segments over many CTAs: the merge in the ring, in L2 and of 64 rows."""
    c = Case(nf.NF_KV_K8V4, [30000], hq=8, hkv=1)
    c.check(20001, 65)
    Case(nf.NF_KV_K8V4, [20000], n_q=8, hq=8, hkv=1).check(15000, 10, torch.bfloat16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq", [4, 8, 20])
def test_decode_window_bytes_of_hidden_keys_do_not_matter(fmt, hq):
    """Pages out of every window may be gone, and hidden keys that share a page
    (and a chunk) with seen ones may hold anything, not-a-number included."""
    window, n_sink, n_q = 300, 5, 3
    c = Case(fmt, [1400, 800], n_q=n_q, hq=hq)
    want = c.check(window, n_sink)
    for b, L in enumerate(c.seqlens):
        first = L - n_q - window + 1
        for e in range(c.np_table.shape[1]):
            for t in range(e * 256, e * 256 + 256):
                if (n_sink <= t < first) or t >= L:
                    page = c.np_table[b, e]
                    if page >= 0:
                        wipe(c.kv, page, t % 256)
            if e * 256 >= n_sink and (e + 1) * 256 <= first:
                c.np_table[b, e] = -1
    got = c.run(window, n_sink)
    assert nf.nf_get_device_error() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q, hq, hkv", [(2, 8, 2), (3, 8, 2), (4, 8, 1), (8, 8, 1)])
def test_decode_window_of_everything_is_causal_attention(fmt, n_q, hq, hkv):
    """With a window of at least the length the call is nf_decode_attn, bit for bit."""
    c = Case(fmt, [2500, 513], n_q=n_q, hq=hq, hkv=hkv)
    got = c.run(2500, 0)
    out = torch.empty_like(got)
    nf.nf_decode_attn(c.kv, c.q, c.table, c.lens, c.max_len, SCALE, True, out, None, c.ws)
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_decode_window_zero_and_tiny_queries():
    for dtype in (torch.float32, torch.bfloat16):
        c = Case(nf.NF_KV_K8V4, [600, 40], dtype=dtype)
        c.q[0, 0, 0] = 0
        c.q[0, 0, 1] = 1e-39
        c.q[1, 0, 2] = 1e-30
        c.check(200, 4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q, hq", [(1, 8), (4, 8), (8, 16)])
def test_decode_window_tiny_queries_of_every_format(fmt, n_q, hq):
    """Rows of zeros and of subnormals, channels of zeros among them, whose inverse is no fp32 number."""
    for dtype in (torch.float32, torch.bfloat16):
        c = Case(fmt, [600, 90], n_q=n_q, hq=hq, dtype=dtype)
        c.q[0, 0, 0] = 0
        c.q[0, 0, 1] = 1e-39
        c.q[0, 0, 2] = 0
        c.q[0, 0, 2, ::3] = -2e-40
        c.q[0, 0, 3] *= 1e-36
        c.q[1, 0, 0] = 2e-38
        c.q[1, 0, 1] *= 1e-30
        c.check(200, 4)


def test_decode_window_bad_pages_are_reported():
    c = Case(nf.NF_KV_K8V4, [900])
    c.np_table[0, 2] = 10 ** 6
    c.run(900, 0)
    assert nf.nf_get_device_error() == nf.NF_DEVERR_BLOCK_ID
    c.np_table[0, 2] = -7
    c.run(900, 0)
    assert nf.nf_get_device_error() == nf.NF_DEVERR_BLOCK_ID
    c.run(100, 4)  # the page is outside the window now
    assert nf.nf_get_device_error() == 0


def test_decode_window_repeats_bitwise_and_on_another_stream():
    c = Case(nf.NF_KV_K8V4, [5000, 1200], n_q=2)
    want = c.run(3000, 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [c.run(3000, 20) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("n_q, seqlens, hq, hkv", [
    (1, [1, 300], 8, 2), (5, [5, 777], 8, 1), (64, [64, 700], 4, 4), (100, [1000], 10, 2), (33, [33, 0, 290], 32, 4),
    (300, [300], 4, 1), (257, [600, 257], 8, 8)])
@pytest.mark.parametrize("window, n_sink", [(1, 0), (64, 4), (100, 65), (256, 300), (2 ** 31 - 1, 0)])
def test_prefill_window(n_q, seqlens, hq, hkv, window, n_sink):
    c = Case(nf.NF_KV_K8V4, seqlens, n_q=n_q, hq=hq, hkv=hkv)
    c.check(window, n_sink, prefill=True)
    c.check(window, n_sink, torch.bfloat16, prefill=True)


def test_prefill_window_of_everything_is_causal_prefill():
    """A window of at least the length is causal attention (each kernel with its own roundings, 1e-3 of the norm)."""
    c = Case(nf.NF_KV_K8V4, [1500, 700], n_q=200)
    got = c.run(1500, 0, prefill=True)
    out = torch.empty_like(got)
    nf.nf_prefill_attn(c.kv, c.q, c.table, c.lens, c.max_len, SCALE, True, out)
    torch.cuda.synchronize()
    assert (got - out).norm() <= 2e-3 * out.norm()


def test_prefill_window_bytes_of_hidden_keys_do_not_matter():
    window, n_sink, n_q = 300, 70, 40
    c = Case(nf.NF_KV_K8V4, [1400, 800], n_q=n_q)
    want = c.check(window, n_sink, prefill=True)
    for b, L in enumerate(c.seqlens):
        first = L - n_q - window + 1
        for e in range(c.np_table.shape[1]):
            page = c.np_table[b, e]
            for t in range(e * 256, e * 256 + 256):
                if page >= 0 and ((n_sink <= t < first) or t >= L):
                    wipe(c.kv, page, t % 256)
            if e * 256 >= n_sink and (e + 1) * 256 <= first:
                c.np_table[b, e] = -1
    got = c.run(window, n_sink, prefill=True)
    assert nf.nf_get_device_error() == 0
    assert torch.equal(got, want)


def test_prefill_window_zero_and_tiny_queries():
    c = Case(nf.NF_KV_K8V4, [600], n_q=70)
    c.q[0, 3] = 0
    c.q[0, 4] = 1e-39
    c.q[0, 69, 1] = 0
    c.check(200, 4, prefill=True)


def test_prefill_window_flat_scores_repeat_bitwise():
    """Scores so close that no running max rises behind the first tile: each tile's weights replace the last
    one's in tensor memory with no rescale of the output between them."""
    c = Case(nf.NF_KV_K8V4, [2900, 1500], n_q=300)
    c.kv = ref.filled_pool(nf.NF_KV_K8V4, c.kv.num_blocks, 2, k_gain=0.02)
    want = c.check(2500, 4, prefill=True)
    outs = [c.run(2500, 4, prefill=True) for _ in range(8)]
    assert all(torch.equal(o, want) for o in outs)


def climb(c, spacing, step=9.0):
    """Fills the case's pool with keys whose scores (in powers of two) climb by `step` at every `spacing`-th key
    and stay at that level or up to 2 below until the next: the keys before a rise weigh about as much as the key
    that brings it, so a row whose last key comes soon behind a rise shows how the earlier sums were rescaled.
    The rises fall on the first and the second half of 64 keys in turn.  Query head g of a group takes gain
    (1, 0.5, -1, 1.8)[g % 4] of the climb."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    B, _, hq, _ = c.q.shape
    hkv = c.kv.num_kv_heads
    u = torch.randn((hkv, 128), generator=gen, device="cuda")
    for b, L in enumerate(c.seqlens):
        if L == 0:
            continue
        t = torch.arange(L, device="cuda")
        k_of = torch.zeros(L, device="cuda")
        for n, at in enumerate(range(spacing, L, spacing)):
            k_of[at // 64 * 64 + 32 * (n % 2) + at % 32:] += 1.0
        dip = 2.0 * torch.rand((L,), generator=gen, device="cuda")
        rise = torch.zeros(L, dtype=torch.bool, device="cuda")
        rise[1:] = k_of[1:] > k_of[:-1]
        level = step * (k_of - k_of.mean()) - torch.where(rise, torch.zeros_like(dip), dip)
        g = level / (SCALE * math.log2(math.e) * 128)
        k = g[:, None, None] * u + 0.02 * torch.randn((L, hkv, 128), generator=gen, device="cuda")
        v = torch.randn((1, L, hkv, 128), generator=gen, device="cuda")
        nf.nf_kv_append_quant(c.kv, k[None].contiguous(), v, c.table[b:b + 1].contiguous(),
                              torch.zeros(1, dtype=torch.int32, device="cuda"))
    gain = torch.tensor([1.0, 0.5, -1.0, 1.8], device="cuda").repeat(hq)[:hq // hkv]
    rows = (u[:, None] * gain[:, None]).reshape(hq, 128)
    c.q = (rows + 0.05 * torch.randn(c.q.shape, generator=gen, device="cuda")).to(c.q.dtype).contiguous()


@pytest.mark.parametrize("window, n_sink", [(3000, 0), (1000, 70)])
def test_prefill_window_rising_scores(window, n_sink):
    """The running max rises by more than 2^8 several times: weights, sums and output are rescaled each time."""
    c = Case(nf.NF_KV_K8V4, [2900, 1300], n_q=700)
    climb(c, 450)
    c.check(window, n_sink, torch.bfloat16, prefill=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q, hq", [(1, 8), (4, 8), (8, 16)])
def test_decode_window_rising_scores(fmt, n_q, hq):
    """The same on every decode kernel, with about a whole segment for each CTA."""
    rng = np.random.default_rng(5)
    c = Case(fmt, [int(n) for n in rng.integers(500, 1100, 80)], n_q=n_q, hq=hq)
    climb(c, 150)
    c.check(1000, 3, torch.bfloat16)


@pytest.mark.parametrize("plane, bits, error", [
    ("k", 0x6007, 0), ("k", 0x6008, nf.NF_DEVERR_RANGE), ("v", 0x7091, 0), ("v", 0x7092, nf.NF_DEVERR_RANGE)])
def test_prefill_window_range_of_scales(plane, bits, error):
    """The largest K and V scales whose codes stay in fp16 (515.5 and 9352) pass, the next ones are reported, on a
    key that some query sees; a hidden key's scale is not looked at."""
    window, n_sink = 300, 5
    for t, err in ((1100, error), (600, 0)):
        c = Case(nf.NF_KV_K8V4, [1200], n_q=20)
        page, slot = int(c.np_table[0, t // 256]), t % 256
        codes, scales, fill = (c.kv.k_codes, c.kv.k_scales, 127) if plane == "k" else (c.kv.v_codes, c.kv.v_scales, 0x77)
        codes[page, :, slot] = fill
        scales.view(torch.int16)[page, :, slot] = bits
        out = c.run(window, n_sink, prefill=True)
        assert nf.nf_get_device_error() == err
        if not err:
            assert torch.isfinite(out).all()


@pytest.mark.parametrize("full", [False, True], ids=["windowed", "full"])
def test_prefill_scores_beyond_its_range_are_reported(full):
    """Both prefill kernels answer for rows whose largest score is below 2^26 (in powers of two) and say where one
    is not; a query that is not a number is not such a row."""
    for gain, err in ((1e6, 0), (1e9, nf.NF_DEVERR_RANGE), (1e30, nf.NF_DEVERR_RANGE), (float("nan"), 0)):
        c = Case(nf.NF_KV_K8V4, [900, 500], n_q=40)
        window, n_sink = (10 ** 6, 0) if full else (300, 4)
        c.q = (c.q.float() * gain).bfloat16()
        if full:
            out = torch.empty(c.q.shape, device="cuda")
            nf.nf_prefill_attn(c.kv, c.q, c.table, c.lens, c.max_len, SCALE, True, out, c.lse)
            torch.cuda.synchronize()
        else:
            out = c.run(window, n_sink, prefill=True)
        assert nf.nf_get_device_error() == err
        if gain == 1e6:
            _, lse, _ = ref.window_attention(c.kv, c.q, c.np_table, c.seqlens, window, n_sink, SCALE)
            assert np.abs(lse).max() < 2.0 ** 26 * math.log(2)
            assert torch.isfinite(out).all() and torch.isfinite(c.lse).all()
            # a mean of values (weights and values rounded to fp16 once each)
            assert out.abs().max().item() <= np.abs(ref.open_pool(c.kv)[1]).max() * (1 + 2.0 ** -9)


def test_prefill_window_errors():
    c = Case(nf.NF_KV_K8V4, [9, 500], n_q=10)
    c.check(64, 4, prefill=True, errors=nf.NF_DEVERR_SEQLEN)
    c = Case(nf.NF_KV_K8V4, [900], n_q=10)
    c.np_table[0, 1] = 10 ** 6
    c.run(900, 0, prefill=True)
    assert nf.nf_get_device_error() == nf.NF_DEVERR_BLOCK_ID


def test_decode_and_prefill_agree():
    """The two forms of the same queries differ by their roundings only."""
    c = Case(nf.NF_KV_K8V4, [3000, 500], n_q=4, hq=8, hkv=2)
    a, b = c.run(700, 30), c.run(700, 30, prefill=True)
    assert (a - b).norm() <= 2e-3 * a.norm()


def test_window_calls_in_a_graph_follow_the_lengths():
    """Captured once, replayed after the lengths and the table changed."""
    c = Case(nf.NF_KV_K8V4, [700, 900], n_q=1, width=6, spare=6)
    table = c.table
    out, ws = torch.empty_like(c.q), c.ws
    c.max_len = 6 * 256

    def call():
        nf.nf_decode_attn_window(c.kv, c.q, table, c.lens, c.max_len, 300, 4, SCALE, out, c.lse, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    with torch.cuda.graph(other):  # a second graph on the same workspace, replayed in turn
        call()
    for seqlens in ([700, 900], [701, 0], [256, 768]):
        c.seqlens = seqlens
        c.lens.copy_(torch.tensor(seqlens, dtype=torch.int32))
        for g in (graph, other):
            out.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            o, _, parts = ref.window_attention(c.kv, c.q, c.np_table, seqlens, 300, 4, SCALE)
            ref.check_out(out, o, ref.decode_tolerance(parts))
    assert nf.nf_get_device_error() == 0


def test_prefill_window_in_a_graph_follows_the_lengths():
    """Captured once, replayed after the lengths changed (an unused row among them)."""
    c = Case(nf.NF_KV_K8V4, [1300, 900], n_q=150)
    table, out = c.table, torch.empty(c.q.shape, device="cuda")

    def call():
        nf.nf_prefill_attn_window(c.kv, c.q, table, c.lens, c.max_len, 400, 70, SCALE, out, c.lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for seqlens in ([1300, 900], [150, 0], [777, 512]):
        c.lens.copy_(torch.tensor(seqlens, dtype=torch.int32))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        o, _, parts = ref.window_attention(c.kv, c.q, c.np_table, seqlens, 400, 70, SCALE)
        ref.check_out(out, o, ref.prefill_tolerance(parts))
    assert nf.nf_get_device_error() == 0


@pytest.mark.parametrize("n_q, hq, hkv", [(1, 300, 1), (5, 300, 1), (3, 513, 3), (1, 70, 70), (2, 4096, 2)])
def test_prefill_window_groups_of_any_size(n_q, hq, hkv):
    """Rows of a position that span tiles, and positions that share one with a fraction of the next."""
    Case(nf.NF_KV_K8V4, [700], n_q=n_q, hq=hq, hkv=hkv).check(200, 5, torch.bfloat16, prefill=True)


def test_far_pages_of_a_large_pool():
    """Blocks behind the first 4 GiB of a plane: append, decode, prefill and copies."""
    heads, blocks = 8, 17000  # K: 256 KiB a block, 4.15 GiB
    kv = nf.KVLayer.empty(nf.NF_KV_K8V4, blocks, heads)
    seqlens, n_q = [700], 2
    ids = [blocks - 1, 3, blocks - 2]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    k, v = (torch.randn((1, 700, heads, 128), generator=gen, device="cuda") for _ in range(2))
    inv = torch.ones(64, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    nf.nf_rope_append_quant(kv, nf.Rope(inv), torch.zeros((1, 700, 1), dtype=torch.int32, device="cuda"), None, k, v, table,
                            zero, None)
    near = nf.KVLayer.empty(nf.NF_KV_K8V4, 3, heads)
    nf.nf_kv_append_quant(near, k, v, torch.arange(3, dtype=torch.int32, device="cuda")[None], zero)
    for far, close in zip(kv.planes(), near.planes()):
        for page, block in enumerate(ids):
            n = min(256, 700 - 256 * page)
            assert torch.equal(far[block, :, :n], close[page, :, :n])
    q = torch.randn((1, n_q, 16, 128), generator=gen, device="cuda").bfloat16()
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    ws = torch.zeros(nf.nf_decode_attn_window_workspace_size(1, n_q, 16, heads, 768), dtype=torch.uint8, device="cuda")
    o, _, parts = ref.window_attention(near, q, np.arange(3)[None], seqlens, 300, 4, SCALE)
    for prefill in (False, True):
        out = torch.empty(q.shape, device="cuda")
        if prefill:
            nf.nf_prefill_attn_window(kv, q, table, lens, 768, 300, 4, SCALE, out)
        else:
            nf.nf_decode_attn_window(kv, q, table, lens, 768, 300, 4, SCALE, out, None, ws)
        torch.cuda.synchronize()
        ref.check_out(out, o, ref.prefill_tolerance(parts) if prefill else ref.decode_tolerance(parts))
    layers = nf.KVLayers([kv])
    nf.nf_kv_copy_blocks(layers, table[0, :1].contiguous(), torch.tensor([blocks - 5], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert all(torch.equal(p[blocks - 5].view(torch.uint8), p[blocks - 1].view(torch.uint8)) for p in kv.planes())
    assert nf.nf_get_device_error() == 0


def test_window_binding_refusals():
    c = Case(nf.NF_KV_K8V4, [300, 300])
    out = torch.empty_like(c.q)

    def call(**over):
        a = dict(q=c.q, table=c.table, lens=c.lens, out=out, lse=None, ws=c.ws, window=10)
        a.update(over)
        nf.nf_decode_attn_window(c.kv, a["q"], a["table"], a["lens"], c.max_len, a["window"], 0, SCALE, a["out"], a["lse"],
                                 a["ws"])

    call()
    for over in (dict(q=c.q.half()), dict(q=c.q.cpu()), dict(q=c.q[:, :, ::2]), dict(q=c.q[:, 0]), dict(out=out[:1]),
                 dict(out=out.half()), dict(lse=c.lse[:1]), dict(lse=c.lse.double()), dict(table=c.table[:1]),
                 dict(table=c.table.long()), dict(lens=c.lens[:1]), dict(lens=c.lens.cpu()), dict(ws=None),
                 dict(ws=c.ws[:256]), dict(window=0)):
        with pytest.raises(nf.NfError):
            call(**over)
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == 0


def test_two_streams_at_once():
    """Decode calls (each with its own workspace) and prefill calls on two streams, not waiting for one another."""
    mtp = Case(nf.NF_KV_K8V4, [9000, 4000], n_q=4, hq=32, hkv=2, q_seed=6)
    one = Case(nf.NF_KV_K8V4, [7000, 20, 3000], n_q=1, q_seed=7)
    chunk = Case(nf.NF_KV_K8V4, [2100], n_q=300, hq=8, hkv=2, q_seed=8)
    want = [mtp.run(2500, 4), one.run(1000, 300), chunk.run(700, 4, prefill=True)]
    outs = [[torch.empty_like(w) for _ in range(6)] for w in want]
    tables = [c.table for c in (mtp, one, chunk)]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for i in range(6):
        with torch.cuda.stream(a):
            nf.nf_decode_attn_window(mtp.kv, mtp.q, tables[0], mtp.lens, mtp.max_len, 2500, 4, SCALE, outs[0][i], None, mtp.ws)
        with torch.cuda.stream(b):
            nf.nf_decode_attn_window(one.kv, one.q, tables[1], one.lens, one.max_len, 1000, 300, SCALE, outs[1][i], None, one.ws)
        with torch.cuda.stream(a if i % 2 else b):
            nf.nf_prefill_attn_window(chunk.kv, chunk.q, tables[2], chunk.lens, chunk.max_len, 700, 4, SCALE, outs[2][i])
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == 0
    assert all(torch.equal(got, w) for w, row in zip(want, outs) for got in row)

"""Rotary positions fused with the quantised append, against extended-precision
angles and the oracle's quantisers: the pool's bytes are equal, the queries
within their rounding."""
import numpy as np
import pytest
import torch

import long_context_quantized_b200 as nf
import oracle
import sessionref as ref

pytestmark = pytest.mark.gpu

FORMATS = [nf.NF_KV_K8V4, nf.NF_KV_K8V8, nf.NF_KV_F8, nf.NF_KV_K4V4, nf.NF_KV_BF16]


class Case:
    def __init__(self, fmt=nf.NF_KV_K8V4, batch=2, n_new=3, hq=4, hkv=2, dtype=torch.bfloat16, rot=128, n_axes=3,
                 layout=nf.NF_ROPE_HALVES, far=1000, strided=True, before=(250, 511, 0, 100, 7), seed=0, axis=None,
                 theta=1e6):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.fmt, self.dtype, self.rot, self.layout = fmt, dtype, rot, layout
        self.before = list(before[:batch])
        pages = [(b + n_new + 255) // 256 + 1 for b in self.before]
        self.kv = nf.KVLayer.empty(fmt, sum(pages) + 2, hkv, fill=0xA5)
        self.pool = oracle.Pool(fmt, sum(pages) + 2, hkv, 128, poison=0xA5)
        self.np_table = ref.make_table([p * 256 for p in pages], sum(pages) + 2)
        self.table = torch.as_tensor(self.np_table, device="cuda")
        heads = hq + 2 * hkv
        x = torch.randn((batch, n_new, heads, 128), generator=gen, device="cuda").to(dtype)
        parts = x.split([hq, hkv, hkv], dim=2)
        self.q, self.k, self.v = parts if strided else [p.contiguous() for p in parts]
        self.np_pos = rng.integers(0, far, (batch, n_new, n_axes)).astype(np.int32)
        self.inv = (theta ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
        self.axis = [i % n_axes for i in range(rot // 2)] if axis is None else axis
        self.rope = nf.Rope(torch.as_tensor(self.inv, device="cuda"), self.axis, n_axes, layout)
        self.q_out = torch.full((batch, n_new, hq, 128), 9.0, dtype=dtype, device="cuda")
        self.lens = torch.tensor(self.before, dtype=torch.int32, device="cuda")

    def run(self, n_valid=None, q_out=None, **over):
        nf.nf_rope_append_quant(self.kv, self.rope, torch.as_tensor(self.np_pos, device="cuda"), self.q, self.k, self.v,
                                self.table, self.lens, self.q_out if q_out is None else q_out, n_valid, **over)
        torch.cuda.synchronize()

    def turned(self, x):
        return ref.rope_rows(x.double().cpu().numpy(), self.np_pos, self.inv, self.axis, self.layout, self.rot)

    def check(self, n_valid=None, errors=0):
        assert nf.nf_get_device_error() == errors
        k, v = self.turned(self.k).astype(np.float32), self.v.float().cpu().numpy()
        for b, n in enumerate([self.k.shape[1]] * self.k.shape[0] if n_valid is None else n_valid):
            if n > 0:
                assert oracle.append(self.pool, k[b:b + 1, :n], v[b:b + 1, :n], self.np_table[b:b + 1],
                                     np.array(self.before[b:b + 1], np.int32)) == 0
        for got, want in zip(self.kv.planes(), self.pool.planes() if self.fmt != nf.NF_KV_BF16 else [self.pool.k, self.pool.v]):
            g = got.contiguous().view(torch.uint8).cpu().numpy().ravel()
            w = np.ascontiguousarray(want).view(np.uint8).ravel()
            assert np.array_equal(g, w), int((g != w).sum())
        self.check_q(n_valid)

    def check_q(self, n_valid=None):
        """(x cos - y sin) in fp32: cos and sin rounded once (2^-24 each), y sin
        rounded, the sum rounded: at most 4 x 2^-24 (|x| + |y|), then one
        rounding to bf16 (2^-8 of the value)."""
        want = self.turned(self.q)
        x = np.abs(self.q.double().cpu().numpy())
        half = self.rot // 2
        pair = x.copy()
        if self.layout == nf.NF_ROPE_PAIRS:
            pair[..., 0:self.rot:2] += x[..., 1:self.rot:2]
            pair[..., 1:self.rot:2] += x[..., 0:self.rot:2]
        else:
            pair[..., :half] += x[..., half:self.rot]
            pair[..., half:self.rot] += x[..., :half]
        tol = 4 * 2.0 ** -24 * pair
        if self.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        got = self.q_out.double().cpu().numpy()
        n = [self.q.shape[1]] * self.q.shape[0] if n_valid is None else n_valid
        for b in range(len(n)):
            m = min(max(n[b], 0), self.q.shape[1])
            assert np.all(np.abs(got[b, :m] - want[b, :m]) <= tol[b, :m])
            assert np.all(got[b, m:] == 9.0)  # padding is left as it was


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", [nf.NF_ROPE_HALVES, nf.NF_ROPE_PAIRS])
def test_formats_types_layouts(fmt, dtype, layout):
    for strided in (False, True):
        c = Case(fmt, dtype=dtype, layout=layout, n_new=17, strided=strided)
        c.run()
        c.check()


@pytest.mark.parametrize("rot", [8, 16, 24, 32, 64, 72, 96, 120, 128])
@pytest.mark.parametrize("layout", [nf.NF_ROPE_HALVES, nf.NF_ROPE_PAIRS])
def test_partial_rotary(rot, layout):
    c = Case(rot=rot, layout=layout, n_axes=1, dtype=torch.float32)
    c.run()
    c.check()


@pytest.mark.parametrize("n_axes", [1, 2, 3, 4])
def test_axes_in_sections_and_interleaved(n_axes):
    half = 64
    for axis in ([min(i * n_axes // half, n_axes - 1) for i in range(half)], [i % n_axes for i in range(half)],
                 [n_axes - 1] * half):
        c = Case(n_axes=n_axes, axis=axis, n_new=5)
        c.run()
        c.check()


@pytest.mark.parametrize("far", [1, 262144, 2 ** 24, 2 ** 31 - 1])
def test_far_positions(far):
    c = Case(far=far, dtype=torch.float32, n_new=40, theta=1e4)
    c.np_pos[0, 0] = far - 1
    c.np_pos[0, 1] = -(far - 1)  # positions may be negative
    c.run()
    c.check()


@pytest.mark.parametrize("pos", [2 ** 31 - 1, -2 ** 31, 1073741789])
def test_angles_at_the_largest_positions(pos):
    """A key of (1, 0) pairs holds its angles' cos and sin: the fp32 keys of a bf16
    pool's rows differ from them by their rounding to bf16 alone, and queries of
    fp32 by 2^-23 -- far below what a rounded product position x frequency leaves
    (2^-22 radians and more)."""
    c = Case(nf.NF_KV_BF16, batch=1, n_new=1, dtype=torch.float32, n_axes=1, theta=3.0, strided=False, before=(5,))
    for x in (c.q, c.k):
        x.zero_()
        x[..., :64] = 1.0
    c.np_pos[:] = pos
    c.run()
    want = c.turned(c.q)
    assert np.abs(c.q_out.double().cpu().numpy() - want).max() <= 2.0 ** -23
    c.check()


@pytest.mark.parametrize("batch, n_new, hq, hkv", [(1, 1, 1, 1), (1, 1, 40, 8), (5, 1, 32, 4), (1, 700, 5, 1), (3, 257, 8, 8)])
def test_sizes(batch, n_new, hq, hkv):
    for fmt in (nf.NF_KV_K8V4, nf.NF_KV_K4V4):
        c = Case(fmt, batch=batch, n_new=n_new, hq=hq, hkv=hkv)
        c.run()
        c.check()


def test_padding_tokens():
    n_valid = [3, 0, 5, -1]
    c = Case(batch=4, n_new=5)
    c.run(torch.tensor(n_valid, dtype=torch.int32, device="cuda"))
    c.check(n_valid)
    c = Case(batch=2, n_new=2)  # more than there are: all
    c.run(torch.tensor([9, 2], dtype=torch.int32, device="cuda"))
    c.check([2, 2])


def test_in_place_and_without_queries():
    c = Case(strided=False, n_new=9, dtype=torch.float32)
    q = c.q.clone()
    nf.nf_rope_append_quant(c.kv, c.rope, torch.as_tensor(c.np_pos, device="cuda"), q, c.k, c.v, c.table, c.lens, q)
    c.q_out = q
    torch.cuda.synchronize()
    c.check()
    d = Case(n_new=9)
    nf.nf_rope_append_quant(d.kv, d.rope, torch.as_tensor(d.np_pos, device="cuda"), None, d.k, d.v, d.table, d.lens, None)
    torch.cuda.synchronize()
    d.q, d.q_out = d.q[:, :, :0], d.q_out[:, :, :0]
    d.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", [nf.NF_ROPE_HALVES, nf.NF_ROPE_PAIRS])
def test_in_place_equals_out_of_place(dtype, layout):
    """Rows of a token in flight (several a half-warp, and over several CTAs) while others are written over q."""
    for n_new, hq, rot in ((300, 64, 96), (1, 40, 128)):
        c = Case(n_new=n_new, hq=hq, rot=rot, layout=layout, dtype=dtype, strided=False)
        c.run()
        want = c.q_out.clone()
        c.run(q_out=c.q)
        assert torch.equal(c.q, want)


def test_position_zero_is_the_plain_append():
    c = Case(n_axes=1, n_new=30, strided=False)
    c.np_pos[:] = 0
    c.run()
    plain = nf.KVLayer.empty(c.fmt, c.kv.num_blocks, c.kv.num_kv_heads, fill=0xA5)
    nf.nf_kv_append_quant(plain, c.k, c.v, c.table, c.lens)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c.kv.planes(), plain.planes()))
    assert torch.equal(c.q_out, c.q)


def test_bad_pages_are_reported_and_skipped():
    c = Case(batch=1, n_new=10, before=(250,))
    was = [p.clone() for p in c.kv.planes()]
    c.table.fill_(-1)
    c.run()
    assert nf.nf_get_device_error() == nf.NF_DEVERR_BLOCK_ID
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(was, c.kv.planes()))
    c.check_q()
    c = Case(batch=1, n_new=10, before=(250,))
    c.lens.fill_(c.table.shape[1] * 256 - 4)
    c.run()
    assert nf.nf_get_device_error() == nf.NF_DEVERR_TABLE
    c.lens.fill_(-4)
    c.run()
    assert nf.nf_get_device_error() == nf.NF_DEVERR_TABLE


def test_side_stream_and_graph():
    c = Case(n_new=4)
    pos = torch.as_tensor(c.np_pos, device="cuda")

    def call(stream=None):
        nf.nf_rope_append_quant(c.kv, c.rope, pos, c.q, c.k, c.v, c.table, c.lens, c.q_out, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.before = [17, 300]
    c.lens.copy_(torch.tensor(c.before, dtype=torch.int32))
    c.np_pos = c.np_pos + 5
    pos.copy_(torch.as_tensor(c.np_pos))
    graph.replay()
    torch.cuda.synchronize()
    c.check()


def test_rope_binding_refusals():
    c = Case(n_new=2)
    pos = torch.as_tensor(c.np_pos, device="cuda")

    def call(**over):
        a = dict(pos=pos, q=c.q, k=c.k, v=c.v, table=c.table, lens=c.lens, out=c.q_out, valid=None)
        a.update(over)
        nf.nf_rope_append_quant(c.kv, c.rope, a["pos"], a["q"], a["k"], a["v"], a["table"], a["lens"], a["out"], a["valid"])

    call()
    for over in (dict(pos=pos[..., :2]), dict(pos=pos.long()), dict(q=c.q.float()), dict(k=c.k[:, :, :1]), dict(v=c.v[..., ::2]),
                 dict(v=c.v[:1]), dict(k=c.k.transpose(1, 2)), dict(table=c.table[:1]), dict(lens=c.lens.cpu()),
                 dict(out=c.q_out[:, :1]), dict(out=None), dict(valid=c.lens[:1]), dict(out=c.q_out.float()),
                 dict(q=torch.empty((2, 2, 8, 128), dtype=torch.bfloat16, device="cuda")[:, :, ::2])):
        with pytest.raises(nf.NfError):
            call(**over)
    with pytest.raises(nf.NfError):
        nf.Rope(c.rope.inv_freq, [0, 3], 3)
    torch.cuda.synchronize()
    assert nf.nf_get_device_error() == 0

"""A windowed session as a server runs it: pages reserved, tokens turned and
appended, attention under the window, pages released behind it, sequences
forked, the pool compacted -- checked at every step against attention over the
whole history."""
import numpy as np
import pytest
import torch

import long_context_quantized_b200 as nf
import sessionref as ref

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5
HQ, HKV, AXES = 8, 2, 3


def dev(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda").contiguous()


class Session:
    def __init__(self, fmt, rows, width, blocks, window, n_sink, layers=2):
        self.rng = np.random.default_rng(1)
        self.rows, self.width, self.window, self.n_sink, self.fmt = rows, width, window, n_sink, fmt
        self.kvs = [nf.KVLayer.empty(fmt, blocks, HKV, fill=0xFF) for _ in range(layers)]
        self.layers = nf.KVLayers(self.kvs)
        self.refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        self.table = dev(np.full((rows, width), -1))
        self.lens = dev(np.zeros(rows))
        self.sinks = dev(np.full(rows, n_sink))
        self.inv = (1e4 ** (-np.arange(64) / 64)).astype(np.float32)
        self.axis = [i % AXES for i in range(64)]
        self.rope = nf.Rope(torch.as_tensor(self.inv, device="cuda"), self.axis, AXES)
        self.ws = torch.zeros(nf.nf_decode_attn_window_workspace_size(rows, 4, HQ, HKV, width * 256), dtype=torch.uint8,
                              device="cuda")
        self.pages_ws = torch.empty(nf.nf_kv_pages_workspace_size(blocks, rows), dtype=torch.uint8, device="cuda")
        self.history = [[(np.zeros((0, HKV, 128), np.float32),) * 2 for _ in range(rows)] for _ in range(layers)]

    def step(self, n_new, active, prefill=False):
        """n_new tokens on the active rows; the others are unused rows of the batch."""
        live = np.asarray(active)
        add = dev(np.where(live, n_new, 0))
        to = self.lens + add
        nf.nf_kv_reserve(self.refs, self.table, self.lens, to)
        pos = self.rng.integers(0, 100000, (self.rows, n_new, AXES)).astype(np.int32)
        seen = torch.where(add > 0, to, torch.zeros_like(to))
        outs = []
        for i, kv in enumerate(self.kvs):
            qkv = torch.as_tensor(self.rng.standard_normal((self.rows, n_new, HQ + 2 * HKV, 128)), dtype=torch.bfloat16,
                                  device="cuda")
            q, k, v = qkv.split([HQ, HKV, HKV], dim=2)
            turned = torch.empty((self.rows, n_new, HQ, 128), dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(turned)
            nf.nf_rope_append_quant(kv, self.rope, torch.as_tensor(pos, device="cuda"), q, k, v, self.table, self.lens, turned,
                                    add)
            if prefill:
                nf.nf_prefill_attn_window(kv, turned, self.table, seen, self.width * 256, self.window, self.n_sink, SCALE, out)
            else:
                nf.nf_decode_attn_window(kv, turned, self.table, seen, self.width * 256, self.window, self.n_sink, SCALE, out,
                                         None, self.ws)
            kt = ref.rope_rows(k.double().cpu().numpy(), pos, self.inv, self.axis, nf.NF_ROPE_HALVES, 128)
            for b in np.nonzero(live)[0]:
                hk, hv = self.history[i][b]
                self.history[i][b] = (np.concatenate([hk, kt[b].astype(np.float32)]),
                                      np.concatenate([hv, v[b].float().cpu().numpy()]))
            outs.append((turned, out))
        self.lens = to.contiguous()
        # the next query, at position len, sees (len - window, len] and the sinks
        nf.nf_kv_release(self.refs, self.table, self.sinks, (self.lens + 1 - self.window).clamp(min=0))
        torch.cuda.synchronize()
        assert nf.nf_get_device_error() == 0
        self.check(outs, live, n_new, prefill)

    def check(self, outs, live, n_new, prefill):
        lens = self.lens.tolist()
        pages = -(-max(lens) // 256)
        for (q, out), rows in zip(outs, self.history):
            # the whole history in a pool of its own
            whole = nf.KVLayer.empty(self.fmt, pages * self.rows, HKV, fill=0)
            table = np.arange(pages * self.rows, dtype=np.int32).reshape(self.rows, pages)
            for b, (k, v) in enumerate(rows):
                if len(k):
                    nf.nf_kv_append_quant(whole, torch.as_tensor(k, device="cuda")[None], torch.as_tensor(v, device="cuda")[None],
                                          dev(table[b:b + 1]), dev([0]))
            o, _, parts = ref.window_attention(whole, q, table, [n if on else 0 for n, on in zip(lens, live)], self.window,
                                               self.n_sink, SCALE)
            ref.check_out(out, o, ref.prefill_tolerance(parts) if prefill else ref.decode_tolerance(parts))

    def held(self):
        t = self.table.cpu().numpy()
        count = np.zeros(len(self.refs), np.int64)
        np.add.at(count, t[t >= 0], 1)
        assert count.tolist() == self.refs.tolist()  # every count stands for table entries
        return int((count > 0).sum())

    def fork(self, src, dst):
        nf.nf_kv_fork(self.layers, self.refs, self.table, dev(src), dev(dst), self.lens, self.pages_ws)
        for hist in self.history:
            for s, d in zip(src, dst):
                hist[d] = hist[s]

    def compact(self):
        nf.nf_kv_compact(self.layers, self.refs, self.table, self.pages_ws)


@pytest.mark.parametrize("fmt", [nf.NF_KV_K8V4, nf.NF_KV_K4V4, nf.NF_KV_F8])
def test_windowed_session(fmt):
    s = Session(fmt, rows=5, width=9, blocks=24, window=300, n_sink=4)
    on = [True, True, False, False, False]
    if fmt == nf.NF_KV_K8V4:
        s.step(700, on, prefill=True)
        s.step(333, on, prefill=True)
    else:
        for _ in range(13):
            s.step(4, [True, True, True, False, False])
        s.step(1, [False, True, True, False, False])
    s.held()
    for _ in range(3):
        s.step(1, on)
    s.step(4, on)                      # drafts
    s.fork([0, 0, 1], [2, 3, 4])       # continuations, over whatever the rows held
    s.held()
    for _ in range(3):
        s.step(1, [True] * 5)
    s.compact()
    n = s.held()
    assert not s.refs[n:].any()
    s.step(2, [True, False, True, True, True])
    # a sequence ends
    end = dev([0] * 5)
    nf.nf_kv_release(s.refs, s.table, end, dev([0, 9 * 256, 0, 0, 0]))
    s.lens[1] = 0
    for hist in s.history:
        hist[1] = (hist[1][0][:0], hist[1][1][:0])
    s.held()
    s.fork([4], [1])
    s.compact()
    s.step(4, [True] * 5)
    s.held()


def test_a_long_session_stays_within_its_pages():
    """Window 300 and 4 sinks hold at most 1 + 3 pages a row, whatever the length."""
    s = Session(nf.NF_KV_K8V4, rows=2, width=40, blocks=12, window=300, n_sink=4, layers=1)
    for _ in range(20):
        s.step(256, [True, True], prefill=True)
        assert s.held() <= 2 * 4
    s.step(1, [True, True])

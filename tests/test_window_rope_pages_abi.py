"""Host-side checks of the windowed-session calls: what they refuse before any
launch.  No GPU is needed; the pointers are never followed."""
import ctypes

import pytest

import long_context_quantized_b200 as nf


@pytest.fixture(scope="module")
def lib():
    from long_context_quantized_b200 import build
    build.build()
    return nf.load_library()


def _layer(fmt=nf.NF_KV_K8V4, heads=2, blocks=4, block=256, ptr=256):
    return nf.nf_kv_layer(fmt, blocks, block, heads, 128, 32, ptr, ptr, ptr, ptr)


INV, UNS, WS = nf.NF_ERR_INVALID_ARG, nf.NF_ERR_UNSUPPORTED, nf.NF_ERR_WORKSPACE


def _window(lib, name, **over):
    a = dict(kv=_layer(), q=256, q_dtype=nf.NF_BF16, batch=1, n_q=1, H_q=4, bt=256, max_blocks=4, seqlens=256,
             max_seqlen=1000, window=128, n_sink=4, scale=0.088, out=256, out_dtype=nf.NF_BF16, lse=None, ws=256,
             ws_bytes=1 << 20)
    a.update(over)
    args = [None if a["kv"] is None else ctypes.byref(a["kv"]), a["q"], a["q_dtype"], a["batch"], a["n_q"], a["H_q"],
            a["bt"], a["max_blocks"], a["seqlens"], a["max_seqlen"], a["window"], a["n_sink"], a["scale"], a["out"],
            a["out_dtype"], a["lse"]]
    if name == "nf_decode_attn_window":
        args += [a["ws"], a["ws_bytes"]]
    return getattr(lib, name)(*args, None)


@pytest.mark.parametrize("name", ["nf_decode_attn_window", "nf_prefill_attn_window"])
@pytest.mark.parametrize("over, status", [
    (dict(kv=None), INV), (dict(window=0), INV), (dict(window=-3), INV), (dict(n_sink=-1), INV), (dict(scale=0.0), INV),
    (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(out_dtype=nf.NF_F16), UNS), (dict(out_dtype=9), UNS), (dict(max_seqlen=(1 << 30) + 1, max_blocks=1 << 23), UNS),
    (dict(max_seqlen=2000), INV), (dict(max_seqlen=0), INV), (dict(H_q=3), INV), (dict(n_q=0), INV), (dict(batch=0), INV),
    (dict(q=None), INV), (dict(out=None), INV), (dict(bt=None), INV), (dict(seqlens=None), INV), (dict(out=264), INV),
    (dict(q=260), INV), (dict(kv=_layer(block=128)), UNS), (dict(kv=_layer(ptr=264)), INV), (dict(q_dtype=nf.NF_F16), UNS)])
def test_window_refusals(lib, name, over, status):
    assert _window(lib, name, **over) == status
    assert lib.nf_last_error()


def test_prefill_window_takes_only_k8v4_and_bf16(lib):
    for fmt in (nf.NF_KV_K8V8, nf.NF_KV_F8, nf.NF_KV_K4V4, nf.NF_KV_BF16):
        assert _window(lib, "nf_prefill_attn_window", kv=_layer(fmt)) == UNS
    assert _window(lib, "nf_prefill_attn_window", q_dtype=nf.NF_F32) == UNS
    assert _window(lib, "nf_prefill_attn_window", H_q=2 << 21) == UNS  # above 2^20 q-heads per kv-head
    assert _window(lib, "nf_prefill_attn_window", H_q=4, n_q=1 << 30, max_seqlen=1 << 30, max_blocks=1 << 23) == UNS


def test_window_workspace_size(lib):
    assert nf.nf_decode_attn_window_workspace_size(2, 4, 32, 4, 90112, 148) \
        == nf.nf_decode_attn_workspace_size(2, 4, 32, 4, 90112, 148) > 0
    assert nf.nf_decode_attn_window_workspace_size(1, 9, 32, 4, 1000, 148) == 0  # 72 rows per kv-head


def _rope(lib, **over):
    a = dict(kv=_layer(), rot=128, layout=0, n_axes=3, axis=[i % 3 for i in range(64)], inv=256, pos=256, q=256, k=256,
             v=256, bs=768, ts=768, dtype=nf.NF_BF16, batch=1, n_new=1, H_q=2, bt=256, max_blocks=4, before=256, valid=None,
             q_out=256, rope=True, rows=True)
    a.update(over)
    rope = nf.nf_rope(a["rot"], a["layout"], a["n_axes"], (ctypes.c_uint8 * 64)(*a["axis"]), a["inv"])
    rows = (nf.nf_heads * 3)(*[nf.nf_heads(a[x], a["bs"], a["ts"]) for x in ("q", "k", "v")])
    return lib.nf_rope_append_quant(None if a["kv"] is None else ctypes.byref(a["kv"]),
                                    ctypes.byref(rope) if a["rope"] else None, a["pos"], rows if a["rows"] else None, a["dtype"], a["batch"],
                                    a["n_new"], a["H_q"], a["bt"], a["max_blocks"], a["before"], a["valid"], a["q_out"], None)


@pytest.mark.parametrize("over, status", [
    (dict(kv=None), INV), (dict(rope=False), INV), (dict(rows=False), INV), (dict(rot=4), UNS), (dict(rot=12), UNS), (dict(rot=136), UNS),
    (dict(rot=0), UNS), (dict(layout=2), UNS), (dict(n_axes=0), UNS), (dict(n_axes=5), UNS), (dict(n_axes=2), INV),
    (dict(batch=-1), INV), (dict(n_new=-1), INV), (dict(H_q=-1), INV), (dict(dtype=nf.NF_F16), UNS), (dict(inv=None), INV),
    (dict(pos=None), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(bt=None), INV),
    (dict(before=None), INV), (dict(q_out=None), INV), (dict(max_blocks=0), INV), (dict(k=260), INV), (dict(q_out=260), INV),
    (dict(ts=770), INV), (dict(bs=2), INV), (dict(dtype=nf.NF_F32, q=264), INV), (dict(batch=2, n_new=1 << 30), INV), (dict(batch=70000), UNS),
    (dict(H_q=1 << 21), INV)])
def test_rope_refusals(lib, over, status):
    assert _rope(lib, **over) == status
    assert lib.nf_last_error()


def test_rope_with_nothing_to_append(lib):
    assert _rope(lib, n_new=0, k=None, v=None, q=None, pos=None) == 0
    assert _rope(lib, batch=0) == 0


def test_page_refusals(lib):
    for name in ("nf_kv_reserve", "nf_kv_release"):
        f = getattr(lib, name)
        assert f(256, 8, 256, 0, 4, None, None, None) == 0  # no rows
        assert f(None, 8, 256, 1, 4, 256, 256, None) == INV
        assert f(256, 8, None, 1, 4, 256, 256, None) == INV
        assert f(256, 8, 256, 1, 4, None, 256, None) == INV
        assert f(256, 0, 256, 1, 4, 256, 256, None) == INV
        assert f(256, (1 << 30) + 1, 256, 1, 4, 256, 256, None) == INV
        assert f(256, 8, 256, -1, 4, 256, 256, None) == INV
        assert f(256, 8, 256, 1, 0, 256, 256, None) == INV
        assert f(258, 8, 256, 1, 4, 256, 256, None) == INV
    layers = (nf.nf_kv_layer * 2)(_layer(), _layer())
    mixed = (nf.nf_kv_layer * 2)(_layer(), _layer(fmt=nf.NF_KV_F8))
    sizes = (nf.nf_kv_layer * 2)(_layer(), _layer(blocks=5))
    wide = (nf.nf_kv_layer * 1)(_layer(heads=60000))
    assert lib.nf_kv_copy_blocks(layers, 2, None, None, 0, None) == 0
    assert lib.nf_kv_copy_blocks(layers, 2, None, 256, 1, None) == INV
    assert lib.nf_kv_copy_blocks(layers, 2, 256, 256, -1, None) == INV
    for bad, n, status in ((None, 1, INV), (layers, 0, UNS), (layers, 129, UNS), (mixed, 2, INV), (sizes, 2, INV),
                           (wide, 1, UNS)):
        assert lib.nf_kv_copy_blocks(bad, n, 256, 256, 1, None) == status
        assert lib.nf_kv_fork(bad, n, 256, 256, 4, 4, 256, 256, 1, 256, 256, 1 << 20, None) == status
        assert lib.nf_kv_compact(bad, n, 256, 256, 4, 4, 256, 1 << 20, None) == status
    assert lib.nf_kv_fork(layers, 2, 256, 256, 4, 4, 256, 256, 0, 256, None, 0, None) == 0  # no pairs
    assert lib.nf_kv_fork(layers, 2, 256, 256, 4, 4, 256, 256, -1, 256, 256, 1 << 20, None) == INV
    assert lib.nf_kv_fork(layers, 2, 256, 256, 4, 4, 256, 256, 1025, 256, 256, 1 << 20, None) == UNS
    assert lib.nf_kv_fork(layers, 2, 256, 256, 4, 4, 256, 256, 3, None, 256, 1 << 20, None) == INV
    assert lib.nf_kv_fork(layers, 2, 256, 256, 4, 4, 256, 256, 3, 256, 256, 59, None) == WS
    assert lib.nf_kv_fork(layers, 2, 256, 256, 4, 4, 256, 256, 3, 256, 264, 1 << 20, None) == INV
    assert lib.nf_kv_compact(layers, 2, 256, 256, 4, 4, 256, 16, None) == WS
    assert lib.nf_kv_compact(layers, 2, 256, 256, 4, 4, 264, 1 << 20, None) == INV
    assert nf.nf_kv_pages_workspace_size(0) == 0 and nf.nf_kv_pages_workspace_size(8, 1025) == 0
    assert nf.nf_kv_pages_workspace_size(720, 32) >= (16 + 2 * 361 + 720) * 4


def test_binding_refusals_without_a_device():
    import torch
    cpu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(nf.NfError):
        nf.nf_kv_reserve(cpu, cpu.view(2, 2), cpu[:2], cpu[:2])
    with pytest.raises(nf.NfError):
        nf.Rope(torch.ones(8), n_axes=1)  # not on a device
    with pytest.raises(nf.NfError):
        nf.KVLayers([])


@pytest.mark.parametrize("wide", [2 ** 31, 2 ** 32 + 16, 2 ** 63, -2 ** 31 - 1])
def test_integers_outside_32_bits_are_refused(wide):
    """ctypes keeps an integer's low 32 bits: a window of 2^32 + 16 would run as one of 16.  Refused before
    anything else is looked at."""
    def window(f, *ws):
        for ints in ((wide, 16, 4), (1000, wide, 4), (1000, 16, wide)):
            with pytest.raises(nf.NfError) as e:
                f(None, None, None, None, *ints, 0.1, None, None, *ws)
            assert e.value.status == INV and str(wide) in str(e.value)

    window(nf.nf_decode_attn_window, None)
    window(nf.nf_prefill_attn_window)
    sizes = (1, 1, 32, 4, 1000, 148)
    calls = [lambda: nf.nf_decode_attn(None, None, None, None, wide, 0.1, True, None),
             lambda: nf.nf_decode_attn_ex(None, None, None, None, 1000, 0.1, True, wide, None),
             lambda: nf.nf_decode_attn_noalloc(None, None, None, None, wide, 0.1, True, None),
             lambda: nf.nf_prefill_attn(None, None, None, None, wide, 0.1, True, None),
             lambda: nf.nf_attn_packed_slot_floats(wide), lambda: nf.nf_attn_packed_slot_floats(8, wide),
             lambda: nf.nf_attn_combine_packed(None, wide, None), lambda: nf.nf_selftest_bounded_wait(wide),
             lambda: nf.nf_kv_pages_workspace_size(wide), lambda: nf.nf_kv_pages_workspace_size(8, wide),
             lambda: nf.Rope(None, n_axes=wide), lambda: nf.Rope(None, layout=wide)]
    for i in range(6):
        for f in (nf.nf_decode_attn_workspace_size, nf.nf_decode_attn_window_workspace_size):
            calls.append(lambda f=f, i=i: f(*sizes[:i], wide, *sizes[i + 1:]))
    for call in calls:
        with pytest.raises(nf.NfError) as e:
            call()
        assert e.value.status == INV and str(wide) in str(e.value)


def test_package_imports_on_a_torch_without_cuda():
    """Shard plans and the CPU tests need no CUDA build, which is what has the raw stream lookup."""
    import os
    import subprocess
    import sys
    code = ("import torch; del torch._C._cuda_getCurrentRawStream; "
            "import long_context_quantized_b200.sharded as s; print(s.local_pool_table.__name__)")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "local_pool_table" in done.stdout, done.stderr

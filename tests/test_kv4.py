"""The paged 4-bit cache without a GPU: refusals of the C ABI and of the binding,
sizes, and the reference the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import kv4_ref as R
from exact_io_aware_40_gb300 import build as fab

FAKE, ODD, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    fab.build()
    from exact_io_aware_40_gb300 import fa
    return fa.load_library()


def call(fn, good, **bad):
    args = dict(good, **bad)
    return fn(*args.values())


PLAN = dict(past=FAKE, new=FAKE, B=4, page=64, pages=100, table=FAKE, width=8, ring=FAKE, state=FAKE,
            tokens=16, kv=FAKE, cu=FAKE, slots=FAKE, out=FAKE, stream=NULL)
APPEND = dict(K=FAKE, V=FAKE, T=4, H=2, d=128, kt=512, kh=128, vt=512, vh=128, slots=FAKE, cache=FAKE,
              pages=10, page=16, group=32, stream=NULL)
GATHER = dict(slots=FAKE, cache=FAKE, pages=10, page=16, group=32, T=4, H=2, d=64, K=FAKE, V=FAKE, stream=NULL)
ATTN = dict(Q=FAKE, cache=FAKE, table=FAKE, cu=FAKE, kv=FAKE, O=FAKE, L=FAKE, B=2, total=4, max_q=2, Hq=8,
            Hkv=2, d=128, qt=1024, qh=128, pages=10, width=4, page=16, group=32,
            scale=ctypes.c_float(0.1), causal=1, window=-1, ws=FAKE, bytes=1 << 30, stream=NULL)


@pytest.mark.parametrize("bad,status", [
    (dict(past=NULL), 1), (dict(out=NULL), 1), (dict(B=0), 1), (dict(pages=0), 1), (dict(width=0), 1),
    (dict(tokens=0), 1), (dict(page=24), 2), (dict(page=256), 2), (dict(B=8193), 2),
    (dict(pages=1 << 26), 2), (dict(width=1 << 26), 2), (dict(slots=ctypes.c_void_p(0x10002)), 1)])
def test_plan_refuses(lib, bad, status):
    assert call(lib.fa_kv4_plan, PLAN, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(K=NULL), 1), (dict(K=ODD), 1), (dict(V=ODD), 1), (dict(cache=ODD), 1), (dict(T=0), 1), (dict(H=0), 1),
    (dict(kt=516), 1), (dict(vh=-128), 1), (dict(d=96), 2), (dict(group=128), 2), (dict(page=8), 2),
    (dict(pages=0), 1), (dict(pages=1 << 28), 2), (dict(H=65536), 2), (dict(T=(1 << 30) + 1), 2)])
def test_append_refuses(lib, bad, status):
    assert call(lib.fa_kv4_append, APPEND, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(K=NULL), 1), (dict(V=ODD), 1), (dict(slots=NULL), 1), (dict(T=0), 1), (dict(d=32), 2), (dict(group=16), 2),
    (dict(T=(1 << 30) + 1), 2)])
def test_gather_refuses(lib, bad, status):
    assert call(lib.fa_kv4_gather, GATHER, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(Q=NULL), 1), (dict(Q=ODD), 1), (dict(ws=NULL), 1), (dict(ws=ctypes.c_void_p(0x10010)), 1),
    (dict(bytes=64), 1), (dict(B=0), 1), (dict(total=0), 1), (dict(max_q=0), 1), (dict(Hq=7), 1),
    (dict(Hq=0), 1), (dict(d=80), 2), (dict(qt=12), 1), (dict(qh=-8), 1), (dict(window=-2), 1),
    (dict(scale=ctypes.c_float(0.0)), 1), (dict(scale=ctypes.c_float(3e38)), 1), (dict(scale=ctypes.c_float(float("nan"))), 1), (dict(width=0), 1),
    (dict(width=1 << 27), 2), (dict(max_q=1 << 29), 2), (dict(page=48), 2), (dict(total=(1 << 30) + 1), 2)])
def test_attention_refuses(lib, bad, status):
    assert call(lib.fa_kv4_attn, ATTN, **bad) == status


def test_sizes(lib):
    from exact_io_aware_40_gb300 import fa
    for d in (64, 128, 256):
        for page in (16, 32, 64, 128):
            for group in (32, 64):
                assert fa.kv4_page_bytes(d, page, group) == R.sections(page, d, group)[-1][1]
    for bad in ((96, 16, 32), (64, 20, 32), (64, 16, 128)):
        assert lib.fa_kv4_page_bytes(*bad) == 0
        with pytest.raises(ValueError):
            fa.kv4_page_bytes(*bad)
    assert fa.kv4_attention_workspace_bytes(8, 2, 128, 1) > 0
    for bad in ((8, 3, 128, 1), (0, 1, 128, 1), (8, 2, 96, 1), (8, 2, 128, 0)):
        assert fa.kv4_attention_workspace_bytes(*bad) == 0


def test_workspace_of_a_call(lib):
    most = lib.fa_kv4_attn_workspace_bytes
    need = lib.fa_kv4_attn_call_workspace_bytes
    # B, total_q, max_q, Hq, Hkv, d, max_pages, page_size, window
    assert need(2, 4, 2, 8, 2, 128, 32, 16, -1) == 0          # 512 tokens
    assert need(2, 4, 2, 8, 2, 128, 33, 16, -1) == most(8, 2, 128, 2)
    assert need(2, 4, 2, 8, 2, 128, 1000, 16, 100) == 0       # a window as short
    assert need(2, 4, 2, 8, 2, 128, 1000, 16, 1000) == most(8, 2, 128, 2)
    assert need(2, 600, 300, 8, 2, 128, 1000, 16, -1) == most(8, 2, 128, 300)
    assert need(2, 4, 2, 8, 3, 128, 32, 16, -1) == 0          # no such heads
    assert call(lib.fa_kv4_attn, ATTN, ws=NULL, bytes=0, width=40) == 1
    assert call(lib.fa_kv4_attn, ATTN, ws=NULL, bytes=0, width=4, B=0) == 1


def test_binding_has_no_cpu_path():
    import torch
    from exact_io_aware_40_gb300 import fa
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    cache = fa.kv4_cache(3, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_plan(i32(2), i32(2), i32(2, 4), i32(9), i32(2), 16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_append(bf(4, 2, 64), bf(4, 2, 64), i32(4), cache, 16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_gather(i32(4), cache, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_attention(bf(2, 4, 64), cache, i32(2, 2), i32(3), i32(2), 1, 16)
    with pytest.raises(ValueError):
        fa.kv4_plan(i32(2), i32(2), i32(8), i32(9), i32(2), 16, 8)


def test_reference_round_trip():
    # pack / unpack, and quantisation within half a step of every value
    rng = np.random.default_rng(0)
    c = rng.integers(0, 16, (5, 128))
    assert np.array_equal(R.unpack(R.pack(c)), c)
    assert R.pack(np.arange(8)[None] % 16).tobytes() == bytes([0x20, 0x64, 0x31, 0x75])
    x = R.bf16_value(R.bf16_bits(rng.standard_normal((7, 128))))
    codes, sb, mb = R.quantise(x, 32)
    off = np.abs(R.values(codes, sb, mb, 32) - x).reshape(7, 4, 32)
    # the largest value may miss by the scale's own rounding: 15 * half a step of it
    assert (off <= R.bf16_value(sb)[..., None] * (0.5 + 15 * 2.0 ** -8)).all()


def test_reference_plan_by_hand():
    # two-token steps on pages of 16: request 0 crosses a page, 1 is finished, 2 fits its page
    table = np.array([[5, 0, 0], [7, 3, 0], [1, 0, 0]], np.int32)
    ring = np.array([9, 8, 2, -1, -1, -1, -1, -1, -1, -1], np.int32)
    kv, cu, slots, state, t, r = R.plan([15, 17, 3], [2, -1, 1], table, ring, 0, 3, 16, 4)
    assert kv.tolist() == [17, 0, 4] and cu.tolist() == [0, 2, 2, 3]
    assert slots.tolist() == [5 * 16 + 15, 9 * 16, 16 + 3, -1]
    assert state.tolist() == [1, 4, 3, 3]
    assert t[0].tolist() == [5, 9, 0] and r[:5].tolist() == [9, 8, 2, 7, 3]

"""The paged 4-bit cache on the GPU against its plain 64-bit restatement."""
import numpy as np
import pytest

import kv4_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from exact_io_aware_40_gb300 import build as fab, fa
    fab.build()
    fa.load_library()
    return fa


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def dev_bf16(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def i32(x):
    return dev(np.asarray(x, np.int32))


# ------------------------------------------------------------------ plan

def plan_case(rng, B, page, width, pool, done=0.1, prompt=0.2, tight=None):
    room = width * page
    past = rng.integers(0, room, B)
    new = np.where(rng.random(B) < prompt, rng.integers(0, room + 1, B), 1)
    new = np.minimum(new, room - past)
    new = np.where(rng.random(B) < done, -1, new)
    held = -(-past // page)
    F = int(held.sum()) + pool
    ids = rng.permutation(F).astype(np.int32)
    table = rng.integers(0, F, (B, width)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    head, count = int(rng.integers(0, F)), F - at
    ring = np.full(F, -1, np.int32)
    ring[(head + np.arange(count)) % F] = ids[at:]
    return past, new, table, ring, head, count


def run_plan(fa, past, new, table, ring, head, count, page, cap):
    t, r = dev(table.copy()), dev(ring.copy())
    args = (i32(past), i32(new), t, r, i32([head, count]), page, cap)
    first = [x.cpu().numpy().copy() for x in fa.kv4_plan(*args)] + [t.cpu().numpy(), r.cpu().numpy()]
    again = [x.cpu().numpy() for x in fa.kv4_plan(*args)] + [t.cpu().numpy(), r.cpu().numpy()]
    for a, b in zip(first, again):  # a repeated call changes nothing
        assert np.array_equal(a, b)
    return first


def check_plan(fa, case, page, cap):
    got = run_plan(fa, *case, page, cap)
    for g, w, name in zip(got, R.plan(*case, page, cap), ("kv_len", "cu_q", "slots", "state", "table", "ring")):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("B,page,width", [(1, 16, 1), (3, 16, 5), (33, 64, 7), (257, 32, 9), (1000, 128, 4),
                                          (1500, 16, 12)])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan(fa, B, page, width, seed):
    rng = np.random.default_rng(100 * B + seed)
    case = plan_case(rng, B, page, width, pool=B * width)
    need = int(np.maximum(case[1], 0).sum())
    check_plan(fa, case, page, max(1, need + 5))
    fa.fa_check_error()


def test_plan_largest_batch(fa):
    rng = np.random.default_rng(9)
    case = plan_case(rng, 8192, 16, 3, pool=8192 * 3)
    check_plan(fa, case, 16, int(np.maximum(case[1], 0).sum()))
    fa.fa_check_error()


@pytest.mark.parametrize("seed", range(4))
def test_plan_stops_at_the_first_request_that_does_not_fit(fa, seed):
    rng = np.random.default_rng(seed)
    case = list(plan_case(rng, 60, 16, 6, pool=25, prompt=0.5))     # the pages run out
    check_plan(fa, case, 16, 4000)
    case = list(plan_case(rng, 60, 16, 6, pool=400, prompt=0.5))    # the places run out
    check_plan(fa, case, 16, 300)
    case[1] = case[1].copy()                                        # lengths that are none
    case[0] = case[0].copy()
    case[1][20] = (-2, 1 << 30, 2147483647, 97)[seed]
    if seed == 3:
        case[0][20] = -1
    check_plan(fa, case, 16, 4000)
    fa.fa_check_error()


def test_plan_reports_a_free_list_that_cannot_be(fa):
    rng = np.random.default_rng(3)
    past, new, table, ring, head, count = plan_case(rng, 5, 16, 4, pool=40, done=0.0)
    bad = ring.copy()
    bad[(head + np.arange(count)) % len(ring)] = len(ring) + 7    # pages that do not exist
    new[:] = 16
    past[:] = 1
    kv, cu, slots, state, t, r = run_plan(fa, past, new, table, bad, head, count, 16, 200)
    assert (slots[:cu[1]] == -1).any()
    with pytest.raises(fa.FAError) as e:
        fa.fa_check_error()
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    fa.fa_check_error()
    out = run_plan(fa, past, new, table, ring, len(ring) + 3, count, 16, 200)  # no such first entry
    assert out[3].tolist()[1:] == [0, 0, 0]
    with pytest.raises(fa.FAError):
        fa.fa_check_error()


# ------------------------------------------------------------------ append, gather

def special_rows(rng, T, H, d):
    """Keys of every kind: ordinary, constant, zero, with ties, tiny, huge, mixed."""
    x = rng.standard_normal((T, H, d))
    kind = np.arange(T) % 9
    x[kind == 1] = 0.75
    x[kind == 2] = 0.0
    x[kind == 3] = np.round(x[kind == 3] * 4) / 4           # many ties
    x[kind == 4] *= 2.0 ** -120
    x[kind == 5] *= 2.0 ** 124
    x[kind == 6] *= 2.0 ** rng.integers(-100, 100, (int((kind == 6).sum()), H, d))
    x[kind == 7] = np.where(rng.random(x[kind == 7].shape) < 0.5, 3.3e38, -3.3e38)
    x[kind == 8] = rng.integers(0, 16, x[kind == 8].shape) * 2.0 ** -130   # subnormal
    return R.bf16_bits(np.clip(x, -3.38e38, 3.38e38))


def expect_rows(bits, group):
    return R.quantise(R.bf16_value(bits), group)


@pytest.mark.parametrize("T,H,d,group,page", [(1, 1, 64, 32, 16), (7, 3, 64, 64, 32), (129, 2, 128, 32, 64),
                                              (65, 5, 128, 64, 128), (33, 2, 256, 32, 16), (18, 1, 256, 64, 64)])
@pytest.mark.parametrize("packed", [False, True])
def test_append_and_gather(fa, T, H, d, group, page, packed):
    import torch
    rng = np.random.default_rng(T * d + group)
    kb, vb = special_rows(rng, T, H, d), special_rows(rng, T, H, d)
    pages = (T + page - 1) // page + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    skip = (rng.random(T) < 0.2) & (T > 1)
    slots = np.where(skip, -1, slots).astype(np.int32)
    fill = rng.integers(0, 256, (pages, H, fa.kv4_page_bytes(d, page, group))).astype(np.uint8)
    cache = dev(fill.copy())
    if packed:  # views of one projection: strides of another layout
        qkv = torch.zeros(T, 2 * H + 4, d + 8, dtype=torch.bfloat16, device="cuda")
        k, v = qkv[:, 1:1 + H, 8:], qkv[:, H + 3:2 * H + 3, :d]
        k.copy_(dev_bf16(kb))
        v.copy_(dev_bf16(vb))
    else:
        k, v = dev_bf16(kb), dev_bf16(vb)
    fa.kv4_append(k, v, dev(slots), cache, page, group)
    fa.fa_check_error()
    got = cache.cpu().numpy()
    keep = slots >= 0
    for part, bits in zip(R.token_rows(got, slots[keep], page, d, group), (kb, vb)):
        want = expect_rows(bits[keep], group)
        for g, w, name in zip(part, want, ("codes", "scale", "minimum")):
            if name == "minimum":  # a minimum of zero has no sign to keep
                g, w = np.where(g == 0x8000, 0, g), np.where(w == 0x8000, 0, w)
            assert np.array_equal(g, w), name
    # nothing else was written
    written = np.zeros((pages, H, page), bool)
    written[slots[keep] // page, :, slots[keep] % page] = True
    for lo, hi in R.sections(page, d, group):
        a = fill[..., lo:hi].reshape(pages, H, page, -1)[~written]
        assert np.array_equal(a, got[..., lo:hi].reshape(pages, H, page, -1)[~written])
    # and back
    ok, ov = (torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.kv4_gather(dev(slots), cache, page, d, group, out_k=ok, out_v=ov)
    fa.fa_check_error()
    for o, bits in ((ok, kb), (ov, vb)):
        o = o.view(torch.int16).cpu().numpy().view(np.uint16)
        assert (o[~keep] == R.bf16_bits(7.0)).all()
        val = R.values(*expect_rows(bits[keep], group), group)
        with np.errstate(over="ignore"):  # past bf16's range: infinity
            want = R.bf16_bits(val)        # rounded once (through fp32 it would be twice)
        assert np.array_equal(np.where(o[keep] == 0x8000, 0, o[keep]), np.where(want == 0x8000, 0, want))


def test_append_marks_groups_that_are_not_numbers(fa):
    import torch
    k = torch.zeros(3, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 5], k[1, 0, 40], k[2, 0, 127] = float("nan"), float("inf"), float("-inf")
    k[:, :, 64] = 1.0
    cache = fa.kv4_cache(1, 1, 16, 128)
    fa.kv4_append(k, k, i32([3, 0, 9]), cache, 16)
    gk, gv = fa.kv4_gather(i32([3, 0, 9]), cache, 16, 128)
    for g in (gk, gv):
        nan = torch.isnan(g).view(3, 4, 32)
        assert nan.all(-1).cpu().tolist() == [[True, False, False, False], [False, True, False, False],
                                              [False, False, False, True]]
        assert (nan.any(-1) == nan.all(-1)).all()
        assert (g[:, 0, 64] == 1).all()


def test_rows_outside_the_cache_are_skipped_and_reported(fa):
    import torch
    cache = torch.zeros(2, 1, fa.kv4_page_bytes(64, 16, 32), dtype=torch.uint8, device="cuda")
    k = torch.randn(4, 1, 64, device="cuda").bfloat16()
    fa.kv4_append(k, k, i32([0, 32, -5, 31]), cache, 16)
    with pytest.raises(fa.FAError) as e:
        fa.fa_check_error()
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    got, _ = fa.kv4_gather(i32([0, 31]), cache, 16, 64)
    assert (got - k[[0, 3]]).abs().max() < 0.3 and got.abs().max() > 0.5
    fa.fa_check_error()
    out = torch.full((3, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.kv4_gather(i32([1 << 30, -1, -7]), cache, 16, 64, out_k=out, out_v=out.clone())
    assert (out == 3).all()
    with pytest.raises(fa.FAError):
        fa.fa_check_error()
    # the word of input errors ends no other kernel's work
    fa.kv4_append(k, k, i32([0, 99, 1, 2]), cache, 16)
    q = torch.randn(1, 1, 200, 64, device="cuda").bfloat16()
    o, _ = fa.attention_fwd(q, q, q)
    want = torch.softmax(q.float() @ q.float().transpose(-1, -2) / 8, -1) @ q.float()
    assert (o.float() - want).abs().max() < 2e-2
    with pytest.raises(fa.FAError):
        fa.fa_check_error()


# ------------------------------------------------------------------ attention

def attention_case(seed, lens, nq, heads, per, d, group, page, spread=1.0, spare=2, table_pad=1):
    rng = np.random.default_rng(seed)
    need = [-(-max(l, 0) // page) for l in lens]
    width = max(max(need), 1) + table_pad
    pages = sum(need) + spare
    cache = R.random_cache(rng, pages, heads, page, d, group, spread)
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    q = R.bf16_value(R.bf16_bits(rng.standard_normal((max(int(cu[-1]), 1), heads * per, d))))
    return dict(q=q, cache=cache, table=table, cu=cu, kv_len=np.asarray(lens, np.int32), page=page, group=group,
                scale=1.0 / np.sqrt(d), causal=True, window=-1)


def run_attention(fa, c, max_q=None, **kw):
    max_q = max(1, int(np.diff(c["cu"]).max())) if max_q is None else max_q
    return fa.kv4_attention(dev_bf16(R.bf16_bits(c["q"])), dev(c["cache"]), dev(c["table"]), dev(c["cu"]),
                            dev(c["kv_len"]), max_q, c["page"], c["group"], causal=c["causal"],
                            scale=float(c["scale"]), window=c["window"], **kw)


def compare(o, l, c, rows=None):
    O, L, tol_o, tol_l = R.attention(c["q"], c["cache"], c["table"], c["cu"], c["kv_len"], c["page"], c["group"],
                                     np.float32(c["scale"]).astype(np.float64), c["causal"], c["window"])
    n = int(c["cu"][-1])
    o, l = o.double().cpu().numpy()[:n], l.double().cpu().numpy()[:n]
    O, L, tol_o, tol_l = O[:n], L[:n], tol_o[:n], tol_l[:n]
    assert np.array_equal(np.isnan(o), np.isnan(O)) and np.array_equal(np.isnan(l), np.isnan(L))
    assert np.array_equal(np.isneginf(l), np.isneginf(L))
    f = np.isfinite(O)
    worst = (np.abs(o - O)[f] / (tol_o[f] + 1e-30)).max() if f.any() else 0.0
    assert worst <= 1.0, "O off by %.3g of its bound" % worst
    f = np.isfinite(L)
    worst = (np.abs(l[f] - L[f]) / tol_l[f]).max() if f.any() else 0.0
    assert worst <= 1.0, "L off by %.3g of its bound" % worst
    assert (o[np.isneginf(l)] == 0).all()


def check(fa, c, **kw):
    o, l = run_attention(fa, c, **kw)
    fa.fa_check_error()
    compare(o, l, c)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attention_formats(fa, d, group, page):
    lens = [1, 15, 16, 17, 63, 64, 65, 200, 300]
    check(fa, attention_case(d + page + group, lens, [1] * 9, 2, 4, d, group, page))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,per", [(1, 1), (3, 2), (2, 3), (1, 7), (2, 8), (1, 12), (1, 16), (1, 29), (1, 40)])
def test_attention_heads(fa, d, heads, per):
    check(fa, attention_case(7 * d + per, [1, 130, 77], [1, 1, 1], heads, per, d, 32, 32))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq", [[2], [1, 5, 3], [9, 1, 0, 4], [33, 2, 70], [128, 130, 1]])
@pytest.mark.parametrize("per", [1, 3, 4])
def test_attention_queries(fa, d, nq, per):
    lens = [n + (37 * i * i) % 150 for i, n in enumerate(nq)]
    check(fa, attention_case(d + per + len(nq), lens, nq, 2, per, d, 64 if per == 3 else 32, 16))


@pytest.mark.parametrize("window", [0, 1, 15, 16, 64, 100, 1 << 30, (1 << 31) - 1])
@pytest.mark.parametrize("nq", [[1, 1, 1], [5, 20, 1], [60, 90, 200]])
def test_attention_window(fa, window, nq):
    c = attention_case(window % 97, [300, 129, 513], nq, 2, 2, 64, 32, 16)
    c["window"] = window
    check(fa, c)
    c["causal"] = False  # the window brings the causal bound with it
    check(fa, c)


@pytest.mark.parametrize("nq", [[1, 3], [40, 70]])
def test_attention_without_causal_mask(fa, nq):
    c = attention_case(5, [91, 200], nq, 2, 2, 128, 32, 32)
    c["causal"] = False
    check(fa, c)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_rows_that_see_nothing(fa, d):
    # no keys at all, a length below zero, more queries than keys
    c = attention_case(11, [0, -3, 2, 64, 3], [1, 2, 5, 1, 50], 2, 2, d, 32, 16)
    check(fa, c)
    c = attention_case(12, [0, 0], [1, 1], 1, 4, d, 64, 64)
    check(fa, c)


@pytest.mark.parametrize("d,nq", [(64, 1), (128, 1), (256, 1), (128, 6), (128, 17), (64, 40), (256, 40)])
def test_attention_long(fa, d, nq):
    # long enough for many shares to cut an item
    check(fa, attention_case(d + nq, [20011, 33], [nq, 1], 1, 2, d, 32, 64))


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_of_rising_scores(fa, nq):
    # every tile raises the running maximum by more than the kernels' threshold
    c = attention_case(21, [700], [nq], 1, 4, 64, 32, 16, spread=4.0)
    c["q"] = R.bf16_value(R.bf16_bits(c["q"] * 6.0))
    check(fa, c)


@pytest.mark.parametrize("nq", [1, 7, 60])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_ignores_what_was_never_written(fa, nq, d):
    import torch
    c = attention_case(31, [70, 40 + nq], [min(nq, 70), nq], 2, 2, d, 32, 64)
    used = np.zeros((c["cache"].shape[0], 64), bool)
    for b in range(2):
        for j in range(int(c["kv_len"][b])):
            used[c["table"][b, j // 64], j % 64] = True
    for lo, hi in R.sections(64, d, 32):
        view = c["cache"][..., lo:hi].reshape(c["cache"].shape[0], 2, 64, -1)
        view = np.where(used[:, None, :, None], view, np.uint8(0xff))   # NaN parameters
        c["cache"][..., lo:hi] = view.reshape(c["cache"].shape[0], 2, -1)
    check(fa, c)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("per", [1, 2, 8, 14])
def test_attention_values_that_are_not_numbers(fa, d, per):
    # the newest tokens hold NaN in some groups: only the rows that see them take it
    c = attention_case(41, [90], [9], 1, per, d, 32, 16)
    for which, token in ((1, 85), (1, 89), (0, 88)):
        slot = int(c["table"][0, token // 16]) * 16 + token % 16
        lo, _ = R.sections(16, d, 32)[2 * which + 1]
        at = lo + (slot % 16) * 4 * (d // 32) + 4 * (token % (d // 32))
        c["cache"][slot // 16, 0, at:at + 4] = [0xc0, 0x7f, 0xc0, 0x7f]
    check(fa, c)


def test_attention_strided_queries_and_untouched_rows(fa):
    import torch
    c = attention_case(51, [100, 30, 64], [3, 0, 2], 2, 3, 128, 32, 32)
    total = 5
    wide = torch.full((total + 4, 14, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 2:14:2, 8:]
    q[:total] = dev_bf16(R.bf16_bits(c["q"]))
    o = torch.full((total + 4, 6, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((total + 4, 6), 5.0, device="cuda")
    fa.kv4_attention(q, dev(c["cache"]), dev(c["table"]), dev(c["cu"]), dev(c["kv_len"]), 3, 32, 32, out=o, lse=l)
    fa.fa_check_error()
    compare(o[:total], l[:total], c)
    assert (o[total:] == 5).all() and (l[total:] == 5).all()


def test_attention_is_deterministic_and_independent_of_the_batch(fa):
    import torch
    c = attention_case(61, [5000, 800, 77], [2, 2, 2], 2, 4, 128, 32, 64)
    o1, l1 = run_attention(fa, c)
    o2, l2 = run_attention(fa, c)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    o3, l3 = run_attention(fa, c, max_q=30)   # another variant, the same answer
    compare(o3, l3, c)
    fa.fa_check_error()


def test_attention_reports_pages_and_offsets_out_of_range(fa):
    import torch
    c = attention_case(71, [100, 100], [1, 1], 1, 2, 64, 32, 16)
    o0, l0 = run_attention(fa, c)
    fa.fa_check_error()
    bad = dict(c, table=c["table"].copy())
    bad["table"][1, 2] = c["cache"].shape[0]
    o, l = run_attention(fa, bad)
    with pytest.raises(fa.FAError) as e:
        fa.fa_check_error()
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    assert torch.equal(o[0], o0[0]) and torch.equal(l[0], l0[0])
    for cu in ([0, 2, 1], [-1, 0, 1], [0, 1, 9]):
        run_attention(fa, dict(c, cu=np.asarray(cu, np.int32)), max_q=1)
        with pytest.raises(fa.FAError):
            fa.fa_check_error()
    # a length past the block table's row stops at the row's end
    long = dict(c, kv_len=np.asarray([100, 1 << 30], np.int32))
    long["table"] = np.where(long["table"] < 0, 0, long["table"])
    check(fa, long)


@pytest.mark.parametrize("nq", [1, 30])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_queries_that_are_not_numbers(fa, nq, d):
    # a query's NaN or infinity stays in its own row
    import torch
    c = attention_case(43, [300, 70], [nq, nq], 2, 4, d, 32, 32)
    clean, _ = run_attention(fa, c)
    q = dev_bf16(R.bf16_bits(c["q"]))
    q[0, 1, 3], q[-1, 5, 7] = float("nan"), float("inf")
    args = [dev(c[x]) for x in ("cache", "table", "cu", "kv_len")]
    o, l = fa.kv4_attention(q, *args, nq, 32, 32)
    fa.fa_check_error()
    hit = torch.zeros(o.shape[:2], dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[-1, 5] = True
    assert torch.isnan(o[0, 1]).all() and torch.isnan(l[0, 1])
    assert torch.equal(o[~hit], clean[~hit]) and not torch.isnan(l[~hit]).any()


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sizes", [(2.0 ** -40, 0), (2.0 ** 40, 0), (2.0 ** -12, 1 / 24), (2.0 ** 12, -1 / 24)])
def test_attention_of_keys_and_values_of_any_size(fa, nq, d, sizes):
    # far from 1, and growing or shrinking along the tokens (the kernels' fp16 units follow)
    base, slope = sizes
    c = attention_case(17, [333], [nq], 1, 2, d, 32, 16)
    page = 16
    sec = R.sections(page, d, 32)
    place = np.zeros(c["cache"].shape[0])
    place[c["table"][0, :21]] = np.arange(21)
    grow = base * 2.0 ** (slope * (place[:, None] * page + np.arange(page)))
    for which, (lo, hi) in ((0, sec[1]), (1, sec[3])):
        par = np.ascontiguousarray(c["cache"][..., lo:hi]).view(np.uint16)
        v = R.bf16_value(par).reshape(par.shape[0], 1, page, -1) * grow[:, None, :, None]
        c["cache"][..., lo:hi] = R.bf16_bits(v).reshape(par.shape).view(np.uint8)
    c["q"] = R.bf16_value(R.bf16_bits(c["q"] / base))   # scores of ordinary size
    check(fa, c)


@pytest.mark.parametrize("B,nq", [(129, 1), (300, 1), (200, 9), (1100, 1)])
def test_attention_of_many_requests(fa, B, nq):
    # more requests than a warp adds up, several to a share, some without queries or keys
    rng = np.random.default_rng(B)
    n = [int(x) for x in rng.integers(0, nq + 1, B)]
    lens = [int(x) if rng.random() < 0.95 else 0 for x in rng.integers(1, 150, B)]
    lens[B // 2] = 1500
    n[0] = nq
    check(fa, attention_case(B, lens, n, 1, 4, 64, 32, 16))
    check(fa, attention_case(B + 1, lens, n, 1, 8, 128, 64, 64))


@pytest.mark.parametrize("d,per,window", [(64, 4, -1), (64, 4, 50), (128, 4, 7), (256, 2, 200)])
@pytest.mark.parametrize("others", [1, 140])
def test_attention_of_many_blocks_of_rows(fa, d, per, window, others):
    # a request of more blocks than a warp has lanes, beside short ones before and behind it
    lens = [40 + 3 * b for b in range(others)]
    n = [b % 5 for b in range(others)]
    at = others // 2
    c = attention_case(d + others, lens[:at] + [2411] + lens[at:], n[:at] + [2203] + n[at:], 1, per, d, 32, 16)
    c["window"] = window
    check(fa, c)


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)])
@pytest.mark.parametrize("window", [-1, 1200])
def test_attention_of_chunks_that_shares_cut(fa, d, group, window):
    # longer than what is left whole: parts of items, some shares with two items, and the merge
    c = attention_case(d + group, [1901, 40, 2603, 1300], [301, 5, 77, 1], 2, 4, d, group, 64)
    c["window"] = window
    check(fa, c)
    c["causal"] = window >= 0
    check(fa, c)


@pytest.mark.parametrize("nq", [1, 12, 100])
def test_attention_is_bitwise_repeatable(fa, nq):
    import torch
    c = attention_case(63, [9000, 700, 1], [nq, min(nq, 5), 1], 2, 4, 128, 32, 64)
    first = run_attention(fa, c)
    for _ in range(3):
        for a, b in zip(first, run_attention(fa, c)):
            assert torch.equal(a, b)
    fa.fa_check_error()


def test_offsets_past_32_bits(fa):
    # a cache of more than 2^32 bytes: its last pages are written, read and attended to
    import torch
    heads, d, page = 16, 128, 128
    record = fa.kv4_page_bytes(d, page, 32)
    pages = (1 << 32) // (heads * record) + 40
    cache = fa.kv4_cache(pages, heads, page, d)
    assert cache.numel() > 1 << 32
    T = 200
    rng = np.random.default_rng(5)
    kb, vb = (R.bf16_bits(rng.standard_normal((T, heads, d))) for _ in range(2))
    ids = np.array([pages - 1, pages - 3], np.int32)
    j = np.arange(T)
    slots = ids[j // page].astype(np.int64) * page + j % page
    fa.kv4_append(dev_bf16(kb), dev_bf16(vb), i32(slots), cache, page)
    k, v = fa.kv4_gather(i32(slots), cache, page, d)
    fa.fa_check_error()
    for x, bits in ((k, kb), (v, vb)):
        want = dev(R.values(*R.quantise(R.bf16_value(bits), 32), 32)).float().bfloat16()
        assert (x == want).all()
    small = np.zeros((2, heads, record), np.uint8)
    small[:] = cache[[pages - 1, pages - 3]].cpu().numpy()
    for nq in (1, 60):
        q = R.bf16_value(R.bf16_bits(rng.standard_normal((nq, heads, d))))
        c = dict(q=q, cache=small, table=np.array([[0, 1]], np.int32), cu=np.array([0, nq], np.int32),
                 kv_len=np.array([T], np.int32), page=page, group=32, scale=1 / np.sqrt(d), causal=True, window=-1)
        o, l = fa.kv4_attention(dev_bf16(R.bf16_bits(q)), cache, dev(ids[None]), dev(c["cu"]), dev(c["kv_len"]), nq,
                                page, 32)
        fa.fa_check_error()
        compare(o, l, c)


def test_the_binding_refuses(fa):
    import torch
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    n32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    cache = torch.zeros(4, 2, fa.kv4_page_bytes(64, 16), dtype=torch.uint8, device="cuda")
    k = bf(8, 2, 64)
    good = dict(k=k, v=k, slots=n32(8), cache=cache, page_size=16)
    for bad in (dict(k=bf(8, 3, 64), v=bf(8, 3, 64)), dict(v=bf(7, 2, 64)), dict(k=k.float()), dict(slots=n32(9)),
                dict(slots=n32(8).long()), dict(cache=cache[:, :, :-16].contiguous()), dict(cache=cache.transpose(0, 1)),
                dict(k=bf(8, 2, 68)[:, :, :64]), dict(k=bf(8, 2, 128)[:, :, ::2]), dict(k=bf(8, 2, 80)[:, :, 4:68]),
                dict(page_size=32), dict(k=k[0]), dict(v=k.cpu())):
        with pytest.raises(ValueError):
            fa.kv4_append(**dict(good, **bad))
    q = bf(3, 4, 64)
    good = dict(q=q, cache=cache, block_table=n32(3, 2), cu_q=n32(4), kv_len=n32(3), max_q=1, page_size=16)
    for bad in (dict(q=bf(3, 5, 64)), dict(cu_q=n32(3)), dict(kv_len=n32(4)), dict(max_q=0), dict(window=-2),
                dict(block_table=n32(6)), dict(block_table=n32(2, 3).T), dict(out=bf(3, 4, 128)), dict(lse=bf(3, 4)),
                dict(group=64), dict(q=q.cpu()), dict(max_q=1 << 32), dict(workspace=n32(4))):
        with pytest.raises(ValueError):
            fa.kv4_attention(**dict(good, **bad))
    with pytest.raises(fa.FAError):
        fa.kv4_attention(**dict(good, scale=0.0))
    with pytest.raises(fa.FAError):
        fa.kv4_attention(**dict(good, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")))
    for bad in (dict(new_len=n32(4)), dict(free_state=n32(1)), dict(block_table=n32(3)), dict(max_tokens=0),
                dict(free_list=n32(9)[::2]), dict(past_len=n32(3).long())):
        with pytest.raises(ValueError):
            fa.kv4_plan(**dict(dict(past_len=n32(3), new_len=n32(3), block_table=n32(3, 2), free_list=n32(9),
                                    free_state=n32(2), page_size=16, max_tokens=4), **bad))
    # nothing to do is not an error
    fa.kv4_append(bf(0, 2, 64), bf(0, 2, 64), n32(0), cache, 16)
    assert fa.kv4_gather(n32(0), cache, 16, 64)[0].shape == (0, 2, 64)
    assert fa.kv4_attention(bf(0, 4, 64), cache, n32(3, 2), n32(4), n32(3), 1, 16)[1].shape == (0, 4)
    fa.fa_check_error()


# ------------------------------------------------------------------ together

def serve(fa, steps, seed, stream=None):
    """A small server: prompts, then single tokens, one request finished on the way.  Yields
    what each step computed and what it should have."""
    import torch
    rng = np.random.default_rng(seed)
    heads, per, d, page, group, B, width, F = 2, 4, 128, 16, 32, 3, 8, 24
    cache = fa.kv4_cache(F, heads, page, d, group)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    ring, state = i32(rng.permutation(F)), i32([0, F])
    kv = i32([0] * B)
    held = [([], []) for _ in range(B)]
    for new in steps:
        T = sum(max(n, 0) for n in new)
        x = rng.standard_normal((max(T, 1), heads * (per + 2), d))
        xb = R.bf16_bits(x)
        qkv = dev_bf16(xb)
        q, k, v = qkv[:, :heads * per], qkv[:, heads * per:heads * (per + 1)], qkv[:, heads * (per + 1):]
        kv, cu, slots, state = fa.kv4_plan(kv, i32(new), table, ring, state, page, max(T, 1))
        fa.kv4_append(k, v, slots, cache, page, group)
        o, l = fa.kv4_attention(q, cache, table, cu, kv, max(max(new), 1), page, group)
        fa.fa_check_error()
        val = R.bf16_value(xb)
        at = 0
        for b, n in enumerate(new):
            if n < 0:
                held[b] = ([], [])
            for t in range(max(n, 0)):
                for side, lo in enumerate((heads * per, heads * (per + 1))):
                    held[b][side].append(R.values(*R.quantise(val[at, lo:lo + heads], group), group))
                at += 1
        yield new, val, held, o.double().cpu().numpy(), l.double().cpu().numpy()


def test_plan_append_and_attention_together(fa):
    heads, per, d = 2, 4, 128
    steps = [[40, 0, 17], [1, 33, 1], [1, 1, -1], [4, 1, 60], [1, 1, 1]]
    for new, val, held, o, l in serve(fa, steps, 5):
        at = 0
        for b, n in enumerate(new):
            for t in range(max(n, 0)):
                upto = len(held[b][0]) - n + t + 1
                K, V = (np.stack(x[:upto]) for x in held[b])
                for h in range(heads * per):
                    z = K[:, h // per] @ val[at, h] / np.sqrt(d)
                    p = np.exp(z - z.max())
                    want = (p / p.sum()) @ V[:, h // per]
                    # three roundings to bf16 (2^-8 each) of weights, values and the result, the
                    # first two under the weighted sum of magnitudes, and the divisor's
                    tol = 2.0 ** -8 * (3.1 * (p / p.sum()) @ np.abs(V[:, h // per]) + np.abs(want)) + 1e-4
                    assert (np.abs(o[at, h] - want) <= tol).all()
                    assert abs(l[at, h] - (z.max() + np.log(p.sum()))) < 1e-3
                at += 1


def test_a_prefix_read_back_serves_the_forward(fa):
    # the cached rows, read back, are what attention over the cache computes with
    import torch
    c = attention_case(81, [256], [256], 2, 1, 128, 32, 64)
    cache = dev(c["cache"])
    j = np.arange(256)
    slots = i32(c["table"][0, j // 64] * 64 + j % 64)
    k, v = fa.kv4_gather(slots, cache, 64, 128)
    q = dev_bf16(R.bf16_bits(c["q"]))
    o1, l1 = fa.attention_fwd(*(x.transpose(0, 1)[None].contiguous() for x in (q, k, v)), causal=True)
    o2, l2 = run_attention(fa, c)
    # the forward's K is rounded to bf16 (2^-8 a value) where the cache's is not
    assert (o1[0].transpose(0, 1).float() - o2.float()).abs().max() < 6e-2
    assert (l1[0].T - l2).abs().max() < 4e-2


def test_captured_step_replays(fa):
    # plan, append and attention in one CUDA graph, replayed on new inputs
    import torch
    rng = np.random.default_rng(91)
    heads, per, d, page, B, F = 2, 4, 128, 16, 4, 64
    cache = fa.kv4_cache(F, heads, page, d)
    table = torch.zeros(B, 8, dtype=torch.int32, device="cuda")
    ring, state, past = i32(rng.permutation(F)), i32([0, F]), i32([0] * B)
    new = i32([1] * B)
    qkv = torch.zeros(B, heads * (per + 2), d, dtype=torch.bfloat16, device="cuda")

    def step():
        kv, cu, slots, st = fa.kv4_plan(past, new, table, ring, state, page, B)
        fa.kv4_append(qkv[:, heads * per:heads * (per + 1)], qkv[:, heads * (per + 1):], slots, cache, page)
        o, l = fa.kv4_attention(qkv[:, :heads * per], cache, table, cu, kv, 1, page)
        return kv, st, o, l

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv, st, o, l = step()
    keys = [[] for _ in range(B)]
    for i in range(40):
        xb = R.bf16_bits(rng.standard_normal((B, heads * (per + 2), d)))
        qkv.copy_(dev_bf16(xb))
        graph.replay()
        past.copy_(kv)
        state.copy_(st[:2])
        val = R.bf16_value(xb)
        for b in range(B):
            keys[b].append([R.values(*R.quantise(val[b, lo:lo + heads], 32), 32)
                            for lo in (heads * per, heads * (per + 1))])
    fa.fa_check_error()
    o = o.double().cpu().numpy()
    for b in range(B):
        K, V = (np.stack([x[s] for x in keys[b]]) for s in (0, 1))
        for h in range(heads * per):
            z = K[:, h // per] @ val[b, h] / np.sqrt(d)
            p = np.exp(z - z.max())
            p /= p.sum()
            want = p @ V[:, h // per]
            tol = 2.0 ** -8 * (3.1 * p @ np.abs(V[:, h // per]) + np.abs(want)) + 1e-4
            assert (np.abs(o[b, h] - want) <= tol).all()


@pytest.mark.parametrize("nq", [9, 60])
def test_captured_attention_replays(fa, nq):
    # two graphs with buffers of their own, replayed in turn on changing inputs
    import torch
    cases = [attention_case(95 + i, [900, 64], [nq, nq], 2, 4, 128, 32, 64) for i in range(2)]
    args = [(dev_bf16(R.bf16_bits(c["q"])), dev(c["cache"]), dev(c["table"]), dev(c["cu"]), dev(c["kv_len"]))
            for c in cases]
    alone = [fa.kv4_attention(*a, nq, 64) for a in args]
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.kv4_attention(*a, nq, 64))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        for o in outs[i]:
            o.zero_()
        graphs[i].replay()
        for o, w in zip(outs[i], alone[i]):
            assert torch.equal(o, w)
    args[0][4].copy_(i32([500, 63]))     # other lengths
    graphs[0].replay()
    compare(*outs[0], dict(cases[0], kv_len=np.array([500, 63], np.int32)))
    fa.fa_check_error()


def test_two_streams_with_workspaces_of_their_own(fa):
    import torch
    cases = [attention_case(101 + i, [3000, 500], [1, 1], 2, 4, 128, 32, 64) for i in range(2)]
    alone = [run_attention(fa, c) for c in cases]
    args = [(dev_bf16(R.bf16_bits(c["q"])), dev(c["cache"]), dev(c["table"]), dev(c["cu"]), dev(c["kv_len"]))
            for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, (a, s) in enumerate(zip(args, streams)):
            got[i] = fa.kv4_attention(*a, 1, 64, 32, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for (o, l), (o1, l1) in zip(alone, got):
        assert torch.equal(o, o1) and torch.equal(l, l1)
    fa.fa_check_error()


def test_two_streams_of_chunks(fa):
    import torch
    cases = [attention_case(111 + i, [1500, 300], [130, 90], 1, 4, d, 32, 64) for i, d in enumerate([64, 128])]
    alone = [run_attention(fa, c) for c in cases]
    args = [(dev_bf16(R.bf16_bits(c["q"])), dev(c["cache"]), dev(c["table"]), dev(c["cu"]), dev(c["kv_len"]))
            for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [fa.kv4_attention(*a, 130, 64, 32, stream=s.cuda_stream) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for (o, l), (o1, l1) in zip(alone, got):
            assert torch.equal(o, o1) and torch.equal(l, l1)
    fa.fa_check_error()


@pytest.mark.parametrize("lens,nq", [([9000, 33], [1, 2]), ([200, 33], [1, 2]), ([1900, 600], [150, 20]), ([300, 64], [90, 64])])
def test_a_workspace_may_hold_anything(fa, lens, nq):
    import torch
    c = attention_case(131, lens, nq, 2, 4, 128, 32, 64)
    o, l = run_attention(fa, c)
    compare(o, l, c)
    size = fa.kv4_attention_workspace_bytes(8, 2, 128, max(nq))
    for byte in (0, 255):
        o1, l1 = run_attention(fa, c, workspace=torch.full((size,), byte, dtype=torch.uint8, device="cuda"))
        assert torch.equal(o, o1) and torch.equal(l, l1)
    fa.fa_check_error()


@pytest.mark.parametrize("d,nq", [(64, 1), (128, 5), (128, 90), (256, 40)])
def test_lengths_past_the_table_are_clamped(fa, d, nq):
    import torch
    c = attention_case(141 + d, [640, 320], [nq, 1], 1, 4, d, 32, 64, table_pad=0)
    c["table"][1, 5:] = c["table"][0, 5:]      # the table's rows are full
    c["kv_len"] = np.asarray([640, 640], np.int32)
    o, l = run_attention(fa, c)
    compare(o, l, c)
    for far in (641, 10**6, 2**31 - 1):
        o1, l1 = run_attention(fa, dict(c, kv_len=np.asarray([far, far], np.int32)))
        assert torch.equal(o, o1) and torch.equal(l, l1)
    fa.fa_check_error()


def test_calls_without_rows(fa):
    import torch
    cache = fa.kv4_cache(4, 2, 16, 64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    fa.kv4_append(none, none, i32([]), cache, 16)
    k, v = fa.kv4_gather(i32([]), cache, 16, 64)
    assert k.shape == v.shape == (0, 2, 64)
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    o, l = fa.kv4_attention(none, cache, table, i32([0, 0, 0]), i32([0, 0]), 1, 16)
    assert o.shape == (0, 2, 64) and l.shape == (0, 2)
    # rows, and no request that has any: nothing is written
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    for max_q in (1, 300):
        o, l = torch.full_like(q, 5.0), torch.full((3, 2), 5.0, device="cuda")
        fa.kv4_attention(q, cache, table, i32([0, 0, 0]), i32([0, 0]), max_q, 16, out=o, lse=l)
        assert (o == 5).all() and (l == 5).all()
    fa.fa_check_error()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_bound_on_queries_only_chooses_the_kernel(fa, d):
    # one query a request, told it might be many: every block of rows, cut and whole
    for lens in ([700, 5, 129], [5000, 64, 1]):
        c = attention_case(d + lens[0], lens, [1, 1, 1], 2, 2, d, 32, 32)
        for max_q in (1, 4, 5, 8, 12, 16, 24, 33, 64, 5000):
            o, l = run_attention(fa, c, max_q=max_q)
            compare(o, l, c)
    fa.fa_check_error()

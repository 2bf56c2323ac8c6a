"""Packed prompt attention on the GPU against plain attention in 64 bits."""
import itertools
import math

import pytest

from int4_quantized_attention_b200 import api, build
from serve_reference import D, check, packed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def op():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return api.PackedAttention()


def cum(lens):
    return [0] + list(itertools.accumulate(lens))


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(seed, tq, tk, hq, hkv, dtype, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    return (gain * r(tq, hq, D)).to(dtype), r(tk, hkv, D).to(dtype), r(tk, hkv, D).to(dtype)


def run_case(op, lq, lk, hq, hkv, dtype, causal, gain=1.0, seed=1, scale=None):
    cq, ck = cum(lq), cum(lk)
    q, k, v = inputs(seed, cq[-1], ck[-1], hq, hkv, dtype, gain)
    o, lse = op.forward(q, k, v, ints(cq), ints(ck), causal=causal, scale=scale or 0.0, return_lse=True)
    op.check()
    want, wl, tol, tl = packed(q, k, v, cq, ck, causal, scale)
    check(o, want, tol, "o")
    check(lse, wl, tl, "lse")
    return q, k, v, cq, ck, o, lse


# lengths of queries and keys: one token, tile borders, odd sizes, none at all
LENS = {
    "one": ([1], [1]),
    "borders": ([127, 128, 129, 1, 256, 257], [127, 128, 129, 1, 256, 257]),
    "odd": ([13, 0, 77, 1, 0, 301], [13, 0, 77, 1, 5, 301]),
    "chunk": ([5, 130, 1], [700, 1000, 2049]),
    "more_queries": ([200, 3, 140], [60, 0, 139]),
    "empty_tail": ([33, 0, 0], [40, 0, 9]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (5, 1), (14, 2), (128, 1)])
@pytest.mark.parametrize("lens", list(LENS))
def test_lengths_and_heads(op, lens, hq, hkv, dtype, causal):
    run_case(op, *LENS[lens], hq, hkv, dtype, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_items(op, dtype, causal):
    # enough query tiles that whole items are dealt out instead of key shares
    lens = [700, 1, 0, 129, 512, 300, 64, 1025]
    p = api.Packed(len(lens), 40, 40, 128, 0, 0, sum(lens), sum(lens), 0.0, *([40 * 128, 128] * 4))
    assert api.packed_workspace_bytes(p) == 256          # no room for partial rows: no split
    run_case(op, lens, [n + (i % 3) * 50 for i, n in enumerate(lens)], 40, 40, dtype, causal)


def test_many_sequences(op):
    lens = [(i * 7) % 40 for i in range(900)]
    run_case(op, lens, lens, 4, 2, BF16, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [31, 32, 33, 128, 129])
def test_item_order(op, n, causal):
    # whole items, longest first, with as many sequences as one, several and too many rounds of lanes hold
    lens = [(i * i * 37) % 400 + (700 if i % 13 == 5 else 0) for i in range(n)]
    past = [(i % 4) * 61 for i in range(n)]
    hq = 12 if n > 100 else 48
    p = api.Packed(n, hq, hq, 128, 0, 0, sum(lens), sum(lens) + sum(past), 0.0, *([hq * 128, 128] * 4))
    assert api.packed_workspace_bytes(p) == 256
    out = run_case(op, lens, [a + b for a, b in zip(lens, past)], hq, hq, F16, causal)
    for _ in range(3):                                   # tickets are set back each time
        assert torch.equal(op.forward(*out[:3], ints(out[3]), ints(out[4]), causal=causal), out[5])


def test_long_keys_few_rows(op):
    run_case(op, [3], [70001], 8, 1, F16, True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gain", [0.0, 40.0])
def test_flat_and_peaked_scores(op, dtype, gain):
    # all weights equal, and rows that one key decides
    run_case(op, [150, 40], [900, 40], 6, 2, dtype, True, gain=gain)


def test_rising_maximum(op):
    # keys whose scores climb tile after tile: the accumulator is rescaled each time
    n = 1500
    q = torch.ones(64, 1, D, device="cuda", dtype=F16)
    k = (torch.arange(n, device="cuda") / n * 6 - 3)[:, None, None].expand(n, 1, D).to(F16).contiguous()
    v = inputs(3, 1, n, 1, 1, F16)[2]
    for lse_only, scale in ((0, 0.1), (1, 0.7)):
        o, lse = op.forward(q, k, v, ints([0, 64]), ints([0, n]), causal=True, scale=scale, return_lse=True)
        want, wl, tol, tl = packed(q, k, v, [0, 64], [0, n], True, scale)
        check(o, want, tol, "o")
        check(lse, wl, tl, "lse")


def test_strides_and_outputs(op):
    # q, k, v as slices of one projection; head-major keys; an output inside a larger buffer
    lens, hq, hkv = [130, 7, 250], 8, 2
    n, cu = sum(lens), cum(lens)
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(n, hq + 2 * hkv, D, generator=g, device="cuda").to(BF16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    want, wl, tol, tl = packed(q, k, v, cu, cu, True)
    big = torch.full((n + 9, hq, 2, D), 7.0, device="cuda", dtype=BF16)
    out = big[4:4 + n, :, 1]
    got = op.forward(q, k, v, ints(cu), ints(cu), out=out)
    assert got is out
    check(out, want, tol, "o")
    assert bool((big[:4] == 7).all()) and bool((big[4 + n:] == 7).all()) and bool((big[:, :, 0] == 7).all())
    kh = k.transpose(0, 1).contiguous().transpose(0, 1)           # [Hkv][tokens][D] in memory
    vh = v.transpose(0, 1).contiguous().transpose(0, 1)
    oh = torch.empty(hq, n, D, device="cuda", dtype=BF16).transpose(0, 1)
    op.forward(q, kh, vh, ints(cu), ints(cu), out=oh)
    assert torch.equal(oh, out)


def test_rows_behind_the_last_sequence_stay(op):
    q, k, v = inputs(9, 300, 300, 4, 4, F16)
    out = torch.full((300, 4, D), 3.0, device="cuda", dtype=F16)
    lse = torch.full((300, 4), 5.0, device="cuda")
    op.forward(q, k, v, ints([0, 100, 170]), ints([0, 100, 170]), out=out, lse=lse)
    op.check()
    assert bool((out[170:] == 3).all()) and bool((lse[170:] == 5).all())
    want, wl, tol, tl = packed(q[:170], k, v, [0, 100, 170], [0, 100, 170], True)
    check(out[:170], want, tol, "o")


@pytest.mark.parametrize("heads", [2, 40])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_hidden_values_do_not_leak(op, dtype, heads):
    # NaN and infinities in keys and values that a row does not see leave it alone,
    # and reach exactly the rows that do see them
    lens = [200, 90, 300] if heads == 2 else [200, 90, 300, 700, 500]
    cu = cum(lens)
    q, k, v = inputs(11, cu[-1], cu[-1], heads, heads, dtype)
    v[199, 0, 5] = math.nan         # the last key of a sequence: only its last token
    v[200 + 40, 1, 7] = math.inf    # from the middle on
    v[200 + 50, 1, 7] = -math.inf   # both: NaN
    v[200 + 60, 0, 100] = -math.inf
    v[290 + 128, 0, 64] = math.inf
    o, lse = op.forward(q, k, v, ints(cu), ints(cu), return_lse=True)
    op.check()
    want, wl, tol, tl = packed(q, k, v, cu, cu, True)
    check(o, want, tol, "o")
    check(lse, wl, tl, "lse")
    # a hidden key: rows before it keep their values, bit for bit
    k2 = k.clone()
    k2[199, 0] = math.nan
    k2[289, 0] = math.inf
    o2 = op.forward(q, k2, v, ints(cu), ints(cu))
    same = [i for i in range(cu[-1]) if i not in (199, 289)]
    a, b = o[same].clone(), o2[same].clone()
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) and torch.equal(torch.isnan(a), torch.isnan(b))
    # rows behind the last sequence's keys hold NaN: no effect
    kk, vv = (torch.cat([x, torch.full((200, heads, D), math.nan, device="cuda", dtype=dtype)]) for x in (k, v))
    o3 = op.forward(q, kk, vv, ints(cu), ints(cu))
    assert torch.equal(torch.nan_to_num(o3), torch.nan_to_num(o)) and torch.equal(torch.isnan(o3), torch.isnan(o))


@pytest.mark.parametrize("nan_q", [True, False])
def test_nan_rows_stay_nan_when_joined(op, nan_q):
    # a NaN query, or a NaN key that every row sees: NaN whether or not the keys are split
    q, k, v = inputs(12, 40, 9000, 2, 1, F16)
    (q if nan_q else k)[3, 0, 9] = math.nan
    o, lse = op.forward(q, k, v, ints([0, 40]), ints([0, 9000]), return_lse=True)
    op.check()
    bad = torch.zeros(40, 2, dtype=torch.bool, device="cuda")
    if nan_q:
        bad[3, 0] = True
    else:
        bad[:] = True
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad)


def test_repeatable_captured_and_on_a_side_stream(op):
    lens = [260, 31, 1]
    q, k, v, cq, ck, o, lse = run_case(op, lens, [n + 400 for n in lens], 8, 2, BF16, True)
    cu_q, cu_k = ints(cq), ints(ck)
    for _ in range(3):
        assert torch.equal(op.forward(q, k, v, cu_q, cu_k), o)
    side, mine = torch.cuda.Stream(), api.PackedAttention()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2 = mine.forward(q, k, v, cu_q, cu_k)
    side.synchronize()
    assert torch.equal(o2, o)
    # captured once, replayed with other lengths and contents
    out = torch.empty_like(o)
    mine.forward(q, k, v, cu_q, cu_k, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mine.forward(q, k, v, cu_q, cu_k, out=out)
    graph.replay()
    assert torch.equal(out, o)
    cu_q.copy_(ints([0, 17, 200, 292]))
    k.mul_(0.5)
    graph.replay()
    mine.check()
    want, _, tol, _ = packed(q, k, v, [0, 17, 200, 292], ck, True)
    check(out, want, tol, "replayed")


def test_two_streams_at_once():
    # calls of two objects may overlap: each has its own workspace
    cases = [([900, 31], 8, 2, BF16), ([500, 700, 300, 2], 40, 40, F16)]
    sets = []
    for lens, hq, hkv, dtype in cases:
        cu = cum(lens)
        q, k, v = inputs(7, cu[-1], cu[-1], hq, hkv, dtype)
        sets.append((api.PackedAttention(), torch.cuda.Stream(), q, k, v, ints(cu), packed(q, k, v, cu, cu, True)))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (mine, stream, q, k, v, cu, _) in enumerate(sets):
            with torch.cuda.stream(stream):
                outs[i].append(mine.forward(q, k, v, cu, cu))
    torch.cuda.synchronize()
    for i, (mine, _, _, _, _, _, (want, _, tol, _)) in enumerate(sets):
        mine.check()
        check(outs[i][0], want, tol, "o")
        assert all(torch.equal(x, outs[i][0]) for x in outs[i])


def test_bad_offsets_are_reported_and_left_out(op):
    q, k, v = inputs(2, 100, 100, 2, 2, F16)
    for cq, ck, fine in (([0, 40, 30], [0, 40, 100], 40), ([0, 40, 101], [0, 40, 100], 40),
                         ([0, 40, 100], [0, 40, 1000], 40), ([0, 40, 100], [0, 40, 20], 40)):
        out = torch.full_like(q, 2.0)
        op.forward(q, k, v, ints(cq), ints(ck), out=out)
        with pytest.raises(api.RotateAttnError) as e:
            op.check()
        assert e.value.status == api.RA_ERR_DEVICE_BOUNDS
        want, _, tol, _ = packed(q[:fine], k, v, [0, fine], [0, fine], True)
        check(out[:fine], want, tol, "the good sequence")
    op.forward(q, k, v, ints([0, 100]), ints([0, 100]))
    op.check()


@pytest.mark.parametrize("n,hq", [(300, 48), (300, 2), (129, 48), (60, 48), (40, 2)])
def test_a_bad_offset_anywhere_is_reported(op, n, hq):
    # among many sequences, whole items or split ones; a plain call afterwards is right
    lens = [40 + i % 7 for i in range(n)]
    cu = cum(lens)
    q, k, v = inputs(2, cu[-1], cu[-1], hq, 2, F16)
    for at in sorted({1, n // 4, n // 2, n // 2 + 1, n - 1, n}):
        for bad in (0, -1, -2 ** 31, cu[at - 1] - 1, cu[-1] + 1, 2 ** 31 - 1):
            if (at, bad) == (1, 0):                     # an empty first sequence
                continue
            for which in "qk":
                wrong = cu[:at] + [bad] + cu[at + 1:]
                out = torch.full_like(q, 2.0)
                op.forward(q, k, v, ints(wrong if which == "q" else cu), ints(wrong if which == "k" else cu), out=out)
                with pytest.raises(api.RotateAttnError) as e:
                    op.check()
                assert e.value.status == api.RA_ERR_DEVICE_BOUNDS, (at, bad, which)
    o, lse = op.forward(q, k, v, ints(cu), ints(cu), return_lse=True)
    op.check()
    want, wl, tol, tl = packed(q, k, v, cu, cu, True)
    check(o, want, tol, "o")
    check(lse, wl, tl, "lse")


def test_segments_that_outlast_a_wait(op):
    # the tiles of one query pair take longer than the limit of a wait alone: 2500 of them some 4 ms, against 1 ms
    tq, tk = 300 * 256, 320000
    q, k, v = inputs(3, tq, tk, 1, 1, BF16)
    p = api.Packed(1, 1, 1, 128, 1, 0, tq, tk, 0.0, *([128, 128] * 4))
    assert api.packed_workspace_bytes(p) == 256          # whole items
    api.debug_set_wait_timeout_us(1000)
    try:
        o, lse = op.forward(q, k, v, ints([0, tq]), ints([0, tk]), causal=False, return_lse=True)
        op.check()
    finally:
        api.debug_set_wait_timeout_us(0)
    for rows in (slice(0, 40), slice(tq - 40, tq)):
        want, wl, tol, tl = packed(q[rows], k, v, [0, 40], [0, tk], False)
        check(o[rows], want, tol, "o")
        check(lse[rows], wl, tl, "lse")


def test_no_tokens(op):
    q, k, v = inputs(2, 0, 4, 2, 2, F16)
    assert op.forward(q, k, v, ints([0, 0]), ints([0, 4])).shape == (0, 2, D)
    q, k, v = inputs(2, 3, 0, 2, 2, F16)
    o, lse = op.forward(q, k, v, ints([0, 3]), ints([0, 0]), return_lse=True)
    op.check()
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())

"""GPU parity of causal grouped-head attention (moe_attn_forward through the C ABI) against the
fp64 oracle (oracle.attention), and the two token mixers run together.

Bar, from the roundings the operator makes, per element with mass = sum_j p_ij |v_j|: half a
bf16 step of the result, 2^-8 |o|; the weights p may be rounded to bf16 before they meet the
values, 2^-8 mass; scores are fp32 sums of at most 128 exact products, at most 128 * 2^-24 of
sum |q||k| scale (below 2^7 for these inputs): 2^-10 of a weight, with the exponential's and
the sums' few 2^-22 inside that: 2^-10 mass."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from int4_expert_gemv_router_b200 import abi, build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def f64(t):
    return t.float().double().cpu().numpy()


def make(Hq, Hkv, d, lens, kv=None, seed=0, gap=3, pad=0, fill=float("nan")):
    """Packed queries and, with kv, slabs of a cache with unused rows (NaN) around each."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *size: torch.randn(*size, device=DEV, generator=gen).to(torch.bfloat16)  # noqa: E731
    T = sum(lens) + 2 * pad
    off = np.concatenate([[pad], pad + np.cumsum(lens)]).astype(np.int32)
    c = dict(shape=abi.moe_attn_shape(Hq, Hkv, d), n=len(lens), T=T, off=torch.from_numpy(off).to(DEV),
             q=normal(max(T, 1), Hq, d), scale=1.0 / math.sqrt(d))
    if kv is None:
        c.update(begin=None, len=None, rows=T, k=normal(max(T, 1), Hkv, d), v=normal(max(T, 1), Hkv, d), max_kv=max(lens))
        return c
    begin, at = [], gap
    for x in kv:
        begin.append(at)
        at += x + gap
    k = torch.full((at, Hkv, d), fill, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    for b, x in zip(begin, kv):
        k[b:b + x], v[b:b + x] = normal(x, Hkv, d), normal(x, Hkv, d)
    c.update(begin=torch.tensor(begin, dtype=torch.int32, device=DEV), rows=at, k=k, v=v, max_kv=max(kv),
             len=torch.tensor(kv, dtype=torch.int32, device=DEV))
    return c


def workspace(c):
    return torch.zeros(abi.moe_attn_workspace_size(c["shape"], c["n"], c["T"], c["max_kv"]), dtype=torch.uint8, device=DEV)


def run(c, ws=None):
    ws = workspace(c) if ws is None else ws
    out = torch.full((max(c["T"], 1), c["shape"].n_q_heads, c["shape"].d), 7.0, dtype=torch.bfloat16, device=DEV)
    abi.moe_attn_forward(c["shape"], c["n"], c["T"], c["off"], c["begin"], c["len"], c["max_kv"], c["q"], c["k"], c["v"],
                         c["rows"], c["scale"], out, ws)
    return out, ws


def check(c, out, seqs=None):
    off = c["off"].tolist()
    for s in range(c["n"]) if seqs is None else seqs:
        at = slice(off[s], off[s + 1])
        b, x = (off[s], off[s + 1] - off[s]) if c["begin"] is None else (int(c["begin"][s]), int(c["len"][s]))
        o, mass = oracle.attention(f64(c["q"][at]), f64(c["k"][b:b + x]), f64(c["v"][b:b + x]), c["scale"])
        err = np.abs(f64(out[at]) - o)
        bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -10) * mass + 1e-30
        assert np.isfinite(f64(out[at])).all()
        assert (err <= bar).all(), (s, (err / bar).max(), np.argwhere(err > bar)[:4].tolist())


@pytest.mark.parametrize("Hq,Hkv,d,lens", [
    (4, 2, 128, [1]),
    (16, 2, 128, [37]),
    (4, 4, 64, [127, 128, 129]),                # one query head per key head
    (4, 4, 128, [255, 256, 257, 0, 1]),
    (8, 1, 128, [1, 2, 15, 16, 17, 31, 32, 33]),
    (6, 2, 64, [100, 43, 85, 86]),              # three query heads per key head: no power of two
    (10, 2, 128, [300]),
    (64, 1, 64, [5, 130]),                      # as many query heads as a key head may have
    (74, 2, 64, [7, 70]),                       # 37 per key head
    (16, 4, 128, [700, 1, 513]),
])
def test_prompts_match_oracle(Hq, Hkv, d, lens):
    c = make(Hq, Hkv, d, lens, seed=Hq + d + len(lens))
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out)


@pytest.mark.parametrize("Hq,Hkv,d,lens,kv", [
    (4, 2, 128, [3, 64, 10], [3, 200, 1000]),          # a prompt, a piece, a piece after a long history
    (16, 2, 128, [1, 1, 1, 1], [1, 127, 128, 129]),    # single tokens
    (16, 2, 64, [1, 1, 1], [4000, 1, 2049]),
    (8, 8, 128, [1, 2], [1500, 700]),
    (12, 4, 128, [1], [5000]),                         # one token, a long axis
    (16, 1, 64, [1], [20000]),                         # ... cut into more than 16 pieces, 16 rows
    (8, 1, 128, [2, 0], [9500, 3]),                    # ... two tokens of it
    (4, 2, 128, [33], [9000]),                         # tiles cut into pieces
    (4, 1, 64, [130, 1], [2000, 3000]),
    (6, 2, 128, [20, 5, 7], [4, 0, 7]),                # more queries than keys: some see nothing
])
def test_histories_and_tokens_match_oracle(Hq, Hkv, d, lens, kv):
    c = make(Hq, Hkv, d, lens, kv, seed=Hq + d + sum(kv))
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out)


@pytest.mark.parametrize("n", [1, 40])
def test_bound_of_the_lengths_may_be_loose(n):
    """max_kv far above the lengths changes nothing but the split."""
    c = make(8, 2, 128, [1] * n, [5 + 9 * i for i in range(n)], seed=n)
    c["max_kv"] = 100000
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out)


def test_growing_scores_rescale():
    """Keys ordered so that the maximum rises in every block of keys, then only falls; scores far
    apart; and scores of one size."""
    c = make(4, 2, 128, [300], seed=21)
    c["q"][:] = c["q"][:1, :1]
    lift = torch.linspace(-4, 4, 300, device=DEV)[:, None, None] * c["q"][:1, :1].float()
    for sign in (1.0, -1.0):
        c["k"] = (c["k"].float() * 0.1 + sign * lift).to(torch.bfloat16)
        out, _ = run(c)
        check(c, out)
    c["k"][:] = 0
    out, _ = run(c)
    check(c, out)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(scale):
    c = make(4, 2, 64, [150], seed=22)
    c["scale"] = scale
    out, _ = run(c)
    check(c, out)


def test_infinities_in_keys_beyond_sight_and_unused_rows():
    """Unused rows hold infinities; a later key's infinity in k does not reach earlier queries."""
    c = make(4, 2, 128, [60, 1], [200, 90], seed=23, fill=float("inf"))
    out, ws = run(c)
    check(c, out)
    base = out.clone()
    c["k"][int(c["begin"][0]) + 199] = float("nan")  # seen by the last query alone
    out, _ = run(c, ws)
    assert torch.equal(out[:59], base[:59]) and torch.isnan(out[59].float()).all() and torch.equal(out[60], base[60])


@pytest.mark.parametrize("Hq,Hkv,d,n,kv,bad", [
    (4, 2, 128, 300, 300, [37, 150, 299]),
    (4, 4, 64, 400, 400, [0, 127, 128, 255, 256, 399]),  # units of 256 positions
    (16, 2, 128, 45, 45, [3, 31, 32]),                   # units of 32
    (4, 2, 128, 33, 9000, [20, 8967, 8968, 8998, 8999]),  # cut into pieces
    (6, 2, 64, 20, 9, [0, 8]),                           # rows that see no key at all
    (4, 2, 128, 8, 8, [0, 5, 7]),                        # few rows
    (4, 2, 64, 8, 135, [126, 127, 128, 134]),            # ... from one tile into the next
    (8, 1, 128, 2, 9500, [9498, 9499]),                  # ... in pieces
])
def test_nonfinite_values_reach_only_the_queries_that_see_them(Hq, Hkv, d, n, kv, bad):
    """Every other element keeps its bits; those columns of the rows that see the key are not finite."""
    c = make(Hq, Hkv, d, [n], [kv], seed=34)
    base, ws = run(c)
    check(c, base)
    first, gone = int(c["begin"][0]), torch.zeros(n, Hq, d, dtype=torch.bool, device=DEV)
    for i, key in enumerate(bad):
        head, col = i % Hkv, (i * 29 + 5) % d
        c["v"][first + key, head, col] = (float("nan"), float("inf"), -float("inf"))[i % 3]
        gone[max(0, key - (kv - n)):, head * (Hq // Hkv):(head + 1) * (Hq // Hkv), col] = True
    out, _ = run(c, ws)
    assert abi.moe_ws_check(ws) == 0
    assert torch.equal(~torch.isfinite(out.float()), gone)
    assert torch.equal(out[~gone], base[~gone])


def test_nonfinite_values_over_many_units():
    """Calls of many units, every one with such values, back to back on one workspace."""
    lens = [1 + (37 * i) % 150 for i in range(120)]
    c = make(8, 2, 128, lens, [x + (i % 3) * 70 for i, x in enumerate(lens)], seed=35)
    base, ws = run(c)
    check(c, base, seqs=range(0, 120, 17))
    off, begin, length = c["off"].tolist(), c["begin"].tolist(), c["len"].tolist()
    gone = torch.zeros(c["T"], 8, 128, dtype=torch.bool, device=DEV)
    for s in range(1, 120, 2):  # every other sequence: the units between stay clean
        c["v"][begin[s] + length[s] - 1, 1, s % 128] = float("nan")
        gone[off[s + 1] - 1, 4:, s % 128] = True
    for _ in range(3):
        out, _ = run(c, ws)
        assert abi.moe_ws_check(ws) == 0
        assert torch.equal(~torch.isfinite(out.float()), gone)
        assert torch.equal(out[~gone], base[~gone])


def test_bad_ranges_are_left_out():
    c = make(4, 2, 128, [30, 10, 5, 6, 7, 8], [40, 10, 5, 6, 7, 8], seed=24)
    c["begin"][1] = -1
    c["len"][2] = -3
    c["begin"][3] = c["rows"] - 5
    c["len"][4] = c["max_kv"] + 1
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == abi.DEVERR_BAD_RANGE
    assert abi.moe_ws_check(ws) == 0
    check(c, out, seqs=(0, 5))
    assert (out[30:58] == 7.0).all()
    c = make(4, 2, 128, [40, 20], seed=25)
    c["off"] = torch.tensor([0, 40, 61], dtype=torch.int32, device=DEV)
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == abi.DEVERR_BAD_RANGE
    check(c, out, seqs=(0,))
    assert (out[40:] == 7.0).all()


@pytest.mark.parametrize("lens,kv", [
    ([1, 2, 1, 1, 3], [300, 20, 70, 9, 3]),               # few rows
    ([1, 2, 1, 1, 3], [3000, 20, 70, 9, 3]),              # ... with keys in pieces
    ([90, 20, 1, 33, 3], [300, 20, 70, 33, 3]),           # tiles
    ([90, 20, 1, 33, 3], [9000, 20, 70, 33, 3]),          # ... with keys in pieces
    ([90, 20, 1, 33, 3] * 8, [300, 20, 70, 33, 3] * 8),   # more sequences than a warp has lanes
    ([1, 2, 1, 1, 3] * 8, [900, 20, 70, 9, 3] * 8),
])
def test_bad_ranges_on_every_path(lens, kv):
    """Keys out of range, then query rows out of order: the sequences concerned, and no others."""
    c = make(8, 2, 128, lens, kv, seed=36)
    ws = workspace(c)
    off = c["off"].tolist()
    begin = c["begin"].clone()
    begin[1], begin[3] = -1, c["rows"] - 2
    out, _ = run(dict(c, begin=begin), ws)
    assert abi.moe_ws_check(ws) == abi.DEVERR_BAD_RANGE and abi.moe_ws_check(ws) == 0
    check(c, out, seqs=[s for s in range(len(lens)) if s not in (1, 3)])
    assert all((out[off[s]:off[s + 1]] == 7.0).all() for s in (1, 3))
    offsets = c["off"].clone()
    offsets[2] = offsets[1] - 1  # sequence 1 would end before it begins; sequence 2 begin in sequence 0's rows
    out, _ = run(dict(c, off=offsets), ws)
    assert abi.moe_ws_check(ws) == abi.DEVERR_BAD_RANGE
    check(c, out, seqs=[s for s in range(len(lens)) if s not in (1, 2)])
    assert all((out[off[s]:off[s + 1]] == 7.0).all() for s in (1, 2))


def test_rows_outside_sequences_and_shared_keys():
    c = make(4, 2, 128, [20, 33], [64, 64], seed=26, pad=6)
    c["begin"][1] = c["begin"][0]  # both read the same keys
    out, ws = run(c)
    check(c, out)
    assert (out[:6] == 7.0).all() and (out[-6:] == 7.0).all()
    again, _ = run(c, ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("lens", [[3, 2], [40, 1]])
def test_no_keys_at_all(lens):
    """kv_rows = 0: no k and v, every query sees nothing."""
    c = make(4, 2, 128, lens, [0, 0], seed=33, gap=0)
    c.update(k=None, v=None)
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == 0 and (out[:sum(lens)] == 0).all()


def test_many_sequences():
    lens = [(i * 5) % 4 for i in range(1400)]
    c = make(4, 2, 64, lens, [x + (i % 90) for i, x in enumerate(lens)], seed=27)
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out, seqs=list(range(60)) + list(range(1015, 1035)) + list(range(1380, 1400)))


def test_cache_rows_past_32_bits():
    Hkv, d = 2, 128
    rows = (1 << 31) // (Hkv * d) + 4000
    c = make(8, Hkv, d, [9, 1], [300, 2000], seed=28, gap=0)
    a = rows - 2300
    for x in ("k", "v"):
        big = torch.zeros(rows, Hkv, d, dtype=torch.bfloat16, device=DEV)
        big[a:] = c[x]
        c[x] = big
    c["begin"] += a
    c["rows"] = rows
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out)


def test_captured_and_on_two_streams():
    cs = [make(8, 2, 128, [130, 1, 0], [400, 900, 5], seed=29, gap=8),
          make(8, 2, 128, [1, 0, 130], [900, 5, 400], seed=30, gap=8)]
    ref = [run(c)[0] for c in cs]
    names = ("q", "k", "v", "off", "begin", "len")
    c = dict(cs[0], **{x: cs[0][x].clone() for x in names})
    ws, s = workspace(c), torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        out, _ = run(c, ws)
    for i in (0, 1, 0):
        for x in names:
            c[x].copy_(cs[i][x])
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[i])
    streams, wss = [torch.cuda.Stream(), torch.cuda.Stream()], [workspace(x) for x in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for st, cc, w in zip(streams, cs, wss):
            with torch.cuda.stream(st):
                got.append(run(cc, w)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, ref[i % 2])


@pytest.mark.parametrize("few", [False, True])
def test_small_calls_captured_with_other_lengths(few):
    """Two small calls without a plan kernel on one workspace in one graph, replayed over other lengths
    (as many rows and room for keys) and over a sequence that went out of range."""
    lens = [[1, 3, 0, 1, 1], [2, 0, 1, 1, 2]] if few else [[40, 3, 0, 70, 1], [5, 60, 44, 0, 5]]
    kv = [[30, 9, 4, 200, 1], [2, 7, 1, 90, 400]] if few else [[40, 90, 4, 70, 300], [5, 60, 100, 7, 5]]
    names = ("q", "k", "v", "off", "begin", "len")
    cs = []
    for i in range(2):
        c = make(8, 2, 64, lens[i], kv[i], seed=37 + i)
        rows = 700
        for x in ("k", "v"):
            c[x] = torch.cat([c[x], c[x].new_full((rows - c["rows"], 2, 64), float("nan"))])
        cs.append(dict(c, rows=rows, max_kv=512))
    assert cs[0]["T"] == cs[1]["T"]
    for c in cs:
        check(c, run(c)[0])
    ref = [run(c)[0] for c in cs]
    c = dict(cs[0], **{x: cs[0][x].clone() for x in names})
    ws, s = workspace(c), torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        first, _ = run(c, ws)
        second, _ = run(c, ws)
    for i in (0, 1, 0):
        for x in names:
            c[x].copy_(cs[i][x])
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, ref[i]) and torch.equal(second, ref[i]) and abi.moe_ws_check(ws) == 0
    c["len"][0] = 513
    gr.replay()
    torch.cuda.synchronize()
    assert abi.moe_ws_check(ws) == abi.DEVERR_BAD_RANGE
    n = lens[0][0]
    assert (first[:n] == 7.0).all() and torch.equal(first[n:], ref[0][n:])


def test_hybrid_prompt_then_token():
    """A prompt through a Gated DeltaNet layer and an attention layer, one workspace for both, then
    one token of each sequence through the decode step and the attention over the grown cache."""
    gen = torch.Generator(device=DEV).manual_seed(31)
    lens, H, d = [70, 9], 4, 128
    T, n, room = sum(lens), 2, 80
    off = torch.tensor([0, 70, 79], dtype=torch.int32, device=DEV)
    gsh, ash = abi.moe_gdn_shape(2, H, d, d), abi.moe_attn_shape(H, 2, d)
    ws = torch.zeros(max(abi.moe_gdn_prefill_workspace_size(gsh, n, T), abi.moe_attn_workspace_size(ash, n, T, room)),
                     dtype=torch.uint8, device=DEV)
    q, k, v, g, beta = (x[:, 0].contiguous() for x in synth.gdn_inputs(2, H, d, d, 1, T, 32, DEV))
    S = torch.empty(n, H, d, d, device=DEV)
    mid = torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV)
    abi.moe_gdn_prefill(gsh, n, T, off, None, S, q, k, v, g, beta, mid, ws)
    cache_k, cache_v = (torch.full((n * room, 2, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kn, vn = (torch.randn(T, 2, d, device=DEV, generator=gen).to(torch.bfloat16) for _ in range(2))
    for s, (a, b) in enumerate(((0, 70), (70, 79))):
        cache_k[s * room:s * room + b - a], cache_v[s * room:s * room + b - a] = kn[a:b], vn[a:b]
    begin = torch.tensor([0, room], dtype=torch.int32, device=DEV)
    length = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = torch.empty_like(mid)
    abi.moe_attn_forward(ash, n, T, off, begin, length, room, mid, cache_k, cache_v, n * room, d ** -0.5, out, ws)
    c = dict(n=n, off=off, begin=begin, len=length, q=mid, k=cache_k, v=cache_v, scale=d ** -0.5, shape=ash)
    check(c, out)
    gc = dict(shape=gsh, n=n, off=off, S=None, q=q, k=k, v=v, g=g, beta=beta)
    from test_gpu_gdn_prefill import check as gdn_check
    gdn_check(gc, mid, S)
    # one more token of each
    q1, k1, v1, g1, b1 = (x[0].contiguous() for x in synth.gdn_inputs(2, H, d, d, n, 1, 33, DEV))
    S0 = S.clone()
    mid1 = torch.empty(n, H, d, dtype=torch.bfloat16, device=DEV)
    abi.moe_gdn_decode_step(gsh, n, S, q1, k1, v1, g1, b1, mid1)
    for s in range(n):
        cache_k[s * room + lens[s]] = torch.randn(2, d, device=DEV, generator=gen).to(torch.bfloat16)
        cache_v[s * room + lens[s]] = torch.randn(2, d, device=DEV, generator=gen).to(torch.bfloat16)
    length += 1
    one = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    out1 = torch.empty_like(mid1)
    abi.moe_attn_forward(ash, n, n, one, begin, length, room, mid1, cache_k, cache_v, n * room, d ** -0.5, out1, ws)
    check(dict(c, off=one, q=mid1), out1)
    for s in range(n):
        _, o, size, _ = oracle.gdn_prompt(S0[s].double().cpu().numpy(), f64(q1[s:s + 1]), f64(k1[s:s + 1]), f64(v1[s:s + 1]),
                                          f64(g1[s:s + 1]), f64(b1[s:s + 1]))
        assert (np.abs(f64(mid1[s]) - o[0]) <= 2.0 ** -8 * np.abs(o[0]) + 2.0 ** -12 * size[0]).all()
    assert abi.moe_ws_check(ws) == 0

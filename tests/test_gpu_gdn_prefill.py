"""GPU parity of the gated delta rule over prompts (moe_gdn_prefill through the C ABI) against
the fp64 recurrence (oracle.gdn_prompt).

Bars, from the roundings the operator makes.  With m_t = alpha m_{t-1} + |write_t| (the size of
what a row of the state is a sum of; oracle `size` is m / sqrt(d_k), a bound of the output's
sums):
  out    half a bf16 step of the result, 2^-8 |o|; the weights q^.k^ of a 64-token block may be
         rounded to bf16 before they meet its writes, 2^-8 size; everything else is carried
         to at least 16 bits, together below 2^-10 size.
  state  held to 24 bits: products of at least 22 bits and fp32 sums of at most 64 + d_k <= 320
         terms, (320 + 8) 2^-24 < 2^-15 of m, twice (once in what the state recalls, once in the
         update): 2^-14 m."""
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


def make(Hk, Hv, dk, dv, lens, seed, start=True, pad=0):
    """Inputs of packed sequences (pad rows before the first and behind the last)."""
    T = sum(lens) + 2 * pad
    q, k, v, g, beta = (x[:, 0].contiguous() for x in synth.gdn_inputs(Hk, Hv, dk, dv, 1, max(T, 1), seed, DEV))
    off = np.concatenate([[pad], pad + np.cumsum(lens)]).astype(np.int32)
    S = synth.gdn_state(Hv, dk, dv, len(lens), seed, DEV) if start else None
    return dict(shape=abi.moe_gdn_shape(Hk, Hv, dk, dv), n=len(lens), T=T, off=torch.from_numpy(off).to(DEV), S=S, q=q, k=k,
                v=v, g=g, beta=beta)


def workspace(c):
    return torch.zeros(abi.moe_gdn_prefill_workspace_size(c["shape"], c["n"], c["T"]), dtype=torch.uint8, device=DEV)


def run(c, ws=None, in_place=False, stream=None):
    sh = c["shape"]
    ws = workspace(c) if ws is None else ws
    out = torch.full((max(c["T"], 1), sh.n_v_heads, sh.d_v), 7.0, dtype=torch.bfloat16, device=DEV)
    S = c["S"].clone() if in_place else torch.full((c["n"], sh.n_v_heads, sh.d_v, sh.d_k), 9.0, device=DEV)
    abi.moe_gdn_prefill(sh, c["n"], c["T"], c["off"], S if in_place else c["S"], S, c["q"], c["k"], c["v"], c["g"],
                        c["beta"], out, ws, stream=stream)
    return out, S, ws


def check(c, out, S, seqs=None):
    sh, off = c["shape"], c["off"].tolist()
    for s in range(c["n"]) if seqs is None else seqs:
        at = slice(off[s], off[s + 1])
        S0 = np.zeros((sh.n_v_heads, sh.d_v, sh.d_k)) if c["S"] is None else c["S"][s].double().cpu().numpy()
        S_ref, o, size, m = oracle.gdn_prompt(S0, f64(c["q"][at]), f64(c["k"][at]), f64(c["v"][at]),
                                              c["g"][at].double().cpu().numpy(), c["beta"][at].double().cpu().numpy())
        err = np.abs(f64(out[at]) - o)
        bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -10) * size + 1e-36
        assert (err <= bar).all(), (s, (err / bar).max(), np.argwhere(err > bar)[:4].tolist())
        err = np.abs(S[s].double().cpu().numpy() - S_ref)
        bar = 2.0 ** -14 * m[..., None] + 1e-36
        assert (err <= bar).all(), (s, (err / bar).max())


@pytest.mark.parametrize("Hk,Hv,dk,dv,lens,start", [
    (2, 4, 128, 128, [1], True),
    (2, 4, 128, 128, [1, 2, 3, 15, 16, 17], True),
    (2, 4, 128, 128, [63, 64, 65], True),
    (2, 4, 128, 128, [127, 128, 129, 0, 1], False),
    (2, 2, 64, 64, [200, 31], True),
    (1, 4, 256, 96, [70, 130], True),      # four value heads on one key head, d_k 256
    (3, 3, 128, 40, [33, 100], False),     # a value width that fills no tile
    (2, 2, 64, 1, [65, 7], True),          # one value element
    (1, 2, 128, 257, [90], True),
    (1, 2, 256, 33, [64, 66], False),
    (16, 32, 128, 128, [150, 20], True),   # the 80B-like shape
    (4, 32, 128, 128, [70, 3, 65], True),  # enough state rows for 64-row CTAs, one long chain
    (4, 32, 128, 128, [65] * 6, True),     # ... and no chain longer than the rest: two slices a warp
    (2, 32, 128, 72, [66, 1, 64, 2, 64, 64, 30], False),
    (1, 32, 128, 33, [64] * 8, True),      # ... with an odd value width
    (2, 32, 256, 96, [65, 64, 10, 1], True),  # d_k 256, two slices a warp
])
def test_prompt_matches_oracle(Hk, Hv, dk, dv, lens, start):
    c = make(Hk, Hv, dk, dv, lens, seed=3 * Hv + dk + len(lens), start=start)
    out, S, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out, S)


def test_long_prompt_and_pieces():
    """700 tokens in one call, and in pieces of 1, 64, 300 and the rest, the state handed on."""
    c = make(2, 4, 128, 128, [700], seed=5)
    out, S, _ = run(c)
    check(c, out, S)
    S2, outs = c["S"], []
    for a, b in ((0, 1), (1, 65), (65, 365), (365, 700)):
        p = dict(c, T=b - a, off=torch.tensor([0, b - a], dtype=torch.int32, device=DEV), S=S2,
                 **{x: c[x][a:b].clone() for x in ("q", "k", "v", "g", "beta")})
        o, S2, _ = run(p)
        outs.append(o)
    check(c, torch.cat(outs), S2)


def test_prompt_then_decode_steps():
    """The decode step goes on from the prompt's state as the recurrence does."""
    c = make(2, 4, 128, 64, [77, 20], seed=6)
    B, extra = 2, 3
    q, k, v, g, beta = synth.gdn_inputs(2, 4, 128, 64, B, extra, 60, DEV)
    out, S, _ = run(c)
    check(c, out, S)
    S0 = S.double().cpu().numpy()
    for t in range(extra):
        o = torch.empty(B, 4, 64, dtype=torch.bfloat16, device=DEV)
        abi.moe_gdn_decode_step(c["shape"], B, S, q[t].contiguous(), k[t].contiguous(), v[t].contiguous(),
                                g[t].contiguous(), beta[t].contiguous(), o)
    for b in range(B):
        S_ref, o_ref, size, m = oracle.gdn_prompt(S0[b], f64(q[:, b]), f64(k[:, b]), f64(v[:, b]), f64(g[:, b]),
                                                  f64(beta[:, b]))
        assert (np.abs(f64(o[b]) - o_ref[-1]) <= 2.0 ** -8 * np.abs(o_ref[-1]) + 2.0 ** -12 * size[-1]).all()
        assert (np.abs(S[b].double().cpu().numpy() - S_ref) <= 2.0 ** -14 * m[..., None]).all()


@pytest.mark.parametrize("kind", ["keep", "forget", "slow", "grow", "write_all", "no_write", "same_key", "zero_key"])
def test_gates_and_keys_at_their_limits(kind):
    c = make(2, 4, 128, 48, [150], seed=11)
    if kind == "keep":
        c["g"].zero_()
    elif kind == "forget":  # the state is dropped at tokens 5, 64 and 100
        c["g"][[5, 64, 100]] = -float("inf")
    elif kind == "slow":
        c["g"].mul_(1e-4)
        c["g"][70] = -60.0
    elif kind == "grow":
        c["g"].fill_(0.01)
    elif kind == "write_all":
        c["beta"].fill_(1.0)
    elif kind == "no_write":
        c["beta"].zero_()
    elif kind == "same_key":  # every entry of the block's system is as large as it gets
        c["k"][:] = c["k"][:1].clone()
        c["g"].zero_()
        c["beta"].fill_(1.0)
    else:
        c["k"][[0, 63, 64, 149]] = 0
        c["q"][[1, 64]] = 0
    out, S, _ = run(c)
    check(c, out, S)


def test_scale_of_values_and_keys():
    """Values of 1e30 and 1e-30 and keys of 1e15 and 1e-3: only the ratios count."""
    c = make(1, 2, 128, 32, [80], seed=12)
    c["v"][:, 0] *= 1e30
    c["v"][:, 1] *= 1e-30
    c["S"][:, 0] *= 1e30
    c["S"][:, 1] *= 1e-30
    c["k"][::2] *= 1e15
    c["k"][1::2] *= 1e-3
    out, S, _ = run(c)
    check(c, out, S)


def test_bad_ranges_are_left_out():
    """Sequences 1 (backwards), 2 (overlaps), 4 and 5 (past T) are left out, the others computed;
    rows of no sequence and their states stay as they were."""
    c = make(2, 4, 128, 64, [40, 0, 0, 20, 0, 0], seed=13)
    c["off"] = torch.tensor([0, 40, 20, 40, 60, 61, 10], dtype=torch.int32, device=DEV)
    out, S, ws = run(c)
    assert abi.moe_ws_check(ws) == abi.DEVERR_BAD_RANGE
    assert abi.moe_ws_check(ws) == 0
    check(c, out, S, seqs=(0, 3))
    assert (S[[1, 2, 4, 5]] == 9.0).all()


def test_rows_outside_and_state_in_place():
    c = make(2, 4, 128, 64, [50, 0, 9], seed=14, pad=5)
    out, S, ws = run(c, in_place=True)
    check(c, out, S)
    assert (out[:5] == 7.0).all() and (out[-5:] == 7.0).all()
    assert torch.equal(S[1], c["S"][1])
    # the same bits out of place, from the same workspace again, and alone
    out2, S2, _ = run(c, ws=ws)
    assert torch.equal(out, out2) and torch.equal(S, S2)
    a, b = c["off"].tolist()[2:4]
    alone = dict(c, n=1, T=b - a, off=torch.tensor([0, b - a], dtype=torch.int32, device=DEV), S=c["S"][2:3],
                 **{x: c[x][a:b].clone() for x in ("q", "k", "v", "g", "beta")})
    check(alone, *run(alone)[:2])


def test_no_tokens_copies_the_states():
    c = make(2, 2, 64, 32, [0, 0], seed=15)
    c["T"] = 0
    _, S, ws = run(c)
    assert torch.equal(S, c["S"]) and abi.moe_ws_check(ws) == 0
    _, S, _ = run(dict(c, S=None))
    assert (S == 0).all()


def test_many_short_sequences():
    lens = [(i * 7) % 5 for i in range(1500)]
    c = make(1, 1, 64, 16, lens, seed=16)
    out, S, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out, S, seqs=list(range(0, 40)) + list(range(1020, 1030)) + list(range(1490, 1500)))


def test_rows_past_32_bits():
    """A sequence whose rows start past 2^31 elements of v and out."""
    Hv, dv, n = 32, 128, 70
    T = (1 << 31) // (Hv * dv) + 200
    c = make(1, Hv, 64, dv, [n], seed=17, start=False)
    a = T - n - 3
    big = {x: torch.zeros(T, *c[x].shape[1:], dtype=c[x].dtype, device=DEV) for x in ("q", "k", "v", "g", "beta")}
    for x in big:
        big[x][a:a + n] = c[x]
    d = dict(c, T=T, off=torch.tensor([a, a + n], dtype=torch.int32, device=DEV), **big)
    out, S, ws = run(d)
    assert abi.moe_ws_check(ws) == 0
    check(c, out[a:a + n], S)
    assert (out[a - 1] == 7.0).all() and (out[a + n:] == 7.0).all()


def test_captured_and_on_two_streams():
    """A captured call replayed on new inputs, and two calls at once on two streams, each with its
    own workspace."""
    c1, c2 = make(2, 4, 128, 64, [300, 20], seed=18), make(2, 4, 128, 64, [20, 300], seed=19)
    ref = [run(c)[:2] for c in (c1, c2)]
    buf = {x: c1[x].clone() for x in ("q", "k", "v", "g", "beta", "off", "S")}
    c = dict(c1, **buf)
    ws, s = workspace(c), torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        out, S, _ = run(c, ws=ws)
    for src, want in ((c1, ref[0]), (c2, ref[1]), (c1, ref[0])):
        for x in buf:
            buf[x].copy_(src[x])
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(S, want[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [workspace(c1), workspace(c2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for st, cc, w in zip(streams, (c1, c2), wss):
            with torch.cuda.stream(st):
                got.append(run(cc, ws=w))
    torch.cuda.synchronize()
    for i, (o, S, _) in enumerate(got):
        assert torch.equal(o, ref[i % 2][0]) and torch.equal(S, ref[i % 2][1])

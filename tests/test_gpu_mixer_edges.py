"""GPU tests of what the token mixers (moe_attn_forward, moe_gdn_prefill) promise beside their
sums: who an infinity or NaN reaches, the same bits from the same call, workspaces sized once.
Inputs and oracle checks are those of the operators' own tests."""
import pytest
import torch

from int4_expert_gemv_router_b200 import abi, build
import test_gpu_gdn_prefill as gdn
from test_gpu_attn import check, make, run

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,lens,kv,max_kv", [
    (9, 1, [3, 0], [40, 5], 40),
    (12, 1, [2, 1, 1, 1], [130, 3, 129, 1], 512),
    (16, 1, [2, 0], [2, 0], 2),                   # a whole prompt of two tokens
    (32, 2, [3, 0, 0], [128, 7, 0], 128),         # the last key of a tile, two key heads
    (16, 1, [2, 0], [129, 9], 129),               # hidden keys are a tile of their own
    (16, 1, [3, 0, 0], [9500, 3, 0], 9500),       # keys in pieces
    (24, 2, [2, 1, 1, 1], [3000, 700, 3, 1], 3000),
    (9, 1, [3, 1, 0, 1], [1, 1, 0, 1], 1),        # queries that see no key at all beside one that does
])
def test_nonfinite_values_with_one_position_a_unit(Hq, Hkv, d, lens, kv, max_kv):
    """More than eight query heads a key head: units of one position, which do not see the last keys of
    their sequence.  Every other element keeps its bits."""
    c = dict(make(Hq, Hkv, d, lens, kv, seed=40 + Hq + d), max_kv=max_kv)
    base, ws = run(c)
    check(c, base)
    off, begin = c["off"].tolist(), c["begin"].tolist()
    gone = torch.zeros(c["T"], Hq, d, dtype=torch.bool, device=DEV)
    for s, n in enumerate(lens):
        for i in range(min(2, n, kv[s])):  # the last key (its query alone sees it) and the one before
            key, head, col = kv[s] - 1 - i, i % Hkv, (s * 29 + i * 7 + 5) % d
            c["v"][begin[s] + key, head, col] = (float("nan"), float("inf"), -float("inf"))[(s + i) % 3]
            at = slice(off[s] + max(0, key - (kv[s] - n)), off[s + 1])
            gone[at, head * (Hq // Hkv):(head + 1) * (Hq // Hkv), col] = True
    out, _ = run(c, ws)
    assert abi.moe_ws_check(ws) == 0
    assert torch.equal(~torch.isfinite(out.float()), gone)
    assert torch.equal(out[~gone], base[~gone])


@pytest.mark.parametrize("n,H", [(48, 32), (300, 8)])
def test_prompts_of_one_length_keep_their_bits(n, H):
    """More sequences than a plan without its kernel takes, all of one length class, and a last round of
    units that is cut: the same call gives the same bits, however busy the GPU is, and sequences of
    the same inputs differ only where the cut falls, in the call's order."""
    c = gdn.make(H // 2, H, 128, 128, [64] * n, seed=50)
    for x in ("q", "k", "v", "g", "beta"):
        c[x] = c[x][:64].repeat(n, *[1] * (c[x].dim() - 1))
    c["S"][:] = c["S"][:1].clone()
    out, S, ws = gdn.run(c)
    gdn.check(c, out, S, seqs=(0, n - 1))
    a, side = torch.randn(2048, 2048, device=DEV), torch.cuda.Stream()
    for i in range(30):
        if i % 2:
            with torch.cuda.stream(side):
                a = (a @ a).clamp(-1, 1)
        again, S_again, _ = gdn.run(c, ws=ws)
        assert torch.equal(out, again) and torch.equal(S, S_again)
    torch.cuda.synchronize()
    # heads of a state from one slice or two: all of the former come last
    for h in range(H):
        same = (S[:, h] == S[0, h]).flatten(1).all(1)
        first = int(same.long().argmin()) if not same.all() else n
        assert same[:first].all() and not same[first:].any()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33])
def test_offsets_checked_around_a_warp_of_sequences(n):
    """A call's offsets are checked a lane a sequence up to 32 of them: one range out of order, at the first,
    a middle and the last place; the sequence is left out and no other."""
    lens = [1 + i % 3 for i in range(n)]
    c = gdn.make(1, 2, 64, 32, lens, seed=51, pad=2)
    ws = gdn.workspace(c)
    for at in sorted({0, n // 2, n - 1}):
        off = c["off"].clone()
        off[at + 1] = off[at] - 1  # this one ends before it begins, the next begins in an earlier one's rows
        d = dict(c, off=off)
        out, S, _ = gdn.run(d, ws=ws)
        assert abi.moe_ws_check(ws) == abi.DEVERR_BAD_RANGE and abi.moe_ws_check(ws) == 0
        left = [s for s in (at, at + 1) if s < n]
        gdn.check(d, out, S, seqs=[s for s in range(n) if s not in left])
        assert all((S[s] == 9.0).all() for s in left)
    out, S, _ = gdn.run(c, ws=ws)
    assert abi.moe_ws_check(ws) == 0
    gdn.check(c, out, S)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("between", ["attention", "prompt", "router", "step"])
def test_early_state_reads_behind_a_kernel_that_writes_another(between, graph):
    """MOE_GDN_EARLY_STATE asks that the kernel right before the step does not write its state.  The one
    before that may: prompt (writes S), one other small call, early step on S, over and over, gives the
    bits of the plain steps."""
    Hk, H, d, n, rounds = 2, 4, 64, 2, 6
    c = gdn.make(Hk, H, d, d, [300, 40], seed=52)
    other = gdn.make(Hk, H, d, d, [3, 1], seed=53)
    at = make(4, 2, 64, [1, 1], [70, 9], seed=54)
    sh, T = c["shape"], c["T"]
    ws, wsb = gdn.workspace(c), torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)
    one = [x[:n].contiguous() for x in (c["q"], c["k"], c["v"], c["g"], c["beta"])]
    mshape = abi.moe_shape(256, 128, 128, 16, 2, 4, 64)
    x, wr = (torch.randn(r, 256, device=DEV).to(torch.bfloat16) for r in (20, 16))
    idx, wts = torch.empty(20, 2, dtype=torch.int32, device=DEV), torch.empty(20, 2, device=DEV)
    assert abi.moe_workspace_size(mshape, 20) <= wsb.numel()

    def chain(flags):
        S, S2, aside = c["S"].clone(), other["S"].clone(), other["S"].clone()
        out = torch.zeros(T, H, d, dtype=torch.bfloat16, device=DEV)
        outs = torch.zeros(rounds, 2, n, H, d, dtype=torch.bfloat16, device=DEV)
        side_out, a_out = torch.zeros(4, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)

        def calls():
            st = torch.cuda.current_stream()
            for r in range(rounds):
                abi.moe_gdn_prefill(sh, n, T, c["off"], S, S, c["q"], c["k"], c["v"], c["g"], c["beta"], out, ws, stream=st)
                for i in range(2):
                    if between == "attention":
                        abi.moe_attn_forward(at["shape"], 2, 2, at["off"], at["begin"], at["len"], at["max_kv"], at["q"], at["k"],
                                             at["v"], at["rows"], at["scale"], a_out, wsb, stream=st)
                    elif between == "prompt":
                        abi.moe_gdn_prefill(sh, 2, 4, other["off"], other["S"], S2, other["q"], other["k"], other["v"], other["g"],
                                            other["beta"], side_out, wsb, stream=st)
                    elif between == "router":
                        abi.moe_router_topk(mshape, x, 20, wr, None, idx, wts, wsb, stream=st)
                    else:
                        abi.moe_gdn_decode_step(sh, n, aside, *one, side_out, stream=st, flags=flags if i else 0)
                    abi.moe_gdn_decode_step(sh, n, S, *one, outs[r, i], stream=st, flags=flags)

        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        if graph:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=stream):
                calls()
            gr.replay()
        else:
            with torch.cuda.stream(stream):
                calls()
        torch.cuda.synchronize()
        assert abi.moe_ws_check(ws) == 0 and abi.moe_ws_check(wsb) == 0
        return S, out, outs

    plain, early = chain(0), chain(abi.MOE_GDN_EARLY_STATE)
    assert all(torch.equal(a, b) for a, b in zip(plain, early))


@pytest.mark.parametrize("Hq,Hkv,d", [(5, 1, 64), (9, 1, 64), (30, 2, 64), (7, 1, 128)])
def test_long_joins_of_an_odd_number_of_rows(Hq, Hkv, d):
    """One token over keys in more than 16 pieces (joined in two steps), rows that fill no warp's halves."""
    c = make(Hq, Hkv, d, [1, 0], [20000, 3], seed=55 + Hq)
    out, ws = run(c)
    assert abi.moe_ws_check(ws) == 0
    check(c, out)
    for _ in range(5):
        assert torch.equal(run(c, ws)[0], out)


def test_one_attention_workspace_for_every_smaller_call():
    """Sized for the largest batch; fewer sequences with as many rows take another kernel and fit all the same."""
    at = abi.moe_attn_shape(16, 2, 128)
    size = abi.moe_attn_workspace_size(at, 64, 64, 4096)
    ws = torch.zeros(size + 256, dtype=torch.uint8, device=DEV)
    ws[size:] = 77
    for lens, kv in (([1] * 64, [50 + 9 * i for i in range(64)]), ([64], [4096]), ([30, 34], [1000, 3000]), ([1], [4096])):
        c = make(16, 2, 128, lens, kv, seed=56 + len(lens))
        out, _ = run(c, ws[:size])
        assert abi.moe_ws_check(ws) == 0
        check(c, out, seqs=range(min(8, len(lens))))
        assert (ws[size:] == 77).all()


def prompt_reference(c):
    """The recurrence in 64 bits with whatever the inputs hold (the normalised keys of a row with an infinity
    or NaN are not finite either)."""
    sh, off = c["shape"], c["off"].tolist()
    rep, outs, states = sh.n_v_heads // sh.n_k_heads, [], []
    for s in range(c["n"]):
        S = torch.zeros(sh.n_v_heads, sh.d_v, sh.d_k, device=DEV, dtype=torch.float64) if c["S"] is None else c["S"][s].double()
        for t in range(off[s], off[s + 1]):
            k, q = (x[t].double() for x in (c["k"], c["q"]))
            k, q = (x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6) for x in (k, q))
            k, q = k.repeat_interleave(rep, 0)[:, None], q.repeat_interleave(rep, 0)[:, None] / sh.d_k ** 0.5
            S = S * c["g"][t].double().exp()[:, None, None]
            S = S + (c["beta"][t].double()[:, None] * (c["v"][t].double() - (S * k).sum(-1)))[..., None] * k
            outs.append((S * q).sum(-1))
        states.append(S)
    return torch.stack(outs), torch.stack(states)


NONFINITE = [  # (input, token, value head or key head, column, value); tokens count over the call
    [("v", 100, 1, 7, float("inf"))], [("v", 100, 1, 7, float("nan"))], [("v", 0, 0, 0, -float("inf"))],
    [("v", 149, 3, 2, float("nan")), ("v", 20, 2, 3, float("inf"))], [("v", 64, 0, 1, float("inf"))],
    [("k", 70, 0, 3, float("nan"))], [("k", 63, 1, 60, -float("inf"))], [("q", 90, 1, 5, float("nan"))],
    [("q", 0, 0, 0, float("inf"))], [("g", 33, 1, None, float("nan"))], [("g", 99, 2, None, float("inf"))],
    [("beta", 127, 0, None, float("nan"))], [("beta", 1, 3, None, float("inf"))],
    [("S", 0, 2, 9, float("inf"))], [("S", 1, 0, 0, float("nan"))],  # the start of sequence 0 or 1
    [("g", 40, 1, None, -float("inf")), ("v", 30, 1, 4, float("nan"))],  # forgetting does not bring it back
]


@pytest.mark.parametrize("bad", NONFINITE, ids=lambda b: "-".join(f"{x[0]}{x[1]}" for x in b))
@pytest.mark.parametrize("Hk,Hv,dk,dv", [(2, 4, 128, 40), (2, 4, 64, 33), (2, 4, 256, 24), (2, 96, 128, 128), (2, 64, 256, 96)])
def test_prompt_infinities_and_nan_reach_the_tokens_behind_them(Hk, Hv, dk, dv, bad):
    """... of their sequence, head and (a value's) column, and nothing else: the rest stays within the bars
    of the same call without them.  The shapes take one and two slices a warp, and one to four warps a slab."""
    c = gdn.make(Hk, Hv, dk, dv, [150, 70], seed=57)
    clean = dict(c)
    c = dict(c, **{x: c[x].clone() for x in ("q", "k", "v", "g", "beta", "S")})
    for name, t, h, col, val in bad:
        if name == "S":
            c["S"][t, h, col % dv, col] = val
        elif col is None:
            c[name][t, h] = val
        else:
            c[name][t, h, col] = val
    want, S_want = prompt_reference(c)
    out, S, ws = gdn.run(c)
    assert abi.moe_ws_check(ws) == 0
    base, S_base, _ = gdn.run(clean, ws=ws)
    gdn.check(clean, base, S_base)
    finite, S_finite = torch.isfinite(want), torch.isfinite(S_want)
    assert not finite.all() and finite.any() and torch.equal(torch.isfinite(out.float()), finite)
    assert torch.equal(torch.isfinite(S), S_finite)
    # within the bars of the clean call where the oracle's sizes are (they do not depend on what was planted)
    off = clean["off"].tolist()
    for s in range(2):
        at = slice(off[s], off[s + 1])
        S_ref, o, size, m = gdn.oracle.gdn_prompt(clean["S"][s].double().cpu().numpy(), *(gdn.f64(clean[x][at]) for x in "qkv"),
                                                  *(clean[x][at].double().cpu().numpy() for x in ("g", "beta")))
        o, size, m, S_ref = (torch.from_numpy(x).to(DEV) for x in (o, size, m, S_ref))
        ok = (out[at].double() - want[at]).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -10) * size + 1e-36
        assert ok[finite[at]].all()
        assert ((S[s].double() - S_want[s]).abs() <= 2.0 ** -14 * m[..., None])[S_finite[s]].all()
    # the same call, the same bits; and the sequence without any keeps its own
    again, S_again, _ = gdn.run(c, ws=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(S.view(torch.int32), S_again.view(torch.int32))
    for s in range(2):
        if finite[off[s]:off[s + 1]].all():
            assert torch.equal(out[off[s]:off[s + 1]], base[off[s]:off[s + 1]]) and torch.equal(S[s], S_base[s])


@pytest.mark.parametrize("big", [2.0 ** 10, 2.0 ** 20, 2.0 ** 30, 1e20])
@pytest.mark.parametrize("order", ["forgotten", "later"])
def test_writes_far_apart_in_one_chunk(order, big):
    """Values `big` times the others' in some columns at one token of a chunk, which a decay then forgets,
    or which comes last.  What shares a scale is good to 2^-30 of the row's largest write in the chunk:
    fp16 pairs of elements scaled to 2^13 .. 2^15 step by 2^-24, so by at most 2^-38 of the largest, in
    R, in T' (whose row meets up to 64 of them) and in W (whose column does): 3 * 64 * 2^-38 < 2^-30.
    The bars of ordinary inputs come on top."""
    c = gdn.make(2, 4, 128, 48, [64], seed=58)
    t = 10 if order == "forgotten" else 60
    c["v"][t, :, 5:9] *= big
    if order == "forgotten":
        c["g"][t + 1] = -float("inf")
    out, S, ws = gdn.run(c)
    assert abi.moe_ws_check(ws) == 0
    S_ref, o, size, m = gdn.oracle.gdn_prompt(c["S"][0].double().cpu().numpy(), *(gdn.f64(c[x]) for x in "qkv"),
                                              *(c[x].double().cpu().numpy() for x in ("g", "beta")))
    top = size.max(0)  # over the chunk
    bar = 2.0 ** -8 * abs(o) + (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -30 * top
    assert (abs(gdn.f64(out) - o) <= bar).all()
    bar = 2.0 ** -14 * m + 2.0 ** -30 * top * 128 ** 0.5
    assert (abs(S[0].double().cpu().numpy() - S_ref) <= bar[..., None]).all()


@pytest.mark.parametrize("g", [0.05, 0.15, 0.2, 0.4, 1.3, 1.4])
def test_prompt_states_that_grow(g):
    """Growth by e^(64 g) inside a chunk, up to what fp32 holds: the tokens before it keep their bars."""
    c = gdn.make(2, 4, 128, 40, [64, 20], seed=59)
    c["g"].fill_(g)
    c["v"] *= 1e-10
    c["S"] *= 1e-10
    out, S, ws = gdn.run(c)
    assert abi.moe_ws_check(ws) == 0 and torch.isfinite(S).all()
    gdn.check(c, out, S)


@pytest.mark.parametrize("beta", [2.0, 20.0, 3000.0])
def test_prompt_writes_that_overshoot(beta):
    """beta of 2 and above, where the rule stops contracting, at two tokens of a chunk."""
    c = gdn.make(2, 4, 128, 40, [64, 20], seed=60)
    c["beta"][[3, 50, 70]] = beta
    out, S, ws = gdn.run(c)
    assert abi.moe_ws_check(ws) == 0
    gdn.check(c, out, S)

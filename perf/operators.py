"""The token mixers of a hybrid model's prompt, as measured cases.

Two operators over packed sequences (sequence s is the token rows offsets[s] .. offsets[s+1]):

  gdn   the gated delta rule over whole prompts (moe_gdn_prefill), per value head with the state
        S (d_v x d_k), k^ = k / max(|k|, 1e-6) and q^ = q / (max(|q|, 1e-6) sqrt(d_k)):
            S_t = e^g_t S_{t-1} + beta_t (v_t - e^g_t S_{t-1} k^_t) k^_t^T,   o_t = S_t q^_t
  attn  causal softmax attention with grouped heads (moe_attn_forward): the queries of a sequence
        are its last tokens, so query i of n sees the keys 0 .. len - n + i; a whole prompt
        (len = n), a chunk of one after its history, or single tokens over a cache
"""
import math

import torch

own = False

# One device buffer of each kind is made per state; the framework's workspace is made by the
# first call on a state and kept with it, as a serving loop keeps it.


def listed():
    return [
        # the last few tokens of a prompt that was fed in pieces: the smallest call, latency alone
        dict(name="gdn tail", op="gdn", lens="17", hk=16, hv=32, dk=128, dv=128, start=True),
        # one ordinary prompt, a new sequence
        dict(name="gdn prompt", op="gdn", lens="1000", hk=16, hv=32, dk=128, dv=128, start=False),
        # a serving batch: prompts of very different lengths, one empty slot among them
        dict(name="gdn ragged", op="gdn", lens="1,700,63,64,0,1531,257,5,1024,33", hk=16, hv=32, dk=128, dv=128,
             start=True),
        # one long document: the sequential axis is all there is
        dict(name="gdn long", op="gdn", lens="8192", hk=16, hv=32, dk=128, dv=128, start=False),
        # a full batch of prompts: throughput
        dict(name="gdn batch", op="gdn", lens=",".join(["1024"] * 16), hk=16, hv=32, dk=128, dv=128, start=False),
        # wide keys and a value width that fills no tile
        dict(name="gdn wide", op="gdn", lens="300,129,511", hk=4, hv=8, dk=256, dv=200, start=True),
        # a short question
        dict(name="attn short", op="attn", lens="37", kv="37", hq=16, hkv=2, d=128),
        # a serving batch of prompts, grouped heads
        dict(name="attn ragged", op="attn", lens="1,700,63,1024,2111,257,5,3000,33,0,128,129",
             kv="1,700,63,1024,2111,257,5,3000,33,0,128,129", hq=16, hkv=4, d=128),
        # one long document, the largest product
        dict(name="attn long", op="attn", lens="16384", kv="16384", hq=16, hkv=2, d=128),
        # pieces of prompts after their histories, narrow heads
        dict(name="attn pieces", op="attn", lens="512,512,300,512", kv="8704,512,4396,2048", hq=16, hkv=8, d=64),
        # one token each for a batch of sequences over their caches
        dict(name="attn tokens", op="attn", lens=",".join(["1"] * 32),
             kv=",".join(str(200 + 251 * i) for i in range(32)), hq=16, hkv=2, d=128),
        # one token of one sequence over a long cache: few rows, a long axis
        dict(name="attn token long", op="attn", lens="1", kv="60001", hq=16, hkv=2, d=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))


def draw(rng):
    if rng.random() < 0.5:
        hk, hv = rng.choice([(16, 32), (16, 16), (4, 8), (2, 2), (1, 4), (8, 32)])
        dk = rng.choice([64, 128, 128, 256])
        dv = rng.choice([128, 64, 256, rng.randint(8, 200)])
        n = _log_int(rng, 1, 16)
        most = 8192 * 32 * 128 // (hv * max(dv, 32)) // n
        lens = [_log_int(rng, 1, max(1, min(4096, most))) for _ in range(n)]
        return dict(op="gdn", lens=",".join(map(str, lens)), hk=hk, hv=hv, dk=dk, dv=dv, start=rng.random() < 0.5)
    hq, hkv = rng.choice([(16, 2), (16, 4), (16, 16), (32, 8), (12, 4), (8, 1), (6, 2)])
    d = rng.choice([64, 128])
    if rng.random() < 0.5:  # prompts, some after a history
        n = _log_int(rng, 1, 12)
        lens = [_log_int(rng, 1, max(16, 6000 // n)) for _ in range(n)]
        kv = [t + (rng.randint(1, 2000) if rng.random() < 0.4 else 0) for t in lens]
    else:  # single tokens over caches
        n = _log_int(rng, 1, 48)
        lens = [1] * n
        kv = [_log_int(rng, 1, 40000 // n) for _ in range(n)]
    return dict(op="attn", lens=",".join(map(str, lens)), kv=",".join(map(str, kv)), hq=hq, hkv=hkv, d=d)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*size):
        return torch.randn(*size, device="cuda", generator=gen).to(torch.bfloat16)

    lens = _ints(case["lens"])
    off = _offsets(lens)
    T, n = off[-1], len(lens)
    s = {"case": case, "n": n, "T": T, "offsets": torch.tensor(off, dtype=torch.int32, device="cuda")}
    if case["op"] == "gdn":
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        s.update(q=normal(T, hk, dk), k=normal(T, hk, dk), v=normal(T, hv, dv))
        # heads that forget within a few tokens and heads that keep hundreds
        reach = 0.3 * torch.exp2(-(torch.arange(hv, device="cuda") % 8).float())
        s["g"] = -reach * torch.rand(T, hv, device="cuda", generator=gen)
        s["beta"] = torch.sigmoid(torch.randn(T, hv, device="cuda", generator=gen))
        s["state"] = 0.1 * torch.randn(n, hv, dv, dk, device="cuda", generator=gen) if case["start"] else None
        s["out"] = torch.empty(T, hv, dv, dtype=torch.bfloat16, device="cuda")
        s["state_out"] = torch.empty(n, hv, dv, dk, device="cuda")
        s["longest"] = max(lens)
        # where the plain form finds token t of sequence b (T: no such token)
        at = torch.arange(max(lens), device="cuda")[None]
        o = s["offsets"].long()
        s["pos"] = torch.where(at < (o[1:] - o[:-1])[:, None], o[:-1, None] + at, T)
        return s
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    kv = _ints(case["kv"])
    # each sequence has a slab of a cache with room to grow
    begin = _offsets([(x + 1 + 63) // 64 * 64 for x in kv])
    rows = begin[-1]
    s.update(q=normal(T, hq, d), k=normal(rows, hkv, d), v=normal(rows, hkv, d), rows=rows, max_kv=max(kv),
             scale=1.0 / math.sqrt(d), kv_begin=torch.tensor(begin[:-1], dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"))
    s["out"] = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    o = s["offsets"].long()
    at = torch.arange(max(lens), device="cuda")[None]
    s["pos"] = torch.where(at < (o[1:] - o[:-1])[:, None], o[:-1, None] + at, T)
    at = torch.arange(max(kv), device="cuda")[None]
    s["kvpos"] = torch.where(at < s["kv_len"][:, None], s["kv_begin"].long()[:, None] + at, rows)
    return s


def run(s):
    if own:
        return _own(s)
    return _plain_gdn(s) if s["case"]["op"] == "gdn" else _plain_attn(s)


def _own(s):
    from int4_expert_gemv_router_b200 import abi

    c = s["case"]
    if c["op"] == "gdn":
        shape = abi.moe_gdn_shape(c["hk"], c["hv"], c["dk"], c["dv"])
        if "ws" not in s:
            size = abi.moe_gdn_prefill_workspace_size(shape, s["n"], s["T"])
            s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        abi.moe_gdn_prefill(shape, s["n"], s["T"], s["offsets"], s["state"], s["state_out"], s["q"], s["k"], s["v"],
                            s["g"], s["beta"], s["out"], s["ws"])
        return {"out": s["out"], "state": s["state_out"]}
    shape = abi.moe_attn_shape(c["hq"], c["hkv"], c["d"])
    if "ws" not in s:
        size = abi.moe_attn_workspace_size(shape, s["n"], s["T"], s["max_kv"])
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    abi.moe_attn_forward(shape, s["n"], s["T"], s["offsets"], s["kv_begin"], s["kv_len"], s["max_kv"], s["q"], s["k"],
                         s["v"], s["rows"], s["scale"], s["out"], s["ws"])
    return {"out": s["out"]}


def _padded(x, pos):
    """Rows of x by sequence [n, longest, ...] in 32 bits, zeros where a sequence has ended."""
    x = x.float()
    return torch.cat([x, x.new_zeros(1, *x.shape[1:])])[pos]


def _plain_gdn(s):
    """The recurrence, one token of every sequence at a time."""
    c, pos = s["case"], s["pos"]
    rep = c["hv"] // c["hk"]
    q, k, v, g, beta = (_padded(s[name], pos) for name in ("q", "k", "v", "g", "beta"))
    q = q / (q.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6) * math.sqrt(c["dk"]))
    k = k / k.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)
    q, k = q.repeat_interleave(rep, 2)[..., None, :], k.repeat_interleave(rep, 2)[..., None, :]
    a, beta = g.exp()[..., None, None], beta[..., None]
    S = torch.zeros_like(s["state_out"]) if s["state"] is None else s["state"]
    o = v.new_empty(v.shape)
    for t in range(s["longest"]):
        S = S * a[:, t]
        S = S + (beta[:, t] * (v[:, t] - (S * k[:, t]).sum(-1)))[..., None] * k[:, t]
        o[:, t] = (S * q[:, t]).sum(-1)
    return {"out": o[pos < s["T"]].to(torch.bfloat16), "state": S}


def _plain_attn(s):
    """Scores, mask, softmax and sum of every sequence, as padded products in 32 bits."""
    c, pos, kvpos = s["case"], s["pos"], s["kvpos"]
    n, longest, most = pos.shape[0], pos.shape[1], kvpos.shape[1]
    hkv, grp, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    q = _padded(s["q"], pos).view(n, longest, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, grp * longest, d)
    k = _padded(s["k"], kvpos).permute(0, 2, 1, 3)
    v = _padded(s["v"], kvpos).permute(0, 2, 1, 3)
    score = ((q * s["scale"]) @ k.transpose(-1, -2)).view(n, hkv, grp, longest, most)
    lens = (s["offsets"][1:] - s["offsets"][:-1]).long()
    last = (s["kv_len"].long() - lens)[:, None] + torch.arange(longest, device="cuda")[None]
    seen = torch.arange(most, device="cuda")[None, None] <= last[..., None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(score.sub_(score.amax(-1, keepdim=True).clamp_min(-1e30)))
    p.div_(p.sum(-1, keepdim=True).clamp_min(1e-30))
    o = (p.view(n, hkv, grp * longest, most) @ v).view(n, hkv, grp, longest, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, longest, c["hq"], d)
    return {"out": o[pos < s["T"]].to(torch.bfloat16)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_gdn(s) if case["op"] == "gdn" else _exact_attn(s)


def _exact_gdn(s):
    """Blocks of 32 tokens in 64 bits: with the decays b_i = e^(g_1 + .. + g_i) inside a block,
    the writes w_i of its tokens solve (I + L) w = beta (v - b S k^), L_ij = beta_i (b_i / b_j) k^_i.k^_j
    for j < i."""
    c = s["case"]
    head = torch.arange(c["hv"], device="cuda") // (c["hv"] // c["hk"])
    outs, states = [], []
    off = s["offsets"].tolist()
    for b in range(s["n"]):
        at = slice(off[b], off[b + 1])
        q, k = s["q"][at].double(), s["k"][at].double()
        q = (q / (torch.linalg.vector_norm(q, dim=-1, keepdim=True).clamp_min(1e-6) * c["dk"] ** 0.5))[:, head]
        k = (k / torch.linalg.vector_norm(k, dim=-1, keepdim=True).clamp_min(1e-6))[:, head]
        v, g, beta = s["v"][at].double(), s["g"][at].double(), s["beta"][at].double()
        S = torch.zeros_like(s["state_out"][b], dtype=torch.float64) if s["state"] is None else s["state"][b].double()
        for t0 in range(0, off[b + 1] - off[b], 32):
            Q, K, V = (x[t0:t0 + 32].transpose(0, 1) for x in (q, k, v))
            G, B = g[t0:t0 + 32].T.cumsum(-1), beta[t0:t0 + 32].T[..., None]
            C = Q.shape[1]
            fade = torch.exp((G[:, :, None] - G[:, None, :]).tril()).tril()
            L = (B * fade * torch.einsum("hid,hjd->hij", K, K)).tril(-1)
            rhs = B * (V - G.exp()[..., None] * torch.einsum("hid,hvd->hiv", K, S))
            w = torch.linalg.solve_triangular(L + torch.eye(C, dtype=L.dtype, device=L.device), rhs, upper=False)
            o = G.exp()[..., None] * torch.einsum("hid,hvd->hiv", Q, S)
            o = o + torch.einsum("hij,hjv->hiv", fade * torch.einsum("hid,hjd->hij", Q, K), w)
            outs.append(o.transpose(0, 1))
            keep = torch.exp(G[:, -1:] - G)[..., None]
            S = torch.exp(G[:, -1])[:, None, None] * S + torch.einsum("hiv,hid->hvd", keep * w, K)
        states.append(S)
    out = torch.cat(outs) if outs else s["v"].double()
    return {"out": out, "state": torch.stack(states)}


def _exact_attn(s):
    """Sequence by sequence and head by head in 64 bits, some rows at a time."""
    c = s["case"]
    out = torch.zeros(s["T"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    off, begin, lens = s["offsets"].tolist(), s["kv_begin"].tolist(), s["kv_len"].tolist()
    for b in range(s["n"]):
        nq = off[b + 1] - off[b]
        for h in range(c["hq"] if nq else 0):
            at = slice(begin[b], begin[b] + lens[b])
            k = s["k"][at, h // (c["hq"] // c["hkv"])].double()
            v = s["v"][at, h // (c["hq"] // c["hkv"])].double()
            for r in range(0, nq, 2048):
                q = s["q"][off[b] + r:min(off[b] + r + 2048, off[b + 1]), h].double()
                m = min(lens[b], lens[b] - nq + r + q.shape[0])
                x = s["scale"] * torch.einsum("id,jd->ij", q, k[:m])
                row = torch.arange(r, r + q.shape[0], device="cuda")[:, None] + (lens[b] - nq)
                x = torch.where(torch.arange(m, device="cuda")[None] > row, -math.inf, x)
                out[off[b] + r:off[b] + r + q.shape[0], h] = torch.softmax(x, -1) @ v[:m]
    return {"out": out}


def work(case):
    lens = _ints(case["lens"])
    T = sum(lens)
    if case["op"] == "gdn":
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        state = 4 * len(lens) * hv * dv * dk * (2 if case["start"] else 1)
        # per token and head: the decay, S k, the update and S q of the recurrence
        return {"bytes": state + T * (2 * 2 * hk * dk + 2 * 2 * hv * dv + 2 * 4 * hv), "flops": 7 * T * hv * dk * dv}
    kv = _ints(case["kv"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(lens, kv))
    read = sum(m for n, m in zip(lens, kv) if n)
    return {"bytes": 2 * (2 * T * hq * d + 2 * read * hkv * d), "flops": 4 * d * hq * pairs}

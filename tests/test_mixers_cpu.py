"""CPU checks of the prompt operators (moe_gdn_prefill, moe_attn_forward): the oracles against
independent formulations, and every refusal of the C ABI (nothing is launched)."""
import numpy as np
import pytest
import torch

import oracle
from int4_expert_gemv_router_b200 import abi, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


# ------------------------------------------------------------------ oracles
def test_gdn_prompt_is_the_steps():
    rng = np.random.default_rng(0)
    T, Hk, Hv, dk, dv = 9, 2, 4, 16, 5
    S0 = rng.normal(size=(Hv, dv, dk))
    q, k, v = rng.normal(size=(T, Hk, dk)), rng.normal(size=(T, Hk, dk)), rng.normal(size=(T, Hv, dv))
    g, beta = -rng.random((T, Hv)), rng.random((T, Hv))
    k[3] = 0.0
    S1, o1 = oracle.gdn_steps(S0, q, k, v, g, beta)
    S2, o2, size, S_size = oracle.gdn_prompt(S0, q, k, v, g, beta)
    np.testing.assert_allclose(S2, S1, rtol=0, atol=1e-12)
    np.testing.assert_allclose(o2, o1, rtol=0, atol=1e-12)
    assert (np.abs(o2) <= size + 1e-12).all() and (np.abs(S2).max(-1) <= S_size + 1e-12).all()


def test_attention_oracle_closed_forms():
    rng = np.random.default_rng(1)
    n, L, Hq, Hkv, d = 5, 8, 4, 2, 6
    k, v = rng.normal(size=(L, Hkv, d)), rng.normal(size=(L, Hkv, d))
    # equal scores: the running mean of the values seen
    out, _ = oracle.attention(np.zeros((n, Hq, d)), k, v, 1.0)
    for i in range(n):
        for h in range(Hq):
            np.testing.assert_allclose(out[i, h], v[:L - n + i + 1, h // 2].mean(0), atol=1e-14)
    # against torch's own softmax in 64 bits, one query at a time
    q = rng.normal(size=(n, Hq, d))
    out, mass = oracle.attention(q, k, v, 0.3)
    for i in range(n):
        for h in range(Hq):
            m = L - n + i + 1
            p = torch.softmax(0.3 * torch.from_numpy(k[:m, h // 2]) @ torch.from_numpy(q[i, h]), 0)
            np.testing.assert_allclose(out[i, h], (p @ torch.from_numpy(v[:m, h // 2])).numpy(), atol=1e-13)
    assert (np.abs(out) <= mass + 1e-14).all()
    # more queries than keys: the first see nothing
    out, _ = oracle.attention(rng.normal(size=(4, Hq, d)), k[:2], v[:2], 1.0)
    assert (out[:2] == 0).all()
    np.testing.assert_allclose(out[2], np.repeat(v[0], 2, 0), atol=1e-14)


# ------------------------------------------------------------------ refusals
def _buf(n=4096):
    return torch.zeros(n, dtype=torch.uint8)


def _gdn(shape=(2, 4, 128, 64), n=1, T=4, offsets=0, state_in=None, state_out=0, q=0, ws=None):
    bufs = [_buf() for _ in range(8)]
    pick = lambda given, i: bufs[i] if isinstance(given, int) and given == 0 else given  # noqa: E731
    sh = None if shape is None else abi.moe_gdn_shape(*shape)
    ws = _buf(1 << 22) if ws is None else ws
    abi.moe_gdn_prefill(sh, n, T, pick(offsets, 0), state_in, pick(state_out, 1), pick(q, 2), bufs[3], bufs[4], bufs[5],
                        bufs[6], bufs[7], ws, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(shape=(2, 3, 128, 64)), -1), (dict(shape=(0, 4, 128, 64)), -1), (dict(shape=(2, 4, 96, 64)), -5),
    (dict(shape=(2, 4, 128, 0)), -1), (dict(n=0), -1), (dict(n=65537), -1), (dict(T=-1), -1), (dict(offsets=None), -1),
    (dict(state_out=None), -1), (dict(q=None), -1), (dict(q=_buf()[2:]), -1), (dict(ws=_buf(64)), -1),
])
def test_gdn_prefill_refuses(kw, status):
    with pytest.raises(abi.MoeError) as ei:
        _gdn(**kw)
    assert ei.value.status == status


def test_gdn_prefill_refuses_overlapping_states():
    states = torch.zeros(2 * 4 * 64 * 128 + 64, dtype=torch.float32)
    with pytest.raises(abi.MoeError) as ei:
        _gdn(state_in=states, state_out=states[64:])
    assert ei.value.status == -1 and "overlap" in str(ei.value)


def _attn(shape=(4, 2, 128), n=1, T=4, off=0, begin=0, length=0, max_kv=8, q=0, k=0, kv_rows=8, scale=0.1, ws=None):
    bufs = [_buf() for _ in range(7)]
    pick = lambda given, i: bufs[i] if isinstance(given, int) and given == 0 else given  # noqa: E731
    ws = _buf(1 << 22) if ws is None else ws
    abi.moe_attn_forward(abi.moe_attn_shape(*shape), n, T, pick(off, 0), pick(begin, 1), pick(length, 2), max_kv,
                         pick(q, 3), pick(k, 4), bufs[5], kv_rows, scale, bufs[6], ws, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(shape=(3, 2, 128)), -1), (dict(shape=(4, 0, 128)), -1), (dict(shape=(4, 2, 96)), -5),
    (dict(shape=(4, 2, 0)), -1), (dict(shape=(130, 2, 64)), -5), (dict(n=0), -1), (dict(n=65537), -1), (dict(T=-1), -1),
    (dict(off=None), -1), (dict(begin=None), -1), (dict(length=None), -1), (dict(max_kv=-1), -1), (dict(kv_rows=-1), -1),
    (dict(begin=None, length=None, kv_rows=3), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(q=_buf()[8:]), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(ws=_buf(64)), -1),
])
def test_attn_refuses(kw, status):
    with pytest.raises(abi.MoeError) as ei:
        _attn(**kw)
    assert ei.value.status == status


def test_workspace_sizes_grow_and_refuse():
    sh, at = abi.moe_gdn_shape(16, 32, 128, 128), abi.moe_attn_shape(16, 2, 128)
    assert abi.moe_gdn_prefill_workspace_size(sh, 1, 0) >= 256
    assert abi.moe_gdn_prefill_workspace_size(sh, 4, 4096) >= abi.moe_gdn_prefill_workspace_size(sh, 1, 64)
    assert abi.moe_attn_workspace_size(at, 1, 0, 0) >= 256
    assert abi.moe_attn_workspace_size(at, 64, 4096, 4096) >= abi.moe_attn_workspace_size(at, 1, 1, 1)
    for bad in ((sh, 0, 4), (sh, 1, -1), (abi.moe_gdn_shape(2, 3, 128, 4), 1, 4)):
        with pytest.raises(abi.MoeError):
            abi.moe_gdn_prefill_workspace_size(*bad)
    for bad in ((at, 0, 4, 4), (at, 1, -1, 4), (at, 1, 4, -1), (abi.moe_attn_shape(4, 2, 32), 1, 4, 4)):
        with pytest.raises(abi.MoeError):
            abi.moe_attn_workspace_size(*bad)


def test_attn_without_queries_is_nothing():
    _attn(T=0, q=None)


@pytest.mark.parametrize("shape", [(16, 2, 128), (16, 16, 64), (24, 2, 64), (64, 1, 128), (6, 2, 64)])
def test_attn_workspace_never_falls(shape):
    """Sized once for the largest numbers, it serves every smaller call."""
    at = abi.moe_attn_shape(*shape)
    size = {(n, T, kv): abi.moe_attn_workspace_size(at, n, T, kv)
            for n in (1, 2, 3, 17, 64, 256, 1000) for T in (0, 1, 2, 16, 128, 512, 5000) for kv in (0, 1, 512, 513, 8192)}
    for (n, T, kv), x in size.items():
        for (m, U, kw), y in size.items():
            assert not (n <= m and T <= U and kv <= kw) or x <= y, ((n, T, kv), (m, U, kw))


def test_gdn_workspace_never_falls():
    sh = abi.moe_gdn_shape(2, 4, 128, 64)
    size = {(n, T): abi.moe_gdn_prefill_workspace_size(sh, n, T) for n in (1, 2, 63, 64, 65, 1000) for T in (0, 1, 63, 64, 65, 4000)}
    for (n, T), x in size.items():
        assert all(x <= y for (m, U), y in size.items() if n <= m and T <= U)


@pytest.mark.parametrize("n,T", [(1, 64), (1, 8192), (16, 16 * 1024), (4096, 4096), (10, 3678), (3, 0)])
def test_gdn_workspace_is_what_the_header_states(n, T):
    """256 d_k H_k + 16,384 H_v + 8 bytes a chunk, T / 64 + min(n_seqs, T) chunks, 16 bytes a sequence, the
    control block and each part's padding to 256 bytes."""
    Hk, Hv, dk = 16, 32, 128
    stated = (T // 64 + min(n, T)) * (256 * dk * Hk + 16384 * Hv + 8) + 16 * n
    got = abi.moe_gdn_prefill_workspace_size(abi.moe_gdn_shape(Hk, Hv, dk, 128), n, T)
    assert stated <= got <= stated + 8 * 256 + 256

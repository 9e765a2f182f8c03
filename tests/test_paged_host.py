"""The paged cache without a GPU: pins of its oracle, host-side refusals of the
C ABI (made before any CUDA call) and of the Python binding."""
import ctypes

import numpy as np
import pytest
import torch

from gen import counter_hash as ch
from oracle import paged as P
from oracle import reference as R
from shared_top_routing_b200 import sa as S


# ----------------------------------------------------------------- oracle

def test_nearest_code_is_nearest_and_ties_go_to_the_even_code():
    vals = R.e4m3_bits_to_f64(np.arange(127))
    x = np.concatenate([np.linspace(-500, 500, 4001), vals, -vals, (vals[1:] + vals[:-1]) / 2,
                        vals * (1 + 2.0 ** -20), [2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -11]])
    got = P.e4m3_nearest(x)
    y = R.e4m3_bits_to_f64(got)
    clipped = np.clip(x, -448, 448)
    best = np.abs(np.abs(clipped)[:, None] - vals[None, :]).min(1)
    assert np.array_equal(np.abs(clipped - y), best)
    ties = (vals[1:] + vals[:-1]) / 2
    assert (P.e4m3_nearest(ties) % 2 == 0).all()
    # torch's conversion, where nothing is clamped
    inside = np.abs(x) <= 448
    t = torch.from_numpy(x[inside]).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    f32 = x[inside].astype(np.float32).astype(np.float64)
    assert np.array_equal(P.e4m3_nearest(f32), t)
    assert list(P.e4m3_nearest([np.inf, -np.inf, np.nan])) == [0x7F] * 3


def test_scale_is_the_least_that_holds_the_row():
    x = R.bf16_bits_to_f64(ch.normal_bf16(5, 1, count=40 * 128)).reshape(40, 128)
    x = x * np.exp2(np.arange(-20, 20))[:, None]
    x[3] = 0.0
    x[4, 7], x[4, 8] = np.inf, np.nan
    e = P.scale_exponent(x)
    top = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
    assert e[3] == -118
    live = top > 0
    assert (top <= 448 * np.exp2(e.astype(float))).all()
    assert (top > 448 * np.exp2(e.astype(float) - 1))[live].all()
    # exact borders: 448 * 2^n needs n, the next bf16 above it n + 1
    edge = np.zeros((2, 128))
    edge[0, 0], edge[1, 0] = 448.0, 450.0
    assert list(P.scale_exponent(edge)) == [0, 1]


@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_a_row_read_back_is_within_half_a_step_and_exact_in_bf16(hkv):
    bits = ch.normal_bf16(6, hkv, count=hkv * 128).reshape(hkv, 128)
    x = R.bf16_bits_to_f64(bits)
    row = P.make_row(bits, P.E4M3)
    assert row.shape == (P.row_bytes(P.E4M3, hkv),) and not row[hkv * 128 + hkv:].any()
    y = P.row_values(row, P.E4M3)
    scale = np.exp2(P.scale_exponent(x).astype(float))[:, None]
    # e4m3's half step: 2^-4 of the value, 2^-10 of the scale below its normal range
    assert (np.abs(x - y) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale)).all()
    assert np.array_equal(R.bf16_bits_to_f64(ch.f32_to_bf16_bits(y.astype(np.float32))), y)
    assert np.array_equal(P.row_values(P.make_row(bits, P.BF16), P.BF16), x)


def test_chunk_attention_equals_dense_causal_attention():
    """One page after another and no prefix: torch's causal attention."""
    T, Hq, hkv, ps = 37, 6, 2, 16
    q, k, v = (ch.normal_bf16(8, i, count=T * h * 128).reshape(T, h, 128) for i, h in ((1, Hq), (2, hkv), (3, hkv)))
    table = np.array([[2, 0, 1]], dtype=np.int32)
    pools = [P.paged_write(x, np.zeros((3, ps, P.row_bytes(P.BF16, hkv)), np.uint8), table, [0, T], [T], P.BF16)
             for x in (k, v)]
    out, lse, mag, _ = P.paged_attention(q, *pools, table, [0, T], [T], P.BF16)
    tq, tk, tv = (torch.from_numpy(R.bf16_bits_to_f64(x)).transpose(0, 1) for x in (q, k, v))
    tk, tv = (x.repeat_interleave(Hq // hkv, 0) for x in (tk, tv))
    ref = torch.nn.functional.scaled_dot_product_attention(tq[None], tk[None], tv[None], is_causal=True)[0]
    assert np.allclose(out, ref.transpose(0, 1).numpy(), atol=1e-12)
    assert (mag >= np.abs(out) - 1e-12).all()
    # the sparse form over every position is the last token's
    sp = P.paged_sparse_attention(q[-1:], *pools, table, np.arange(T)[None], [T], P.BF16)
    assert np.allclose(sp[0][0], out[-1]) and np.allclose(sp[1][0], lse[-1])


# --------------------------------------------------------------- refusals

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x100008)
SIZES = dict(B=2, max_pages=4, num_pages=9, page_size=16, Hkv=2, D=128, kv_type=S.SA_KV_E4M3)


def _write(**kw):
    a = {**SIZES, **dict(k=FAKE, v=FAKE, ks=256, vs=256, qs=FAKE, kl=FAKE, bt=FAKE, N=3, kp=FAKE, vp=FAKE), **kw}
    return S.lib().sa_paged_kv_write(a["k"], a["v"], a["ks"], a["vs"], a["qs"], a["kl"], a["bt"], a["B"], a["N"],
                                     a["max_pages"], a["num_pages"], a["page_size"], a["Hkv"], a["D"], a["kv_type"],
                                     a["kp"], a["vp"], None)


def _gather(**kw):
    a = {**SIZES, **dict(kp=FAKE, vp=FAKE, bt=FAKE, idx=FAKE, cnt=FAKE, kr=FAKE, vr=FAKE, k=8), **kw}
    return S.lib().sa_paged_kv_gather(a["kp"], a["vp"], a["bt"], a["idx"], a["cnt"], a["B"], a["max_pages"],
                                      a["num_pages"], a["page_size"], a["Hkv"], a["D"], a["k"], a["kv_type"],
                                      a["kr"], a["vr"], None)


def _attn(**kw):
    a = {**SIZES, **dict(q=FAKE, qs=1024, kp=FAKE, vp=FAKE, bt=FAKE, st=FAKE, kl=FAKE, N=5, max_q=4, Hq=8, out=FAKE,
                         lse=None, ws=FAKE, wsn=1 << 40), **kw}
    return S.lib().sa_paged_attn(a["q"], a["qs"], a["kp"], a["vp"], a["bt"], a["st"], a["kl"], a["B"], a["N"],
                                 a["max_q"], a["max_pages"], a["num_pages"], a["page_size"], a["Hq"], a["Hkv"],
                                 a["D"], a["kv_type"], 0.0, a["out"], a["lse"], a["ws"], a["wsn"], None)


def _sparse(**kw):
    a = {**SIZES, **dict(q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, idx=FAKE, cnt=FAKE, Hq=8, k=8, out=FAKE, lse=None,
                         ws=FAKE, wsn=1 << 40), **kw}
    return S.lib().sa_paged_sparse_attn_decode(a["q"], a["kp"], a["vp"], a["bt"], a["idx"], a["cnt"], a["B"],
                                               a["max_pages"], a["num_pages"], a["page_size"], a["Hq"], a["Hkv"],
                                               a["D"], a["k"], a["kv_type"], 0.0, a["out"], a["lse"], a["ws"],
                                               a["wsn"], None)


@pytest.mark.parametrize("call", [_write, _gather, _attn, _sparse])
def test_sizes_are_refused_on_the_host(call):
    bad, uns = S.SA_ERR_INVALID_ARG, S.SA_ERR_UNSUPPORTED
    assert call(B=-1) == bad and call(max_pages=0) == bad and call(num_pages=0) == bad and call(Hkv=0) == bad
    assert call(kv_type=2) == bad and call(kv_type=-1) == bad
    assert "kv_type" in S.last_error()
    assert call(D=64) == uns
    assert call(Hkv=9, Hq=9) == uns
    for ps in (0, 8, 24, 512):
        assert call(page_size=ps) == uns
    assert "page_size" in S.last_error()
    assert call(num_pages=1 << 27) == uns and call(max_pages=1 << 27) == uns   # 2^31 rows
    assert call(kp=None) == bad and call(vp=None) == bad and call(bt=None) == bad
    assert call(kp=ODD) == bad and call(vp=ODD) == bad
    assert call(bt=ctypes.c_void_p(0x100002)) == bad
    assert call(B=0) == S.SA_OK                                                # nothing to do, no launch


def test_write_and_gather_refusals():
    bad, uns = S.SA_ERR_INVALID_ARG, S.SA_ERR_UNSUPPORTED
    assert _write(N=-1) == bad and _write(N=0) == S.SA_OK
    assert _write(ks=255) == bad and _write(ks=260) == bad and _write(vs=248) == bad
    assert "stride" in S.last_error()
    assert _write(k=None) == bad and _write(v=ODD) == bad and _write(qs=None) == bad and _write(kl=None) == bad
    assert _gather(k=0) == bad and _gather(k=(1 << 20) + 1) == uns and _gather(B=65536) == uns
    assert _gather(idx=None) == bad and _gather(cnt=None) == bad and _gather(kr=ODD) == bad and _gather(vr=None) == bad
    assert S.lib().sa_paged_row_bytes(S.SA_KV_BF16, 8) == 2064
    assert S.lib().sa_paged_row_bytes(S.SA_KV_E4M3, 8) == 1040
    for args in ((2, 8), (0, 0), (0, 9)):
        assert S.lib().sa_paged_row_bytes(*args) == 0


def test_attention_refusals():
    bad, uns = S.SA_ERR_INVALID_ARG, S.SA_ERR_UNSUPPORTED
    for call in (_attn, _sparse):
        assert call(Hq=0) == bad and call(Hq=7) == bad and call(Hq=34) == uns
        assert call(q=None) == bad and call(q=ODD) == bad and call(out=None) == bad and call(out=ODD) == bad
        assert call(lse=ctypes.c_void_p(0x100002)) == bad
        assert call(ws=None, wsn=0) == S.SA_ERR_WORKSPACE
        assert call(ws=ctypes.c_void_p(0x100010)) == S.SA_ERR_WORKSPACE
        assert call(wsn=16) == S.SA_ERR_WORKSPACE
    assert _attn(N=-1) == bad and _attn(max_q=-1) == bad and _attn(qs=1000) == bad and _attn(qs=1028) == bad
    assert _attn(N=1 << 28, Hq=32, qs=4096) == uns
    assert _attn(N=0) == S.SA_OK and _attn(max_q=0) == S.SA_OK
    assert _attn(st=None) == bad and _attn(kl=None) == bad
    assert _sparse(k=0) == bad and _sparse(k=(1 << 20) + 1) == uns
    assert _sparse(idx=None) == bad and _sparse(cnt=None) == bad


def test_workspace_sizes():
    L = S.lib()
    def ws(B=8, N=8, max_q=1, pages=512, page=64, Hq=32, Hkv=8, kv_type=S.SA_KV_E4M3, lib=L):
        return lib.sa_paged_attn_workspace(B, N, max_q, pages, page, Hq, Hkv, 128, kv_type)

    assert 0 < ws() < 64 << 20 and ws(kv_type=S.SA_KV_BF16) > 0
    # a bound far above the tokens there are asks for no more than the tokens do
    assert ws(max_q=1 << 20) == ws(max_q=8)
    for kw in (dict(B=0), dict(N=0), dict(max_q=0), dict(Hkv=9), dict(Hq=33), dict(pages=0), dict(page=0)):
        assert ws(**kw) == 0
    # long chunks of E4M3 caches: the rows in bf16, a window of at most 1 GiB at a time
    long = dict(N=4096, max_q=4096)
    small = ws(**long, kv_type=S.SA_KV_BF16)
    assert ws(**long) - small == 8 * 512 * 64 * 8 * 512        # all of 8 x 32K positions, 8 heads
    assert ws(**long, pages=1 << 14) - small <= 1 << 30        # 8 x 1M positions
    assert ws(**long, pages=1 << 14) - small > 1 << 28
    assert L.sa_paged_sparse_attn_decode_workspace(8, 32, 8, 128, 2048, 1) > 0
    assert ws(lib=S.lib_debug()) == ws() + 256


def test_the_binding_refuses_what_it_cannot_pass_on():
    """Checked before any CUDA call (the tensors are on the CPU)."""
    with pytest.raises(ValueError, match="kv heads"):
        S.sa_paged_kv_alloc(2, 16, 9)
    k, v = S.sa_paged_kv_alloc(2, 16, 3, S.SA_KV_E4M3)
    assert k.shape == (2, 16, 400) and k.dtype == torch.uint8 and not v.any()
    assert S.sa_paged_kv_alloc(2, 16, 3)[0].shape == (2, 16, 392)
    dev = -1   # the CPU's ordinal
    assert S._pools(k, v, dev) == (S.SA_KV_E4M3, 3)
    with pytest.raises(ValueError, match="one shape"):
        S._pools(k, v[:1], dev)
    with pytest.raises(ValueError, match="bfloat16"):
        S._pools(k.float(), v.float(), dev)
    with pytest.raises(ValueError, match="rows"):
        S._pools(k[..., 1:].contiguous(), v[..., 1:].contiguous(), dev)
    with pytest.raises(ValueError, match="contiguous"):
        S._pools(k[:, ::2], v[:, ::2], dev)
    with pytest.raises(ValueError, match="CUDA"):
        S._tokens(torch.zeros(2, 3, 128, dtype=torch.bfloat16), "q")
    with pytest.raises(ValueError, match="int32"):
        S._ints32(torch.zeros(2, dtype=torch.int64), "kv_len", dev, (2,))
    with pytest.raises(ValueError, match="shape"):
        S._ints32(torch.zeros(2, dtype=torch.int32), "kv_len", dev, (3,))
    with pytest.raises(ValueError, match="out"):
        S._result(torch.zeros(2), "out", dev, (2,), torch.bfloat16)


def test_two_threads_on_one_stream_take_the_shared_workspace_in_turn(monkeypatch):
    """A call's kernels hand results to one another through the stream's
    workspace: no other thread's call is enqueued between them, and the buffer
    is not replaced under one."""
    import threading
    import time

    S._names()
    seen = {"inside": 0, "most": 0, "calls": 0, "replaced": 0}
    alive = {}

    class Torch:
        @staticmethod
        def zeros(n, dtype, device):
            t = torch.zeros(n, dtype=dtype)
            seen["replaced"] += seen["inside"]
            alive[t.data_ptr()] = n
            return t

    class Cuda:
        @staticmethod
        def _cuda_isCurrentStreamCapturing():
            return False

    class Lib:
        _handle = 0

        @staticmethod
        def sa_paged_attn_workspace(B, N, max_q, *_):
            return 256 * max_q

        @staticmethod
        def sa_paged_attn(*args):
            ws, nbytes = args[-3], args[-2]
            assert alive[ws] >= nbytes
            seen["inside"] += 1
            seen["most"] = max(seen["most"], seen["inside"])
            time.sleep(2e-3)          # (between the launches of two kernels)
            seen["inside"] -= 1
            seen["calls"] += 1
            return S.SA_OK

    monkeypatch.setattr(S, "_torch", lambda: Torch)
    monkeypatch.setattr(S, "_cuda", Cuda)
    monkeypatch.setattr(S, "_lib", Lib)
    monkeypatch.setattr(S, "_paged_ws", {})
    monkeypatch.setattr(S, "_paged_ws_need", {})
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    ints = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(4, 16, 264, dtype=torch.bfloat16)
    errors = []

    def work(t):
        try:
            out = torch.empty_like(q)
            for i in range(12):
                S._attn(q, pool, pool, ints, ints, ints, 1 + i + t, 0.0, out, False, None, -1, q.shape, 1024, S.SA_KV_BF16,
                        2, 4, 16, 2, 2, 77)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert seen["calls"] == 48 and seen["most"] == 1 and seen["replaced"] == 0


def test_a_workspace_with_less_memory_than_elements_is_refused(monkeypatch):
    """An expanded tensor's size says nothing of its memory; kernels would write
    beyond it."""
    S._names()
    calls = []

    class Lib:
        _handle = 1
        sa_paged_attn_workspace = staticmethod(lambda *a: 4096)
        sa_paged_attn = staticmethod(lambda *a: calls.append(a[-3:-1]) or S.SA_OK)

    monkeypatch.setattr(S, "_lib", Lib)
    monkeypatch.setattr(S, "_paged_ws_need", {})
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    ints = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(4, 16, 264, dtype=torch.bfloat16)

    def call(ws):
        S._attn(q, pool, pool, ints, ints, ints, 1, 0.0, torch.empty_like(q), False, ws, -1, q.shape, 1024, S.SA_KV_BF16, 2,
                4, 16, 2, 2, 77)

    good = torch.zeros(4096, dtype=torch.uint8)
    call(good)
    assert calls == [(good.data_ptr(), 4096)]
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            call(ws)
    assert len(calls) == 1

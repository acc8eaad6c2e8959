"""The float64 statements of oracle/latent.py against independent ones: torch's autograd in float64, central
differences, closed forms, and the binding's refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_25_b200 as kda
from oracle import latent as O

CASES = [([3, 0, 5], [3, 2, 9], True), ([4, 1], [2, 0], True), ([3, 2], [1, 4], False)]


def _inputs(lens_q, lens_k, H=2, R=3, seed=0):
    g = np.random.default_rng(seed)
    T, Tk = sum(lens_q), sum(lens_k)
    cu = lambda ls: np.cumsum([0] + ls)  # noqa: E731
    return (g.standard_normal((T, H, 128 + R)), g.standard_normal((Tk, H, 128)), g.standard_normal((Tk, H, 128)),
            g.standard_normal((Tk, R)), g.standard_normal((T, H, 128)), cu(lens_q), cu(lens_k))


def _autograd(q, k, v, r, dout, cu_q, cu_k, scale, causal):
    q, k, v, r = (torch.tensor(x, requires_grad=True) for x in (q, k, v, r))
    outs = []
    for q0, q1, k0, k1 in O.spans(cu_q, cu_k):
        i, j = torch.arange(q1 - q0)[:, None], torch.arange(k1 - k0)[None]
        seen = (j <= i + (k1 - k0) - (q1 - q0)) if causal else torch.ones(q1 - q0, k1 - k0, dtype=torch.bool)
        key = torch.cat([k[k0:k1], r[k0:k1, None].expand(-1, k.shape[1], -1)], -1)
        x = torch.einsum("ihd,jhd->hij", q[q0:q1], key) * scale
        e = torch.where(seen, torch.exp(x), 0.0)
        s = e.sum(-1, keepdim=True)
        outs.append(torch.einsum("hij,jhd->ihd", e / torch.where(s == 0, 1.0, s), v[k0:k1]))
    out = torch.cat(outs)
    (out * torch.tensor(dout)).sum().backward()
    return out.detach().numpy(), [x.grad.numpy() for x in (q, k, v, r)]


@pytest.mark.parametrize("lens_q,lens_k,causal", CASES)
def test_attention_against_autograd(lens_q, lens_k, causal):
    q, k, v, r, dout, cu_q, cu_k = _inputs(lens_q, lens_k)
    out, lse, _, _ = O.forward(q, k, v, r, cu_q, cu_k, 0.1, causal)
    g = O.backward(q, k, v, r, dout, cu_q, cu_k, 0.1, causal)
    ref, grads = _autograd(q, k, v, r, dout, cu_q, cu_k, 0.1, causal)
    np.testing.assert_allclose(out, ref, atol=1e-12)
    for name, want in zip(("dq", "dk", "dv", "dr"), grads):
        np.testing.assert_allclose(g[name], want, atol=1e-12, err_msg=name)
    assert np.all((lse == -np.inf) == (np.abs(out).sum(-1) == 0))


def test_attention_gradients_against_differences():
    q, k, v, r, dout, cu_q, cu_k = _inputs([3, 2], [4, 2], seed=3)
    loss = lambda q, k, v, r: float((O.forward(q, k, v, r, cu_q, cu_k, 0.1, True)[0] * dout).sum())  # noqa: E731
    g = O.backward(q, k, v, r, dout, cu_q, cu_k, 0.1, True)
    rng = np.random.default_rng(1)
    for i, name in enumerate(("dq", "dk", "dv", "dr")):
        args = [q, k, v, r]
        d = rng.standard_normal(args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
        slope = (loss(*up) - loss(*down)) / 2e-5
        assert abs(slope - float((g[name] * d).sum())) < 1e-6 * max(1.0, abs(slope)), name


def test_absorbed_form_is_the_expanded_one():
    """With W_k, W_v the expansions, q (W_k c) = (W_k^T q) c and sum p (W_v c) = W_v (sum p c)."""
    g = np.random.default_rng(2)
    L, H, R = 7, 2, 4
    c, r = g.standard_normal((L, 512)), g.standard_normal((L, R))
    wk, wv = g.standard_normal((H, 128, 512)) / 22, g.standard_normal((H, 128, 512)) / 22
    q = g.standard_normal((1, H, 128 + R))
    k, v = np.einsum("hdc,jc->jhd", wk, c), np.einsum("hdc,jc->jhd", wv, c)
    out, lse, _, _ = O.forward(q, k, v, r, np.array([0, 1]), np.array([0, L]), 0.1, True)
    qa = np.concatenate([np.einsum("hdc,thd->thc", wk, q[..., :128]), q[..., 128:]], -1)
    cache = np.concatenate([c, r], -1).reshape(1, L, -1)
    o2, lse2, _, _ = O.decode(qa[None], cache, np.zeros((1, 1), int), [L], 0.1)
    np.testing.assert_allclose(np.einsum("hdc,thc->thd", wv, o2[0]), out, atol=1e-12)
    np.testing.assert_allclose(lse2[0], lse, atol=1e-12)


def test_norm_against_autograd_and_closed_forms():
    g = np.random.default_rng(4)
    h, w, dy = g.standard_normal((5, 16)), g.standard_normal(16), g.standard_normal((5, 16))
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = th / (th.square().mean(-1, keepdim=True) + 1e-5).sqrt() * tw
    (y * torch.tensor(dy)).sum().backward()
    np.testing.assert_allclose(O.rms_norm(h, w, 1e-5), y.detach().numpy(), atol=1e-14)
    dx, dw, _ = O.rms_norm_backward(dy, h, w, 1e-5)
    np.testing.assert_allclose(dx, th.grad.numpy(), atol=1e-13)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-13)
    assert np.allclose(O.rms_norm(np.full((1, 8), 3.0), np.ones(8), 0.0), 1.0)


def test_round_e4m3_against_torch():
    x = np.concatenate([np.linspace(-500, 500, 20001), np.exp2(np.linspace(-12, 9, 5001))])
    want = torch.tensor(np.clip(x, -448, 448), dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    got = O.round_e4m3(x.astype(np.float32).astype(np.float64))
    assert np.array_equal(got, want)


# ---- refusals: every call below returns before its first CUDA call

A = 0x10000     # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_25_b200 import build
    build.build()
    return kda.load()


def _fwd(lib, **kw):
    a = dict(q=A, k=A, v=A, r=A, cu=None, cuk=None, out=A, lse=A, B=1, T=8, Tk=8, H=2, N=1, dk=128, dv=128, dr=64, kt=256,
             kh=128, vt=256, vh=128, rt=64, causal=1, scale=0.1, dtype=1, ws=A, wsb=256)
    a.update(kw)
    return lib.kda_latent_fwd(*a.values(), None)


def _bwd(lib, **kw):
    a = dict(q=A, k=A, v=A, r=A, cu=None, cuk=None, out=A, lse=A, dout=A, dq=A, dko=A, dvo=A, dr_out=A, B=1, T=8, Tk=8, H=2,
             N=1, dk=128, dv=128, dr=64, kt=256, kh=128, vt=256, vh=128, rt=64, causal=1, scale=0.1, dtype=1, ws=A,
             wsb=1 << 20)
    a.update(kw)
    return lib.kda_latent_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_latent_host_checks(lib, call):
    bad, unsup = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(r=None), dict(out=None), dict(lse=None), dict(q=A + 2),
               dict(k=A + 8), dict(out=A + 4), dict(lse=A + 2), dict(N=2), dict(cu=A), dict(cu=A, cuk=A, B=2),
               dict(cu=A + 1, cuk=A), dict(H=0), dict(T=-1), dict(Tk=-1), dict(kt=250), dict(vh=4), dict(rt=0), dict(kt=-256),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=9), dict(ws=None),
               dict(wsb=16), dict(ws=A + 8)):
        assert call(lib, **kw) == bad, kw
    for kw in (dict(dtype=0), dict(dk=64), dict(dv=64), dict(H=65536, kt=65536 * 128, wsb=1 << 40),
               dict(cu=A, cuk=A, N=65536)):
        assert call(lib, **kw) == unsup, kw
    assert call(lib, dr=32) in (bad, unsup)
    if call is _bwd:
        for kw in (dict(dout=None), dict(dq=None), dict(dko=None), dict(dvo=None), dict(dr_out=None), dict(dq=A + 8),
                   dict(wsb=256)):
            assert call(lib, **kw) == bad, kw


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_latent_tokens_of_no_sequence_are_refused(lib, call):
    for kw in (dict(T=8, Tk=8), dict(T=8, Tk=0), dict(T=0, Tk=8)):
        assert call(lib, cu=A, cuk=A, N=0, **kw) == kda.KDA_ERR_INVALID_ARG, kw


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_latent_more_blocks_than_a_launch_takes_are_unsupported(lib, call):
    for kw in (dict(T=1 << 30, H=1024), dict(T=1 << 24, H=65535), dict(T=64, Tk=64, H=65535, N=65535, cu=A, cuk=A)):
        assert call(lib, wsb=1 << 50, **kw) == kda.KDA_ERR_UNSUPPORTED, kw


def _dec(lib, **kw):
    a = dict(q=A, cache=A, table=A, lens=A, out=A, lse=A, N=2, Tq=1, H=4, dc=512, dr=64, page=64, pages=8, maxp=4, scale=0.1,
             dtype=1, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.kda_latent_decode_step(*a.values(), None)


def test_decode_host_checks(lib):
    bad, unsup = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(cache=None), dict(table=None), dict(lens=None), dict(out=None), dict(lse=None), dict(q=A + 8),
               dict(cache=A + 2), dict(table=A + 2), dict(N=-1), dict(Tq=0), dict(H=0), dict(page=0), dict(pages=-1),
               dict(scale=-1.0), dict(scale=float("nan")), dict(dtype=5), dict(ws=None), dict(wsb=8)):
        assert _dec(lib, **kw) == bad, kw
    for kw in (dict(dtype=0), dict(dc=256), dict(dr=32), dict(page=24), dict(pages=1 << 28), dict(maxp=1 << 28)):
        assert _dec(lib, **kw) == unsup, kw
    assert lib.kda_latent_decode_workspace_size(-1, 1, 4) == 0


def _app(lib, **kw):
    a = dict(c=A, r=A, slots=A, w=A, cache=A, cs=576, rs=576, rows=64, T=4, dc=512, dr=64, eps=1e-5, dtype=1)
    a.update(kw)
    return lib.kda_latent_append(*a.values(), None)


def test_append_host_checks(lib):
    bad, unsup = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
    for kw in (dict(c=None), dict(r=None), dict(slots=None), dict(cache=None), dict(c=A + 2), dict(slots=A + 4), dict(cs=571),
               dict(rs=-8), dict(T=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=4)):
        assert _app(lib, **kw) == bad, kw
    for kw in (dict(dtype=0), dict(dc=256), dict(dr=32)):
        assert _app(lib, **kw) == unsup, kw
    assert _app(lib, T=0) == kda.KDA_OK


def test_norm_host_checks(lib):
    P, bad, unsup = ctypes.c_void_p, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED

    def norm(x=A, res=A, w=A, y=A, h=A, rows=4, D=256, eps=1e-5, dtype=1):
        return lib.kda_rms_norm(P(x), P(res), P(w), P(y), P(h), rows, D, eps, dtype, None)

    def norm8(scale=A, D=256):
        return lib.kda_rms_norm_e4m3(P(A), None, P(A), P(A), P(scale), None, 4, D, 1e-5, 1, None)

    def bwd(dy=A, h=A, w=A, dx=A, dw=A, rows=4, D=256, ws=A, wsb=1 << 20):
        return lib.kda_rms_norm_bwd(P(dy), P(h), P(w), None, P(dx), P(dw), rows, D, 1e-5, 1, P(ws), wsb, None)

    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(h=None), dict(x=A + 2), dict(rows=-1), dict(D=0), dict(eps=-1.0),
               dict(dtype=2)):
        assert norm(**kw) == bad, kw
    for kw in (dict(D=100), dict(D=16392)):
        assert norm(**kw) == unsup, kw
    assert norm(rows=0) == kda.KDA_OK and norm8(scale=None) == bad and norm8(D=136) == unsup
    for kw in (dict(dy=None), dict(h=None), dict(w=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(wsb=64)):
        assert bwd(**kw) == bad, kw
    assert kda.rms_norm_bwd_workspace_size(4, 100) == 0 and kda.rms_norm_bwd_workspace_size(4, 256) == 4 * 256 * 4


def test_norm_e4m3_refuses_an_output_over_its_inputs(lib):
    """The 8-bit rows lie elsewhere than the rows they come from, so writing them in place would race."""
    P, size = ctypes.c_void_p, 4 * 256 * 2
    far = A + 64 * size
    for x, res, h, y in ((A, None, None, A), (A, None, None, A + size - 16), (A + 512, None, None, A), (far, A, far + size, A + 256),
                         (far, far + size, A, A)):
        assert lib.kda_rms_norm_e4m3(P(x), P(res), P(A), P(y), P(far + 8 * size), P(h), 4, 256, 1e-5, 1, None) == kda.KDA_ERR_INVALID_ARG


def test_strides_of_batch_rows():
    """Token and head strides of views, rows of one token among them (whose token stride is the batch's)."""
    from kimi_delta_attention_25_b200 import latent
    t = torch.zeros(3, 5, 2, 256)
    rows = lambda x: latent._rows("k", x, *x.shape)  # noqa: E731
    assert rows(t) == (512, 256) and rows(t[..., :128]) == (512, 256)
    assert rows(t[:, :1]) == (2560, 256) and rows(t[:, 2:3, :, 128:]) == (2560, 256) and rows(t[:1, :1])[1] == 256
    assert rows(t[:, :0])[0] > 0
    for bad in (t[:, :2], t[:, 1:4], t.transpose(0, 1), t[..., ::2]):
        with pytest.raises(ValueError):
            rows(bad)


def test_binding_refuses_cpu_tensors_types_and_shapes():
    b = torch.bfloat16
    q, k = torch.zeros(1, 4, 2, 192, dtype=b), torch.zeros(1, 4, 2, 128, dtype=b)
    r = torch.zeros(1, 4, 64, dtype=b)
    with pytest.raises(ValueError):
        kda.latent_fwd(q, k, k, r)
    with pytest.raises(TypeError):
        kda.latent_fwd(q.float(), k, k, r)
    with pytest.raises(ValueError):
        kda.latent_fwd(q[0], k, k, r)
    with pytest.raises(ValueError):
        kda.latent_decode_step(torch.zeros(2, 1, 4, 576, dtype=b), torch.zeros(3, 16, 576, dtype=b),
                               torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.latent_append(torch.zeros(2, 512, dtype=b), None, torch.zeros(1, 16, 512, dtype=b), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        kda.rms_norm(torch.zeros(2, 64), torch.zeros(64))
    with pytest.raises(TypeError):
        kda.rms_norm(torch.zeros(2, 64, dtype=torch.float16), torch.zeros(64))
    with pytest.raises(ValueError):
        kda.rms_norm_bwd(torch.zeros(2, 64), torch.zeros(2, 64), torch.zeros(64))

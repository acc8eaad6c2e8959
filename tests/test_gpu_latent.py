"""GPU parity of the latent attention (expanded form and its backward pass, absorbed form over a paged
cache, cache append) and of the norm in front of a layer, against the float64 statements of oracle/latent.py.

Bounds, element by element. A value stored in bf16 is off by at most 2^-8 of itself. P (and dS) enter the
second product rounded to bf16, which moves each term by at most 2^-8 of itself: 2^-8 (P|V|) in an output.
fp32 sums of n products are off by at most n 2^-24 of the sum of their absolute values; a score's error is
relative in P (twice: once in the term, once in the sum), exp2's and the sums' own errors are below 2^-18.
"""
import numpy as np
import pytest
import torch

import kimi_delta_attention_25_b200 as kda
from oracle import latent as O
from tests.kda_check import np32

pytestmark = pytest.mark.gpu
DEV = "cuda"
B16 = torch.bfloat16
HALF = 2.0 ** -8                   # half a bf16 step, relative


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_25_b200 import build
    build.build()
    kda.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def f64(t):
    return np32(t).astype(np.float64)


def within(x, ref, bound, what):
    """|x - ref| <= bound + half a bf16 step of the result, element by element; non-finite values equal."""
    x = np.asarray(x, dtype=np.float64)
    assert x.shape == ref.shape, what
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(x)), "%s: non-finite values" % what
    assert np.array_equal(x[~fine], ref[~fine]), what
    slack = np.abs(x - ref, where=fine, out=np.zeros_like(ref)) - (bound * (1 + HALF) + HALF * np.abs(np.where(fine, ref, 0)) + 1e-30)
    assert slack.max(initial=-1.0) <= 0, "%s: exceeds its bound by %.3e at %s (bound there %.3e)" % (
        what, slack.max(), np.unravel_index(slack.argmax(), slack.shape), np.broadcast_to(bound, slack.shape).ravel()[slack.argmax()])


def score_error(big, width):
    return 2 * (width + 8) * 2.0 ** -24 * big + 2.0 ** -18


def cu_of(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=DEV)


def expanded(lens_q, lens_k, H, R, seed=0, std=1.5):
    """Packed inputs on the GPU; k and v are views of one tensor, k_shared a view of a wider one."""
    g = torch.Generator().manual_seed(seed)
    T, Tk = sum(lens_q), sum(lens_k)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, kv = (n(1, T, H, 128 + R) * std).to(B16).to(DEV), n(1, Tk, H, 256).to(B16).to(DEV)
    wide = n(1, Tk, 512 + 64).to(B16).to(DEV)
    return q, kv[..., :128], kv[..., 128:], (wide[..., 512:] if R else None), n(1, T, H, 128).to(B16).to(DEV)


def check_forward(q, k, v, r, lens_q, lens_k, causal, out, lse, scale=None):
    W = q.shape[-1]
    scale = W ** -0.5 if scale is None else scale
    cu_q, cu_k = np.cumsum([0] + list(lens_q)), np.cumsum([0] + list(lens_k))
    ro, rl, wide, big = O.forward(f64(q)[0], f64(k)[0], f64(v)[0], None if r is None else f64(r)[0], cu_q, cu_k,
                                  float(np.float32(scale)), causal)
    d = score_error(big, W)
    within(f64(out)[0], ro, (HALF + d + max(lens_k) * 2.0 ** -24)[..., None] * wide, "out")
    fine = np.isfinite(rl)
    x = f64(lse)[0]
    assert np.array_equal(fine, np.isfinite(x)) and np.all(x[~fine] == -np.inf)
    assert np.all(np.abs(x[fine] - rl[fine]) <= (d + max(lens_k) * 2.0 ** -24 + 2.0 ** -22 * np.abs(rl) + 2.0 ** -18)[fine]), "lse"
    return ro


def check_backward(q, k, v, r, dout, lens_q, lens_k, causal, g, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    cu_q, cu_k = np.cumsum([0] + list(lens_q)), np.cumsum([0] + list(lens_k))
    ref = O.backward(f64(q)[0], f64(k)[0], f64(v)[0], None if r is None else f64(r)[0], f64(dout)[0], cu_q, cu_k,
                     float(np.float32(scale)), causal, rounding=HALF * 1.01 + 2.0 ** -18)
    for key, name in (("dq", "dq"), ("dk", "dk"), ("dv", "dv"), ("dk_shared", "dr")):
        if g[key] is not None:
            within(f64(g[key])[0], ref[name], ref[name + "_bound"], key)


LENGTHS = [
    ([1], [1]), ([1], [130]), ([5], [5]), ([64], [64]), ([127], [127]), ([128], [128]), ([129], [129]), ([255], [300]),
    ([257], [257]), ([300], [200]),                       # more queries than keys: the first hundred see nothing
    ([0, 3, 1, 0, 70, 129], [0, 3, 64, 5, 70, 200]),       # empty sequences, and keys that no query sees
    ([40, 60], [0, 60]),                                   # a sequence without keys
    ([513, 2, 250], [513, 700, 251]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("R", [64, 0])
@pytest.mark.parametrize("lens_q,lens_k", LENGTHS)
def test_expanded_forward_and_backward(lens_q, lens_k, R, causal):
    q, k, v, r, dout = expanded(lens_q, lens_k, 2, R, seed=len(lens_q) + sum(lens_k))
    cu = (cu_of(lens_q), cu_of(lens_k))
    out, lse, ws = kda.latent_fwd(q, k, v, r, *cu, causal=causal, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    ro = check_forward(q, k, v, r, lens_q, lens_k, causal, out, lse)
    out = torch.tensor(ro, dtype=torch.float32, device=DEV).to(B16)[None]       # the bound's D: out rounded once
    g, ws = kda.latent_bwd(q, k, v, r, out, lse, dout, *cu, causal=causal, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    check_backward(q, k, v, r, dout, lens_q, lens_k, causal, g)


@pytest.mark.parametrize("H,T,Tk", [(1, 100, 100), (5, 33, 290), (3, 200, 200)])
def test_expanded_batch_rows_without_offsets(H, T, Tk):
    B = 3
    q, k, v, r, dout = expanded([T] * B, [Tk] * B, H, 64, seed=H)
    shape = lambda x, n: x.reshape(B, n, *x.shape[2:]) if x.is_contiguous() else x.unflatten(1, (B, n))[0]  # noqa: E731
    qb, kb, vb, rb, db = shape(q, T), shape(k, Tk), shape(v, Tk), shape(r, Tk), shape(dout, T)
    out, lse = kda.latent_fwd(qb, kb, vb, rb)
    check_forward(q, k, v, r, [T] * B, [Tk] * B, True, out.reshape(1, B * T, H, 128), lse.reshape(1, B * T, H))
    packed = kda.latent_fwd(q, k, v, r, cu_of([T] * B), cu_of([Tk] * B))
    assert torch.equal(packed[0].reshape(out.shape), out) and torch.equal(packed[1].reshape(lse.shape), lse)
    g = kda.latent_bwd(qb, kb, vb, rb, out, lse, db)
    p = kda.latent_bwd(q, k, v, r, packed[0], packed[1], dout, cu_of([T] * B), cu_of([Tk] * B))
    for key in g:
        assert torch.equal(g[key].reshape(p[key].shape), p[key]), key


def test_expanded_batch_rows_of_one_key_or_none():
    """Views whose batch rows hold one key each (``t[:, :1]``), and batch rows without keys."""
    B, H = 3, 2
    q, kv, wide, dout = (torch.randn(*s, device=DEV).to(B16) for s in ((B, 4, H, 192), (B, 5, H, 256), (B, 5, 576), (B, 4, H, 128)))
    k, v, r = kv[:, :1, :, :128], kv[:, :1, :, 128:], wide[:, :1, 512:]
    for causal in (True, False):
        out, lse = kda.latent_fwd(q, k, v, r, causal=causal)
        want = kda.latent_fwd(q, k.contiguous(), v.contiguous(), r.contiguous(), causal=causal)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        g, w = (kda.latent_bwd(q, *a, out, lse, dout, causal=causal) for a in ((k, v, r), (k.contiguous(), v.contiguous(), r.contiguous())))
        assert all(torch.equal(g[x], w[x]) for x in g)
    out, lse = kda.latent_fwd(q, kv[:, :0, :, :128], kv[:, :0, :, 128:], wide[:, :0, 512:])
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


def test_expanded_head_major_and_dense_layouts_agree():
    lens = [130, 77]
    q, k, v, r, dout = expanded(lens, lens, 4, 64, seed=9)
    cu = cu_of(lens)
    want = kda.latent_fwd(q, k, v, r, cu)
    kc, vc, rc = k.contiguous(), v.contiguous(), r.contiguous()
    kh = kc.transpose(1, 2).contiguous().transpose(1, 2)              # [H, T, 128] in memory
    vh = vc.transpose(1, 2).contiguous().transpose(1, 2)
    for a in ((kc, vc, rc), (kh, vh, rc), (kh, vc, r)):
        got = kda.latent_fwd(q, *a, cu)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        g, w = kda.latent_bwd(q, *a, *want, dout, cu), kda.latent_bwd(q, k, v, r, *want, dout, cu)
        assert all(torch.equal(g[x], w[x]) for x in g)


@pytest.mark.parametrize("scale,std", [(1.0, 0.2), (2.0, 3.0), (1e-3, 1.0)])
def test_expanded_scales(scale, std):
    """Up to scores of several hundred, where one key takes all of the softmax."""
    lens = [150]
    q, k, v, r, dout = expanded(lens, lens, 2, 64, seed=3, std=std)
    out, lse = kda.latent_fwd(q, k, v, r, scale=scale)
    ro = check_forward(q, k, v, r, lens, lens, True, out, lse, scale)
    g = kda.latent_bwd(q, k, v, r, torch.tensor(ro, dtype=torch.float32, device=DEV).to(B16)[None], lse, dout, scale=scale)
    check_backward(q, k, v, r, dout, lens, lens, True, g, scale)


def test_expanded_neighbours_do_not_leak():
    """Infinities and NaN in one sequence, and behind the tensors' used part, stay there."""
    lens_q, lens_k = [60, 70, 50], [90, 70, 131]
    q, k, v, r, dout = expanded(lens_q, lens_k, 2, 64, seed=5)
    cu = (cu_of(lens_q), cu_of(lens_k))
    clean = kda.latent_fwd(q, k, v, r, *cu)
    gc = kda.latent_bwd(q, k, v, r, *clean, dout, *cu)
    bad = float("nan"), float("inf")
    q2, d2 = q.clone(), dout.clone()
    kv2 = torch.cat([k, v], -1)
    r2 = r.clone()
    q2[:, 60:130], d2[:, 60:130] = bad[0], bad[1]
    kv2[:, 90:160], r2[:, 90:160] = bad[1], bad[0]
    out, lse = kda.latent_fwd(q2, kv2[..., :128], kv2[..., 128:], r2, *cu)
    for a, b in ((slice(0, 60), slice(0, 90)), (slice(130, 180), slice(160, 291))):
        assert torch.equal(out[:, a], clean[0][:, a]) and torch.equal(lse[:, a], clean[1][:, a])
    g = kda.latent_bwd(q2, kv2[..., :128], kv2[..., 128:], r2, out, lse, d2, *cu)
    for a, b in ((slice(0, 60), slice(0, 90)), (slice(130, 180), slice(160, 291))):
        assert torch.equal(g["dq"][:, a], gc["dq"][:, a])
        for key in ("dk", "dv", "dk_shared"):
            assert torch.equal(g[key][:, b], gc[key][:, b]), key


def test_expanded_bad_offsets_are_reported_and_skipped():
    lens = [100, 28]
    q, k, v, r, dout = expanded(lens, lens, 2, 64, seed=6)
    for offs in ([0, 100, 50, 128], [0, 60, 400], [0, -5, 128], [3, 100, 128], [0, 100, 120]):
        cu = torch.tensor(offs, dtype=torch.int32, device=DEV)
        out, lse, ws = kda.latent_fwd(q, k, v, r, cu, return_workspace=True)
        assert kda.workspace_status(ws) == kda.KDA_ERR_INVALID_ARG, offs
        out, lse = torch.zeros_like(out), torch.zeros_like(lse)
        _, ws = kda.latent_bwd(q, k, v, r, out, lse, dout, cu, return_workspace=True)
        assert kda.workspace_status(ws) == kda.KDA_ERR_INVALID_ARG, offs
    out, lse, ws = kda.latent_fwd(q, k, v, r, cu_of(lens), return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    check_forward(q, k, v, r, lens, lens, True, out, lse)


def test_expanded_offsets_are_checked_where_there_is_no_query():
    for keys, offs_q, offs_k, status in (
            (5, [0, 0], [0, 5], kda.KDA_OK), (5, [0, 0], [0, 3], kda.KDA_ERR_INVALID_ARG), (5, [0, 0, 0], [0, 6, 5], kda.KDA_ERR_INVALID_ARG),
            (5, [0, 1], [0, 5], kda.KDA_ERR_INVALID_ARG), (0, [0, 0], [0, 0], kda.KDA_OK), (0, [0, 0], [0, 1], kda.KDA_ERR_INVALID_ARG),
            (0, [2, 0], [0, 0], kda.KDA_ERR_INVALID_ARG)):
        q, k, v, r, dout = expanded([0], [keys], 2, 64)
        cu = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (offs_q, offs_k)]
        ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
        out, lse = kda.latent_fwd(q, k, v, r, *cu, workspace=ws)
        assert kda.workspace_status(ws) == status, (offs_q, offs_k)
        ws = torch.full((kda.latent_bwd_workspace_size(1, 0, keys, 2, len(offs_q) - 1),), 255, dtype=torch.uint8, device=DEV)
        kda.latent_bwd(q, k, v, r, out, lse, dout, *cu, workspace=ws)
        assert kda.workspace_status(ws) == status, (offs_q, offs_k)


def test_expanded_empty_sizes():
    q, k, v, r, dout = expanded([4], [0], 2, 64)
    out, lse = kda.latent_fwd(q, k, v, r, cu_of([4]), cu_of([0]))
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))
    g = kda.latent_bwd(q, k, v, r, out, lse, dout, cu_of([4]), cu_of([0]))
    assert torch.all(g["dq"] == 0) and g["dk"].numel() == 0
    q, k, v, r, dout = expanded([0], [5], 2, 64)
    out, lse = kda.latent_fwd(q, k, v, r, cu_of([0]), cu_of([5]))
    g = kda.latent_bwd(q, k, v, r, out, lse, dout, cu_of([0]), cu_of([5]))
    assert all(torch.all(g[x] == 0) for x in ("dk", "dv", "dk_shared"))


@pytest.mark.parametrize("R", [64, 0])
def test_expanded_backward_over_many_query_tiles(R):
    """Blocks of dk and dv that walk twelve tiles of queries, whose statistics go through two buffers in turn."""
    lens_q, lens_k = [1500], [70]
    q, k, v, r, dout = expanded(lens_q, lens_k, 2, R, seed=31)
    cu = (cu_of(lens_q), cu_of(lens_k))
    for causal in (True, False):
        out, lse = kda.latent_fwd(q, k, v, r, *cu, causal=causal)
        ro = check_forward(q, k, v, r, lens_q, lens_k, causal, out, lse)
        out = torch.tensor(ro, dtype=torch.float32, device=DEV).to(B16)[None]
        g, ws = kda.latent_bwd(q, k, v, r, out, lse, dout, *cu, causal=causal, return_workspace=True)
        assert kda.workspace_status(ws) == kda.KDA_OK
        check_backward(q, k, v, r, dout, lens_q, lens_k, causal, g)


@pytest.mark.parametrize("N", [40, 60, 70, 380, 390, 1100])
def test_expanded_many_sequences(N):
    """More sequences than a warp's first look at the offsets, and so many blocks that they are no longer
    ranked; empty sequences and ones without queries or without keys among them."""
    rng = np.random.default_rng(N)
    lens_q = np.minimum(rng.integers(0, 3, N) * rng.integers(0, 6, N), 9)
    lens_k = np.where(rng.random(N) < 0.1, 0, lens_q + rng.integers(0, 4, N))
    if N == 40:
        lens_q, lens_k = lens_q * 30, lens_k * 31
    elif N == 380:
        lens_q = np.minimum(lens_q, 3)
    lens_q, lens_k = lens_q.tolist(), lens_k.tolist()
    q, k, v, r, dout = expanded(lens_q, lens_k, 2, 64, seed=N)
    cu = (cu_of(lens_q), cu_of(lens_k))
    out, lse, ws = kda.latent_fwd(q, k, v, r, *cu, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    ro = check_forward(q, k, v, r, lens_q, lens_k, True, out, lse)
    out = torch.tensor(ro, dtype=torch.float32, device=DEV).to(B16)[None]
    g, ws = kda.latent_bwd(q, k, v, r, out, lse, dout, *cu, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    check_backward(q, k, v, r, dout, lens_q, lens_k, True, g)


@pytest.mark.parametrize("R", [64, 0])
@pytest.mark.parametrize("lens_q,lens_k", [([70], [900]), ([300, 130], [700, 800])])
def test_expanded_growing_scores(lens_q, lens_k, R):
    """Scores that rise by some 13 (19 in the log2 domain) over each tile of 128 keys, so that every row's maximum moves
    in every tile by more than the 2^15 that the forward pass lets pass."""
    H, W = 2, 128 + R
    q, k, v, r, dout = expanded(lens_q, lens_k, H, R, seed=17)
    g = torch.Generator().manual_seed(18)
    sign = torch.randn(128, generator=g).sign()
    ramp = torch.cat([torch.arange(n) / 128.0 for n in lens_k])[None, :, None, None]
    k = (ramp * sign + 0.05 * torch.randn(1, sum(lens_k), H, 128, generator=g)).to(B16).to(DEV)
    q = torch.cat([(sign + 0.05 * torch.randn(1, sum(lens_q), H, 128, generator=g)), 0.2 * torch.randn(1, sum(lens_q), H, R, generator=g)], -1).to(B16).to(DEV)
    cu = (cu_of(lens_q), cu_of(lens_k))
    for causal in (True, False):
        out, lse = kda.latent_fwd(q, k, v, r, *cu, causal=causal, scale=0.1)
        ro = check_forward(q, k, v, r, lens_q, lens_k, causal, out, lse, 0.1)
        grads = kda.latent_bwd(q, k, v, r, torch.tensor(ro, dtype=torch.float32, device=DEV).to(B16)[None], lse, dout, *cu, causal=causal, scale=0.1)
        check_backward(q, k, v, r, dout, lens_q, lens_k, causal, grads, 0.1)


@pytest.mark.parametrize("lens_q,lens_k", [([130], [6000]), ([64], [131072]), ([2100], [2100])])
def test_expanded_long(lens_q, lens_k):
    """A few queries behind a long history, and a prompt of several blocks."""
    q, k, v, r, dout = expanded(lens_q, lens_k, 1, 64, seed=lens_k[0])
    cu = (cu_of(lens_q), cu_of(lens_k))
    out, lse, ws = kda.latent_fwd(q, k, v, r, *cu, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    ro = check_forward(q, k, v, r, lens_q, lens_k, True, out, lse)
    out = torch.tensor(ro, dtype=torch.float32, device=DEV).to(B16)[None]
    g, ws = kda.latent_bwd(q, k, v, r, out, lse, dout, *cu, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    check_backward(q, k, v, r, dout, lens_q, lens_k, True, g)


def test_expanded_gradients_of_short_rows():
    """Rows that see one key have no gradient through the softmax (exactly), and those that see a few keep their
    accuracy although ``out`` was rounded: over all rows two roundings to bf16, each at most 2^-8 of a value and of
    2^-8 / sqrt(3) in the mean square, stay below 2^-8 of the gradients' 2-norm."""
    for lens_q, lens_k in (([1] * 16, [1] * 16), ([1, 2, 1, 3, 2, 4, 5, 2, 9, 17, 3, 2], [1, 2, 1, 3, 2, 4, 5, 2, 9, 17, 3, 2]),
                           ([3, 40, 5], [1, 2, 4]), ([2, 200], [3, 201])):
        for causal in (True, False):
            q, k, v, r, dout = expanded(lens_q, lens_k, 3, 64, seed=21)
            cu = (cu_of(lens_q), cu_of(lens_k))
            out, lse = kda.latent_fwd(q, k, v, r, *cu, causal=causal)
            g = kda.latent_bwd(q, k, v, r, out, lse, dout, *cu, causal=causal)
            ref = O.backward(f64(q)[0], f64(k)[0], f64(v)[0], f64(r)[0], f64(dout)[0], cu[0].cpu().numpy(), cu[1].cpu().numpy(),
                             float(np.float32(192 ** -0.5)), causal)
            for key, name in (("dq", "dq"), ("dk", "dk"), ("dv", "dv"), ("dk_shared", "dr")):
                off, size = np.linalg.norm(f64(g[key])[0] - ref[name]), np.linalg.norm(ref[name])
                if size < 1e-12:
                    assert off == 0, (key, lens_q, causal)
                else:
                    assert off <= 2.0 ** -8 * size, (key, lens_q, causal, off / size)


def test_expanded_gradients_against_differences():
    """The directional derivative of the forward itself, taken by central differences in its inputs."""
    lens = [90, 45]
    q, k, v, r, dout = expanded(lens, lens, 2, 64, seed=11, std=1.0)
    cu = cu_of(lens)
    out, lse = kda.latent_fwd(q, k, v, r, cu)
    g = kda.latent_bwd(q, k, v, r, out, lse, dout, cu)
    gen = torch.Generator().manual_seed(1)
    loss = lambda *a: float((kda.latent_fwd(*a, cu)[0].double() * dout.double()).sum())  # noqa: E731
    args = [q, k.contiguous(), v.contiguous(), r.contiguous()]
    for i, key in enumerate(("dq", "dk", "dv", "dk_shared")):
        up, down = list(args), list(args)
        d = torch.randn(args[i].shape, generator=gen).to(DEV).sign() * g[key].sign().float()
        d = d.abs() * g[key].sign().float()                  # along the gradient's signs: every term adds up
        up[i], down[i] = (args[i].float() + 0.0625 * d).to(B16), (args[i].float() - 0.0625 * d).to(B16)
        step = (up[i].double() - down[i].double())
        slope, want = loss(*up) - loss(*down), float((g[key].double() * step).sum())
        # each output carries half a bf16 step twice (its own and P's), at random signs: sums of 135*2*128 of them
        noise = 4 * HALF * float((out.double().abs() * dout.double().abs()).square().sum().sqrt()) * 2
        curve = 0.05 * abs(want)                             # the third derivative's share at steps of 1/16
        assert abs(slope - want) <= noise + curve, (key, slope, want, noise)


def test_expanded_repeats_bitwise_and_on_other_streams_and_graphs():
    lens = [260, 131]
    q, k, v, r, dout = expanded(lens, lens, 3, 64, seed=12)
    cu = cu_of(lens)
    out, lse = kda.latent_fwd(q, k, v, r, cu)
    g = kda.latent_bwd(q, k, v, r, out, lse, dout, cu)
    for _ in range(3):
        o2, l2 = kda.latent_fwd(q, k, v, r, cu)
        g2 = kda.latent_bwd(q, k, v, r, o2, l2, dout, cu)
        assert torch.equal(o2, out) and torch.equal(l2, lse) and all(torch.equal(g2[x], g[x]) for x in g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o3, l3 = kda.latent_fwd(q, k, v, r, cu)
        g3 = kda.latent_bwd(q, k, v, r, o3, l3, dout, cu)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o3, out) and all(torch.equal(g3[x], g[x]) for x in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o4, l4 = kda.latent_fwd(q, k, v, r, cu)
        g4 = kda.latent_bwd(q, k, v, r, o4, l4, dout, cu)
    for _ in range(2):
        o4.zero_(), g4["dk"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o4, out) and all(torch.equal(g4[x], g[x]) for x in g)


# ------------------------------------------------------------------------------------------- decode

def paged(lens, H, R, Tq, page, seed=0, extra=3, std=1.0):
    """A cache whose pages lie in a random order, filled with NaN wherever no sequence has a row."""
    g = torch.Generator().manual_seed(seed)
    W, per = 512 + R, [-(-n // page) for n in lens]
    pages = sum(per) + extra
    order = torch.randperm(pages, generator=g)
    cache = torch.full((pages, page, W), float("nan"))
    table = torch.full((len(lens), max(per + [1]) + 1), -1, dtype=torch.int32)     # entries behind the end: not read
    at = 0
    for n, length in enumerate(lens):
        for i in range(per[n]):
            table[n, i] = order[at]
            rows = min(page, length - i * page)
            cache[order[at], :rows] = torch.randn(rows, W, generator=g)
            cache[order[at], rows:, ::3] = float("inf")
            at += 1
    q = torch.randn(len(lens), Tq, H, W, generator=g) * std
    return (q.to(B16).to(DEV), cache.to(B16).to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))


def check_decode(q, cache, table, lens, out, lse, scale):
    ro, rl, wide, big = O.decode(f64(q), np.nan_to_num(f64(cache), posinf=0.0), table.cpu().numpy(), lens.cpu().numpy(),
                                 float(np.float32(scale)))
    d = score_error(big, q.shape[-1])
    n = float(lens.max())
    within(f64(out), ro, (HALF + d + n * 2.0 ** -24)[..., None] * wide, "out")
    x, fine = f64(lse), np.isfinite(rl)
    assert np.array_equal(fine, np.isfinite(x)) and np.all(x[~fine] == -np.inf)
    assert np.all(np.abs(x[fine] - rl[fine]) <= (d + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(rl) + 2.0 ** -18)[fine]), "lse"


@pytest.mark.parametrize("R", [64, 0])
@pytest.mark.parametrize("lens,H,Tq,page", [
    ([1], 8, 1, 16), ([64], 16, 1, 64), ([65], 16, 1, 16), ([63, 0, 1, 200], 32, 1, 32), ([130], 64, 1, 128),
    ([333, 17, 64], 16, 3, 16), ([700, 3], 20, 1, 80), ([257], 128, 1, 48), ([129, 128, 2], 32, 4, 64), ([5, 1], 8, 4, 64),
    ([1500], 1, 1, 112), ([300] * 7, 5, 2, 256),
])
def test_absorbed(lens, H, Tq, page, R):
    a = paged(lens, H, R, Tq, page, seed=len(lens) + H)
    scale = (128 + R) ** -0.5
    out, lse, ws = kda.latent_decode_step(*a, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    check_decode(*a, out, lse, scale)


def test_absorbed_many_sequences_of_all_lengths():
    lens = [(i * 37) % 200 for i in range(310)]
    a = paged(lens, 4, 64, 1, 16, seed=2)
    out, lse = kda.latent_decode_step(*a, scale=0.3)
    check_decode(*a, out, lse, 0.3)


def test_absorbed_long_sequence_split_over_the_gpu():
    """A length that many blocks share, against the expanded statement on one head; others are checked by
    giving every head the same query."""
    n = 20011
    q, cache, table, lens = paged([n], 16, 64, 1, 64, seed=4)
    q[:, :, 1:] = q[:, :, :1]
    out, lse = kda.latent_decode_step(q, cache, table, lens)
    assert all(torch.equal(out[0, 0, h], out[0, 0, 0]) for h in range(16))
    check_decode(q[:, :, :1], cache, table, lens, out[:, :, :1], lse[:, :, :1], 192 ** -0.5)


@pytest.mark.parametrize("H", [8, 48, 128])
def test_absorbed_short_sequences_beside_a_long_one(H):
    """As many sequences as shares of the GPU, nearly, and one of them cut into many parts: the join goes by share and
    takes a block to a row."""
    lens = [(i * 37) % 160 for i in range(60)] + [20000] + [(i * 53) % 160 for i in range(45)]
    a = paged(lens, H, 64, 1, 64, seed=H)
    out, lse, ws = kda.latent_decode_step(*a, return_workspace=True)
    assert kda.workspace_status(ws) == kda.KDA_OK
    check_decode(*a, out, lse, 192 ** -0.5)
    again = kda.latent_decode_step(*a)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_absorbed_peaked_and_growing_scores():
    """Scores that grow along the sequence, so that the running maximum moves in every tile."""
    q, cache, table, lens = paged([900], 8, 64, 1, 64, seed=8)
    rows = cache[table[0, :15].long()].reshape(-1, 576)[:900]
    ramp = torch.linspace(-4, 4, 900, device=DEV)[:, None]
    rows = (torch.randn(900, 576, device=DEV) * 0.1 + ramp * torch.sign(q[0, 0, 0].float())).to(B16)
    flat = cache.view(-1, 576)
    at = (table[0].long()[torch.arange(900, device=DEV) // 64] * 64 + torch.arange(900, device=DEV) % 64)
    flat[at] = rows
    for scale in (0.02, 0.3):
        out, lse = kda.latent_decode_step(q, cache, table, lens, scale=scale)
        check_decode(q, cache, table, lens, out, lse, scale)


def test_absorbed_bad_lengths_and_pages_are_reported():
    q, cache, table, lens = paged([100, 60, 30], 8, 64, 1, 16, seed=7)
    want = kda.latent_decode_step(q, cache, table, lens)
    for n, value in ((0, 16 * table.shape[1] + 1), (1, -3)):
        bad = lens.clone()
        bad[n] = value
        out, lse, ws = kda.latent_decode_step(q, cache, table, bad, return_workspace=True)
        assert kda.workspace_status(ws) == kda.KDA_ERR_INVALID_ARG
        assert torch.all(out[n] == 0) and torch.all(lse[n] == -float("inf"))
        for other in {0, 1, 2} - {n}:
            assert torch.equal(out[other], want[0][other])
    for page in (-1, cache.shape[0], 2 ** 30):
        bad = table.clone()
        bad[1, 2] = page
        out, lse, ws = kda.latent_decode_step(q, cache, bad, lens, return_workspace=True)
        assert kda.workspace_status(ws) == kda.KDA_ERR_INVALID_ARG
        assert torch.equal(out[0], want[0][0]) and torch.equal(out[2], want[0][2])


@pytest.mark.parametrize("width", [0, 3])
def test_absorbed_empty_cache(width):
    """A cache without a page: idle slots get zeros, a length above zero is reported."""
    q = torch.randn(3, 1, 8, 576, device=DEV).to(B16)
    cache, table = torch.empty(0, 64, 576, dtype=B16, device=DEV), torch.zeros(3, width, dtype=torch.int32, device=DEV)
    for lens, status in (([0, 0, 0], kda.KDA_OK), ([0, 5, 0], kda.KDA_ERR_INVALID_ARG)):
        out, lse, ws = kda.latent_decode_step(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), return_workspace=True)
        assert kda.workspace_status(ws) == status
        assert torch.all(out == 0) and torch.all(lse == -float("inf"))


def test_absorbed_streams_graphs_and_two_workspaces():
    a, b = paged([500, 77], 16, 64, 1, 64, seed=1), paged([90, 333], 16, 64, 1, 64, seed=2)
    wa, wb = kda.latent_decode_step(*a), kda.latent_decode_step(*b)
    size = kda.latent_decode_workspace_size(2, 1, 16)
    ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    graphs, outs = [], []
    for x, w in ((a, ws[0]), (b, ws[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kda.latent_decode_step(*x, workspace=w))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, (wa, wb)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------------ norm and append

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(1, 8), (3, 72), (37, 256), (5, 1000), (2, 1032), (130, 2048), (9, 4096), (3, 4104),
                                    (4, 8192), (2, 16384), (700, 128)])
def test_rms_norm(rows, D, dtype):
    dt = B16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(rows * D)
    x, res, dy, dh = (torch.randn(rows, D, generator=g).to(dt).to(DEV) for _ in range(4))
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(DEV)
    half = HALF if dt == B16 else 0.0
    # fp32: D products in the mean of squares (relative error D 2^-24 at most, halved by the root), five roundings more
    rel = (D / 2 + 8) * 2.0 ** -24
    for r in (None, res):
        y, h = kda.rms_norm(x, w, residual=r)
        want_h = x if r is None else (x.float() + r.float()).to(dt)
        assert torch.equal(h, want_h)
        ref = O.rms_norm(f64(h), f64(w), 1e-5)
        assert np.all(np.abs(f64(y) - ref) <= (half + rel) * (1 + half) * np.abs(ref) + 1e-30)
    # in place on the residual stream
    stream = res.clone()
    y2, h2 = kda.rms_norm(x, w, residual=stream, residual_out=stream)
    assert h2 is stream and torch.equal(h2, h) and torch.equal(y2, y)
    for extra in (None, dh):
        dx, dw = kda.rms_norm_bwd(dy, h, w, dh=extra)
        rx, rw, wide = O.rms_norm_backward(f64(dy), f64(h), f64(w), 1e-5)
        ad = 0.0 if extra is None else f64(extra)
        hh, gg = f64(h), np.abs(f64(dy) * f64(w))
        rms = np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-5)
        size = gg / rms + np.abs(hh) / rms ** 3 * (gg * np.abs(hh)).mean(-1, keepdims=True)
        assert np.all(np.abs(f64(dx) - rx - ad) <= half * np.abs(rx + ad) + (3 * rel * size + 2.0 ** -23 * np.abs(ad)) * (1 + half) + 1e-30)
        assert np.all(np.abs(f64(dw) - rw) <= (rel * 2 + (rows + 8) * 2.0 ** -24) * wide + 1e-30)


@pytest.mark.parametrize("rows,D,dtype", [
    (20003, 128, "bf16"), (6001, 1000, "bf16"), (3001, 2048, "bf16"), (1531, 4096, "bf16"), (743, 8192, "bf16"), (743, 4096, "f32"),
    (1501, 4104, "f32"), (1501, 10000, "bf16"), (650, 16384, "f32")])
def test_rms_norm_backward_of_many_rows(rows, D, dtype):
    """More rows than blocks: each block walks several, the last of them not all as many, for every number of threads
    that holds a row; bounds as in ``test_rms_norm``."""
    dt, half = (B16, HALF) if dtype == "bf16" else (torch.float32, 0.0)
    g = torch.Generator().manual_seed(rows)
    h, dy, dh = (torch.randn(rows, D, generator=g).to(dt).to(DEV) for _ in range(3))
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(DEV)
    rel = (D / 2 + 8) * 2.0 ** -24
    rx, rw, wide = O.rms_norm_backward(f64(dy), f64(h), f64(w), 1e-5)
    hh, gg = f64(h), np.abs(f64(dy) * f64(w))
    rms = np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-5)
    size = gg / rms + np.abs(hh) / rms ** 3 * (gg * np.abs(hh)).mean(-1, keepdims=True)
    for extra in (None, dh):
        dx, dw = kda.rms_norm_bwd(dy, h, w, dh=extra)
        ad = 0.0 if extra is None else f64(extra)
        assert np.all(np.abs(f64(dx) - rx - ad) <= half * np.abs(rx + ad) + (3 * rel * size + 2.0 ** -23 * np.abs(ad)) * (1 + half) + 1e-30)
        assert np.all(np.abs(f64(dw) - rw) <= (rel * 2 + (rows + 8) * 2.0 ** -24) * wide + 1e-30)
    # in place over each of its inputs
    want = kda.rms_norm_bwd(dy, h, w, dh=dh)
    for over in range(3):
        a = [t.clone() for t in (dy, h, dh)]
        got = kda.rms_norm_bwd(a[0], a[1], w, dh=a[2], dx=a[over])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(1, 128), (37, 256), (5, 1152), (3, 4096), (2, 16384)])
def test_rms_norm_e4m3(rows, D, dtype):
    dt = B16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(D)
    x, res = (torch.randn(rows, D, generator=g).to(dt).to(DEV) for _ in range(2))
    x[0, :128] = 0
    res[0, :128] = 0                                   # a group of zeros: scale 0, values 0
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(DEV)
    for r in (None, res):
        q, scale, h = kda.rms_norm_e4m3(x, w, residual=r)
        assert torch.equal(h, x if r is None else (x.float() + r.float()).to(dt))
        y = O.rms_norm(f64(h), f64(w), 1e-5).reshape(rows, -1, 128)
        s = f64(scale)
        rel = (D / 2 + 12) * 2.0 ** -24
        amax = np.abs(y).max(-1)
        assert np.all(np.abs(s - amax / 448) <= rel * amax / 448 + 1e-30)
        assert s[0, 0] == 0 and torch.all(q.float()[0, :128] == 0)
        # the stored value is the nearest one to y / scale: half a step of e4m3, 2^-4 relative (2^-10 below 2^-6)
        got, want = f64(q).reshape(y.shape), y / np.where(s == 0, 1, s)[..., None]
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 448 * 4 * rel)
        exact = O.round_e4m3(want)
        assert np.mean(exact != got) <= 1e-3            # only ties within the fp32 error may fall the other way


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(2051, 512), (700, 4096), (300, 8320)])
def test_rms_norm_e4m3_of_many_rows(rows, D, dtype):
    test_rms_norm_e4m3(rows, D, dtype)


def test_rms_norm_e4m3_non_finite_groups_say_so():
    x = torch.randn(3, 384, device=DEV)
    x[1, 130] = float("nan")
    q, scale, _ = kda.rms_norm_e4m3(x, torch.ones(384, device=DEV))
    assert torch.all(torch.isfinite(scale[[0, 2]])) and not torch.isfinite(scale[1]).any()


def test_rms_norm_no_rows_and_bitwise_repeats():
    w = torch.ones(256, device=DEV)
    y, _ = kda.rms_norm(torch.empty(0, 256, device=DEV), w)
    assert y.shape == (0, 256)
    _, dw = kda.rms_norm_bwd(torch.empty(0, 256, device=DEV), torch.empty(0, 256, device=DEV), w)
    assert torch.all(dw == 0)
    h, dy = torch.randn(5000, 256, device=DEV), torch.randn(5000, 256, device=DEV)
    a = kda.rms_norm_bwd(dy, h, w)
    for _ in range(3):
        b = kda.rms_norm_bwd(dy, h, w)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,R,page", [(1, 64, 16), (7, 0, 32), (300, 64, 48)])
def test_append(T, R, page):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 512 + R, generator=g).to(B16).to(DEV)
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(DEV)
    pages = T // page + 3
    cache = torch.randn(pages, page, 512 + R, generator=g).to(B16).to(DEV)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::5] = -1                                      # padding
    if T > 2:
        slots[2] = pages * page                          # outside: skipped as well
    before = cache.clone()
    got = kda.latent_append(x[:, :512], x[:, 512:] if R else None, cache, slots.to(DEV), weight=w)
    assert got is cache
    flat, old = f64(cache).reshape(-1, 512 + R), f64(before).reshape(-1, 512 + R)
    ref = O.rms_norm(f64(x)[:, :512], f64(w), 1e-5)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            assert np.all(np.abs(flat[s, :512] - ref[t]) <= (HALF + 300 * 2.0 ** -24) * np.abs(ref[t]) + 1e-30)
            assert np.array_equal(flat[s, 512:], f64(x)[t, 512:])
            old[s] = flat[s]
    assert np.array_equal(flat, old)                     # every other row as it was
    plain = kda.latent_append(x[:, :512], x[:, 512:] if R else None, before.clone(), slots.to(DEV))
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            assert torch.equal(plain.view(-1, 512 + R)[s], x[t])


@pytest.mark.parametrize("R", [64, 0])
@pytest.mark.parametrize("T", [1, 2, 9])
def test_append_of_the_first_token(T, R):
    """Every token has a row, the first and only one too; with the norm and as it is."""
    g = torch.Generator().manual_seed(T + R)
    x = torch.randn(T, 640, generator=g).to(B16).to(DEV)
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(DEV)
    before = torch.randn(3, 16, 512 + R, generator=g).to(B16).to(DEV)
    slots = torch.randperm(48, generator=g)[:T]
    c, r = x[:, :512], x[:, 512:512 + R] if R else None
    cache = kda.latent_append(c, r, before.clone(), slots.to(DEV), weight=w)
    want = f64(before).reshape(48, -1)
    ref, got = O.rms_norm(f64(c), f64(w), 1e-5), f64(cache).reshape(48, -1)
    assert np.all(np.abs(got[slots, :512] - ref) <= (HALF + 300 * 2.0 ** -24) * np.abs(ref) + 1e-30)
    want[slots, :512] = got[slots, :512]
    want[slots, 512:] = f64(x)[:, 512:512 + R]
    assert np.array_equal(got, want)                     # the shared part as it is, every other row as it was
    plain = kda.latent_append(c, r, before.clone(), slots.to(DEV))
    assert torch.equal(plain.view(48, -1)[slots], x[:, :512 + R])


# ------------------------------------------------------------------------------------ used together

def test_layer_prompt_and_decode_together():
    """One attention layer over a packed prompt and then a decode step: norm, projections, cache append, the
    expanded form for the prompt, the absorbed form for the next token, which must agree with the expanded
    form run over the whole sequences."""
    H, R, D, page = 4, 64, 256, 32
    g = torch.Generator().manual_seed(5)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DEV)  # noqa: E731
    wq, wc = n(D, H * 192, std=D ** -0.5), n(D, 512 + R, std=D ** -0.5)
    wk, wv = n(H, 128, 512, std=512 ** -0.5), n(H, 128, 512, std=512 ** -0.5)
    norm_w, latent_w = 1 + n(D, std=0.1), 1 + n(512, std=0.1)
    lens = [70, 33, 129]
    total = [x + 1 for x in lens]
    x, res = n(sum(total), D).to(B16), n(sum(total), D).to(B16)
    starts = np.cumsum([0] + total)
    new = torch.tensor([int(s) - 1 for s in starts[1:]], device=DEV)               # each sequence's last token
    y, _ = kda.rms_norm(x, norm_w, residual=res)
    q = (y.float() @ wq).to(B16).reshape(1, -1, H, 192)
    down = (y.float() @ wc).to(B16)
    per = [-(-t // page) for t in total]
    cache = torch.full((sum(per), page, 512 + R), float("nan"), dtype=B16, device=DEV)
    table = torch.zeros(3, max(per), dtype=torch.int32, device=DEV)
    slots, base = [], 0
    for i, t in enumerate(total):
        table[i, :per[i]] = torch.arange(base, base + per[i])
        slots += [base * page + j for j in range(t)]
        base += per[i]
    kda.latent_append(down[:, :512], down[:, 512:], cache, torch.tensor(slots, device=DEV), weight=latent_w)
    c = cache.view(-1, 576)[torch.tensor(slots, device=DEV)]
    up = torch.cat([wk, wv], 1)                                                     # [H, 256, 512]
    kv = torch.einsum("hdc,tc->thd", up, c[:, :512].float()).to(B16)[None]
    whole, _ = kda.latent_fwd(q, kv[..., :128], kv[..., 128:], c[None, :, 512:], cu_of(total))
    qn = q[0, new].float()
    qa = torch.cat([torch.einsum("hdc,thd->thc", wk, qn[..., :128]), qn[..., 128:]], -1).to(B16)[:, None]
    o, _ = kda.latent_decode_step(qa, cache, table, torch.tensor(total, dtype=torch.int32, device=DEV))
    absorbed = torch.einsum("hdc,thc->thd", wv, o[:, 0].float())
    want = whole[0, new].float()
    # the two differ by the roundings of k, v, q, P and the outputs: each at most 2^-8 of its value, of random sign;
    # six of them at four standard deviations of a uniform error (2^-8 / sqrt 3) stay below 2^-4 of the output's size
    size = want.square().mean().sqrt()
    assert float((absorbed - want).abs().max()) <= 2.0 ** -4 * 4 * float(size)
    assert float((absorbed - want).square().mean().sqrt()) <= 2.0 ** -5 * float(size)


@pytest.mark.parametrize("N,H", [(3, 16), (40, 32)])
def test_calls_that_read_one_anothers_results(N, H):
    """A chain in which each call reads what the call before it wrote, without a pause: the same bits as with the
    device idle between the calls, and as in a graph whose first nodes are a memset and copies."""
    rows, page, D = N * H, 32, 576
    g = torch.Generator().manual_seed(9)
    x0 = torch.randn(rows, D, generator=g).to(B16).to(DEV)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(DEV)
    pages = -(-rows // page)
    slots = torch.randperm(rows, generator=g).to(DEV)
    table = torch.randint(0, pages, (N, 5), generator=g, dtype=torch.int32).to(DEV)
    lens = torch.randint(1, 5 * page, (N,), generator=g, dtype=torch.int32).to(DEV)
    x, cache = torch.empty_like(x0), torch.empty(pages, page, D, dtype=B16, device=DEV)

    def chain(pause):
        cache.zero_()
        x.copy_(x0)
        y, h, kept = x, x, []
        for _ in range(4):
            y, h = kda.rms_norm(y, w, residual=h)
            pause()
            kda.latent_append(y[:, :512], y[:, 512:], cache, slots)
            pause()
            o, _ = kda.latent_decode_step(y.view(N, 1, H, D), cache, table, lens)
            pause()
            q, kv = y.view(1, 3 * rows, 1, 192), o.view(1, 4 * rows, 1, 128)
            k, v, r = kv[:, :3 * rows], kv[:, rows:], h.view(1, 9 * rows, 64)[:, :3 * rows]
            out, lse = kda.latent_fwd(q, k, v, r)
            pause()
            grads = kda.latent_bwd(q, k, v, r, out, lse, out)
            pause()
            y, dw = kda.rms_norm_bwd(grads["dq"].view(rows, D), h, w, dh=grads["dk"].view(-1)[:rows * 128].repeat(5)[:rows * D].view(rows, D))
            pause()
            kept += [o, out, lse, grads["dk_shared"], grads["dv"], dw, y, kda.rms_norm_e4m3(out.view(-1, 128), w[:128])[1]]
        return kept

    want = [t.clone() for t in chain(torch.cuda.synchronize)]
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)
    for _ in range(3):
        for a, b in zip(chain(lambda: None), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(3):
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_offsets_and_inputs_rewritten_between_calls():
    """One buffer of offsets and one of each input, rewritten on the stream in front of every call without a pause:
    each call has the values written last (the same bits as with the device idle before and after it)."""
    g = torch.Generator().manual_seed(13)
    T, H, N = 700, 4, 5
    sets = []
    for i in range(4):
        cut = sorted(torch.randint(0, T + 1, (N - 1,), generator=g).tolist())
        q, k, v, r, dout = expanded([T], [T], H, 64, seed=40 + i)
        sets.append((torch.tensor([0] + cut + [T], dtype=torch.int32, device=DEV), q, k.contiguous(), v.contiguous(), r.contiguous(), dout))
    here = [t.clone() for t in sets[0]]

    def round_trip(pause):
        kept = []
        for new in sets + sets[::-1]:
            for a, b in zip(here, new):
                a.copy_(b)
            pause()
            cu, q, k, v, r, dout = here
            out, lse = kda.latent_fwd(q, k, v, r, cu)
            pause()
            for a, b in zip(here, new):      # written again, directly in front of the backward pass
                a.zero_()
                a.copy_(b)
            pause()
            grads = kda.latent_bwd(q, k, v, r, out, lse, dout, cu)
            pause()
            kept += [out, lse, *grads.values()]
        return kept

    want = round_trip(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(round_trip(lambda: None), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = round_trip(lambda: None)
    for _ in range(3):
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)

"""The vocabulary operators on the CPU: the 64-bit reference forms against
closed forms and differences, and the library's refusals (no kernel runs)."""

from __future__ import annotations

import ctypes as C
import os

import numpy as np
import pytest

import dspark_draft_sampling_amd as ds
from tests import _vocab_ref as ref

FAKE = C.c_void_p(4096)  # a non-NULL, 16-byte aligned pointer that is never dereferenced
OTHER = C.c_void_p(1 << 40)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ds.LIB_PATH):
        pytest.skip("libdspark.so not built")
    return ds.lib()


# ---- the reference forms ------------------------------------------------------------


def test_reference_top_logits():
    x = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4])
    v, i, rest, lse = ref.top_logits(x, 2)
    assert i.tolist() == [[1, 2], [-1, -1]] and v[0].tolist() == [3.0, 3.0]
    assert rest[0] == 1.0 and np.isclose(lse[0], np.log(np.e + 2 * np.e ** 3))
    assert np.isneginf(rest[1]) and np.isneginf(lse[1])


@pytest.mark.parametrize("with_rest", [False, True])
def test_reference_distill_is_zero_for_the_teacher_itself(with_rest):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 12)) * 2
    v, i, r, _ = ref.top_logits(x.reshape(6, 12), 12 if not with_rest else 4, 2.0)
    K = v.shape[1]
    out = ref.distill(x, v.reshape(2, 3, K), i.reshape(2, 3, K), r.reshape(2, 3) if with_rest else None, T=2.0)
    assert np.all(np.abs(out["kl"]) < 1e-12) and np.allclose(out["sums"][1], 6)


@pytest.mark.parametrize("with_rest,dup", [(False, False), (True, False), (True, True), (False, True)])
def test_reference_gradient_against_differences(with_rest, dup):
    rng = np.random.default_rng(1)
    N, G, V, K, T = 2, 2, 9, 4, 1.7
    x = rng.standard_normal((N, G, V)) * 1.5
    t = rng.standard_normal((N * G, V)) * 1.5
    v, i, r, _ = ref.top_logits(t, K, T)
    v, i, r = v.reshape(N, G, K), i.reshape(N, G, K), r.reshape(N, G)
    if dup:
        i[0, 0, 2] = i[0, 0, 0]
        i[1, 1, 3] = -1
    a = (v, i, r if with_rest else None, np.array([1, 1], np.uint8), T, 0.7)
    g = ref.distill_grad(x, *a, scale=1.3)
    for at in np.ndindex(N, G, V):
        h = 1e-5
        p, m = x.copy(), x.copy()
        p[at] += h
        m[at] -= h
        d = 1.3 * (ref.distill(p, *a)["sums"][0] - ref.distill(m, *a)["sums"][0]) / (2 * h)
        # a central difference is off by h^2 f''' / 6 and by rounding / h, both under 1e-9
        assert abs(d - g[at]) < 1e-8, at


# ---- refusals -----------------------------------------------------------------------


def top(L, logits=FAKE, dtype=1, R=4, V=1024, K=8, T=1.0, out=FAKE, ws=FAKE, wsb=1 << 30):
    return L.dspark_top_logits(logits, dtype, R, V, K, T, out, FAKE, FAKE, FAKE, FAKE, ws, wsb, None)


def test_top_logits_refusals(L):
    assert top(L, R=-1) == ds.DSPARK_EINVAL
    assert top(L, V=0) == ds.DSPARK_EINVAL
    assert top(L, K=0) == ds.DSPARK_EINVAL
    assert top(L, dtype=5) == ds.DSPARK_EDTYPE
    assert top(L, K=ds.DSPARK_MAX_TOP + 1) == ds.DSPARK_ESHAPE
    assert top(L, V=ds.DSPARK_MAX_TOP_VOCAB + 1) == ds.DSPARK_ESHAPE
    for T in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -21, 2.0 ** 21):
        assert top(L, T=T) == ds.DSPARK_EINVAL, T
    assert top(L, logits=None) == ds.DSPARK_EINVAL
    assert top(L, out=None) == ds.DSPARK_EINVAL
    assert top(L, logits=C.c_void_p(4097)) == ds.DSPARK_EINVAL
    assert top(L, logits=C.c_void_p(4098), dtype=2) == ds.DSPARK_EINVAL
    assert top(L, R=0, logits=None, out=None, ws=None) == ds.DSPARK_OK
    assert ds.dspark_workspace_size(ds.DSPARK_OP_TOP, 1, 1, 1000000, 8) > 0
    assert top(L, R=1, V=1000000, ws=None) == ds.DSPARK_EWORKSPACE
    assert top(L, R=1, V=1000000, wsb=64) == ds.DSPARK_EWORKSPACE
    assert ds.dspark_workspace_size(ds.DSPARK_OP_TOP, 4, 1, 1024, 0) == 0
    assert ds.dspark_workspace_size(ds.DSPARK_OP_TOP, 4, 1, 1024, ds.DSPARK_MAX_TOP + 1) == 0


def distill(L, draft=FAKE, dtype=1, values=FAKE, N=4, gamma=5, V=1024, K=8, T=1.0, sums=FAKE, ws=FAKE, wsb=1 << 30):
    return L.dspark_distill(draft, dtype, values, FAKE, None, None, N, gamma, V, K, T, 1.0, FAKE, FAKE, FAKE, FAKE,
                            sums, ws, wsb, None)


def grad(L, draft=FAKE, dtype=1, values=FAKE, rest=FAKE, N=4, gamma=5, V=1024, K=8, T=1.0, out=OTHER):
    return L.dspark_distill_backward(draft, dtype, values, FAKE, rest, None, None, N, gamma, V, K, T, 1.0, None, out,
                                     None)


@pytest.mark.parametrize("call", [distill, grad])
def test_distill_refusals(L, call):
    assert call(L, N=-1) == ds.DSPARK_EINVAL
    assert call(L, gamma=0) == ds.DSPARK_EINVAL
    assert call(L, V=0) == ds.DSPARK_EINVAL
    assert call(L, K=0) == ds.DSPARK_EINVAL
    assert call(L, dtype=3) == ds.DSPARK_EDTYPE
    assert call(L, gamma=17) == ds.DSPARK_ESHAPE
    assert call(L, V=(1 << 30) + 1) == ds.DSPARK_ESHAPE
    assert call(L, K=ds.DSPARK_MAX_TOP + 1) == ds.DSPARK_ESHAPE
    assert call(L, N=1 << 30) == ds.DSPARK_ESHAPE
    assert call(L, T=0.0) == ds.DSPARK_EINVAL
    assert call(L, T=float("nan")) == ds.DSPARK_EINVAL
    assert call(L, draft=None) == ds.DSPARK_EINVAL
    assert call(L, values=None) == ds.DSPARK_EINVAL
    assert call(L, draft=C.c_void_p(4097)) == ds.DSPARK_EINVAL


def test_distill_workspace_and_overlap(L):
    assert distill(L, sums=None) == ds.DSPARK_EINVAL
    assert distill(L, ws=None) == ds.DSPARK_EWORKSPACE
    assert distill(L, wsb=16) == ds.DSPARK_EWORKSPACE
    assert grad(L, rest=None) == ds.DSPARK_EINVAL
    assert grad(L, out=None) == ds.DSPARK_EINVAL
    assert grad(L, out=FAKE) == ds.DSPARK_EINVAL  # the gradient over the logits
    assert grad(L, out=C.c_void_p(4096 + 4 * 5 * 1024 * 2 - 2)) == ds.DSPARK_EINVAL  # one element of them
    assert grad(L, out=C.c_void_p(4096 + 2 * 1024 + 1)) == ds.DSPARK_EINVAL  # misaligned
    assert grad(L, N=0, draft=None, out=None) == ds.DSPARK_OK


def beam(L, logits=FAKE, dtype=1, scores=FAKE, finished=None, eos=0, B=2, W=4, V=1024, M=8, out=OTHER, ws=FAKE,
         wsb=1 << 30):
    return L.dspark_beam_select(logits, dtype, scores, finished, eos, B, W, V, M, FAKE, FAKE, out, FAKE, ws, wsb, None)


def test_beam_select_refusals(L):
    assert beam(L, B=-1) == ds.DSPARK_EINVAL
    for kw in (dict(W=0), dict(V=0), dict(M=0), dict(logits=None), dict(scores=None), dict(out=None),
               dict(out=FAKE), dict(logits=C.c_void_p(4099)), dict(finished=FAKE, eos=-1),
               dict(finished=FAKE, eos=1024)):
        assert beam(L, **kw) == ds.DSPARK_EINVAL, kw
    assert beam(L, dtype=0) == ds.DSPARK_EDTYPE
    for kw in (dict(W=33), dict(M=129), dict(V=ds.DSPARK_MAX_TOP_VOCAB + 1), dict(B=1 << 30)):
        assert beam(L, **kw) == ds.DSPARK_ESHAPE, kw
    assert beam(L, ws=None) == ds.DSPARK_EWORKSPACE
    assert beam(L, wsb=16) == ds.DSPARK_EWORKSPACE
    assert beam(L, B=0, logits=None, scores=None, out=None, ws=None) == ds.DSPARK_OK
    assert ds.dspark_workspace_size(ds.DSPARK_OP_BEAM, 2, 33, 1024, 8) == 0


def move(L, src=FAKE, dst=OTHER, parents=FAKE, lengths=None, n=1, B=2, W=4, M=4, S=1, T=8, size=16):
    return L.dspark_beam_reorder(src, dst, parents, lengths, n, B, W, M, S, T, size, None)


def test_beam_reorder_refusals(L):
    for kw in (dict(n=-1), dict(B=-1), dict(W=-1), dict(M=-1), dict(S=-1), dict(T=-1), dict(size=-1),
               dict(src=None), dict(dst=None), dict(parents=None), dict(dst=FAKE, M=3),
               dict(dst=C.c_void_p(4096 + 16)), dict(dst=C.c_void_p(4096 - 2 * 4 * 8 * 16 + 1))):
        assert move(L, **kw) == ds.DSPARK_EINVAL, kw
    assert move(L, dst=FAKE, W=33, M=33) == ds.DSPARK_ESHAPE
    assert move(L, T=2 ** 31 - 1, size=2 ** 40) == ds.DSPARK_ESHAPE
    for kw in (dict(n=0), dict(B=0), dict(W=0), dict(M=0), dict(S=0), dict(T=0), dict(size=0)):
        assert move(L, src=None, dst=None, parents=None, **kw) == ds.DSPARK_OK, kw


def test_binding_refuses_cpu_tensors(L):
    import torch

    x = torch.zeros(1, 2, 8)
    i = torch.zeros(1, 2, 4, dtype=torch.int32)
    v = torch.zeros(1, 2, 4)
    for call in (lambda: ds.dspark_top_logits(x, 4), lambda: ds.dspark_distill(x, v, i),
                 lambda: ds.dspark_distill_backward(x, v, i, v[..., 0]),
                 lambda: ds.dspark_beam_select(x, x[..., 0], 2),
                 lambda: ds.dspark_beam_reorder(x, i[..., 0]), lambda: ds.dspark_beam_reorder(None, i)):
        with pytest.raises(ds.DSparkError):
            call()


def test_limits_match_the_header():
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "dspark.h")).read()
    defines = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define\s+(DSPARK_MAX_\w+)\s+(\d+)", text)}
    for name in ("DSPARK_MAX_TOP", "DSPARK_MAX_TOP_VOCAB", "DSPARK_MAX_BEAMS"):
        assert defines[name] == getattr(ds, name)

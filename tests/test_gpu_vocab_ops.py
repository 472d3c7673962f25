"""The vocabulary operators (highest logits, distillation and its gradient, beam
selection and reordering) on the GPU against their 64-bit forms
(tests/_vocab_ref.py, with the tolerances derived there)."""

from __future__ import annotations

import math
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import dspark_draft_sampling_amd as ds  # noqa: E402
from tests import _gpu as G  # noqa: E402
from tests import _vocab_ref as ref  # noqa: E402
from workloads import bf16_to_f32, to_bf16  # noqa: E402

NEG = -np.inf
LOWEST = {"f32": np.finfo(np.float32).min, "bf16": np.float32(-3.3895314e38)}


def values_of(x, dtype):
    """float32 values as the logits type holds them."""
    if dtype == "f32":
        return x.astype(np.float32)
    inf = np.isinf(x)
    return np.where(inf, x, bf16_to_f32(to_bf16(np.where(inf, 0, x).astype(np.float32)))).astype(np.float32)


def dev(x, dtype, shift=0):
    """x on the device; shift: elements by which its start is off an aligned address."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=G.DEV)
    buf[shift:] = t.flatten().to(G.DEV)
    return buf[shift:].view(t.shape)


def host(d):
    torch.cuda.synchronize()
    return {k: (v.float() if v.dtype == torch.bfloat16 else v).cpu().numpy() for k, v in d.items()}


def check_top(x, dtype, K, T=1.0, shift=0):
    x = values_of(x, dtype)
    got = host(ds.dspark_top_logits(dev(x, dtype, shift), K, T))
    v, i, rest, lse = ref.top_logits(x, K, T)
    assert np.array_equal(got["top_ids"], i)
    assert np.array_equal(got["top_values"], v.astype(np.float32))
    assert ref.near(got["rest"], rest), np.max(np.abs(got["rest"] - rest))
    assert ref.near(got["lse"], lse)
    assert np.array_equal(got["flags"], np.where(np.all(x == NEG, axis=1), ds.FLAG_EMPTY_ROW, 0))
    return got


# ---- highest logits -----------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,K,T,shift", [
    (1, 1, 1, 1.0, 0), (2, 1, 5, 1.0, 1), (3, 7, 3, 1.0, 0), (5, 64, 64, 0.5, 0), (4, 100, 128, 2.0, 3),
    (2, 1000, 8, 1.0, 0), (3, 1025, 128, 1.0, 1), (2, 4095, 1, 1.0, 5), (2, 8192, 17, 1.0, 0), (2, 8193, 64, 1.0, 2),
    (1, 16387, 100, 1.0, 0), (3, 32003, 20, 0.7, 0), (2, 50257, 128, 1.0, 7), (1, 129280, 8, 1.0, 0),
    (600, 20000, 12, 1.0, 0), (2, 131072, 64, 1.0, 0), (2, 131072, 64, 1.0, 1), (1, 300001, 50, 1.0, 0)])
def test_top_logits(dtype, R, V, K, T, shift):
    rng = np.random.default_rng(R * 1000003 + V * 131 + K)
    check_top(rng.standard_normal((R, V), dtype=np.float32) * 3, dtype, K, T, shift)


def test_top_logits_many_rows_and_splits():
    # more rows than fill the GPU: every split of a row there is
    rng = np.random.default_rng(7)
    for R, V in [(700, 33000), (1100, 9000), (40, 129280)]:
        x = values_of(rng.standard_normal((R, V), dtype=np.float32) * 3, "bf16")
        got = host(ds.dspark_top_logits(dev(x, "bf16"), 9))
        for r in (0, 1, R // 2, R - 1):
            one = check_top(x[r:r + 1], "bf16", 9)
            for k in ("top_values", "top_ids"):  # the same whatever the split
                assert np.array_equal(got[k][r], one[k][0])
            v, i, rest, lse = ref.top_logits(x[r:r + 1], 9)
            assert ref.near(got["rest"][r], rest[0]) and ref.near(got["lse"][r], lse[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [500, 5000, 40000, 140001])
@pytest.mark.parametrize("kind", ["constant", "two_values", "few_finite", "lowest", "lowest_all", "one", "none", "sorted",
                                  "peak", "far_rest", "signed_zero", "head", "block"])
def test_top_logits_odd_rows(dtype, V, kind):
    rng = np.random.default_rng(V)
    K = 24
    x = rng.standard_normal((2, V)).astype(np.float32) * 3
    if kind == "constant":  # nearly every index ties: the lowest ones count
        x[:] = 0.25
    elif kind == "two_values":
        x = np.where(rng.random((2, V)) < 0.5, 1.5, -2.0)
    elif kind == "few_finite":
        keep = rng.permutation(V)[:10]
        x[0] = NEG
        x[0, keep] = rng.standard_normal(10)
    elif kind == "lowest":  # masked by the type's lowest value, not by -inf
        x[:, rng.permutation(V)[: V - 30]] = LOWEST[dtype]
    elif kind == "lowest_all":
        x[:] = LOWEST[dtype]
    elif kind == "one":
        x[:] = NEG
        x[1, V - 1] = -3.0
        x[0, 0] = 1e30
    elif kind == "none":
        x[0] = NEG
    elif kind == "sorted":
        x.sort(axis=1)
        x[1] = x[1][::-1]
    elif kind == "peak":  # one token holds everything
        x[:, 3] = 120.0
    elif kind == "far_rest":  # the others' mass is far below what exp() of the top's scale holds
        x -= 400.0
        x[:, V // 2: V // 2 + K] += 800.0
    elif kind == "signed_zero":
        x = np.where(rng.random((2, V)) < 0.5, 0.0, -0.0)
    elif kind == "head":  # the best tokens side by side at the start
        x[:, :200] += 30.0
    else:  # a long run of finite tokens in a masked row
        x[:, : V // 3] = NEG
        x[:, V // 2:] = NEG
    check_top(x, dtype, K)
    check_top(x, dtype, 1)
    check_top(x, dtype, 128)


@pytest.mark.parametrize("V", [1000, 30000, 200000])
def test_top_logits_bad_values(V):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, V)).astype(np.float32)
    x[0, V // 2] = np.nan
    x[1, V - 1] = np.inf
    x[2] = np.nan
    x[4, 0] = -np.inf
    got = host(ds.dspark_top_logits(dev(x, "f32"), 6))
    assert got["flags"].tolist() == [ds.FLAG_NONFINITE] * 3 + [0, 0]
    assert np.all(got["top_ids"][:3] == -1) and np.all(np.isneginf(got["top_values"][:3]))
    assert np.all(np.isnan(got["rest"][:3])) and np.all(np.isnan(got["lse"][:3]))
    v, i, rest, lse = ref.top_logits(x[3:], 6)
    assert np.array_equal(got["top_ids"][3:], i) and ref.near(got["lse"][3:], lse) and ref.near(got["rest"][3:], rest)


def test_top_logits_is_reproducible_and_batch_independent():
    rng = np.random.default_rng(11)
    x = dev(rng.standard_normal((300, 50257)).astype(np.float32) * 3, "f32")
    a = host(ds.dspark_top_logits(x, 40))
    for _ in range(4):
        b = host(ds.dspark_top_logits(x, 40))
        assert all(np.array_equal(a[k], b[k]) for k in a)


def test_top_logits_shapes():
    x = dev(np.random.default_rng(1).standard_normal((6, 900)).astype(np.float32), "bf16")
    flat = host(ds.dspark_top_logits(x, 5))
    cube = host(ds.dspark_top_logits(x.view(2, 3, 900), 5))
    row = host(ds.dspark_top_logits(x[4], 5))
    for k in flat:
        assert np.array_equal(flat[k].reshape(cube[k].shape), cube[k])
        assert np.array_equal(flat[k][4], row[k])
    empty = ds.dspark_top_logits(torch.empty(0, 900, device=G.DEV), 5)
    assert empty["top_ids"].shape == (0, 5)


@pytest.mark.parametrize("dtype,R,V,K", [("bf16", 2100, 9000, 9), ("bf16", 2100, 30011, 32), ("f32", 2100, 5003, 30),
                                         ("bf16", 2100, 9000, 40), ("f32", 600, 129280, 20), ("bf16", 600, 140001, 33)])
def test_top_logits_every_way_to_take_a_row(dtype, R, V, K):
    # a wave a row, workgroups of 256, rows in several segments: rows alone (few) and in a batch (many)
    g = torch.Generator(device=G.DEV).manual_seed(V)
    x = (torch.randn(R, V, generator=g, device=G.DEV) * 3).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    got = host(ds.dspark_top_logits(x, K))
    for r in (0, 1, R // 2, R - 1):
        one = check_top(x[r:r + 1].float().cpu().numpy(), dtype, K)
        for k in ("top_values", "top_ids", "flags"):
            assert np.array_equal(got[k][r], one[k][0])
        for k in ("rest", "lse"):
            assert ref.near(got[k][r], np.float64(one[k][0]), 2 * ref.MASS_TOL)


def test_more_rows_than_a_grid_takes():
    """Counts past the 2^22 workgroups of one launch."""
    R = (1 << 22) + 5
    x = torch.randint(-8, 8, (R, 3), device=G.DEV).to(torch.float32)
    got = ds.dspark_top_logits(x, 2)
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    assert torch.equal(got["top_values"], v[:, :2]) and torch.equal(got["top_ids"].long(), i[:, :2])
    N, g = 300_000, 16
    d = torch.randn(N, g, 4, device=G.DEV)
    top = ds.dspark_top_logits(torch.randn(N, g, 4, device=G.DEV), 2)
    a = (top["top_values"], top["top_ids"])
    loss = ds.dspark_distill(d, *a, teacher_rest=top["rest"])
    grad = ds.dspark_distill_backward(d, *a, loss["rest"], teacher_rest=top["rest"])["grad_draft"]
    n = slice(N - 3, N)
    part = ds.dspark_distill(d[n].clone(), a[0][n].clone(), a[1][n].clone(), teacher_rest=top["rest"][n].clone())
    pg = ds.dspark_distill_backward(d[n].clone(), a[0][n].clone(), a[1][n].clone(), part["rest"],
                                    teacher_rest=top["rest"][n].clone())["grad_draft"]
    assert torch.equal(loss["kl"][n], part["kl"]) and torch.equal(grad[n], pg)
    w = torch.exp(-torch.arange(1, g + 1, device=G.DEV).double() / g)
    # the losses as written are the summands: only the 64-bit sums' rounding is between
    assert ref.near(float(loss["sums"][0]), float((loss["kl"].double() * w).sum()), 1e-3)
    assert float(loss["sums"][3]) == N * g
    B = (1 << 22) + 3
    pick = ds.dspark_beam_select(torch.randint(-8, 8, (B, 1, 2), device=G.DEV).float(), torch.zeros(B, 1, device=G.DEV), 2)
    assert torch.all(pick["tokens"].sum(1) == 1) and not pick["parents"].any()
    state = torch.arange(2 * B, device=G.DEV, dtype=torch.int32).view(B, 2)
    swap = torch.tensor([[1, 0]], dtype=torch.int32, device=G.DEV).expand(B, 2).contiguous()
    assert torch.equal(ds.dspark_beam_reorder(state, swap), state.flip(1))


def test_distill_sums_past_2_to_the_28_rows():
    N = (1 << 28) + 5
    d = torch.zeros(N, 1, 2, dtype=torch.bfloat16, device=G.DEV)
    v = torch.zeros(N, 1, 1, device=G.DEV)
    i = torch.zeros(N, 1, 1, dtype=torch.int32, device=G.DEV)
    mask = torch.zeros(N, dtype=torch.uint8, device=G.DEV)
    on = [7, N - 3, N - 1]
    for n in on:
        mask[n] = 1
        d[n, 0, 1] = 1.0
    got = ds.dspark_distill(d, v, i, block_mask=mask)
    kl = [float(got["kl"][n, 0]) for n in on]
    # the losses as written are the summands; one rounding of the sum to 32 bits
    assert ref.near(float(got["sums"][0]), math.exp(-1.0) * sum(kl), 2.0 ** -23)
    assert ref.near(float(got["sums"][2]), sum(kl), 2.0 ** -23)
    assert float(got["sums"][1]) == float(got["sums"][3]) == len(on)
    assert all(abs(k - math.log(1 + math.e)) < 1e-5 for k in kl)


def test_top_logits_past_32_bit_offsets():
    V, R = 129280, 16700  # R V passes 2^31 elements
    x = torch.zeros((R, V), dtype=torch.bfloat16, device=G.DEV)
    rng = np.random.default_rng(5)
    tail = rng.standard_normal((2, V)).astype(np.float32) * 3
    x[-2:] = dev(tail, "bf16")
    got = ds.dspark_top_logits(x, 7)
    one = host(ds.dspark_top_logits(dev(tail, "bf16"), 7))
    assert np.array_equal(got["top_ids"][-2:].cpu().numpy(), one["top_ids"])
    assert torch.equal(got["top_ids"][0].cpu(), torch.arange(7, dtype=torch.int32))  # a constant row


# ---- distillation -------------------------------------------------------------------


def distill_case(dtype, N, g, V, K, T, with_rest, masked, seed, shift=0):
    rng = np.random.default_rng(seed)
    x = values_of(rng.standard_normal((N, g, V), dtype=np.float32) * 2.5, dtype)
    t = (x + rng.standard_normal((N, g, V), dtype=np.float32)).astype(np.float32)
    v, i, r, _ = ref.top_logits(t.reshape(N * g, V), K, T)
    v, i = v.reshape(N, g, K).astype(np.float32), i.reshape(N, g, K).astype(np.int32)
    r = r.reshape(N, g).astype(np.float32) if with_rest else None
    m = (rng.random(N) < 0.7).astype(np.uint8) if masked else None
    return x, v, i, r, m, dev(x, dtype, shift)


def check_distill(x, v, i, r, m, xd, dtype, T=1.0, weight=1.0, scale=None):
    N, g, V = x.shape
    a = (torch.from_numpy(v).to(G.DEV), torch.from_numpy(i).to(G.DEV))
    kw = dict(teacher_rest=None if r is None else torch.from_numpy(r).to(G.DEV),
              block_mask=None if m is None else torch.from_numpy(m).to(G.DEV), temperature=T, weight=weight)
    out = ds.dspark_distill(xd, *a, **kw)
    sc = None if scale is None else torch.tensor([scale], device=G.DEV)
    grad = host(ds.dspark_distill_backward(xd, *a, out["rest"], grad_scale=sc, **kw))["grad_draft"]
    got = host(out)
    want = ref.distill(x, v, i, r, m, T, weight)
    assert ref.near(got["lse"], want["lse"]) and ref.near(got["rest"], want["rest"])
    # d kl / d log(rest) = s_r - t_r lies in [-1, 1]: kl is off by no more than rest is
    assert ref.near(got["kl"], want["kl"])
    count = max(1.0, want["sums"][1])
    assert np.array_equal(got["sums"][[1, 3]], want["sums"][[1, 3]].astype(np.float32))
    assert ref.near(got["sums"][0], want["sums"][0], abs(weight) * count * ref.MASS_TOL)
    assert ref.near(got["sums"][2], want["sums"][2], count * ref.MASS_TOL)
    s = 1.0 if scale is None else float(np.float32(scale))
    g64 = ref.distill_grad(x, v, i, r, m, T, weight, s, rest=got["rest"])
    tol = ref.grad_tol(x, got["rest"], g64, T, dtype)
    # at listed tokens the value is a difference in 64 bits, rounded to fp32 and to the type
    assert np.all(np.abs(grad - g64) <= tol + 1e-12 * np.max(np.abs(g64))), np.max(np.abs(grad - g64) - tol)
    # against the row's own normaliser: rest is off by MASS_TOL and its rounding, and s_v, s_r by that factor
    own = ref.distill_grad(x, v, i, r, m, T, weight, s)
    off = ref.MASS_TOL + 2.0 ** -24 * np.abs(np.where(np.isfinite(want["rest"]), want["rest"], 0))
    w = abs(s * weight / T)
    assert np.all(np.abs(grad - own) <= tol + 3 * w * off[..., None])
    return got, grad


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,g,V,K,T,with_rest,masked,shift", [
    (1, 1, 1, 1, 1.0, False, False, 0), (1, 1, 2, 1, 1.0, True, False, 0), (2, 3, 5, 5, 1.0, True, False, 1),
    (3, 5, 64, 7, 2.0, False, True, 0), (4, 2, 129, 128, 0.5, True, False, 0), (2, 16, 1000, 3, 1.0, True, True, 3),
    (3, 1, 2049, 64, 1.0, False, False, 0), (2, 2, 4101, 65, 1.0, True, False, 1), (1, 1, 33000, 128, 1.0, True, False, 0),
    (2, 7, 20011, 20, 2.0, False, True, 0), (1, 2, 129280, 64, 1.0, True, False, 0), (1, 1, 280001, 9, 1.0, True, False, 5),
    (300, 5, 700, 16, 1.0, True, True, 0)])
def test_distill(dtype, N, g, V, K, T, with_rest, masked, shift):
    case = distill_case(dtype, N, g, V, min(K, 128), T, with_rest, masked, N + V + K, shift)
    check_distill(*case, dtype, T, weight=T * T, scale=0.37)


def test_distill_rounds_to_nearest_even_everywhere():
    # every element against the rounding of the 64-bit value, beside the bound of its 32-bit form
    x, v, i, r, m, xd = distill_case("bf16", 2, 3, 9001, 12, 1.0, True, False, 99)
    a = (torch.from_numpy(v).to(G.DEV), torch.from_numpy(i).to(G.DEV))
    kw = dict(teacher_rest=torch.from_numpy(r).to(G.DEV))
    out = ds.dspark_distill(xd, *a, **kw)
    g16 = host(ds.dspark_distill_backward(xd, *a, out["rest"], **kw))["grad_draft"]
    g32 = host(ds.dspark_distill_backward(xd.float(), *a, out["rest"], **kw))["grad_draft"]
    assert np.array_equal(g16, bf16_to_f32(to_bf16(g32)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_rest", [False, True])
def test_distill_ids_twice_and_missing(dtype, with_rest):
    x, v, i, r, m, xd = distill_case(dtype, 3, 2, 3001, 10, 1.0, with_rest, False, 5)
    i[0, 0, 3] = i[0, 0, 1]           # a token twice
    i[0, 1, 2:6] = i[0, 1, 2]         # four times
    i[1, 0, 4] = -1                   # missing entries, by a token outside the vocabulary
    i[1, 1, 0] = 3001
    i[2, 0, 5] = np.iinfo(np.int32).min
    i[2, 1, 9] = np.iinfo(np.int32).max
    v[1, 0, 4] = np.nan               # not read as a value
    v[2, 0, 1] = NEG                  # listed without mass
    check_distill(x, v, i, r, m, xd, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 12007])
def test_distill_masked_vocabularies(dtype, V):
    x, v, i, r, m, _ = distill_case(dtype, 4, 2, V, 6, 1.0, True, False, 17)
    x = x.copy()
    outside = np.ones(V, bool)
    outside[i[0, 0]] = False
    x[0, 0, outside] = NEG                 # the draft has nothing beside the list
    r[0, 0] = NEG                          # and neither has the teacher
    outside = np.ones(V, bool)
    outside[i[0, 1]] = False
    x[0, 1, outside] = LOWEST[dtype]       # masked by the type's lowest value
    r[0, 1] = NEG
    x[1, 0, i[1, 0, 2]] = NEG              # the draft excludes what the teacher keeps: +inf
    x[1, 1] = NEG                          # an empty draft row
    v[2, 0] = NEG                          # a teacher with mass nowhere
    r[2, 0] = NEG
    x[2, 1, i[2, 1]] = LOWEST[dtype]       # the list at the lowest value
    x[3, 0] += 90.0                        # far from zero
    x = values_of(x, dtype)  # what the device holds
    got, grad = check_distill(x, v, i, r, m, dev(x, dtype), dtype)
    assert got["flags"].tolist() == [[0, 0], [0, ds.FLAG_EMPTY_ROW], [ds.FLAG_EMPTY_ROW, 0], [0, 0]]
    assert np.isposinf(got["kl"][1, 0]) and np.all(np.isfinite(grad))
    assert not grad[1, 1].any() and not grad[2, 0].any()
    assert got["kl"][1, 1] == 0 and got["kl"][2, 0] == 0


def test_distill_confident_rows_keep_their_accuracy():
    # one probability is 1 - 1e-9: its logarithm and its difference from 1 are the tail's mass
    V, K = 4000, 1
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 2, V)).astype(np.float32)
    x[..., 77] = 30.0
    i = np.full((1, 2, K), 77, np.int32)
    v = np.full((1, 2, K), 5.0, np.float32)
    xd = dev(x, "f32")
    a = (torch.from_numpy(v).to(G.DEV), torch.from_numpy(i).to(G.DEV))
    out = ds.dspark_distill(xd, *a)
    grad = host(ds.dspark_distill_backward(xd, *a, out["rest"]))["grad_draft"]
    want = ref.distill(x, v, i)
    g = ref.distill_grad(x, v, i)
    assert np.all(want["kl"] < 1e-9) and np.allclose(host(out)["kl"], want["kl"], rtol=ref.MASS_TOL + 1e-6)
    assert np.allclose(grad[..., 77], g[..., 77], rtol=ref.MASS_TOL + 1e-6)


def test_distill_bad_values():
    x, v, i, r, m, _ = distill_case("f32", 3, 2, 2500, 8, 1.0, True, False, 23)
    x, m = x.copy(), np.array([1, 1, 0], np.uint8)
    x[0, 0, 2499] = np.nan
    x[0, 1, int(i[0, 1, 3])] = np.inf
    v[1, 0, 2] = np.nan
    r[1, 1] = np.inf
    x[2, 0, 5] = np.nan  # in a masked block
    a = (torch.from_numpy(v).to(G.DEV), torch.from_numpy(i).to(G.DEV))
    kw = dict(teacher_rest=torch.from_numpy(r).to(G.DEV), block_mask=torch.from_numpy(m).to(G.DEV))
    xd = dev(x, "f32")
    got = host(ds.dspark_distill(xd, *a, **kw))
    assert got["flags"].tolist() == [[2, 2], [2, 2], [2, 0]]
    assert np.all(np.isnan(got["kl"][got["flags"] == 2])) and np.isfinite(got["kl"][2, 1])
    grad = host(ds.dspark_distill_backward(xd, *a, torch.from_numpy(got["rest"]).to(G.DEV), **kw))["grad_draft"]
    assert not grad[2].any()  # a masked block gives zeros whatever it holds


def test_distill_empty_batch_and_reproducible():
    e = torch.empty((0, 5, 100), device=G.DEV)
    out = ds.dspark_distill(e, torch.empty((0, 5, 4), device=G.DEV), torch.empty((0, 5, 4), dtype=torch.int32, device=G.DEV))
    assert not host(out)["sums"].any()
    x, v, i, r, m, xd = distill_case("bf16", 40, 7, 30011, 32, 1.0, True, True, 31)
    i[:, :, 5] = i[:, :, 4]
    a = (torch.from_numpy(v).to(G.DEV), torch.from_numpy(i).to(G.DEV))
    kw = dict(teacher_rest=torch.from_numpy(r).to(G.DEV), block_mask=torch.from_numpy(m).to(G.DEV))
    first = host(ds.dspark_distill(xd, *a, **kw))
    for _ in range(4):
        again = host(ds.dspark_distill(xd, *a, **kw))
        assert all(np.array_equal(first[k], again[k]) for k in first)


def test_distill_gradient_against_differences_of_the_loss():
    x, v, i, r, m, xd = distill_case("f32", 1, 2, 40, 6, 1.3, True, False, 3)
    a = (torch.from_numpy(v).to(G.DEV), torch.from_numpy(i).to(G.DEV))
    kw = dict(teacher_rest=torch.from_numpy(r).to(G.DEV), temperature=1.3)
    out = ds.dspark_distill(xd, *a, **kw)
    g = host(ds.dspark_distill_backward(xd, *a, out["rest"], **kw))["grad_draft"]
    h = 2.0 ** -5
    for at in np.ndindex(1, 2, 40):
        f = []
        for d in (h, -h):
            y = x.copy()
            y[at] += d
            step = float(y[at]) - float(x[at])
            f.append((float(ds.dspark_distill(dev(y, "f32"), *a, **kw)["sums"][0]), step))
        d = (f[0][0] - f[1][0]) / (f[0][1] - f[1][1])
        # h^2 / 6 of the third derivative (under 1), and the loss's error (MASS_TOL a row) over 2 h
        assert abs(d - g[at]) < h * h / 6 + 2 * ref.MASS_TOL / h


# ---- beam selection -----------------------------------------------------------------


def check_beam(x, scores, M, dtype, finished=None, eos=0, shift=0):
    x = values_of(x, dtype)
    B, W, V = x.shape
    out = ds.dspark_beam_select(dev(x, dtype, shift), torch.from_numpy(scores).to(G.DEV), M,
                                None if finished is None else torch.from_numpy(finished).to(G.DEV), eos)
    got = host(out)
    for b in range(B):
        s = ref.beam_scores(x[b], scores[b], None if finished is None else finished[b], eos)
        order = np.argsort(-s.ravel(), kind="stable")[:M]
        want = s.ravel()[order]
        n = int(np.sum(want > NEG))
        tok, par, sc = got["tokens"][b], got["parents"][b], got["scores"][b]
        assert np.all(tok[n:] == -1) and np.all(par[n:] == -1) and np.all(np.isneginf(sc[n:]))
        assert np.all(tok[:n] >= 0) and np.all((par[:n] >= 0) & (par[:n] < W))
        assert len({(p, t) for p, t in zip(par[:n], tok[:n])}) == n
        # each pick's own 64-bit score is that of its rank: two picks trade places only where
        # their scores are nearer than the normalisers' error
        assert np.all(np.abs(s[par[:n], tok[:n]] - want[:n]) <= 2 * ref.MASS_TOL)
        assert ref.near(sc[:n], s[par[:n], tok[:n]])
        gaps = np.abs(np.diff(np.sort(s[s > NEG])[::-1][: M + 1]))
        if n and (len(gaps) == 0 or gaps.min() > 2 * ref.MASS_TOL):
            assert np.array_equal(par[:n] * V + tok[:n], order[:n])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V,M,shift", [
    (1, 1, 1, 1, 0), (2, 1, 3, 5, 0), (1, 4, 32000, 8, 0), (3, 4, 1001, 4, 1), (2, 16, 5003, 32, 0),
    (2, 32, 600, 128, 0), (5, 3, 50257, 6, 3), (1, 32, 140000, 128, 0), (64, 4, 9000, 8, 0), (1, 2, 300007, 128, 0)])
def test_beam_select(dtype, B, W, V, M, shift):
    rng = np.random.default_rng(B + W + V + M)
    x = rng.standard_normal((B, W, V), dtype=np.float32) * 3
    scores = (rng.standard_normal((B, W)) * 0.7 - 20).astype(np.float32)
    check_beam(x, scores, M, dtype, shift=shift)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 3001, 30000])
def test_beam_select_first_step_and_ended_beams(dtype, V):
    rng = np.random.default_rng(V)
    x = rng.standard_normal((4, 5, V), dtype=np.float32) * 2
    scores = (rng.standard_normal((4, 5)) - 4).astype(np.float32)
    scores[0, 1:] = NEG                   # the first step: one beam
    scores[1] = NEG                       # no beam at all
    finished = np.zeros((4, 5), np.uint8)
    finished[2, 1] = finished[2, 3] = 1   # ended beams
    finished[3] = 1                       # all of them
    x[2, 1] = np.nan                      # an ended beam's logits are not read
    x[0, 2] = np.inf                      # nor a dead one's
    got = check_beam(np.where(np.isfinite(x), x, 0), scores, 7, dtype, finished, eos=V - 1)
    raw = host(ds.dspark_beam_select(dev(x, dtype), torch.from_numpy(scores).to(G.DEV), 7,
                                     torch.from_numpy(finished).to(G.DEV), V - 1))
    for k in got:
        assert np.array_equal(got[k], raw[k]), k
    assert np.all(raw["flags"] == 0)
    assert np.all(raw["tokens"][1] == -1)
    n = 5
    assert np.array_equal(np.sort(raw["parents"][3][:n]), np.arange(5)) and np.all(raw["tokens"][3][:n] == V - 1)


def test_beam_select_ties_and_bad_rows():
    V = 2000
    x = np.zeros((3, 4, V), np.float32)
    x[0, :, 10] = x[0, :, 500] = 2.0      # equal beams: the lower beam, then the lower token
    scores = np.full((3, 4), -1.0, np.float32)
    x[1, 1, 7] = np.nan
    x[1, 2] = NEG
    scores[2, 0] = np.nan
    scores[2, 1] = np.inf
    got = host(ds.dspark_beam_select(dev(x, "f32"), torch.from_numpy(scores).to(G.DEV), 9))
    assert got["parents"][0].tolist() == [0, 0, 1, 1, 2, 2, 3, 3, 0]
    assert got["tokens"][0].tolist() == [10, 500] * 4 + [0]
    assert got["flags"].tolist() == [[0, 0, 0, 0], [0, 2, 8, 0], [2, 2, 0, 0]]
    assert got["parents"][1].tolist() == [0] * 9 and got["tokens"][1].tolist() == list(range(9))
    assert got["parents"][2].tolist() == [2] * 9
    # all equal, with as many picks as there may be
    big = host(ds.dspark_beam_select(torch.zeros((1, 32, 3001), device=G.DEV), torch.zeros((1, 32), device=G.DEV), 128))
    assert big["parents"][0].tolist() == [0] * 128 and big["tokens"][0].tolist() == list(range(128))


# ---- reordering ---------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int64])
@pytest.mark.parametrize("lead,B,W,M,tail,length_dim", [
    ((), 2, 4, 4, (), None), ((), 3, 4, 7, (64,), None), ((2,), 2, 3, 3, (5, 33), None), ((3,), 2, 5, 5, (2, 17, 3), 4),
    ((), 1, 32, 32, (300,), None), ((2, 2), 3, 4, 8, (2, 70, 64), 5), ((), 4, 2, 2, (1, 1), 2), ((1,), 2, 16, 16, (4, 40, 8), 4),
    ((), 2, 40, 40, (9,), None)])
def test_beam_reorder(dtype, lead, B, W, M, tail, length_dim):
    rng = np.random.default_rng(B * 100 + W + M)
    d = len(lead)
    shape = (*lead, B, W, *tail)
    state = torch.from_numpy(rng.integers(0, 120, shape)).to(dtype).to(G.DEV)
    parents = rng.integers(0, W, (B, M)).astype(np.int32)
    parents[0, 0] = -1
    parents[-1, -1] = W
    lengths = None
    if length_dim is not None:
        T = shape[length_dim]
        lengths = np.array([(0, 1, T, T + 5, -3, T // 2)[(b + 2) % 6] for b in range(B)], np.int32)
    args = dict(batch_dim=d, lengths=None if lengths is None else torch.from_numpy(lengths).to(G.DEV),
                length_dim=length_dim)
    p = torch.from_numpy(parents).to(G.DEV)
    old = torch.full((*lead, B, M, *tail), 121, dtype=torch.int64).to(dtype).to(G.DEV)
    host64 = lambda t: t.to(torch.int64).cpu().numpy()  # noqa: E731
    for out in (None, old.clone()):
        before = None if out is None else host64(out)
        got = ds.dspark_beam_reorder(state, p, out=out, **args)
        want = ref.reorder(host64(state), parents, d, lengths, length_dim, before)
        assert np.array_equal(host64(got), want)
    if M == W and W <= ds.DSPARK_MAX_BEAMS:  # in place
        want = ref.reorder(host64(state), parents, d, lengths, length_dim, host64(state))
        assert ds.dspark_beam_reorder(state, p, out=state, **args) is state
        assert np.array_equal(host64(state), want)


def test_beam_reorder_at_odd_addresses():
    for shift in (1, 2, 4, 8):
        buf = torch.arange(4000, device=G.DEV).to(torch.uint8)
        src = buf[shift:shift + 2 * 3 * 160].view(2, 3, 160)
        dst = torch.zeros(4000, dtype=torch.uint8, device=G.DEV)[3 * shift:3 * shift + 960].view(2, 3, 160)
        p = torch.tensor([[2, 0, 1], [1, 1, 0]], dtype=torch.int32, device=G.DEV)
        want = torch.stack([src[b][p[b].long()] for b in range(2)])
        assert torch.equal(ds.dspark_beam_reorder(src, p, out=dst), want)


@pytest.mark.parametrize("T", [13, 47, 48, 1100])
def test_beam_reorder_every_last_byte(T):
    """Lengths in bytes from none on, to new states and in place."""
    B, W = 40, 5
    rng = np.random.default_rng(T)
    state = torch.from_numpy(rng.integers(0, 256, (2, B, W, T)).astype(np.uint8)).to(G.DEV)
    parents = rng.integers(0, W, (B, W)).astype(np.int32)
    lengths = np.minimum(np.arange(B) + (T - B if T > 100 else 0), T).astype(np.int32)
    args = dict(batch_dim=1, lengths=torch.from_numpy(lengths).to(G.DEV), length_dim=3)
    p = torch.from_numpy(parents).to(G.DEV)
    fill = torch.full_like(state, 77)
    want = ref.reorder(state.cpu().numpy(), parents, 1, lengths, 3, fill.cpu().numpy())
    assert np.array_equal(ds.dspark_beam_reorder(state, p, out=fill, **args).cpu().numpy(), want)
    want = ref.reorder(state.cpu().numpy(), parents, 1, lengths, 3, state.cpu().numpy())
    assert np.array_equal(ds.dspark_beam_reorder(state, p, out=state, **args).cpu().numpy(), want)


def test_beam_reorder_past_32_bit_offsets():
    T = 36_000_000  # a beam of 2.3 GB
    state = torch.zeros((1, 2, T, 64), dtype=torch.uint8, device=G.DEV)
    state[0, 1, -5:] = 7
    state[0, 0, -1] = 9
    p = torch.tensor([[1, 0]], dtype=torch.int32, device=G.DEV)
    ds.dspark_beam_reorder(state, p, lengths=torch.tensor([T - 1], dtype=torch.int32, device=G.DEV), length_dim=2, out=state)
    torch.cuda.synchronize()
    assert state[0, 0, -6:, 0].tolist() == [0, 7, 7, 7, 7, 9]
    assert state[0, 1, -6:, 0].tolist() == [0, 0, 0, 0, 0, 7]


def test_bindings_refuse_bad_arguments():
    x = torch.zeros(2, 3, 40, device=G.DEV)
    v = torch.zeros(2, 3, 4, device=G.DEV)
    i = torch.zeros(2, 3, 4, dtype=torch.int32, device=G.DEV)
    sc = torch.zeros(2, 3, device=G.DEV)
    p = torch.zeros(2, 3, dtype=torch.int32, device=G.DEV)
    ok = ds.dspark_distill(x, v, i)
    calls = [
        lambda: ds.dspark_top_logits(x.half(), 4), lambda: ds.dspark_top_logits(x.transpose(1, 2), 4),
        lambda: ds.dspark_top_logits(x, 0), lambda: ds.dspark_top_logits(x, -1), lambda: ds.dspark_top_logits(x, 129),
        lambda: ds.dspark_top_logits(x, 4, temperature=0.0), lambda: ds.dspark_top_logits(x, 4, out=ok),
        lambda: ds.dspark_distill(x[0], v, i), lambda: ds.dspark_distill(x, v[:1], i), lambda: ds.dspark_distill(x, v, i.long()),
        lambda: ds.dspark_distill(x, v, i[..., :3].contiguous()), lambda: ds.dspark_distill(x, v.double(), i),
        lambda: ds.dspark_distill(x, v, i, teacher_rest=sc.T.contiguous()), lambda: ds.dspark_distill(x, v, i, block_mask=p),
        lambda: ds.dspark_distill(x, v[..., :0], i[..., :0]), lambda: ds.dspark_distill_backward(x, v, i, sc[:1]),
        lambda: ds.dspark_distill_backward(x, v, i, sc, grad_scale=sc), lambda: ds.dspark_distill_backward(x, v, i, sc, out=dict(grad_draft=x)),
        lambda: ds.dspark_beam_select(x[0], sc, 2), lambda: ds.dspark_beam_select(x, sc[0], 2),
        lambda: ds.dspark_beam_select(x, sc, 0), lambda: ds.dspark_beam_select(x, sc, 200),
        lambda: ds.dspark_beam_select(x, sc, 2, finished=p), lambda: ds.dspark_beam_select(x, sc, 3, out=dict(
            tokens=p, parents=p.clone(), scores=sc, flags=torch.zeros(2, 3, dtype=torch.uint8, device=G.DEV))),
        lambda: ds.dspark_beam_reorder(x, p.long()), lambda: ds.dspark_beam_reorder(x, p, batch_dim=2),
        lambda: ds.dspark_beam_reorder(x, p[:1]), lambda: ds.dspark_beam_reorder(x, p, lengths=p[:, 0].contiguous()),
        lambda: ds.dspark_beam_reorder(x, p, lengths=p[:, 0].contiguous(), length_dim=1),
        lambda: ds.dspark_beam_reorder(x, p[:, :2].contiguous(), out=x), lambda: ds.dspark_beam_reorder(x, p, out=x.flatten()[:-1]),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(ds.DSparkError):
            call()
            pytest.fail(f"call {n} was not refused")
    torch.cuda.synchronize()


def test_bindings_refuse_what_32_bits_would_cut():
    """Numbers whose lower 32 bits would be valid."""
    x = torch.zeros(2, 3, 40, device=G.DEV)
    sc = torch.zeros(2, 3, device=G.DEV)
    done = torch.zeros(2, 3, dtype=torch.uint8, device=G.DEV)
    wide = torch.empty(1, 1, (1 << 32) + 8, dtype=torch.bfloat16, device=G.DEV)
    one = torch.zeros(1, 1, 1, device=G.DEV)
    calls = [
        lambda: ds.dspark_top_logits(x, (1 << 32) + 4), lambda: ds.dspark_beam_select(x, sc, (1 << 32) + 4),
        lambda: ds.dspark_beam_select(x, sc, 2, finished=done, eos_token=(1 << 32) + 1),
        lambda: ds.dspark_beam_select(x, sc, 2, finished=done, eos_token=-1),
        lambda: ds.dspark_top_logits(wide, 4), lambda: ds.dspark_beam_select(wide, one[0], 2),
        lambda: ds.dspark_distill(wide, one, one.int()), lambda: ds.dspark_distill_backward(wide, one, one.int(), one[0]),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(ds.DSparkError):
            call()
            pytest.fail(f"call {n} was not refused")
    ds.dspark_beam_select(x, sc, 2, eos_token=-1)  # not read without finished
    torch.cuda.synchronize()


# ---- together -----------------------------------------------------------------------


def test_teacher_pass_to_gradient():
    """A teacher's rows kept as their highest logits, the loss and its gradient: a
    step down the gradient lowers the loss, and with every token listed the loss is
    the full divergence."""
    rng = np.random.default_rng(8)
    N, g, V, T = 6, 5, 2003, 2.0
    x = dev(rng.standard_normal((N, g, V)).astype(np.float32), "f32")
    t = dev(rng.standard_normal((N, g, V)).astype(np.float32) * 2, "bf16")
    top = ds.dspark_top_logits(t, 32, T)
    kw = dict(teacher_rest=top["rest"], temperature=T, weight=T * T)
    a = (top["top_values"], top["top_ids"])
    out = ds.dspark_distill(x, *a, **kw)
    grad = ds.dspark_distill_backward(x, *a, out["rest"], **kw)["grad_draft"]
    less = ds.dspark_distill(x - 0.1 * grad, *a, **kw)
    assert float(less["sums"][0]) < float(out["sums"][0])
    # a coarser view of two distributions is never further apart than they are
    lt, ls = (torch.log_softmax(y.double() / T, -1) for y in (t, x))
    full = (lt.exp() * (lt - ls)).sum(-1)
    assert torch.all(out["kl"].double() <= full + 2 * ref.MASS_TOL)
    small = ds.dspark_top_logits(t[..., :100].contiguous(), 100, T)
    every = ds.dspark_distill(x[..., :100].contiguous(), small["top_values"], small["top_ids"], temperature=T)
    lt, ls = (torch.log_softmax(y[..., :100].double() / T, -1) for y in (t, x))
    assert ref.near(host(every)["kl"], (lt.exp() * (lt - ls)).sum(-1).cpu().numpy())


def test_beam_search_finds_the_best_sequence():
    """A search over a small bigram table with as many beams as there are prefixes is
    exhaustive: selection, states reordered in place, histories and scores against
    every sequence."""
    rng = np.random.default_rng(12)
    V, steps, B, W = 5, 3, 3, 25
    table = rng.standard_normal((B, V + 1, V)).astype(np.float32) * 2  # row V: the start
    td = torch.from_numpy(table).to(G.DEV)
    state = torch.zeros((2, B, W, steps, 8), dtype=torch.int32, device=G.DEV)  # a history, eight copies of each token
    last = torch.full((B, W), V, dtype=torch.int64, device=G.DEV)
    scores = torch.full((B, W), float("-inf"), device=G.DEV)
    scores[:, 0] = 0
    for k in range(steps):
        logits = td[torch.arange(B, device=G.DEV)[:, None], last].contiguous()
        pick = ds.dspark_beam_select(logits, scores, W)
        ds.dspark_beam_reorder(state, pick["parents"], batch_dim=1,
                               lengths=torch.full((B,), k, dtype=torch.int32, device=G.DEV), length_dim=3, out=state)
        state[:, :, :, k] = pick["tokens"][None, :, :, None]
        last = torch.where(pick["tokens"] < 0, V, pick["tokens"].long())
        scores = pick["scores"]
    got, sc = state[1, ..., 5].cpu().numpy(), scores.cpu().numpy()
    lp = table.astype(np.float64) - ref.lse(table)[..., None]
    for b in range(B):
        every = sorted(((lp[b, V, i] + lp[b, i, j] + lp[b, j, k], (i, j, k)) for i in range(V) for j in range(V)
                        for k in range(V)), reverse=True)[:W]
        assert [tuple(h) for h in got[b]] == [s for _, s in every]
        assert ref.near(sc[b], [s for s, _ in every], 4 * ref.MASS_TOL)


# ---- streams and graphs -------------------------------------------------------------


def _everything(x, t, scores, parents):
    """One pass of every call, outputs as a flat dict."""
    top = ds.dspark_top_logits(t, 16, 1.5)
    a = (top["top_values"], top["top_ids"])
    loss = ds.dspark_distill(x, *a, teacher_rest=top["rest"], temperature=1.5)
    grad = ds.dspark_distill_backward(x, *a, loss["rest"], teacher_rest=top["rest"], temperature=1.5)
    pick = ds.dspark_beam_select(t, scores, 6)
    state = ds.dspark_beam_reorder(x, pick["parents"])
    return ({f"top_{k}": v for k, v in top.items()} | {f"loss_{k}": v for k, v in loss.items()} | grad
            | {f"pick_{k}": v for k, v in pick.items()} | {"state": state})


def _inputs(seed, N=3, W=4, V=40009):
    rng = np.random.default_rng(seed)
    return (dev(rng.standard_normal((N, W, V)).astype(np.float32) * 2, "bf16"),
            dev(rng.standard_normal((N, W, V)).astype(np.float32) * 3, "bf16"),
            torch.from_numpy(rng.standard_normal((N, W)).astype(np.float32)).to(G.DEV), None)


def test_captured_and_replayed():
    srcs = [_inputs(s) for s in (1, 2)]
    refs = [host(_everything(*s)) for s in srcs]
    bufs = [t.clone() if t is not None else None for t in srcs[0]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _everything(*bufs)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs captured on one stream have workspaces of their own
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs = _everything(*bufs)
        graphs.append((gr, outs))
    # an eager call that needs a larger workspace comes between
    big = _inputs(9, N=40)
    _everything(*big)
    torch.cuda.synchronize()
    for rep in range(6):
        gr, outs = graphs[rep % 2]
        which = rep % 3 % 2
        for b, v in zip(bufs, srcs[which]):
            if b is not None:
                b.copy_(v)
        gr.replay()
        got = host(outs)
        for k in got:
            assert np.array_equal(got[k], refs[which][k], equal_nan=True), (rep, k)
        _everything(*srcs[1 - which])  # the program's own work between the replays
        torch.cuda.synchronize()


def test_two_streams_at_once():
    ins = [_inputs(s, V=129280) for s in (3, 4)]
    refs = [host(_everything(*i)) for i in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(3):
        for s, i in zip(streams, ins):
            with torch.cuda.stream(s):
                outs.append(_everything(*i))
    torch.cuda.synchronize()
    for n, o in enumerate(outs):
        got = host(o)
        for k in got:
            assert np.array_equal(got[k], refs[n % 2][k], equal_nan=True), (n, k)


def test_two_threads_on_one_stream():
    ins = [(torch.randn(3, 4, 20000 + n, device=G.DEV), torch.randn(3, 4, device=G.DEV), 8 + n) for n in range(2)]
    refs = [host(ds.dspark_beam_select(*i)) for i in ins]
    outs = [[] for _ in ins]
    start = threading.Barrier(len(ins))

    def work(n):
        start.wait()
        for _ in range(200):
            outs[n].append(ds.dspark_beam_select(*ins[n]))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(ins))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for n, results in enumerate(outs):
        assert len(results) == 200
        for o in results:
            got = host(o)
            for k in got:
                assert np.array_equal(got[k], refs[n][k]), (n, k)

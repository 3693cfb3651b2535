"""Logit shaping, the shaped log-prob and its gradient against the fp64 oracle.

Tolerances follow from the arithmetic, eps = 2^-24 (half an ulp, fp32):
 * z': at most 8 roundings of terms bounded by the row's magnitude M
   (penalty, two products, two differences, bias, inverse and product with
   1/T): 8 eps M, and half an ulp of the type when the output is bf16;
 * LSE: the error of the z' (16 eps max M: they pass to base 2 as well), the
   sum's relative error (about 60 sequential additions and a 2-ulp exponential:
   80 eps), and the rounding of the result itself (8 eps |LSE|);
 * the gradient: p's relative error is that of z' and LSE in the exponent.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import shaping_oracle as so
from synth import f32_to_bf16_bits, bf16_bits_to_f32

from gpu_helpers import gpu_lib  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
HALF_ULP = 2.0 ** -8     # half an ulp of bf16 (8 significant bits), at most, relative to the value
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _batch(rng, n, V, hist=40, features=("hist", "bias", "allow", "temp"), shared=False):
    b = {}
    if "hist" in features:
        if shared:      # one sequence: row i sees i tokens
            b["tokens"] = rng.integers(0, V, n).astype(np.int32)
            b["hist_begin"] = np.zeros(n, np.int64)
            b["hist_len"] = np.arange(n, dtype=np.int32)
            b["prompt_len"] = np.full(n, n // 3, np.int32)
        else:
            length = rng.integers(0, hist + 1, n)
            length[rng.integers(0, n)] = 0
            length[rng.integers(0, n)] = 1
            b["hist_begin"] = np.concatenate([[0], np.cumsum(length)[:-1]]).astype(np.int64)
            b["hist_len"] = length.astype(np.int32)
            t = rng.integers(-2, V + 2, max(1, int(length.sum())))
            hot = rng.integers(0, V, 4)
            b["tokens"] = np.where(rng.random(t.size) < 0.4, hot[rng.integers(0, 4, t.size)], t).astype(np.int32)
            b["prompt_len"] = rng.integers(-1, hist + 3, n).astype(np.int32)
        b["repetition"] = rng.uniform(0.7, 1.6, n).astype(np.float32)
        b["presence"] = rng.uniform(-0.5, 0.8, n).astype(np.float32)
        b["frequency"] = rng.uniform(-0.2, 0.5, n).astype(np.float32)
        off = rng.random(n) < 0.1
        b["repetition"][off], b["presence"][off], b["frequency"][off] = 1, 0, 0
    if "bias" in features:
        cnt = rng.integers(0, 9, 5)
        b["bias_offsets"] = np.concatenate([[0], np.cumsum(cnt)]).astype(np.int32)
        b["bias_tokens"] = rng.integers(-1, V + 1, int(cnt.sum())).astype(np.int32)
        if cnt[0] > 1:
            b["bias_tokens"][1] = b["bias_tokens"][0]        # the last entry of a token counts
        b["bias_values"] = rng.uniform(-5, 5, int(cnt.sum())).astype(np.float32)
        b["bias_set"] = rng.integers(-1, 5, n).astype(np.int32)
        if shared:
            b["bias_set"][:] = 0
    if "allow" in features:
        words = (V + 31) // 32
        bits = rng.integers(0, 1 << 32, (4, words), dtype=np.uint32)
        bits[1] &= rng.integers(0, 1 << 32, words, dtype=np.uint32) & rng.integers(0, 1 << 32, words, dtype=np.uint32)
        bits[2] = 0                                           # leaves nothing
        bits[3] = 0xffffffff
        b["allow_bits"] = bits.view(np.int32)
        b["allow_row"] = rng.integers(-1, 4, n).astype(np.int32)
    if "temp" in features:
        b["temperature"] = rng.uniform(0.4, 1.8, n).astype(np.float32)
    return b


def _shaping(b, n, V):
    import gspo_logprob_gb300 as g
    return g.make_shaping(n, V, **{k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in b.items()})


def _values(rng, n, V, dtype):
    x = (rng.standard_normal((n, V)) * 3).astype(np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)) if dtype == "bf16" else x


def _device(x, dtype, ld=None, shift=0):
    """[n, V] device view with row stride ld, starting `shift` elements into its storage."""
    n, V = x.shape
    ld = V if ld is None else ld
    flat = torch.full((n * ld + shift,), float("nan"), dtype=TYPES[dtype], device="cuda")
    v = torch.as_strided(flat, (n, V), (ld, 1), shift)
    v.copy_(torch.from_numpy(x).cuda())
    return v


def _np(t):
    return t.detach().double().cpu().numpy()


def _targets(rng, n, V):
    y = rng.integers(0, V, n).astype(np.int32)
    m = (rng.random(n) < 0.8).astype(np.uint8)
    m[0] = 1
    return y, m


def _check_shape(got, zp, mag, dtype):
    fin = np.isfinite(zp)
    assert np.array_equal(got == -np.inf, zp == -np.inf)
    tol = 8 * EPS * mag + (HALF_ULP * np.abs(np.where(fin, zp, 0)) * 1.01 if dtype == "bf16" else 0)
    err = np.abs(got[fin] - zp[fin])
    assert np.all(err <= tol[fin] + 1e-30), float(np.max(err - tol[fin]))


def _lse_tol(mag, lse):
    fin = np.where(np.isfinite(lse), np.abs(lse), 0)
    return 16 * EPS * mag.max(1) + 80 * EPS + 8 * EPS * fin


def _check_logp(logp, lse, want_logp, want_lse, tol):
    for got, want, t in ((lse, want_lse, tol), (logp, want_logp, 2 * tol + 4 * EPS * np.abs(np.nan_to_num(want_logp, posinf=0, neginf=0)))):
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got == -np.inf, want == -np.inf)
        fin = np.isfinite(want)
        assert np.all(np.abs(got[fin] - want[fin]) <= t[fin]), float(np.max(np.abs(got[fin] - want[fin]) - t[fin]))


def _check_grad(got, want, zp, slope, lse, coef, mag, dtype):
    lse0 = np.where(np.isfinite(lse), lse, 0)
    p = np.exp(np.minimum(np.where(np.isfinite(zp), zp, -np.inf) - lse0[:, None], 50))
    rel = (24 * EPS * mag.max(1) + 16 * EPS * np.abs(lse0) + 8 * EPS)[:, None]
    tol = np.abs(coef[:, None]) * slope * p * rel + 8 * EPS * np.abs(want)
    if dtype == "bf16":
        tol = tol + HALF_ULP * 1.01 * np.abs(want) + 1e-38
    err = np.abs(got - want)
    assert np.all(err <= tol + 1e-37), float(np.max(err - tol))


def _run_all(b, x, y, m, dtype, ld=None, shift=0, out_dtype=None, grad_out=None):
    """All three calls and their checks; returns the device results."""
    import gspo_logprob_gb300 as g
    from gspo_logprob_gb300 import ops
    n, V = x.shape
    sh = _shaping(b, n, V)
    z = _device(x, dtype, ld, shift)
    zp, slope, mag, bad = so.shape_logits(x, b)
    assert not bad.any()
    out = None if ld is None else _device(np.zeros_like(x), out_dtype or dtype, ld, shift)
    r = g.grpo_shape_logits(z, sh, out=out, out_dtype=TYPES[out_dtype or dtype])
    _check_shape(_np(r["logits"]), zp, mag, out_dtype or dtype)
    ops.raise_on_status(r["status"])
    yd, md = torch.from_numpy(y).cuda(), torch.from_numpy(m).cuda()
    want_logp, want_lse = so.shaped_logp(zp, y, m)
    f = g.grpo_shaped_logp(z, yd, md, sh)
    _check_logp(_np(f["logp"]), _np(f["lse"]), want_logp, want_lse, _lse_tol(mag, want_lse))
    rng = np.random.default_rng(3)
    coef = (rng.standard_normal(n) * m).astype(np.float32)
    coef[rng.random(n) < 0.15] = 0
    go = None if grad_out is None else torch.tensor([grad_out], device="cuda")
    lse32 = _np(f["lse"])
    dz = None if ld is None else _device(np.zeros_like(x), dtype, ld, shift)
    bw = g.grpo_shaped_logp_backward(z, yd, md, sh, f["lse"], torch.from_numpy(coef).cuda(), grad_out=go, dlogits=dz)
    want = so.shaped_logp_grad(zp, slope, y, m, lse32, coef.astype(np.float64), grad_out or 1.0)
    _check_grad(_np(bw["dlogits"]), want, zp, slope, lse32, coef.astype(np.float64) * (grad_out or 1.0), mag, dtype)
    return r["logits"], f, bw["dlogits"]


# rows, V, dtype, row stride beyond V, offset of the first element
_SHAPES = [
    (1, 1, "fp32", 0, 0), (1, 7, "bf16", 0, 0), (3, 31, "bf16", 0, 0), (5, 33, "fp32", 0, 1), (9, 255, "bf16", 1, 0),
    (17, 1000, "bf16", 0, 0), (4, 1024, "fp32", 0, 0), (33, 1025, "bf16", 7, 3), (6, 5001, "bf16", 0, 0),
    (6, 5001, "bf16", 7, 0), (3, 16384, "bf16", 0, 0), (2, 16385, "fp32", 3, 0), (3, 40008, "bf16", 0, 1),
    (2, 33001, "fp32", 0, 2),
]


@pytest.mark.parametrize("n,V,dtype,pad,shift", _SHAPES)
def test_against_oracle(gpu_lib, n, V, dtype, pad, shift):
    rng = np.random.default_rng(n * 131 + V)
    y, m = _targets(rng, n, V)
    _run_all(_batch(rng, n, V), _values(rng, n, V, dtype), y, m, dtype, V + pad, shift)


@pytest.mark.parametrize("features", [(), ("temp",), ("hist",), ("bias",), ("allow",), ("bias", "allow")])
def test_each_feature_alone(gpu_lib, features):
    rng = np.random.default_rng(len(features))
    n, V = 11, 3001
    y, m = _targets(rng, n, V)
    _run_all(_batch(rng, n, V, features=features), _values(rng, n, V, "bf16"), y, m, "bf16", grad_out=0.37)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_output_types(gpu_lib, dtype, out):
    rng = np.random.default_rng(5)
    y, m = _targets(rng, 7, 2050)
    _run_all(_batch(rng, 7, 2050), _values(rng, 7, 2050, dtype), y, m, dtype, out_dtype=out)


@pytest.mark.parametrize("hist", [0, 1, 5000, 70000])
def test_history_lengths(gpu_lib, hist):
    rng = np.random.default_rng(hist)
    n, V = 3, 20000
    y, m = _targets(rng, n, V)
    b = _batch(rng, n, V, hist=max(hist, 1))
    if hist == 0:
        b["hist_len"][:] = 0
    else:
        b["hist_len"][0], b["hist_begin"][0] = min(hist, b["tokens"].size), 0
    _run_all(b, _values(rng, n, V, "bf16"), y, m, "bf16")


def test_more_distinct_tokens_than_a_set_holds(gpu_lib):
    # enough rows for wide column ranges, histories with thousands of distinct tokens in each of them
    rng = np.random.default_rng(70)
    n, V = 320, 33001
    b = _batch(rng, n, V, hist=3)
    b["tokens"] = np.concatenate([b["tokens"], rng.permutation(V)[:25000]]).astype(np.int32)
    for i, k in ((3, 25000), (4, 25000), (5, 9000), (77, 24000), (319, 25000)):
        b["hist_begin"][i], b["hist_len"][i], b["prompt_len"][i] = b["tokens"].size - k, k, k // 2
    y, m = _targets(rng, n, V)
    _run_all(b, _values(rng, n, V, "bf16"), y, m, "bf16")


def test_training_sequence_grows_its_counts(gpu_lib):
    # enough rows that a CTA takes many consecutive ones: additions of one token, of several, rebuilds
    rng = np.random.default_rng(8)
    n, V = 24000, 96
    b = _batch(rng, n, V, shared=True)
    start = np.sort(rng.integers(0, n, 700))
    seq = np.searchsorted(start, np.arange(n), side="right")
    first = np.concatenate([[0], start])[seq]
    b["hist_begin"] = first.astype(np.int64)
    b["hist_len"] = (np.arange(n) - first).astype(np.int32)
    b["prompt_len"] = rng.integers(0, 20, 701)[seq].astype(np.int32)
    for k in ("repetition", "presence", "frequency", "temperature"):
        b[k] = b[k][seq]
    b["bias_set"] = b["bias_set"][seq]
    y, m = _targets(rng, n, V)          # inactive rows leave gaps of several tokens
    x = _values(rng, n, V, "bf16")
    z, f, dz = _run_all(b, x, y, m, "bf16")
    # the same rows in reverse order, each rebuilt, give the same bits
    import gspo_logprob_gb300 as g
    rev = {k: (v[::-1].copy() if v.shape[:1] == (n,) and k != "tokens" else v) for k, v in b.items()}
    sh = _shaping(rev, n, V)
    zr = _device(x[::-1].copy(), "bf16")
    assert torch.equal(g.grpo_shape_logits(zr, sh)["logits"].flip(0).view(torch.int16), z.view(torch.int16))
    fr = g.grpo_shaped_logp(zr, torch.from_numpy(y[::-1].copy()).cuda(), torch.from_numpy(m[::-1].copy()).cuda(), sh)
    assert torch.equal(fr["logp"].flip(0).view(torch.int32), f["logp"].view(torch.int32))
    assert torch.equal(fr["lse"].flip(0).view(torch.int32), f["lse"].view(torch.int32))


def test_bits_do_not_depend_on_the_batch_or_the_stride(gpu_lib):
    import gspo_logprob_gb300 as g
    rng = np.random.default_rng(9)
    n, V = 700, 33003
    b = _batch(rng, n, V)
    x = _values(rng, n, V, "bf16")
    y = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    m = torch.ones(n, dtype=torch.uint8, device="cuda")
    coef = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    ref = None
    for ld, rows in ((V, slice(0, n)), (V + 5, slice(0, n)), (V, slice(13, 14)), (V + 5, slice(100, 160))):
        k = rows.stop - rows.start
        sub = {q: (v[rows] if v.shape[:1] == (n,) and q not in ("tokens", "bias_tokens", "bias_values") else v)
               for q, v in b.items()}
        sh = _shaping(sub, k, V)
        z = _device(x[rows], "bf16", ld)
        f = g.grpo_shaped_logp(z, y[rows], m[rows], sh)
        dz = g.grpo_shaped_logp_backward(z, y[rows], m[rows], sh, f["lse"], coef[rows])["dlogits"]
        s = g.grpo_shape_logits(z, sh)["logits"]
        got = [f["logp"].view(torch.int32), f["lse"].view(torch.int32), dz.contiguous().view(torch.int16),
               s.contiguous().view(torch.int16)]
        if ref is None:
            ref = got
        for a, c in zip(got, ref):
            assert torch.equal(a, c[rows])


@pytest.mark.parametrize("n,V,dtype", [(1024, 1000, "fp32"), (2100, 2049, "bf16"), (4001, 500, "bf16"),
                                       (1030, 40000, "bf16")])
def test_micro_batches_of_packed_sequences(gpu_lib, n, V, dtype):
    # rows per CTA from two to four, whole rows per CTA (one launch) and ranges of them (two): the oracle's values,
    # and the bits of rows that are called by themselves
    import gspo_logprob_gb300 as g
    rng = np.random.default_rng(n)
    b = _batch(rng, n, V, features=("hist", "bias", "temp"), shared=True)
    first = np.arange(n) // 97 * 97
    b["hist_begin"] = first.astype(np.int64)
    b["hist_len"] = (np.arange(n) - first).astype(np.int32)
    b["prompt_len"] = np.full(n, 9, np.int32)
    for k in ("repetition", "presence", "frequency", "temperature"):
        b[k] = b[k][first]
    y, m = _targets(rng, n, V)
    x = _values(rng, n, V, dtype)
    z, f, dz = _run_all(b, x, y, m, dtype)
    for at, k in ((0, 1), (90, 20), (n - 30, 30)):
        rows = slice(at, at + k)
        sub = {q: (v[rows] if v.shape[:1] == (n,) and q != "tokens" else v) for q, v in b.items()}
        fs = g.grpo_shaped_logp(_device(x[rows], dtype), torch.from_numpy(y[rows]).cuda(),
                                torch.from_numpy(m[rows]).cuda(), _shaping(sub, k, V))
        assert torch.equal(fs["logp"].view(torch.int32), f["logp"][rows].view(torch.int32))
        assert torch.equal(fs["lse"].view(torch.int32), f["lse"][rows].view(torch.int32))


def test_in_place(gpu_lib):
    import gspo_logprob_gb300 as g
    rng = np.random.default_rng(10)
    n, V = 9, 5003
    b = _batch(rng, n, V)
    x = _values(rng, n, V, "bf16")
    sh = _shaping(b, n, V)
    z = _device(x, "bf16")
    want = g.grpo_shape_logits(z, sh)["logits"]
    got = g.grpo_shape_logits(z, sh, out=z)["logits"]
    assert got.data_ptr() == z.data_ptr() and torch.equal(got.view(torch.int16), want.view(torch.int16))
    z = _device(x, "bf16")
    y, m = (torch.from_numpy(t).cuda() for t in _targets(rng, n, V))
    f = g.grpo_shaped_logp(z, y, m, sh)
    coef = torch.ones(n, device="cuda")
    want = g.grpo_shaped_logp_backward(z, y, m, sh, f["lse"], coef)["dlogits"]
    got = g.grpo_shaped_logp_backward(z, y, m, sh, f["lse"], coef, dlogits=z)["dlogits"]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_nonfinite_logits(gpu_lib):
    # NaN, infinities and the type's lowest value in barred places are not seen; -inf elsewhere is a barred token;
    # NaN elsewhere spoils its own row only
    import gspo_logprob_gb300 as g
    from gspo_logprob_gb300 import _abi
    rng = np.random.default_rng(11)
    n, V = 8, 2000
    x = _values(rng, n, V, "bf16")
    bits = np.full((1, (V + 31) // 32), -1, np.int32)
    bits[0, 3] = 0                                              # tokens 96..127
    x[:, 96:128] = np.array([np.nan, np.inf, -np.inf, -3.3895314e38])[np.arange(32) % 4]
    x[1, 5] = -np.inf
    x[2, 7] = np.nan
    x[3, :] = -3.3895314e38                                     # the lowest finite bf16 everywhere
    b = dict(allow_bits=bits, allow_row=np.zeros(n, np.int32), temperature=np.ones(n, np.float32))
    y = np.array([0, 5, 0, 0, 100, 1, 2, -4], np.int32)
    m = np.ones(n, np.uint8)
    sh = _shaping(b, n, V)
    z = _device(x, "bf16")
    f = g.grpo_shaped_logp(z, torch.from_numpy(y).cuda(), torch.from_numpy(m).cuda(), sh)
    zp = so.shape_logits(x, b)[0]
    logp, lse = _np(f["logp"]), _np(f["lse"])
    assert np.isnan(logp[2]) and np.isnan(lse[2])
    keep = [0, 1, 3, 4, 5, 6, 7]
    want_logp, want_lse = so.shaped_logp(zp[keep], y[keep], m[keep])
    assert want_logp[1] == -np.inf and want_logp[3] == -np.inf and np.isnan(want_logp[-1])
    mag = np.where(np.isfinite(zp[keep]), np.abs(zp[keep]), 0)
    _check_logp(logp[keep], lse[keep], want_logp, want_lse, _lse_tol(mag, want_lse))
    word = int(f["status"].item())
    assert word == _abi.GH_DEV_TARGET_OOR | _abi.GH_DEV_NONFINITE
    s = _np(g.grpo_shape_logits(z, sh)["logits"])
    assert np.all(s[:, 96:128] == -np.inf) and s[1, 5] == -np.inf and np.isnan(s[2, 7])
    coef = torch.ones(n, device="cuda")
    dz = _np(g.grpo_shaped_logp_backward(z, torch.from_numpy(y).cuda(), torch.from_numpy(m).cuda(), sh, f["lse"],
                                         coef)["dlogits"])
    assert np.all(dz[:, 96:128] == 0) and np.all(np.isfinite(dz[[0, 1, 3, 4, 5, 6, 7]]))


def test_rows_outside_their_arrays_are_reported_and_left_out(gpu_lib):
    import gspo_logprob_gb300 as g
    from gspo_logprob_gb300 import _abi
    rng = np.random.default_rng(12)
    n, V = 16, 1500
    b = _batch(rng, n, V)
    T = b["tokens"].size
    b["hist_begin"][0], b["hist_len"][0] = T - 3, 4             # past the end
    b["hist_begin"][1] = -1
    b["hist_len"][2] = -5
    b["hist_begin"][3], b["hist_len"][3] = 2 ** 62, 2 ** 31 - 1
    b["repetition"][:4] = 1.5
    b["repetition"][4], b["repetition"][5], b["temperature"][6], b["temperature"][7] = 0, np.nan, -1, np.inf
    b["bias_set"][8], b["bias_set"][9] = 5, -2
    b["allow_row"][10], b["allow_row"][11] = 4, -7
    x = _values(rng, n, V, "fp32")
    zp, slope, mag, bad = so.shape_logits(x, b)
    assert np.array_equal(np.nonzero(bad)[0], np.arange(12))
    sh = _shaping(b, n, V)
    z = _device(x, "fp32")
    r = g.grpo_shape_logits(z, sh)
    _check_shape(_np(r["logits"]), zp, mag, "fp32")
    assert int(r["status"].item()) == _abi.GH_DEV_BAD_ROW
    y, m = np.zeros(n, np.int32), np.ones(n, np.uint8)
    f = g.grpo_shaped_logp(z, torch.from_numpy(y).cuda(), torch.from_numpy(m).cuda(), sh)
    wl, ws = so.shaped_logp(zp, y, m)
    _check_logp(_np(f["logp"]), _np(f["lse"]), wl, ws, _lse_tol(mag, ws))
    # bias offsets that are not bounds of the list
    b2 = _batch(rng, 2, V, features=("bias",))
    b2["bias_offsets"] = np.array([0, 10 ** 9, -3], np.int32)
    b2["bias_set"] = np.array([0, 1], np.int32)
    r = g.grpo_shape_logits(z[:2], _shaping(b2, 2, V))
    assert int(r["status"].item()) == _abi.GH_DEV_BAD_ROW
    assert torch.equal(r["logits"], z[:2])


def test_longest_bias_list(gpu_lib):
    rng = np.random.default_rng(13)
    V = 9000
    b = dict(bias_offsets=np.array([0, so.MAX_BIAS], np.int32),
             bias_tokens=rng.permutation(V)[:so.MAX_BIAS].astype(np.int32),
             bias_values=rng.uniform(-9, 9, so.MAX_BIAS).astype(np.float32), bias_set=np.zeros(2, np.int32))
    y, m = _targets(rng, 2, V)
    _run_all(b, _values(rng, 2, V, "bf16"), y, m, "bf16")


def test_gradient_by_differences_of_the_kernel(gpu_lib):
    # the fp32 kernel's own log-prob, differenced: central differences with h = 2^-6 have an error of
    # h^2 / 6 times a third derivative below 1 (4.1e-5) and rounding 2 (LSE tolerance) / 2h
    import gspo_logprob_gb300 as g
    rng = np.random.default_rng(14)
    V = 300
    h = 2.0 ** -6
    x = (rng.standard_normal(V) * 2).astype(np.float32)
    x[np.abs(x) < 2 * h] += 4 * h                               # stay clear of the penalty's kink
    one = _batch(rng, 1, V, hist=60, features=("hist", "bias", "temp"))
    one["repetition"][:], one["hist_len"][:] = 1.3, one["tokens"].size
    one["hist_begin"][:], one["temperature"][:] = 0, 0.8
    n = 2 * V
    rep = {k: (np.repeat(v, n) if v.shape == (1,) and k not in ("tokens", "bias_tokens", "bias_values") else v)
           for k, v in one.items()}
    X = np.repeat(x[None], n, 0)
    X[np.arange(V), np.arange(V)] += h
    X[V + np.arange(V), np.arange(V)] -= h
    y, m = np.full(n, 17, np.int32), np.ones(n, np.uint8)
    lp = _np(g.grpo_shaped_logp(_device(X, "fp32"), torch.from_numpy(y).cuda(), torch.from_numpy(m).cuda(),
                                _shaping(rep, n, V))["logp"])
    diff = (lp[:V] - lp[V:]) / (2 * h)
    sh = _shaping(one, 1, V)
    z = _device(x[None], "fp32")
    f = g.grpo_shaped_logp(z, torch.from_numpy(y[:1]).cuda(), torch.from_numpy(m[:1]).cuda(), sh)
    dz = _np(g.grpo_shaped_logp_backward(z, torch.from_numpy(y[:1]).cuda(), torch.from_numpy(m[:1]).cuda(), sh,
                                         f["lse"], torch.ones(1, device="cuda"))["dlogits"])[0]
    mag = so.shape_logits(x[None], one)[2]
    tol = 5 * h * h / 6 + 3 * float(_lse_tol(mag, _np(f["lse"]))[0]) / h     # slope up to 1.3 / 0.8: its cube is below 5
    assert np.max(np.abs(dz - diff)) <= tol


def test_status_streams_graphs_and_refusals(gpu_lib):
    import gspo_logprob_gb300 as g
    from gspo_logprob_gb300 import ops
    rng = np.random.default_rng(15)
    n, V = 5, 3000
    b = _batch(rng, n, V)
    x = _values(rng, n, V, "bf16")
    sh = _shaping(b, n, V)
    z = _device(x, "bf16")
    y, m = (torch.from_numpy(t).cuda() for t in _targets(rng, n, V))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(sh.workspace_bytes, dtype=torch.uint8, device="cuda")
    want = g.grpo_shaped_logp(z, y, m, sh)
    # another stream than the tensors' own, and a captured step replayed after the batch changed in place
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = {}
    with torch.cuda.stream(side):
        for _ in range(2):
            out = g.grpo_shaped_logp(z, y, m, sh, status=st, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out["logp"].view(torch.int32), want["logp"].view(torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.grpo_shaped_logp(z, y, m, sh, status=st, workspace=ws, out=out)
    sh.tensors["hist_len"].zero_()
    z.mul_(0.5)
    graph.replay()
    want = g.grpo_shaped_logp(z, y, m, sh)
    assert torch.equal(out["logp"].view(torch.int32), want["logp"].view(torch.int32))
    assert torch.equal(out["lse"].view(torch.int32), want["lse"].view(torch.int32))
    # refusals
    with pytest.raises(ValueError, match="shape"):
        g.grpo_shape_logits(z[:, 1:], sh)
    with pytest.raises(ValueError, match="contiguous rows"):
        g.grpo_shape_logits(torch.empty(V, n, dtype=torch.bfloat16, device="cuda").t(), sh)
    with pytest.raises(ValueError, match="overlap"):
        g.grpo_shape_logits(z[:1].expand(n, V), sh)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        g.grpo_shape_logits(z.half(), sh)
    big = torch.empty(n * V + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(g.ops._abi.GhError, match="overlaps"):
        g.grpo_shape_logits(big[:n * V].view(n, V), sh, out=big[8:].view(n, V))
    with pytest.raises(ValueError, match="workspace holds"):
        g.grpo_shaped_logp(z, y, m, sh, workspace=ws[:16])
    with pytest.raises(ValueError, match="together"):
        g.make_shaping(n, V, hist_len=b["hist_len"])
    with pytest.raises(ValueError, match="allow_bits"):
        g.make_shaping(n, V, allow_bits=torch.zeros(1, 3, dtype=torch.int32, device="cuda"),
                       allow_row=torch.zeros(n, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="temperature"):
        g.make_shaping(n, V, temperature=torch.ones(n, dtype=torch.float64, device="cuda"))
    # no rows: nothing to do
    e = g.make_shaping(0, V)
    assert g.grpo_shape_logits(z[:0], e)["logits"].shape == (0, V)
    assert ops.raise_on_status(g.grpo_shaped_logp(z[:0], y[:0], m[:0], e)["status"]) == 0


def test_row_offsets_past_32_bits(gpu_lib):
    # rows 2^31 elements apart: the last row starts past 2^32 bytes and 2^31 elements
    import gspo_logprob_gb300 as g
    V, ld, n = 1003, (1 << 31) + 8, 3
    rng = np.random.default_rng(16)
    b = _batch(rng, n, V)
    x = _values(rng, n, V, "bf16")
    sh = _shaping(b, n, V)
    flat = torch.empty((n - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(flat, (n, V), (ld, 1))
    z.copy_(torch.from_numpy(x).cuda())
    got = g.grpo_shape_logits(z, sh, out=z)["logits"]
    want = g.grpo_shape_logits(_device(x, "bf16"), sh)["logits"]
    assert torch.equal(got.contiguous().view(torch.int16), want.view(torch.int16))

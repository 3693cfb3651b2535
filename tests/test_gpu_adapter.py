"""Head logits with low-rank adapters against the fp64 oracle.

Tolerances, with eps = 2^-24 and M the sum of the absolute terms of a logit:
 * products of bf16 values are exact in fp32; the sums of K terms in fp32 are
   within K eps M of exact in the worst case and sqrt(K) eps M typically: 4
   sqrt(D + rank) eps M is allowed (tensor cores may align a group of products
   before they add it: the factor 4);
 * u is carried in two or three bf16 terms: 2^-16 of the adapter's part, at most M;
   fp32 calls have neither and the same sum bound;
 * a bf16 output: half an ulp, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from oracle.adapter_oracle import adapter_logits
from synth import bf16_bits_to_f32, f32_to_bf16_bits

from gpu_helpers import gpu_lib  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _draw(rng, shape, std, dtype):
    x = (rng.standard_normal(shape) * std).astype(np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)) if dtype == "bf16" else x


def _problem(n, D, V, adapters, rank, dtype, seed, prompts=False):
    rng = np.random.default_rng(seed)
    p = dict(H=_draw(rng, (n, D), 1.0, dtype), W=_draw(rng, (V, D), D ** -0.5, dtype),
             A=_draw(rng, (adapters, rank, D), D ** -0.5, dtype), B=_draw(rng, (adapters, V, rank), rank ** -0.5, dtype),
             scale=rng.uniform(-2, 2, adapters).astype(np.float32),
             adapter_id=rng.integers(-1, adapters, n).astype(np.int32))
    if prompts:
        p["adapter_id"] = np.sort(p["adapter_id"])
    return p


def _device(p, dtype):
    d = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in p.items()}
    for k in ("H", "W", "A", "B"):
        d[k] = d[k].to(TYPES[dtype])
    return d


def _check(got, p, dtype, out):
    want, mag, _ = adapter_logits(**p)
    D, r = p["H"].shape[1], p["A"].shape[1]
    tol = 4 * np.sqrt(D + r) * EPS * mag + (2.0 ** -16 * mag if dtype == "bf16" else 0)
    if out == "bf16":
        tol = tol + 2.0 ** -8 * 1.01 * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol + 1e-30), float(np.max(err - tol))


# n, D, V, adapters, rank: one token to several row tiles, ragged everything
_CASES = [
    (1, 8, 1, 1, 8), (1, 64, 40, 1, 16), (1, 1024, 5000, 4, 16), (7, 72, 300, 3, 8), (37, 1000, 5000, 5, 8),
    (64, 256, 1025, 16, 16), (127, 136, 77, 40, 24), (128, 64, 513, 128, 8), (129, 128, 600, 3, 32),
    (256, 200, 1000, 200, 16), (300, 320, 999, 7, 40), (1100, 256, 700, 5, 64), (1031, 64, 257, 9, 256),
]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("n,D,V,adapters,rank", _CASES)
def test_against_oracle(gpu_lib, n, D, V, adapters, rank, out):
    import gspo_logprob_gb300 as g
    p = _problem(n, D, V, adapters, rank, "bf16", n + V, prompts=n > 1000)
    r = g.grpo_adapter_logits(**_device(p, "bf16"), out_dtype=TYPES[out])
    assert r["logits"].shape == (n, V) and int(r["status"].item()) == 0
    _check(r["logits"], p, "bf16", out)


@pytest.mark.parametrize("n,D,V,adapters,rank", [(1, 5, 3, 1, 1), (9, 65, 130, 3, 7), (70, 300, 401, 6, 16)])
def test_fp32(gpu_lib, n, D, V, adapters, rank):
    import gspo_logprob_gb300 as g
    p = _problem(n, D, V, adapters, rank, "fp32", n)
    r = g.grpo_adapter_logits(**_device(p, "fp32"))
    assert r["logits"].dtype == torch.float32
    _check(r["logits"], p, "fp32", "fp32")


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_output_strides(gpu_lib, n, out):
    # rows off 16-byte boundaries, a gap between rows that stays as it was
    import gspo_logprob_gb300 as g
    p = _problem(n, 128, 203, 4, 16, "bf16", n)
    for ld, shift in ((203, 0), (208, 0), (211, 1)):
        flat = torch.full((n * ld + shift,), 7.0, dtype=TYPES[out], device="cuda")
        z = torch.as_strided(flat, (n, 203), (ld, 1), shift)
        g.grpo_adapter_logits(**_device(p, "bf16"), logits=z)
        _check(z, p, "bf16", out)
        gap = torch.as_strided(flat, (n - 1, ld - 203), (ld, 1), shift + 203) if ld > 203 else flat[:0]
        assert torch.all(gap == 7.0)


def test_adapters_all_none_and_one(gpu_lib):
    import gspo_logprob_gb300 as g
    p = _problem(40, 256, 500, 3, 16, "bf16", 5)
    for ids in (np.full(40, -1), np.full(40, 2)):
        p["adapter_id"] = ids.astype(np.int32)
        _check(g.grpo_adapter_logits(**_device(p, "bf16"), out_dtype=torch.float32)["logits"], p, "bf16", "fp32")


def test_bad_ids_are_reported_and_left_out(gpu_lib):
    import gspo_logprob_gb300 as g
    from gspo_logprob_gb300 import _abi
    for n, dtype in ((20, "bf16"), (400, "bf16"), (20, "fp32")):
        p = _problem(n, 64, 100, 3, 8, dtype, 6)
        p["adapter_id"][[0, n - 1]] = [3, -2]
        p["adapter_id"][n // 2] = 2 ** 31 - 1
        r = g.grpo_adapter_logits(**_device(p, dtype), out_dtype=torch.float32)
        assert int(r["status"].item()) == _abi.GH_DEV_BAD_ROW
        _check(r["logits"], p, dtype, "fp32")


def test_nonfinite_rows_stay_their_own(gpu_lib):
    import gspo_logprob_gb300 as g
    p = _problem(150, 64, 90, 3, 8, "bf16", 7)
    ref = g.grpo_adapter_logits(**_device(p, "bf16"), out_dtype=torch.float32)["logits"].clone()
    p["H"][3, 5], p["H"][140, 0] = np.nan, np.inf
    z = g.grpo_adapter_logits(**_device(p, "bf16"), out_dtype=torch.float32)["logits"]
    keep = torch.ones(150, dtype=torch.bool, device="cuda")
    keep[[3, 140]] = False
    assert torch.equal(z[keep], ref[keep])
    assert torch.isnan(z[3]).all() and not torch.isfinite(z[140]).any()


def test_rows_do_not_depend_on_the_batch(gpu_lib):
    # another tile form, other neighbours, other slots: the same bits
    import gspo_logprob_gb300 as g
    p = _problem(300, 512, 1000, 9, 16, "bf16", 8)
    d = _device(p, "bf16")
    whole = g.grpo_adapter_logits(**d, out_dtype=torch.float32)["logits"]
    for rows in (slice(0, 1), slice(40, 168), slice(290, 300)):
        part = dict(d, H=d["H"][rows].contiguous(), adapter_id=d["adapter_id"][rows].contiguous())
        assert torch.equal(g.grpo_adapter_logits(**part, out_dtype=torch.float32)["logits"], whole[rows])


@pytest.mark.parametrize("n,V,rank", [(5, 50000, 8), (64, 60000, 16), (300, 45000, 32), (1500, 9000, 16)])
def test_calls_queued_one_behind_the_other(gpu_lib, n, V, rank):
    # many tiles per CTA, and calls on different rows and adapters that nothing waits between: each call's u and list
    # take the workspace over from the call before
    import gspo_logprob_gb300 as g
    p = _problem(n, 64, V, 6, rank, "bf16", n)
    d = _device(p, "bf16")
    rng = np.random.default_rng(n)
    sets = []
    for k in range(5):
        q = dict(p, H=_draw(rng, (n, 64), 1.0, "bf16"),
                 adapter_id=np.sort(rng.integers(-1, 6, n)).astype(np.int32) if k % 2 else
                 rng.integers(-1, 6, n).astype(np.int32))
        sets.append((q, dict(d, H=torch.from_numpy(q["H"]).cuda().bfloat16(),
                             adapter_id=torch.from_numpy(q["adapter_id"]).cuda())))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    out = [g.grpo_adapter_logits(**s, status=st)["logits"] for _, s in sets + sets]
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for k in range(5):
        assert torch.equal(out[k], out[k + 5])
        alone = g.grpo_adapter_logits(**sets[k][1])["logits"]
        torch.cuda.synchronize()
        assert torch.equal(out[k], alone)
    _check(out[0], sets[0][0], "bf16", "bf16")


def test_graph_stream_and_refusals(gpu_lib):
    import gspo_logprob_gb300 as g
    p = _problem(30, 128, 400, 4, 16, "bf16", 9)
    d = _device(p, "bf16")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = torch.empty(30, 400, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.grpo_adapter_logits(**d, logits=z, workspace=ws, status=st)
    torch.cuda.current_stream().wait_stream(side)
    _check(z, p, "bf16", "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.grpo_adapter_logits(**d, logits=z, workspace=ws, status=st)
    p["adapter_id"] = np.roll(p["adapter_id"], 3)
    d["adapter_id"].copy_(torch.from_numpy(p["adapter_id"]))
    z.zero_()
    graph.replay()
    _check(z, p, "bf16", "bf16")
    with pytest.raises(ValueError, match="workspace holds"):
        g.grpo_adapter_logits(**d, workspace=ws[:64])
    with pytest.raises(ValueError, match="A must be|shape"):
        g.grpo_adapter_logits(**dict(d, A=d["A"][:, :, :64]))
    with pytest.raises(ValueError, match="shape"):
        g.grpo_adapter_logits(**dict(d, B=d["B"][:, :100].contiguous()))
    with pytest.raises(TypeError, match="adapter_id"):
        g.grpo_adapter_logits(**dict(d, adapter_id=d["adapter_id"].long()))
    with pytest.raises(TypeError, match="W must be"):
        g.grpo_adapter_logits(**dict(d, W=d["W"].float()))
    with pytest.raises(g.ops._abi.GhError, match="rank % 8"):
        g.grpo_adapter_logits(**dict(d, A=d["A"][:, :5].contiguous(), B=d["B"][:, :, :5].contiguous()))
    e = g.grpo_adapter_logits(**dict(d, H=d["H"][:0], adapter_id=d["adapter_id"][:0]))
    assert e["logits"].shape == (0, 400)

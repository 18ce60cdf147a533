"""How close the float parts come to 64 bits, in bounds that a product or a weight of fewer bits
(2^-11 and coarser) breaks by two orders.

Attention, fp32, norm-wise over the rows of a sequence: with q and k of unit variance the partial
sums of a score's D terms grow as the root of their number, so their roundings add up to about
0.41 sqrt(D) u of the score in units of sqrt(D), and with the scale 1/sqrt(D) to 0.41 sqrt(D) u of
a weight's exponent (u = 2^-24).  The score's scaling and the difference to the maximum (of size 2
to 10), the exponential (2 ulp), the step's chain of 64 products and the joins add 8 u at most,
taken together as independent errors.  Output and log-sum-exp are averages of such errors; the
bound is four times them: 4 (0.41 sqrt(D) + 8) u of the norm, 45 u to 58 u.

Rotation: per pair, 2^-19 of the pair's own size (2^-19 = 32 u: the norm's sum of squares in
chains of at most 15 additions, halved by the root, its reciprocal root, three products and a
sum); an element that is not rotated by its own size; bf16 adds its rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import AttentionPlan, _lib  # noqa: E402
from oracle import attention_oracle as O  # noqa: E402
from test_gpu_attention import ROPE, Case, U, f64, rope_inputs  # noqa: E402


@pytest.mark.parametrize("shape", [
    dict(new=(40, 1, 17), length=(300, 77, 1000)),
    dict(new=(64, 30), length=(500, 90), window=50),
    dict(new=(200,), length=(200,), heads=4, heads_kv=4),
    dict(new=(33, 20), length=(100, 400), causal=False),
    dict(new=(25, 60), length=(90, 200), causal=False, window=70, heads=6, heads_kv=2),
    dict(new=(1, 2, 3), length=(700, 90, 4000)),
    dict(new=(1, 3), length=(1500, 60), window=200, heads=8, heads_kv=2),
], ids=["chunks", "window", "prefill", "full", "full_window", "few", "few_window"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_fp32_attention_is_as_close_as_float(D, shape):
    c = Case(seed=41, dtype="f32", D=D, page=32, **shape)
    out, lse = (f64(t) for t in c.run())
    ref, ref_lse, _ = O.attention(f64(c.q), c.k.double().numpy(), c.v.double().numpy(), c.start, c.length, c.table,
                                  D ** -0.5, c.causal, c.window)
    bound = 4 * (0.41 * D ** 0.5 + 8) * U
    for b in range(len(c.length)):
        rows = slice(c.start[b], c.start[b + 1])
        assert np.linalg.norm(out[rows] - ref[rows]) <= bound * np.linalg.norm(ref[rows]), b
        assert np.linalg.norm(lse[rows] - ref_lse[rows]) <= bound * np.linalg.norm(1 + np.abs(ref_lse[rows])), b
    assert c.plan.get_error()[0] == _lib.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["halves", "adjacent"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", ROPE, ids=[str(i) for i in range(len(ROPE))])
def test_rotation_is_as_close_as_float_pair_by_pair(shape, norm, style, dtype):
    H, Hkv, D, r = shape["heads"], shape["heads_kv"], shape["D"], shape["r"]
    q, k, _, gq, gk = rope_inputs(dtype, H, Hkv, D, 150, 51)
    plan = AttentionPlan(heads=H, heads_kv=Hkv, head_dim=D, dtype=dtype, rotary_dim=r, rope_style=style)
    rope = plan.rope_table(500) if r else None
    pos = torch.randint(0, 500, (150,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    got = plan.qk_norm_rope(q, k, pos if r else None, rope, g_q=gq if norm else None, g_k=gk if norm else None)
    lo = np.arange(0, r, 2) if style == "adjacent" else np.arange(r // 2)
    hi = lo + 1 if style == "adjacent" else lo + r // 2
    for y, x, g in zip(got, (q, k), (gq, gk)):
        ref = O.norm_rope(f64(x), f64(g) if norm else None, plan.eps, pos.cpu().numpy(),
                          rope.cpu().numpy() if r else None, style == "adjacent")
        size = np.abs(ref)
        size[..., lo] = size[..., hi] = np.hypot(ref[..., lo], ref[..., hi])
        bound = 2.0 ** -19 * size + (2.0 ** -8 * 1.001 * np.abs(ref) if dtype == "bf16" else 0) + 1e-30
        worst = (np.abs(f64(y) - ref) / bound).max()
        assert worst <= 1.0, f"{worst:.3g} of its bound"
    assert plan.get_error()[0] == _lib.OK

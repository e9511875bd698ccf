"""Inputs and comparisons of the sequence and tree tests.

Tolerances.  Device results are float32 chains of products summed in float32: a dot
product of n terms is off by at most about sqrt(n) 2^-24 of its terms' norm (rounding
errors of either sign), a product of up to 64 decays by 64 2^-24, and a result passes
through at most six such products, 6 (sqrt(128) + 64) 2^-24 < 3e-5 if all of them leaned
one way.  F32 = 2e-5 of the norm is below that; a value then rounded to a 16-bit type is
off by at most half a step more, eps / 2 of itself.
"""

import numpy as np
import torch

from workloads import FORM_GDN, FORM_KDA, FORM_MAMBA2

F32 = 2e-5
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FORMS = {"gdn": FORM_GDN, "kda": FORM_KDA, "mamba2": FORM_MAMBA2}


def close(got, ref, what=""):
    """Relative Frobenius error within the type's half step plus F32."""
    eps = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    x = got.double().cpu().numpy()
    assert np.isfinite(x).all(), f"{what}: not finite"
    ref = np.asarray(ref, dtype=np.float64)
    den = np.linalg.norm(ref)
    err = np.linalg.norm(x.reshape(ref.shape) - ref)
    assert err <= (F32 + eps) * den + 1e-30, f"{what}: {err / max(den, 1e-300):.3e} > {F32 + eps:.1e}"


def token_values(form, shape, h_k, h, dk, dv, rng):
    """q, k (*shape, h_k, dk), v, alpha, beta as the synthetic workloads draw them."""
    q, k = rng.normal(size=(2, *shape, h_k, dk))
    v = rng.normal(size=(*shape, h, dv)) + 1.0
    if form == FORM_MAMBA2:
        q, k = q / dk ** 0.5, k / dk ** 0.5
        beta = np.log1p(np.exp(-2 + 0.5 * rng.normal(size=(*shape, h))))
        alpha = np.exp(-beta * rng.uniform(1, 16, size=h))
    else:
        q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
        beta = 1 / (1 + np.exp(-rng.normal(size=(*shape, h))))
        if form == FORM_GDN:
            alpha = np.exp(-np.log1p(np.exp(-3 + 0.5 * rng.normal(size=(*shape, h)))))
        else:
            alpha = rng.uniform(0.85, 1.0, size=(*shape, h, dk))
    return q, k, v, alpha, beta


def device(x, dtype=torch.float32):
    """x rounded to dtype on the GPU, and the float64 values it then holds."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
    return t.cuda(), t.double().numpy()

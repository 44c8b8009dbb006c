"""kvc_chunk_attn, and the form of kvc_q8_attn that goes through it, with scores far above one: every key
of a (b, l, h) is the same, so that its scores are equal, in whichever tile they stand."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import DT, EPS, Chunk
from tests.test_gpu_q8_large_scores import _check_averages, _run, _same_keys

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


MODS = {"plain": {}, "window": dict(window=2.0 ** 30), "cap": dict(softcap=2.0 ** 40)}


@pytest.mark.parametrize("power", [16, 26, 28, 31])
@pytest.mark.parametrize("n,dtype", [(1, "bf16"), (9, "bf16"), (70, "bf16"), (9, "f32")])
@pytest.mark.parametrize("mod", list(MODS))
def test_equal_scores_in_all_tiles(kvc, mod, n, dtype, power):
    """out is the average of the values seen: the numerators are equal, each rounded (bf16: 2^-8, the
    same way, while their sum is of unrounded ones), and the fp32 sums of N values and numerators and the result are
    rounded.  lse is the score and log2 N, to the score's error and the sum's."""
    c = Chunk(kvc, np.linspace(2500, 4500, 32), [n] * 2, B=2, H=16, dtype=dtype, seed=power, **MODS[mod])
    rng = np.random.default_rng(power)
    key = torch.from_numpy(rng.choice([-1.0, 1.0], c.d) * rng.uniform(0.5, 2.0, c.d)).to(DT[dtype])
    c.q = (c.q.double() * 2.0 ** power).to(c.q.dtype)
    c.k_new[:] = key
    for u in range(32):                                    # several tiles a CTA
        r = c.rows(u, int(c.lens[u]))
        c.K[r], c.logm[r] = key, 0.0
    s = c.upload()
    c.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    rounded = EPS["bf16"] if dtype == "bf16" else 0.0
    out, lse = s["out"].double().cpu().numpy(), s["lse"].double().cpu().numpy()
    for u in c.units:
        K, V, lm, pos, q, (b, lr, hs, n_b, n0) = c.entries(u)
        sc = q @ key.double().numpy() / np.sqrt(c.d)
        dots = np.abs(q) @ np.abs(key.double().numpy()) / np.sqrt(c.d)
        if c.softcap:
            sc = c.softcap * np.tanh(sc / c.softcap)
        for t in {0, n_b // 2, n_b - 1}:
            N = n0 + t + 1
            o, size = V[:N].mean(0), np.abs(V[:N]).mean(0)
            tol = (N * 2.0 ** -23 + 2.0 ** -20 + rounded) * size + (N * 2.0 ** -24 + 2.0 ** -21 + 1.01 * EPS[dtype]) * np.abs(o) + 1e-30
            err = np.abs(out[b, lr, hs, t] - o)
            assert (err <= tol).all(), (u, t, err.max(), (err / tol).max())
            tol_l = ((c.d * 2.0 ** -23 + 2.0 ** -20) * dots[:, t] + 2.0 ** -20) / np.log(2)
            assert (np.abs(lse[b, lr, hs, t] - (sc[:, t] / np.log(2) + np.log2(N))) <= tol_l).all(), (u, t)


@pytest.mark.parametrize("power", [23, 26, 28, 31])
def test_equal_scores_over_expanded_rows(kvc, power):
    c, pick = _same_keys(kvc, "expanded", "bf16", 5 + power, power, v_exps=(0, -1, -3, -2, 0, 2, 1, -1))
    _check_averages(c, *_run(c, pick), numerator=EPS["bf16"])

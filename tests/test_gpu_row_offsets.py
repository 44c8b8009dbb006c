"""Row offsets of any 64-bit size: a (b, l, h) whose rows lie outside the cache is skipped and reported,
whatever its offset and length add up to; the others are served."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import Chunk

pytestmark = pytest.mark.gpu

OFFSETS = [2 ** 63 - 1, 2 ** 63 - 95, 2 ** 62, -2 ** 63, -1]


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


def _done(kvc, code):
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == code


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", OFFSETS)
def test_chunk_attention_and_mass(kvc, off, dtype):
    ch = Chunk(kvc, [100, 90, 300, 64], [5, 3], B=2, H=2, dtype=dtype)
    good, s = ch.upload(), ch.upload()
    s["off"].view(-1)[1] = off
    ch.attn(good)
    _done(kvc, 0)
    ch.attn(s)
    _done(kvc, kvc.KVC_EDEVICE)
    assert (s["out"][0, 0, 4:] == 7.0).all() and s["len_out"][0, 0, 1] == 90
    assert torch.equal(s["out"][0, 0, :4], good["out"][0, 0, :4]) and torch.equal(s["out"][1], good["out"][1])
    s["lse"].copy_(good["lse"])
    ch.run_mass(good, 0.5)
    _done(kvc, 0)
    ch.run_mass(s, 0.5)
    _done(kvc, kvc.KVC_EDEVICE)
    for u in (0, 2, 3):
        r = torch.from_numpy(ch.rows(u, int(ch.lens[u]))).cuda()
        assert torch.equal(s["mass"][r], good["mass"][r]), u
    r = torch.from_numpy(ch.rows(1, 90)).cuda()
    np.testing.assert_array_equal(s["mass"][r].cpu().numpy(), ch.mass[ch.rows(1, 90)])


@pytest.mark.parametrize("off", OFFSETS)
def test_mass_eviction(kvc, off):
    ch = Chunk(kvc, [700, 300, 64, 90], [0], H=4, T=1)
    s = ch.upload()
    s["off"].view(-1)[1] = off
    before = s["mass"].clone()
    keep = torch.tensor([350, 100, 32, 45], dtype=torch.int32, device="cuda").view(1, 1, 4)
    ws = torch.empty(kvc.kvc_mass_evict_workspace_bytes(s["p"], s["c"], 700), dtype=torch.uint8, device="cuda")
    kvc.kvc_mass_evict(s["p"], s["c"], s["mass"], keep, 4, s["pos_new"], s["K"], s["V"], s["logm"], s["pos"], s["len"],
                       s["off"], s["len_out"], 700, ws)
    _done(kvc, kvc.KVC_EDEVICE)
    assert s["len_out"].view(-1).tolist() == [350, 300, 32, 45]
    r = torch.from_numpy(ch.rows(1, 300)).cuda()
    assert torch.equal(s["mass"][r], before[r])


@pytest.mark.parametrize("off", OFFSETS)
def test_decode(kvc, off):
    """The bf16 form, which checks rows against the extent."""
    ch = Chunk(kvc, [100, 90, 300, 64], [1], H=4, reserve=4)
    outs = []
    for bad in (False, True):
        s = ch.upload()
        if bad:
            s["off"].view(-1)[1] = off
        ws = kvc.workspace(kvc.KVC_WS_DECODE, s["p"], zero=True)
        q, k, v = (s[n][:, :, :, 0].contiguous() for n in ("q", "k_new", "v_new"))
        out = torch.full_like(q, 7.0)
        kvc.kvc_decode_attn(s["p"], q, k, v, None, s["K"], s["V"], s["logm"], s["pos"], s["len"], s["cap"], s["off"], out, ws)
        _done(kvc, kvc.KVC_EDEVICE if bad else 0)
        outs.append((out, s["len"].view(-1).tolist()))
    (a, n0), (b, n1) = outs
    assert n0 == [101, 91, 301, 65] and n1 == [101, 90, 301, 65]
    assert (b[0, 0, 4:8] == 7.0).all()
    assert torch.equal(a[0, 0, :4], b[0, 0, :4]) and torch.equal(a[0, 0, 8:], b[0, 0, 8:])

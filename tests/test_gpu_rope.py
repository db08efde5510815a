"""GPU parity of rope_append against its float64 form.

Tolerances, per element: the fraction of a turn is rounded once to float32 (at most 2^-25 half turns,
1.6 * 2^-24 radians), cos and sin are good to 2 units in the last place (2^-23 at most 1), times the
magnitude, two products and a sum round once each: at most 8 * 2^-24 * magnitude * (|x| + |y|); a
bfloat16 result adds half a step, 2^-8 relative.
"""
import pytest
import torch

from _parity import Guarded, check_guards, gpu_or_skip, is_poison
from _plain64 import rope, rope_radians
from long_context_speculative_split_gb300 import mgd, ops

pytestmark = pytest.mark.gpu

SCALINGS = {
    "plain": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=8.0),
    "llama3": dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_len=8192),
    "yarn": dict(kind="yarn", factor=16.0, beta_fast=32.0, beta_slow=1.0, original_len=4096),
}


def _fused(dev, B, T, Hq, Hkv, D, dtype, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((B, T, Hq + 2 * Hkv, D), generator=g, device=dev).to(dtype)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]


def _expect(x, pos, inv, mag, interleaved, got):
    ref = rope(x, pos, inv, mag, interleaved)
    half = len(inv)
    i0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    size = torch.zeros_like(ref)
    size[..., i0] = size[..., i1] = x.double()[..., i0].abs() + x.double()[..., i1].abs()
    tol = 8 * 2.0 ** -24 * mag * size + (2.0 ** -8 * ref.abs() if got.dtype == torch.bfloat16 else 0.0)
    assert bool(((got.double() - ref).abs() <= tol).all()), float(((got.double() - ref).abs() - tol).max())


def _run(dev, B, T, Hq, Hkv, D, rot, cap, dtype, interleaved, scaling, base=10000.0, lens=None, new=None, offset=None,
         seed=0):
    q, kn, vn = _fused(dev, B, T, Hq, Hkv, D, dtype, seed)
    new = [T] * B if new is None else new
    lens = [cap] * B if lens is None else lens
    i32 = dict(dtype=torch.int32, device=dev)
    k, v, qo = (Guarded(s, dtype, dev) for s in ((B, Hkv, cap, D), (B, Hkv, cap, D), (B, T, Hq, D)))
    ws = ops.workspace(mgd.mgd_rope_workspace_size(B), dev)
    table = ops.rope_table(rot, base, SCALINGS[scaling], device=dev)
    off = None if offset is None else torch.tensor(offset, **i32)
    ops.rope_append(q, kn, vn, table, k.t, v.t, torch.tensor(lens, **i32), new_len=torch.tensor(new, **i32),
                    pos_offset=off, interleaved=interleaved, q_out=qo.t, ws=ws)
    assert mgd.mgd_workspace_errors(ws) == 0
    check_guards(k=k, v=v, q_out=qo)
    inv, mag = rope_radians(rot, base, SCALINGS[scaling])
    for b in range(B):
        n, start = new[b], lens[b] - new[b]
        o = 0 if offset is None else offset[b % len(offset)]
        pos = torch.arange(start + o, start + o + n, device=dev)
        _expect(q[b, :n], pos, inv, mag, interleaved, qo.t[b, :n])
        _expect(kn[b, :n], pos, inv, mag, interleaved, k.t[b, :, start:start + n].transpose(0, 1))
        assert torch.equal(v.t[b, :, start:start + n].transpose(0, 1), vn[b, :n])
        assert bool(is_poison(qo.t[b, n:]).all()), "rows past new_len were written"
        for c in (k.t, v.t):
            assert bool(is_poison(c[b, :, :start]).all()) and bool(is_poison(c[b, :, lens[b]:]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot", [
    (1, 1, 1, 1, 64, 64), (3, 5, 32, 8, 128, 128), (2, 7, 6, 2, 128, 64), (2, 3, 4, 4, 64, 16), (2, 2, 3, 1, 80, 20),
    (1, 9, 5, 5, 72, 2), (2, 33, 8, 1, 256, 256), (1, 3, 2, 2, 96, 96), (1, 2, 2, 1, 64, 6)])
def test_layouts_and_types(B, T, Hq, Hkv, D, rot, interleaved, dtype):
    dev = gpu_or_skip()
    _run(dev, B, T, Hq, Hkv, D, rot, T + 5, dtype, interleaved, "plain", lens=[T + b for b in range(B)], seed=T)


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("offset", [[0], [131072], [1000003], [2 ** 31 - 200], [-50]], ids=lambda o: "at%d" % o[0])
def test_scalings_at_near_and_far_positions(scaling, offset):
    """Positions up to 2^31: a float32 angle there would be off by hundreds of radians."""
    dev = gpu_or_skip()
    _run(dev, 2, 6, 4, 2, 128, 128, 60, torch.float32, False, scaling, base=500000.0, lens=[60, 6], offset=offset)


def test_ragged_batches_with_their_own_offsets():
    dev = gpu_or_skip()
    _run(dev, 5, 9, 8, 2, 64, 64, 40, torch.bfloat16, False, "llama3", lens=[9, 40, 3, 0, 17], new=[9, 1, 3, 0, 5],
         offset=[0, 100, 7, 5, 32768])


def test_a_long_prefill():
    dev = gpu_or_skip()
    _run(dev, 2, 4100, 8, 2, 128, 128, 5000, torch.bfloat16, True, "yarn", lens=[4100, 4777], new=[4099, 4100])


def test_one_token_each_of_a_large_batch():
    dev = gpu_or_skip()
    B = 700
    _run(dev, B, 1, 8, 2, 64, 64, 20, torch.bfloat16, False, "plain", lens=[1 + b % 20 for b in range(B)])


def test_bad_sequences_are_flagged_and_untouched():
    dev = gpu_or_skip()
    B, T, Hq, Hkv, D, cap = 4, 3, 4, 2, 64, 16
    q, kn, vn = _fused(dev, B, T, Hq, Hkv, D, torch.bfloat16, 1)
    table = ops.rope_table(64, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    for lens, new in (([5, 17, 5, 5], [3] * 4), ([5, 2, 5, 5], [3] * 4), ([5, 5, 5, 5], [3, 4, 3, 3]),
                      ([5, 5, 5, 5], [3, -1, 3, 3]), ([5, -1, 5, 5], [3, 0, 3, 3])):
        k, v = Guarded((B, Hkv, cap, D), torch.bfloat16, dev), Guarded((B, Hkv, cap, D), torch.bfloat16, dev)
        qo = Guarded((B, T, Hq, D), torch.bfloat16, dev)
        ws = ops.workspace(mgd.mgd_rope_workspace_size(B), dev)
        args = (q, kn, vn, table, k.t, v.t, torch.tensor(lens, **i32))
        ops.rope_append(*args, new_len=torch.tensor(new, **i32), q_out=qo.t, ws=ws)
        assert mgd.mgd_workspace_errors(ws) == mgd.MGD_DEVERR_KV_LEN
        check_guards(k=k, v=v, q=qo)
        assert bool(is_poison(k.t[1]).all()) and bool(is_poison(v.t[1]).all()) and bool(is_poison(qo.t[1]).all())
        assert not bool(is_poison(qo.t[0]).any()) and not bool(is_poison(k.t[2, :, 2:5]).any())
        ops.rope_append(*args[:6], torch.full((B,), 6, **i32), q_out=qo.t, ws=ws)
        assert mgd.mgd_workspace_errors(ws) == 0, "an error outlived its call"


def test_in_place_and_strided_caches():
    dev = gpu_or_skip()
    B, T, Hq, Hkv, D, cap = 2, 4, 6, 2, 128, 10
    q, kn, vn = (x.contiguous() for x in _fused(dev, B, T, Hq, Hkv, D, torch.bfloat16, 3))
    table = ops.rope_table(128, device=dev)
    lens = torch.tensor([10, 4], dtype=torch.int32, device=dev)
    wide = torch.zeros((2, B, Hkv + 1, cap + 3, D), dtype=torch.bfloat16, device=dev)
    k, v = wide[0, :, :Hkv, :cap], wide[1, :, :Hkv, :cap]
    k2, v2 = torch.zeros((B, Hkv, cap, D), dtype=q.dtype, device=dev), torch.zeros((B, Hkv, cap, D), dtype=q.dtype, device=dev)
    ref = ops.rope_append(q, kn, vn, table, k2, v2, lens)
    got = ops.rope_append(q, kn, vn, table, k, v, lens, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, ref)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert int(wide[:, :, Hkv:].count_nonzero()) == 0 and int(wide[:, :, :, cap:].count_nonzero()) == 0


def test_captured_call_follows_the_lengths():
    dev = gpu_or_skip()
    B, T, Hq, Hkv, D, cap = 3, 2, 4, 2, 64, 30
    q, kn, vn = _fused(dev, B, T, Hq, Hkv, D, torch.float32, 5)
    table = ops.rope_table(64, device=dev)
    lens = torch.full((B,), 2, dtype=torch.int32, device=dev)
    k, v = torch.zeros((B, Hkv, cap, D), device=dev), torch.zeros((B, Hkv, cap, D), device=dev)
    ws = ops.workspace(mgd.mgd_rope_workspace_size(B), dev)
    out = ops.rope_append(q, kn, vn, table, k, v, lens, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.rope_append(q, kn, vn, table, k, v, lens, q_out=out, ws=ws)
    inv, mag = rope_radians(64, 10000.0)
    for L in (2, 9, 30):
        lens.fill_(L)
        g.replay()
        pos = torch.arange(L - T, L, device=dev)
        for b in range(B):
            _expect(q[b], pos, inv, mag, False, out[b])
            _expect(kn[b], pos, inv, mag, False, k[b, :, L - T:L].transpose(0, 1))

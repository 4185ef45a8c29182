"""Head norms and rotary positions in one pass (duo_qk_norm_rope): refusals on the CPU
with launches skipped; results against the formula in 64 bits on the GPU.

Tolerance, element y of a pair (u, v) after the norm, scale s: one rounding to the output
type (eps / 2 relative to y) plus fp32 arithmetic.  The norm costs at most 16 roundings
(13 in a sum of 128 squares by tree, the product with 1/d, + eps, rsqrt's two, two
products, halved under the root), the rotation 3, cos and sin 2 units of the last place,
and the angle at most pi 2^-25 + 2 pi 2^-32: under 40 units of 2^-24 of s (|u| + |v|)."""
import math

import pytest
import torch

from head_split_kv_duo_b200 import duo, inputs
from head_split_kv_duo_b200.duo import DuoRope

FAKE = 1 << 40
DEV = "cuda"


def freqs(rot, base=10000.0):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


# ---------------------------------------------------------------- host side

@pytest.fixture
def dry_run():
    assert duo.duo_debug_launch_controls(1, -1) == duo.DUO_OK
    yield
    assert duo.duo_debug_launch_controls(0, -1) == duo.DUO_OK


@pytest.mark.parametrize("kw", [
    dict(head_dim=96, rot_dim=96), dict(rot_dim=0, inv_freq=[1.0]), dict(rot_dim=24), dict(rot_dim=144),
    dict(axes=0), dict(axes=9), dict(pair_axis=[2] * 64, axes=2), dict(interleaved=2), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(inv_freq=[-1.0] + [1.0] * 63),
    dict(inv_freq=[math.nan] * 64), dict(inv_freq=[math.inf] * 64), dict(inv_freq=[1e7] * 64),
])
def test_rope_create_refuses(kw):
    a = dict(head_dim=128, rot_dim=128, inv_freq=[1.0] * 72, pair_axis=None, axes=1, interleaved=0, scale=1.0)
    a.update(kw)
    st, h = duo.duo_rope_create(**a)
    assert st == duo.DUO_ERR_INVALID and not h


def _call(h, n=4, hq=4, hkv=2, dtype=duo.DUO_BF16, q=FAKE, qs=None, k=FAKE + (1 << 20), ks=None, v=FAKE + (2 << 20),
          vs=None, wq=None, wk=None, eps=1e-6, pos=FAKE + (3 << 20), qo=FAKE + (4 << 20), ko=FAKE + (5 << 20),
          vo=FAKE + (6 << 20)):
    return duo.duo_qk_norm_rope(h, n, hq, hkv, dtype, q, hq * 128 if qs is None else qs, k,
                                hkv * 128 if ks is None else ks, v, hkv * 128 if vs is None else vs, wq, wk, eps, pos,
                                qo, ko, vo)


def test_norm_rope_argument_checks(dry_run):
    st, h = duo.duo_rope_create(128, 128, freqs(128))
    assert st == duo.DUO_OK
    w = FAKE + (7 << 20)
    ok = [dict(), dict(q=None, qo=None), dict(k=None, ko=None, v=None, vo=None), dict(v=None, vo=None),
          dict(k=None, ko=None), dict(wq=w, wk=w), dict(eps=0.0), dict(qs=1024), dict(q=FAKE, qo=FAKE),
          dict(v=FAKE, vo=FAKE, q=None, qo=None), dict(k=FAKE + 1024, ks=1024, v=FAKE + 1536, vs=1024, qs=1024)]
    for kw in ok:
        assert _call(h, **kw) == duo.DUO_OK, kw
    bad = [dict(n=0), dict(n=-1), dict(q=None, qo=None, k=None, ko=None), dict(pos=None), dict(pos=FAKE + (3 << 20) + 2),
           dict(dtype=7), dict(hq=0), dict(hkv=0), dict(hq=5000), dict(q=None), dict(qo=None), dict(v=None),
           dict(vo=None), dict(q=FAKE + 8), dict(ko=FAKE + (5 << 20) + 4), dict(qs=511), dict(qs=516), dict(ks=0),
           dict(vs=-256), dict(wq=w, eps=0.0), dict(wk=w, eps=-1.0), dict(wk=w, eps=math.nan),
           dict(wq=w, eps=math.inf), dict(wq=w + 8), dict(q=None, qo=None, wq=w),
           # overlaps: an output over another input or output, its own input shifted or strided, weights, positions
           dict(qo=FAKE + (1 << 20)), dict(qo=FAKE + 256), dict(q=FAKE, qo=FAKE, qs=1024), dict(ko=FAKE),
           dict(ko=FAKE + (4 << 20) + 1024), dict(wq=FAKE + (4 << 20)), dict(qo=FAKE + (3 << 20) - 4096 + 16)]
    for kw in bad:
        assert _call(h, **kw) == duo.DUO_ERR_INVALID, kw
    assert duo.duo_qk_norm_rope(None, 4, 4, 2, duo.DUO_BF16, FAKE, 512, None, 0, None, 0, None, None, 1e-6,
                                FAKE + (3 << 20), FAKE + (4 << 20), None, None) == duo.DUO_ERR_INVALID
    assert duo.duo_debug_launch_controls(1, 0) == duo.DUO_OK  # a launch that fails is reported
    assert _call(h) == duo.DUO_ERR_CUDA
    assert duo.duo_debug_launch_controls(1, -1) == duo.DUO_OK
    duo.duo_rope_destroy(h)
    duo.duo_rope_destroy(None)


# ---------------------------------------------------------------- results

def reference(x, w, eps, pos, inv_freq, pair_axis, interleaved, scale):
    """The formula in 64 bits: (result, |u| + |v| of each element's pair times scale)."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    pairs = len(inv_freq)
    f = torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
    a = (pos.double()[torch.tensor(pair_axis, device=x.device)].t() * f)[:, None]  # [n][1][pairs]
    i = torch.arange(pairs, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    u, v = x[..., first], x[..., second]
    y, size = x.clone(), x.abs()
    y[..., first] = scale * (u * a.cos() - v * a.sin())
    y[..., second] = scale * (u * a.sin() + v * a.cos())
    size[..., first] = size[..., second] = scale * (u.abs() + v.abs())
    return y, size


def check(got, want, size, dtype):
    assert got.dtype == dtype and got.is_contiguous()
    err = (got.double() - want).abs()
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 40 * 2.0 ** -24 * size
    assert bool((err <= tol).all()), f"off by {float((err - tol).max())} beyond the tolerance"


CASES = [
    # n, hq, hkv, d, rot, axes, interleaved, normed, scale, v
    (1, 32, 8, 128, 128, 1, False, "", 1.0, True),
    (1, 1, 1, 64, 64, 1, True, "qk", 1.0, True),
    (3, 7, 1, 128, 16, 2, False, "q", 1.0, False),
    (2, 5, 5, 64, 48, 3, False, "k", 1.0, True),
    (129, 12, 4, 128, 80, 3, True, "qk", 1.25, True),
    (97, 32, 8, 128, 64, 1, False, "qk", 1.0, True),
    (1000, 3, 1, 64, 32, 8, True, "", 0.5, False),
    (4099, 16, 2, 128, 128, 3, False, "qk", 1.0, True),
    (20011, 8, 8, 64, 64, 1, True, "qk", 1.0, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hq,hkv,d,rot,axes,inter,normed,scale,with_v", CASES)
def test_norm_rope_matches_the_formula(n, hq, hkv, d, rot, axes, inter, normed, scale, with_v, dtype):
    """Packed rows (q, k and v side by side, and a gap behind them), positions over the
    whole int32 range, each side normed or not; nothing past the rows is written."""
    gap = 16
    packed = inputs.randn((n, (hq + 2 * hkv) * d + gap), 5, dtype=dtype, device=DEV)
    heads = packed[:, :(hq + 2 * hkv) * d].unflatten(1, (hq + 2 * hkv, d))
    q, k, v = heads[:, :hq], heads[:, hq:hq + hkv], heads[:, hq + hkv:]
    if n > 2:
        packed[1] = 0  # a row of zeros stays one
        packed[2] *= 1000
    g = inputs.generator(7, DEV)
    wq = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dtype) if "q" in normed else None
    wk = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dtype) if "k" in normed else None
    pos = torch.randint(-(2 ** 31), 2 ** 31, (axes, n), generator=g, device=DEV).to(torch.int32)
    pos[:, 0] = torch.tensor([0, 1, 2 ** 31 - 1, -(2 ** 31), 5, 6, 7, 8][:axes], dtype=torch.int32)
    f = freqs(rot)
    pair_axis = [i % axes for i in range(rot // 2)]
    rope = DuoRope(d, f, pair_axis=pair_axis, interleaved=inter, scale=scale)
    before = packed.clone()
    qo, ko, vo = rope.norm_rope(q, k, pos, v=v if with_v else None, q_weight=wq, k_weight=wk, eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(packed, before)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        want, size = reference(x, w, 1e-5, pos, f, pair_axis, inter, scale)
        check(got, want, size, dtype)
    assert (vo is None) == (not with_v)
    if with_v:
        assert torch.equal(vo, v)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope_in_place_and_one_side(dtype):
    """In place gives the bits that separate outputs give; queries alone, keys alone; the
    rows around the tensors keep their values."""
    n, hq, hkv, d = 33, 6, 2, 128
    buf = inputs.randn((3, n, hq, d), 11, dtype=dtype, device=DEV)
    q, k = buf[1], inputs.randn((n, hkv, d), 12, dtype=dtype, device=DEV)
    w = inputs.randn((d,), 13, dtype=dtype, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV) + 70000
    rope = DuoRope(d, freqs(64))
    qo, ko, _ = rope.norm_rope(q, k, pos, q_weight=w, k_weight=w)
    only_q = rope.norm_rope(q, None, pos, q_weight=w)
    only_k = rope.norm_rope(None, k, pos, k_weight=w)
    assert torch.equal(only_q[0], qo) and only_q[1:] == (None, None) and torch.equal(only_k[1], ko)
    around = buf[[0, 2]].clone()
    rope.norm_rope(q, k, pos, q_weight=w, k_weight=w, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(buf[[0, 2]], around)


@pytest.mark.gpu
def test_norm_rope_binding_refuses():
    n, d = 4, 128
    x = torch.zeros(n, 2, d, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(n, dtype=torch.int32, device=DEV)
    rope = DuoRope(d, freqs(d))
    axes = DuoRope(d, freqs(d), pair_axis=[i % 3 for i in range(64)])
    for call in (lambda: rope.norm_rope(None, None, pos), lambda: rope.norm_rope(x.half(), None, pos),
                 lambda: rope.norm_rope(x.cpu(), None, pos), lambda: rope.norm_rope(x, None, pos.long()),
                 lambda: rope.norm_rope(x, None, pos[:3]), lambda: axes.norm_rope(x, None, pos),
                 lambda: rope.norm_rope(x, x.float(), pos), lambda: rope.norm_rope(x[:, :, :64], None, pos),
                 lambda: rope.norm_rope(x.transpose(0, 1), None, pos[:2]), lambda: rope.norm_rope(x, x[:3], pos),
                 lambda: rope.norm_rope(x, x, pos, v=x[:, :1]), lambda: rope.norm_rope(x, None, pos, q_weight=pos),
                 lambda: rope.norm_rope(x, None, pos, q_out=x[:, :1]), lambda: DuoRope(d, freqs(d), pair_axis=[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(duo.DuoError):  # an overlap that the library refuses
        rope.norm_rope(x, x, pos, q_out=x, k_out=x)


@pytest.mark.gpu
def test_norm_rope_captured_and_replayed():
    """A captured call follows its buffers: replayed on new contents it gives theirs."""
    n, d = 5, 64
    q = inputs.randn((n, 4, d), 21, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    rope = DuoRope(d, freqs(d), interleaved=True)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rope.norm_rope(q, None, pos, q_out=out)
    q.copy_(inputs.randn((n, 4, d), 22, device=DEV))
    pos += 100000
    graph.replay()
    torch.cuda.synchronize()
    want, size = reference(q, None, 0.0, pos[None], freqs(d), [0] * (d // 2), True, 1.0)
    check(out, want, size, torch.bfloat16)

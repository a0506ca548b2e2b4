"""Rotary positions on the GPU, against the formula in 64 bits, element by element.

Bound of an element's error, by arithmetic, with a and b its pair: the reduced
angle is at most half a turn, rounded to fp32 (pi 2^-24 off at most), sine and
cosine are good to 2 units (2^-22), each product and the sum round once (3 *
2^-24): together below (|a| + |b|) 2^-20. The angle before is the rounded product of
three 64-bit numbers: |theta| 2^-51 off at most. A norm before adds the sum of D
squares (8 in a lane, then at most 6 sums: 14 * 2^-24, half of it in the root), the
mean, the sum with eps (its conversion included), the root, the quotient and two products: below 2^-20 of a
value. Then half a step of the output's type, for fp16 at least half of its smallest step."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DTYPES = ("f32", "f16", "bf16")
EPS = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_qmat_amd as qmat
    qmat.library_path()
    return qmat


def torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def formula(x, pos, freq, axis, neighbours, weight, eps, out_dtype):
    """(values, bounds) in numpy fp64: x [n, heads, D], pos [axes, n], axis [pairs] (-1: unturned)."""
    x = x.astype(np.float64)
    D, pairs = x.shape[2], len(freq)
    unit = 2.0 ** -20
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
        unit *= 2
    there = (axis >= 0) & (axis < pos.shape[0])
    theta = np.where(there, pos[np.where(there, axis, 0)].T * freq, 0.0)[:, None]  # [n, 1, pairs]
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if neighbours else (slice(0, pairs), slice(pairs, 2 * pairs))
    out, bound = x.copy(), np.abs(x) * unit
    out[..., a] = x[..., a] * np.cos(theta) - x[..., b] * np.sin(theta)
    out[..., b] = x[..., b] * np.cos(theta) + x[..., a] * np.sin(theta)
    both = (np.abs(x[..., a]) + np.abs(x[..., b])) * (unit + np.abs(theta) * 2.0 ** -51)
    bound[..., a] = bound[..., b] = both
    return out, bound + np.abs(out) * EPS[out_dtype] / 2 * (1 + 2.0 ** -8) + (2.0 ** -25 if out_dtype == "f16" else 1e-38)


def run(lib, n, heads, kv_heads, D, rot, axes=1, neighbours=False, norm=False, dtype="f32", out="f32", far=4000, pad=8, seed=0, axis=None,
        in_place=False, freq=None):
    import torch
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(n, heads + kv_heads, D + 0, generator=g)
    buf = torch.cat((qkv.flatten(1), torch.full((n, pad), 7.0)), 1).to(torch_type(dtype)).cuda()
    q = buf[:, :heads * D].unflatten(1, (heads, D))
    k = buf[:, heads * D:(heads + kv_heads) * D].unflatten(1, (kv_heads, D)) if kv_heads else None
    pos = torch.randint(-far // 8, far, (axes, n), generator=g, dtype=torch.int64).to(torch.int32)
    pairs = rot // 2
    freq = lib.rope_freq(rot) if freq is None else freq
    axis = np.arange(pairs) % axes if axis is None else axis
    w = [(1 + 0.3 * torch.randn(D, generator=g)).cuda() if norm else None for _ in range(2)]
    q0, k0 = q.float().cpu().numpy(), None if k is None else k.float().cpu().numpy()
    outs = {}
    if in_place:
        outs = {"q_out": q, "k_out": k}
    else:
        obuf = torch.full((n, (heads + kv_heads) * D + pad), 7.0, dtype=torch_type(out), device="cuda")
        outs["q_out"] = obuf[:, :heads * D].unflatten(1, (heads, D))
        if kv_heads:
            outs["k_out"] = obuf[:, heads * D:(heads + kv_heads) * D].unflatten(1, (kv_heads, D))
    a = None if axes == 1 and (axis == 0).all() else torch.from_numpy(axis.astype(np.int32)).cuda()
    got = lib.rope(q, k, (pos[0] if axes == 1 else pos).cuda(), freq, axis=a, neighbours=neighbours, q_norm=w[0], k_norm=w[1], eps=1e-5,
                   dtype=torch_type(out), **outs)
    for x, y, weight in ((q0, got[0], w[0]), (k0, got[1], w[1])):
        if x is None:
            assert y is None
            continue
        want, bound = formula(x, pos.numpy(), freq.cpu().numpy(), axis, neighbours, None if weight is None else weight.cpu().numpy(), 1e-5, out)
        err = np.abs(y.double().cpu().numpy() - want)
        assert np.all(err <= bound), f"{(err / bound).max()} of the bound"
    tail = (buf if in_place else obuf)[:, (heads + kv_heads) * D:]
    assert torch.all(tail == 7.0).item()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("n,heads,kv_heads,D,rot", [(1, 1, 0, 8, 8), (1, 32, 8, 128, 128), (3, 5, 1, 64, 32), (7, 4, 2, 72, 72), (2, 3, 3, 80, 40),
                                                    (5, 2, 1, 256, 64), (33, 7, 1, 128, 64), (3, 2, 2, 512, 512), (2, 1, 1, 264, 256)])
def test_shapes(lib, n, heads, kv_heads, D, rot, neighbours, norm):
    run(lib, n, heads, kv_heads, D, rot, neighbours=neighbours, norm=norm, seed=n + D)


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_types(lib, dtype, out):
    run(lib, 19, 6, 2, 128, 128, dtype=dtype, out=out, norm=True, axes=3)
    run(lib, 19, 6, 2, 64, 64, dtype=dtype, out=out, neighbours=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("neighbours", [False, True])
def test_in_place(lib, dtype, neighbours):
    run(lib, 21, 8, 2, 128, 96, dtype=dtype, out=dtype, neighbours=neighbours, norm=True, in_place=True)


@pytest.mark.parametrize("axes", [2, 3, 4])
def test_axes(lib, axes):
    import torch
    for cycle in (False, True):
        axis = lib.rope_axis([32 // axes + (a < 32 % axes) for a in range(axes)], cycle=cycle, device="cpu").numpy()
        run(lib, 40, 4, 2, 64, 64, axes=axes, axis=axis, seed=axes)
    odd = np.array([0, -1, axes, axes - 1] * 8)  # axes that are not there: pairs stay
    run(lib, 9, 3, 1, 64, 64, axes=axes, axis=odd)
    run(lib, 9, 3, 1, 64, 64, axes=axes, axis=np.full(32, axes - 1))


def test_far_positions(lib):
    """Angles of positions up to int32's largest."""
    run(lib, 300, 2, 1, 128, 128, far=2 ** 31 - 1)
    run(lib, 300, 2, 1, 128, 128, far=2 ** 20, out="f16", dtype="f32")


@pytest.mark.parametrize("n", [2000, 20000])
def test_many_tokens(lib, n):
    """Fewer groups of lanes for a token, down to one that goes through all heads."""
    run(lib, n, 5, 2, 64, 64, axes=3, norm=True, dtype="bf16", out="bf16")


def test_no_turn(lib):
    """rot_dim 0: the norm alone; no positions matter."""
    import torch
    run(lib, 4, 3, 1, 64, 0, norm=True, freq=torch.zeros(0, dtype=torch.float64, device="cuda"))


def test_other_rows_stay_clean(lib):
    """NaN and infinities of a head stay in that head."""
    import torch
    q = torch.randn(4, 3, 64, generator=torch.Generator().manual_seed(2)).cuda()
    w = torch.ones(64, device="cuda")
    pos, freq = torch.arange(4, dtype=torch.int32, device="cuda"), lib.rope_freq(64)
    want, _ = lib.rope(q, None, pos, freq, q_norm=w)
    q[1, 1, 7], q[2, 0, 9] = float("nan"), float("inf")
    got, _ = lib.rope(q, None, pos, freq, q_norm=w)
    keep = torch.ones(4, 3, dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = False
    assert torch.equal(got.cpu()[keep], want.cpu()[keep]) and torch.isnan(got[1, 1]).all().item()


def test_nothing_to_do(lib):
    import torch
    q = torch.zeros((0, 2, 64), device="cuda")
    got = lib.rope(q, q, torch.zeros(0, dtype=torch.int32, device="cuda"), lib.rope_freq(64), dtype=torch.float16)
    assert got[0].shape == (0, 2, 64) and got[1].dtype == torch.float16


@pytest.mark.parametrize("n,heads,kv_heads,D,rot", [(300, 7, 0, 128, 128), (301, 5, 1, 72, 64), (129, 11, 2, 512, 512), (1000, 3, 0, 8, 8),
                                                    (9000, 1, 2, 8, 8), (4097, 7, 4, 64, 64)])
def test_tokens_across_workgroups(lib, n, heads, kv_heads, D, rot):
    """Heads shared out in parts that do not divide a workgroup's groups of lanes: its tokens begin and end within it."""
    run(lib, n, heads, kv_heads, D, rot, axes=2, seed=n)
    run(lib, n, heads, kv_heads, D, rot, neighbours=True, norm=True, in_place=True, dtype="bf16", out="bf16", seed=n)


def test_keys_alone(lib):
    import torch
    g = torch.Generator().manual_seed(4)
    k = torch.randn(5, 2, 64, generator=g).cuda()
    pos, freq = torch.arange(5, dtype=torch.int32, device="cuda"), lib.rope_freq(64)
    none, got = lib.rope(k[:, :0], k, pos, freq)
    assert none.shape == (5, 0, 64) and torch.equal(got, lib.rope(k, None, pos, freq)[0])

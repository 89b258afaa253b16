"""MXFP8 operators on the GPU against the float64 definitions (oracle/mx8.py): row conversions,
RMS norm with residual and combine, entry conversions, and the expert FFN with MXFP8
activations, alone and as one chain."""
import numpy as np
import pytest

import expert_ffn_cache_amd as moe
import gen
from gen import configs
from gen.arena import device_arena_all_experts, fill_entries_ptr
import oracle
from oracle import mx8
from tests._helpers import dev, dev_bf16, np_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TD = {moe.MOE_F32: torch.float32, moe.MOE_BF16: torch.bfloat16}
DT = [moe.MOE_F32, moe.MOE_BF16]


def _bytes(n, fill=0xA5):
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda")


def _as(a, dt):
    """float array -> device tensor in dt, and the float64 values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(TD[dt])
    return t, np_of(t.float()).astype(np.float64)


def _awkward_rows(T, d, seed):
    """Normal rows with blocks of zeros, tiny and subnormal and huge values, exact ties, a largest
    magnitude just below and at a power of two, negative zeros."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, d)).astype(np.float32) * np.exp2(r.integers(-20, 20, (T, 1))).astype(np.float32)
    b = x.reshape(-1, 32)
    for i, kind in zip(r.permutation(len(b)), range(min(len(b), 8))):
        if kind == 0:
            b[i] = 0
        elif kind == 1:
            b[i] = np.where(np.arange(32) % 3, -0.0, 2.0 ** -126)
        elif kind == 2:
            b[i] = (r.integers(0, 1 << 23, 32).astype(np.float64) * 2.0 ** -149).astype(np.float32)
        elif kind == 3:
            b[i] *= np.float32(3e37) / max(np.abs(b[i]).max(), np.float32(1e-30))
        elif kind == 4:
            b[i] = (np.arange(32) - 16) * 17.0   # ties at scale 1
            b[i, 0] = 272.0
        elif kind == 5:
            b[i] = np.linspace(-1, 1, 32)
            b[i, 5] = np.nextafter(np.float32(2), np.float32(0))
        elif kind == 6:
            b[i] = np.linspace(-1, 1, 32)
            b[i, 31] = -2.0
        else:
            b[i] = 2.0 ** -135
    return x


# ---------------------------------------------------------------- row conversions
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,d", [(1, 64), (3, 320), (17, 4096), (301, 192), (5, 16448)])
def test_quantize_and_dequantize_are_exact(T, d, dt):
    x, v = _as(_awkward_rows(T, d, T + d), dt)
    n = moe.moe_mxfp8_bytes(T, d)
    x8 = _bytes(n + 64)
    moe.moe_mxfp8_quantize(x, dt, T, d, x8)
    got = x8.cpu().numpy()
    want = mx8.pack(*mx8.quantize(v))
    assert np.all(got[n:] == 0xA5)
    np.testing.assert_array_equal(got[:n], want)
    for odt in DT:
        out = torch.full((T, d), float("nan"), dtype=TD[odt], device="cuda")
        moe.moe_mxfp8_dequantize(x8, T, d, out, odt)
        ref = torch.from_numpy(mx8.dequantize(*mx8.unpack(got, T, d))).to(TD[odt])
        np.testing.assert_array_equal(np_of(out.float()), np_of(ref.float()))


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_block_that_is_not_finite_is_nan_and_leaves_the_others(bad):
    x = np.random.default_rng(1).standard_normal((4, 128)).astype(np.float32)
    x[1, 40] = x[3, 127] = bad
    x8 = _bytes(moe.moe_mxfp8_bytes(4, 128))
    moe.moe_mxfp8_quantize(dev(x), moe.MOE_F32, 4, 128, x8)
    np.testing.assert_array_equal(x8.cpu().numpy(), mx8.pack(*mx8.quantize(x)))
    for odt in DT:
        out = torch.empty((4, 128), dtype=TD[odt], device="cuda")
        moe.moe_mxfp8_dequantize(x8, 4, 128, out, odt)
        nan = np.zeros((4, 128), dtype=bool)
        nan[1, 32:64] = nan[3, 96:] = True
        np.testing.assert_array_equal(np.isnan(np_of(out)), nan)


# ---------------------------------------------------------------- norms
def _half(dt):
    return {moe.MOE_F32: 2.0 ** -24, moe.MOE_BF16: 2.0 ** -8}[dt]


def _check_norm(s, gamma, eps, y, ydt, y8):
    """y and y8 of rows s (values of the stored sum) against the definition."""
    ref, err = mx8.rmsnorm(s, gamma, eps)
    if y is not None:
        assert np.all(np.abs(np_of(y).astype(np.float64) - ref) <= err + _half(ydt) * (np.abs(ref) + err))
    if y8 is not None:
        T, d = s.shape
        buf = y8.cpu().numpy()
        got = mx8.dequantize(*mx8.unpack(buf, T, d))
        lo, hi = mx8.span(ref, err)
        assert np.all(got >= lo) and np.all(got <= hi)
        assert np.mean(got != mx8.dequantize(*mx8.quantize(ref))) < 1e-3
        pad = buf[T * d:].reshape(T, -1)[:, d // 32:]
        assert np.all(pad == 0)


@pytest.mark.parametrize("xdt", DT)
@pytest.mark.parametrize("ddt", [None] + DT)
@pytest.mark.parametrize("T,d", [(1, 64), (7, 320), (3, 2048), (2, 2112), (5, 4096), (3, 7680), (2, 8256),
                                 (1, 32768), (2, 33344)])
def test_rmsnorm(T, d, xdt, ddt):
    """Every row-length class (a wave, 256 and 1024 threads, the loop) at its edges."""
    r = np.random.default_rng(T * d)
    x, xv = _as(3 * r.standard_normal((T, d)) * (1 + 20 * (r.random((1, d)) > 0.99)), xdt)
    gdt = moe.MOE_F32 if ddt == moe.MOE_BF16 else moe.MOE_BF16
    g, gv = _as(1 + 0.2 * r.standard_normal(d), gdt)
    delta, s = None, xv
    if ddt is not None:
        delta, dv = _as(r.standard_normal((T, d)), ddt)
        s = np_of((x.float() + delta.float()).to(TD[xdt]).float()).astype(np.float64)
    for ydt, with8 in ((moe.MOE_F32, True), (moe.MOE_BF16, False), (None, True)):
        out = torch.full((T, d), float("nan"), dtype=TD[xdt], device="cuda")
        y = None if ydt is None else torch.full((T, d), float("nan"), dtype=TD[ydt], device="cuda")
        y8 = _bytes(moe.moe_mxfp8_bytes(T, d)) if with8 else None
        moe.moe_rmsnorm(x, xdt, delta, ddt or moe.MOE_F32, g, gdt, 1e-5, T, d, out, y, ydt or moe.MOE_F32, y8)
        np.testing.assert_array_equal(np_of(out.float()).astype(np.float64), s)
        _check_norm(s, gv, 1e-5, y, ydt, y8)


@pytest.mark.parametrize("d", [512, 4096, 33344])
def test_rmsnorm_in_place(d):
    """x_out may be x or delta; the results do not change."""
    r = np.random.default_rng(d)
    x, _ = _as(r.standard_normal((3, d)), moe.MOE_F32)
    delta, _ = _as(r.standard_normal((3, d)), moe.MOE_F32)
    g, _ = _as(r.standard_normal(d), moe.MOE_F32)
    res = []
    for alias in (None, "x", "delta"):
        xi, di = x.clone(), delta.clone()
        out = {None: torch.empty_like(x), "x": xi, "delta": di}[alias]
        y = torch.empty_like(x)
        moe.moe_rmsnorm(xi, moe.MOE_F32, di, moe.MOE_F32, g, moe.MOE_F32, 1e-6, 3, d, out, y, moe.MOE_F32, None)
        res.append((out.clone(), y))
    for o, y in res[1:]:
        assert torch.equal(o, res[0][0]) and torch.equal(y, res[0][1])


@pytest.mark.parametrize("d", [256, 4096])
def test_rmsnorm_rows_do_not_affect_one_another(d):
    """NaN, infinite, zero and huge rows beside ordinary ones; eps = 0 too."""
    r = np.random.default_rng(d)
    x = r.standard_normal((6, d)).astype(np.float32)
    x[1, 3], x[2, 5] = np.nan, np.inf
    x[3], x[4] = 0, x[4] * np.float32(1e30)   # 1e60 overflows fp32: the sum is inf, y is 0
    g = np.ones(d, dtype=np.float32)
    for eps in (1e-6, 0.0):
        y = torch.empty((6, d), device="cuda")
        y8 = _bytes(moe.moe_mxfp8_bytes(6, d))
        moe.moe_rmsnorm(dev(x), moe.MOE_F32, None, moe.MOE_F32, dev(g), moe.MOE_F32, eps, 6, d, None, y, moe.MOE_F32, y8)
        y, v8 = np_of(y), mx8.dequantize(*mx8.unpack(y8.cpu().numpy(), 6, d))
        for t in (0, 5):
            ref, err = mx8.rmsnorm(x[t:t + 1], g, eps)
            assert np.all(np.abs(y[t] - ref[0]) <= err[0] + 2.0 ** -24 * np.abs(ref[0]))
            assert np.isfinite(v8[t]).all()
        assert np.isnan(y[1]).all() and np.isnan(v8[1]).all()
        assert np.isnan(y[2, 5]) and np.all(np.delete(y[2], 5) == 0)
        assert np.all(y[3] == 0) if eps else np.isnan(y[3]).all()
        assert np.all(y[4] == 0)


@pytest.mark.parametrize("T,k,d", [(1, 1, 64), (8, 6, 4096), (5, 16, 2048), (9, 9, 8256), (3, 2, 33344)])
@pytest.mark.parametrize("xdt,ydt", [(moe.MOE_BF16, moe.MOE_F32), (moe.MOE_F32, moe.MOE_BF16)])
def test_combine_rmsnorm_is_combine_then_rmsnorm(T, k, d, xdt, ydt):
    """Bit for bit, in place on the residual too."""
    r = np.random.default_rng(T + k + d)
    yp, _ = _as(r.standard_normal((T * k, d)), ydt)
    inv = dev(r.permutation(T * k).astype(np.int32))
    w = dev(r.random((T, k)).astype(np.float32))
    x, _ = _as(r.standard_normal((T, d)), xdt)
    g, gv = _as(r.standard_normal(d), moe.MOE_BF16)
    comb = torch.empty((T, d), device="cuda")
    moe.moe_combine(yp, ydt, inv, w, T, k, d, comb)
    a = [torch.empty_like(x), torch.empty((T, d), device="cuda"), _bytes(moe.moe_mxfp8_bytes(T, d))]
    moe.moe_rmsnorm(x, xdt, comb, moe.MOE_F32, g, moe.MOE_BF16, 1e-6, T, d, a[0], a[1], moe.MOE_F32, a[2])
    b = [x.clone(), torch.empty((T, d), device="cuda"), _bytes(moe.moe_mxfp8_bytes(T, d))]
    moe.moe_combine_rmsnorm(yp, ydt, inv, w, k, b[0], xdt, g, moe.MOE_BF16, 1e-6, T, d, b[0], b[1], moe.MOE_F32, b[2])
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    _check_norm(np_of(a[0].float()).astype(np.float64), gv, 1e-6, a[1], moe.MOE_F32, a[2])


# ---------------------------------------------------------------- entries
def _plain_entries(n, d, f, seed):
    r = np.random.default_rng(seed)
    v = (r.standard_normal((n, 3 * d * f)) * d ** -0.5).astype(np.float32)
    b = v.reshape(-1, 32)
    for i, kind in zip(r.permutation(len(b)), range(min(len(b), 7))):
        b[i] = [np.zeros(32), (r.integers(0, 1 << 23, 32) * 2.0 ** -149), (np.arange(32) - 16) * 0.25 + 0.25,
                np.linspace(-7.9, 7.9, 32), np.full(32, 2.0 ** -127), b[i] * 1e38, np.linspace(-1, 2, 32)][kind]
    return v


def _mx_bytes(v, d, f):
    """The MXFP4 entry of one plain entry, block by block with the generator's conversion."""
    out = np.full(moe.moe_entry_bytes(d, f, moe.MOE_MXFP4), 0xA5, dtype=np.uint8)
    fd = d * f
    for m, (R, K) in enumerate(((f, d), (f, d), (d, f))):
        w = v[m * fd:(m + 1) * fd].reshape(R, K)
        for r in range(R):
            for b in range(K // 32):
                codes, s = gen.mxfp4_block(w[r, 32 * b:32 * b + 32])
                at = K // 2 * (r // 16) + 64 * (b // 4) + 16 * (b % 4) + r % 16
                out[m * fd // 2 + 16 * at:m * fd // 2 + 16 * at + 16] = codes
                out[3 * fd // 2 + m * fd // 32 + at] = s
    return out


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("n,d,f,gap", [(1, 64, 64, 0), (2, 320, 192, 0), (3, 128, 64, 48), (1, 256, 448, 16)])
def test_entry_quantize_and_dequantize_are_exact(n, d, f, gap, dt):
    src, v = _as(_plain_entries(n, d, f, n + d + f), dt)
    el, ne, eb = src.element_size(), 3 * d * f, moe.moe_entry_bytes(d, f, moe.MOE_MXFP4)
    padded = torch.full((n, ne + 2 * gap), float("nan"), dtype=TD[dt], device="cuda")
    padded[:, :ne] = src
    mx = _bytes(n * (eb + gap)).reshape(n, eb + gap)
    moe.moe_entry_quantize(padded, dt, (ne + 2 * gap) * el, n, d, f, mx, eb + gap)
    got = mx.cpu().numpy()
    assert np.all(got[:, eb:] == 0xA5)
    for i in range(n):
        want = _mx_bytes(v[i].astype(np.float32), d, f)
        # a zero keeps its sign here, the generator drops it: compare values' codes
        lo, hi = got[i, :3 * d * f // 2] & 15, got[i, :3 * d * f // 2] >> 4
        plain = np.where(lo == 8, 0, lo) | np.where(hi == 8, 0, hi) << 4
        wlo, whi = want[:3 * d * f // 2] & 15, want[:3 * d * f // 2] >> 4
        np.testing.assert_array_equal(plain, np.where(wlo == 8, 0, wlo) | np.where(whi == 8, 0, whi) << 4)
        np.testing.assert_array_equal(got[i, 3 * d * f // 2:eb], want[3 * d * f // 2:])
    for odt in DT:
        out = torch.full((n, ne + 2 * gap), 7.0, dtype=TD[odt], device="cuda")
        moe.moe_entry_dequantize(mx, eb + gap, n, d, f, out, odt, (ne + 2 * gap) * out.element_size())
        o = np_of(out.float())
        assert np.all(o[:, ne:] == 7.0)
        ref = mx_values(got, n, d, f)
        np.testing.assert_array_equal(o[:, :ne], np_of(torch.from_numpy(ref).to(TD[odt]).float()))


def mx_values(mx, n, d, f):
    """Values of MXFP4 entries in plain order, from the documented layout."""
    out, fd = np.zeros((n, 3 * d * f)), d * f
    for m, (R, K) in enumerate(((f, d), (f, d), (d, f))):
        c = mx[:n, m * fd // 2:(m + 1) * fd // 2].reshape(n, R // 16, K // 32, 16, 16)
        s = mx[:n, 3 * fd // 2 + m * fd // 32:3 * fd // 2 + (m + 1) * fd // 32].reshape(n, R // 16, K // 32, 16)
        c, s = c.transpose(0, 1, 3, 2, 4).reshape(n * R, K // 2), s.transpose(0, 1, 3, 2).reshape(n * R, K // 32)
        out[:, m * fd:(m + 1) * fd] = oracle.mxfp4_dequant(np.ascontiguousarray(c), np.ascontiguousarray(s)).reshape(n, fd)
    return out


def test_entry_conversions_of_a_block_that_is_not_finite():
    d = f = 64
    v = np.random.default_rng(2).standard_normal((1, 3 * d * f)).astype(np.float32)
    v[0, 33], v[0, d * f + 5] = np.nan, -np.inf
    for dt in DT:
        src, _ = _as(v, dt)
        eb = moe.moe_entry_bytes(d, f, moe.MOE_MXFP4)
        mx = _bytes(eb)
        moe.moe_entry_quantize(src, dt, src.numel() * src.element_size(), 1, d, f, mx, eb)
        assert int((mx[3 * d * f // 2:] == 255).sum()) == 2
        for odt in DT:
            out = torch.empty((1, 3 * d * f), dtype=TD[odt], device="cuda")
            moe.moe_entry_dequantize(mx, eb, 1, d, f, out, odt, out.numel() * out.element_size())
            nan = np.zeros(3 * d * f, dtype=bool)
            nan[32:64] = nan[d * f:d * f + 32] = True
            np.testing.assert_array_equal(np.isnan(np_of(out.float()))[0], nan)


# ---------------------------------------------------------------- expert FFN
def _mx_weights(w, experts):
    return {e: tuple(oracle.mxfp4_dequant(c, s) for c, s in configs.gen_expert(w, 0, e)) for e in experts}


def _ffn(w, x8, perm, offsets, arena, stride, ydt=moe.MOE_F32, path=moe.MOE_PATH_AUTO, mask=None, slots=None,
         keys=None, stream=None, noalloc=False):
    A = w.T * w.k
    y = torch.full((A, w.d), float("nan"), dtype=TD[ydt], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if noalloc:
        moe.moe_expert_ffn_noalloc(x8, moe.MOE_MXFP8, perm, offsets, w.T, w.k, w.E, w.d, w.f, slots, arena, stride,
                                   moe.MOE_MXFP4, mask, keys, 0, y, ydt, path, status, stream)
    else:
        nws = moe.moe_expert_ffn_workspace_bytes(w.T, w.k, w.f, moe.MOE_MXFP8)
        ws = _bytes(nws + 256)
        moe.moe_expert_ffn(x8, moe.MOE_MXFP8, perm, offsets, w.T, w.k, w.E, w.d, w.f, slots, arena, stride,
                           moe.MOE_MXFP4, mask, keys, 0, ws, nws, y, ydt, path, status, stream)
        assert bool((ws[nws:] == 0xA5).all())
    torch.cuda.synchronize()
    return y, int(status.item())


def _case(w, ids=None):
    """(values of the MXFP8 rows, their buffer on the GPU, perm, offsets, ids) of a workload."""
    x = gen.bf16_bits_to_f32(configs.gen_x(w))
    c, s = mx8.quantize(x)
    if ids is None:
        ids, _ = oracle.route(configs.gen_logits(w), w.k)
    counts, offsets, perm, inv = oracle.permute(ids, w.E)
    return mx8.dequantize(c, s), dev(mx8.pack(c, s)), perm, offsets, ids


def _check_ffn(y, ydt, ref, tol, rows=slice(None)):
    got, ref, tol = np_of(y.float()).astype(np.float64)[rows], ref[rows], tol[rows]
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    bad = ~(np.abs(got - ref) <= tol + _half(ydt) * (np.abs(ref) + tol)) & ~np.isnan(ref)
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(np.abs(got - ref) / tol)))
    # the intervals are wide beside the usual error: most elements keep every unit's E4M3 value
    fine = ~np.isnan(ref)
    rms = np.sqrt(np.mean(ref[fine] ** 2))
    assert np.sqrt(np.mean((got - ref)[fine] ** 2)) <= (2e-3 if ydt == moe.MOE_F32 else 4e-3) * rms


def _mx_workload(T, E, k, d, f, alpha=0.5, seed=5):
    return configs.Workload("mx8", seed=seed + T, T=T, d=d, E=E, k=k, f=f, dtype=gen.MXFP4, alpha=alpha)


PATHS = [moe.MOE_PATH_AUTO, moe.MOE_PATH_GEMV, moe.MOE_PATH_GEMM]


@pytest.mark.parametrize("ydt", DT)
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,E,k,d,f,alpha", [
    (1, 8, 2, 64, 64, 0.2),        # one 64-element tile each way
    (1, 16, 6, 512, 256, 0.5),
    (5, 1, 1, 192, 128, 0.0),      # one expert: a dense FFN; short last tile of gate/up
    (6, 4, 4, 128, 192, 0.0),      # every token to every expert; short last tile of down
    (13, 37, 4, 1088, 320, 0.5),   # short last tiles on both sides
    (64, 16, 4, 320, 448, 1.0),
    (200, 5, 3, 256, 576, 1.0),    # over 100 rows for an expert
    (700, 3, 1, 128, 128, 0.2),    # several 128-row tiles
    (2, 4, 2, 8320, 64, 0.2),      # token rows staged over two slices of K, gate/up and down
    (2, 4, 2, 64, 8320, 0.2),
    (9, 4, 2, 4224, 64, 0.2),
    (40, 4, 2, 1088, 64, 0.2)])
def test_ffn_mxfp8(T, E, k, d, f, alpha, path, ydt):
    w = _mx_workload(T, E, k, d, f, alpha)
    x, x8, perm, offsets, ids = _case(w)
    arena = device_arena_all_experts(w)
    y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, ydt, path)
    assert st == 0
    ref, tol = mx8.expert_ffn(x, perm, k, offsets, _mx_weights(w, range(E)))
    _check_ffn(y, ydt, ref, tol)


@pytest.mark.parametrize("T,d,f", [(64, 128, 2048), (64, 2048, 128), (16, 128, 2048), (16, 2048, 128),
                                   (3, 128, 2048)])
def test_ffn_mxfp8_waves_per_strip(T, d, f):
    """256 experts: enough strips for one and two waves to a strip pair, at up to 16 rows a pass and
    up to 32 (fewer experts take four)."""
    w = _mx_workload(T, 256, 6, d, f, 0.2)
    x, x8, perm, offsets, ids = _case(w)
    arena = device_arena_all_experts(w)
    y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_F32, moe.MOE_PATH_GEMV)
    assert st == 0
    used = sorted(set(ids.ravel().tolist()))[::5]
    rows = np.zeros(T * w.k, dtype=bool)
    for e in used:
        rows[offsets[e]:offsets[e + 1]] = True
    ref, tol = mx8.expert_ffn(x, perm, w.k, offsets, _mx_weights(w, used))
    _check_ffn(y, moe.MOE_F32, ref, tol, rows)


@pytest.mark.parametrize("T", [1, 20, 100, 600])
def test_ffn_mxfp8_at_maximum_experts_and_k(T):
    w = _mx_workload(T, 1024, 16, 128, 64)
    x, x8, perm, offsets, ids = _case(w)
    arena = device_arena_all_experts(w)
    ref, tol = mx8.expert_ffn(x, perm, w.k, offsets, _mx_weights(w, sorted(set(ids.ravel().tolist()))))
    for path in PATHS:
        y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_F32, path)
        assert st == 0
        _check_ffn(y, moe.MOE_F32, ref, tol)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [5, 50, 300])
def test_ffn_mxfp8_without_any_expert(T, path):
    """Every expert masked: nothing is written."""
    w = _mx_workload(T, 8, 2, 128, 64)
    x, x8, perm, offsets, ids = _case(w)
    arena = device_arena_all_experts(w)
    mask = torch.zeros(w.E, dtype=torch.uint8, device="cuda")
    y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_F32, path, mask)
    assert st == 0 and bool(torch.isnan(y).all())


def _ids_with(counts, T, k):
    """Ids [T, k] that give expert e counts[e] rows (each at most T, their sum T * k)."""
    ids, free = np.full((T, k), -1, dtype=np.int32), [0] * T
    for e in np.argsort(-np.asarray(counts), kind="stable"):
        for t in sorted(range(T), key=lambda t: (free[t], t))[:counts[e]]:
            ids[t, free[t]] = e
            free[t] += 1
    assert (ids >= 0).all()
    return ids


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("counts,T,k", [
    ([0, 4, 0, 5, 8, 9, 15, 16, 17, 0], 37, 2), ([31, 32, 33, 0, 64], 80, 2), ([65, 0, 65, 0, 0], 65, 2),
    ([127, 128, 129, 0], 192, 2), ([255, 0, 256, 257], 384, 2), ([0, 0, 513, 0, 1], 514, 1)])
def test_ffn_mxfp8_row_counts(counts, T, k, path):
    """Experts without rows and row counts on both sides of every block the kernels take."""
    w = _mx_workload(T, len(counts), k, 192, 128)
    x, x8, perm, offsets, ids = _case(w, _ids_with(counts, T, k))
    arena = device_arena_all_experts(w)
    y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_F32, path)
    assert st == 0
    ref, tol = mx8.expert_ffn(x, perm, k, offsets, _mx_weights(w, range(w.E)))
    _check_ffn(y, moe.MOE_F32, ref, tol)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,k", [(15, 1), (31, 1), (11, 3)])
def test_ffn_mxfp8_work_list_of_single_rows_ends_with_its_workspace(T, k, path):
    """Every row an expert of its own (the longest work list for its rows), sizes at which the
    intermediate ends on an odd multiple of 64 bytes."""
    w = _mx_workload(T, 40, k, 128, 64)
    x, x8, perm, offsets, ids = _case(w, np.arange(T * k, dtype=np.int32).reshape(T, k))
    arena = device_arena_all_experts(w)
    y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_F32, path)
    assert st == 0
    ref, tol = mx8.expert_ffn(x, perm, k, offsets, _mx_weights(w, range(w.E)))
    _check_ffn(y, moe.MOE_F32, ref, tol)


@pytest.mark.parametrize("T,d,f,alpha", [(1, 4096, 2048, 0.2), (8, 4096, 2048, 0.2), (24, 4096, 2048, 1.0)])
def test_ffn_mxfp8_decode_layer(T, d, f, alpha):
    """The decode layer's own sizes: the rows of six experts against the definition."""
    w = _mx_workload(T, 256, 6, d, f, alpha, seed=2)
    x, x8, perm, offsets, ids = _case(w)
    used = sorted(set(ids.ravel().tolist()))
    arena = torch.zeros((w.E, w.entry_bytes), dtype=torch.uint8, device="cuda")
    buf = np.empty((len(used), w.entry_bytes), dtype=np.uint8)
    fill_entries_ptr(w, [(0, e) for e in used], buf.ctypes.data, w.entry_bytes)
    arena[torch.tensor(used, device="cuda")] = torch.from_numpy(buf).cuda()
    ref, tol = mx8.expert_ffn(x, perm, w.k, offsets, _mx_weights(w, used[:6]))
    rows = np.zeros(T * w.k, dtype=bool)
    for e in used[:6]:
        rows[offsets[e]:offsets[e + 1]] = True
    for path in PATHS:
        y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_BF16, path)
        assert st == 0
        _check_ffn(y, moe.MOE_BF16, ref, tol, rows)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [6, 40, 300])
def test_ffn_mxfp8_mask_stale_slots_and_far_entries(T, path):
    """Masked experts and experts with a stale or negative slot leave their rows as they were (the
    latter set MOE_ERANGE); entries sit past 4 GiB of the arena, with a stride above their size."""
    w = _mx_workload(T, 12, 3, 128, 192)
    x, x8, perm, offsets, ids = _case(w)
    stride = w.entry_bytes + 48
    first = (5 << 30) // stride
    arena = torch.empty((first + w.E) * stride, dtype=torch.uint8, device="cuda")
    buf = np.empty((w.E, stride), dtype=np.uint8)
    fill_entries_ptr(w, [(0, e) for e in range(w.E)], buf.ctypes.data, stride)
    order = np.random.default_rng(3).permutation(w.E)
    for e in range(w.E):
        at = (first + int(order[e])) * stride
        arena[at:at + stride] = torch.from_numpy(buf[e]).cuda()
    slots = (first + order).astype(np.int32)
    keys = np.zeros(first + w.E, dtype=np.int32)
    keys[slots] = np.arange(w.E)
    mask = np.ones(w.E, dtype=np.uint8)
    mask[4] = 0
    ref, tol = mx8.expert_ffn(x, perm, w.k, offsets, _mx_weights(w, range(w.E)))
    for stale in ((), (2, 7)):
        k2, s2 = keys.copy(), slots.copy()
        if stale:
            k2[slots[2]] = -9
            s2[7] = -1
        y, st = _ffn(w, x8, dev(perm), dev(offsets), arena, stride, moe.MOE_F32, path, dev(mask), dev(s2), dev(k2))
        off = np.zeros(len(perm), dtype=bool)
        for e in (4,) + stale:
            off[offsets[e]:offsets[e + 1]] = True
        assert off.any() and st == (moe.MOE_ERANGE if stale else 0)
        assert np.isnan(np_of(y)[off]).all()
        _check_ffn(y, moe.MOE_F32, ref, tol, ~off)
    del arena


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [7, 150])
def test_ffn_mxfp8_nan_rows_stay_by_themselves(T, path):
    w = _mx_workload(T, 6, 2, 192, 128)
    x, x8, perm, offsets, ids = _case(w)
    buf = x8.cpu().numpy()
    bad = [0, T // 2, T - 1]
    buf[bad[0] * w.d + 70] = 0x7F                                       # a NaN code
    buf[w.T * w.d + bad[1] * mx8.scale_stride(w.d) + 5] = 255           # a NaN scale, last block
    buf[bad[2] * w.d + 191] = 0xFF
    x = mx8.dequantize(*mx8.unpack(buf, w.T, w.d))
    arena = device_arena_all_experts(w)
    y, st = _ffn(w, dev(buf), dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_F32, path)
    ref, tol = mx8.expert_ffn(x, perm, w.k, offsets, _mx_weights(w, range(w.E)))
    assert st == 0 and np.isnan(ref).any() and not np.isnan(ref).all()
    _check_ffn(y, moe.MOE_F32, ref, tol)


@pytest.mark.parametrize("path", PATHS)
def test_ffn_mxfp8_zero_rows_and_zero_tokens(path):
    """Rows of zeros give zeros; T = 0 writes nothing."""
    w = _mx_workload(9, 4, 2, 128, 64)
    x, x8, perm, offsets, ids = _case(w)
    arena = device_arena_all_experts(w)
    z = torch.zeros_like(x8)
    y, st = _ffn(w, z, dev(perm), dev(offsets), arena, w.entry_bytes, moe.MOE_BF16, path)
    assert st == 0 and bool((y == 0).all())
    y = torch.full((1, w.d), 3.0, device="cuda")
    moe.moe_expert_ffn(x8, moe.MOE_MXFP8, dev(perm), dev(offsets), 0, w.k, w.E, w.d, w.f, None, arena, w.entry_bytes,
                       moe.MOE_MXFP4, None, None, 0, _bytes(256), 256, y, moe.MOE_F32, path)
    torch.cuda.synchronize()
    assert bool((y == 3.0).all())


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_ffn_mxfp8_noalloc_and_other_stream_give_the_same_bits(T):
    w = _mx_workload(T, 24, 4, 512, 256)
    x, x8, perm, offsets, ids = _case(w)
    arena = device_arena_all_experts(w)
    a, _ = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes)
    b, st = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, noalloc=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c, _ = _ffn(w, x8, dev(perm), dev(offsets), arena, w.entry_bytes, stream=s)
    assert st == 0 and torch.equal(a, b) and torch.equal(a, c)


# ---------------------------------------------------------------- as they are used together
@pytest.mark.parametrize("T", [1, 8, 40, 600])
def test_layer_chain(T):
    """Entries quantised on the GPU; residual norm -> router logits -> routing -> FFN -> combine,
    residual and next norm, through MoeLayer.  Each step equals its definition on the inputs that
    it was given, and a captured graph of the chain replays to the same bits on new inputs, with
    eager work between the replays."""
    from expert_ffn_cache_amd.layer import MoeLayer
    E, k, d, f = 16, 3, 256, 192
    r = np.random.default_rng(T)
    entries, _ = _as(r.standard_normal((E, 3 * d * f)) * d ** -0.5, moe.MOE_BF16)
    eb = moe.moe_entry_bytes(d, f, moe.MOE_MXFP4)
    arena = torch.empty((E, eb), dtype=torch.uint8, device="cuda")
    moe.moe_entry_quantize(entries, moe.MOE_BF16, 3 * d * f * 2, E, d, f, arena, eb)
    wr, _ = _as(r.standard_normal((E, d)) * d ** -0.5, moe.MOE_F32)
    g1, _ = _as(1 + 0.1 * r.standard_normal(d), moe.MOE_BF16)
    g2, g2v = _as(1 + 0.1 * r.standard_normal(d), moe.MOE_F32)
    L = MoeLayer(T, E, k, d, f, dtype=moe.MOE_MXFP8)
    assert L.w_dtype == moe.MOE_MXFP4 and not L.fusable
    f32 = dict(dtype=torch.float32, device="cuda")
    res, add, s1, s2 = (torch.empty((T, d), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    y1, y2, lg = torch.empty((T, d), **f32), torch.empty((T, d), **f32), torch.empty((T, E), **f32)
    y8 = _bytes(moe.moe_mxfp8_bytes(T, d))

    def chain(stream=None):
        L.norm(res, g1, 1e-6, delta=add, x_out=s1, y=y1, stream=stream)
        moe.moe_router_logits(y1, wr, moe.MOE_F32, T, d, E, lg, stream)
        L.route_permute(lg, stream)
        L.ffn(L.x8, arena, eb, stream=stream)
        L.combine_norm(s1, g2, 1e-6, x_out=s2, y=y2, x8=y8, stream=stream)

    def inputs(seed):
        q = np.random.default_rng(seed)
        res.copy_(_as(q.standard_normal((T, d)), moe.MOE_BF16)[0])
        add.copy_(_as(q.standard_normal((T, d)), moe.MOE_BF16)[0])

    def state():
        return [t.clone() for t in (s1, y1, L.x8, lg, L.ids, L.y_perm, s2, y2, y8)]
    eager = []
    for i in range(3):
        inputs(100 + i)
        chain()
        torch.cuda.synchronize()
        eager.append(state())
    # the last eager run, step by step
    x = mx8.dequantize(*mx8.unpack(L.x8.cpu().numpy(), T, d))
    perm, offsets = L.perm.cpu().numpy(), L.offsets.cpu().numpy()
    mx = mx_values(arena.cpu().numpy(), E, d, f)
    wts = {e: (mx[e, :d * f].reshape(f, d), mx[e, d * f:2 * d * f].reshape(f, d), mx[e, 2 * d * f:].reshape(d, f))
           for e in range(E)}
    ref, tol = mx8.expert_ffn(x, perm, k, offsets, wts)
    _check_ffn(L.y_perm, moe.MOE_F32, ref, tol)
    L.combine()
    s = np_of((s1.float() + L.out).bfloat16().float())
    np.testing.assert_array_equal(np_of(s2.float()), s)
    _check_norm(s.astype(np.float64), g2v, 1e-6, y2, moe.MOE_F32, y8)
    # forward() from bf16 rows: quantised by the layer
    out = L.forward(y1, lg, arena, eb)
    L.quantize(y1)
    assert torch.equal(L.x8, eager[-1][2]) and torch.isfinite(out).all() and int(L.status.item()) == 0
    # captured and replayed
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        chain(st)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            chain(st)
    torch.cuda.current_stream().wait_stream(st)
    for i in (0, 1, 2, 1):
        inputs(100 + i)
        y2.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(state(), eager[i]):
            assert torch.equal(u, v)
        assert float((y2 * 0).sum()) == 0.0


def test_two_layers_side_by_side_on_two_streams():
    """Calls that share nothing but the weights may overlap."""
    w = _mx_workload(64, 24, 4, 512, 256)
    arena = device_arena_all_experts(w)
    cases = [_case(configs.with_(w, seed=w.seed + i)) for i in range(2)]
    want = [_ffn(w, c[1], dev(c[2]), dev(c[3]), arena, w.entry_bytes)[0] for c in cases]
    args = [(c[1], dev(c[2]), dev(c[3])) for c in cases]
    A = w.T * w.k
    ws = [_bytes(moe.moe_expert_ffn_workspace_bytes(w.T, w.k, w.f, moe.MOE_MXFP8)) for _ in cases]
    y = [torch.zeros((A, w.d), device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            moe.moe_expert_ffn(args[i][0], moe.MOE_MXFP8, args[i][1], args[i][2], w.T, w.k, w.E, w.d, w.f, None, arena,
                               w.entry_bytes, moe.MOE_MXFP4, None, None, 0, ws[i], ws[i].numel(), y[i], moe.MOE_F32,
                               moe.MOE_PATH_AUTO, None, s)
    torch.cuda.synchronize()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])

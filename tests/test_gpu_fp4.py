"""GPU parity of the block-scaled 4-bit KV cache: the quantising append byte for
byte, the load value for value, and attention over it against the float64
oracle.  Unwritten rows hold bytes that stand for nothing (NaN scales)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_18_gb300 as pkv
from oracle import fp4
from paged_kv_cache_18_gb300 import workloads as W
from tests.gpu_util import TORCH_DT, dev_tensor, half_ulp, host_f64, tuning

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
K_SCALE, V_SCALE = 0.0091, 0.0047


def wide(a, dtype):
    return W.storage_to_f64(a, dtype).astype(np.float32)


def caches_of(b, k_scale=K_SCALE, v_scale=V_SCALE):
    dt = b.wl.dtype
    return (fp4.pack(wide(b.k_cache, dt), k_scale, True),
            fp4.pack(wide(b.v_cache, dt), v_scale, False))


def bound(q, k, v, table, lens, scale, dtype, out):
    """What the float arithmetic may add to the exact result, from the data.

    A score is a sum of D products and a few further float32 operations, so it
    is off by at most (D + 8) 2^-24 sum |q_d k_d| scale; a weight then by twice
    that (its own and the row maximum's), 2^-20 for the exponential and its
    argument's rounding, and (keys) 2^-24 for the sums; with 16-bit queries by
    2^-11 more (weights rounded to f16 for the products), plus 2^-13 for the
    tails of query elements that underflow when a row is shifted into f16.  The
    output is off by that times the largest value in its column, and by half a
    unit of its type."""
    B, Q, Hq, D = q.shape
    group = Hq // k.shape[1]
    extra = np.zeros((B, 1, Hq, D))
    for i in range(B):
        L = int(lens[i])
        if L <= 0:
            continue
        rows = lambda c: c[table[i, :-(-L // 16)]].transpose(1, 0, 2, 3).reshape(  # noqa: E731
            c.shape[1], -1, D)[:, :L]
        kk, vv = np.abs(rows(k)), np.abs(rows(v))
        top = np.einsum("jhgd,hnd->hgjn", np.abs(q[i]).reshape(Q, k.shape[1], group, D), kk)
        delta = 2 * (D + 8) * 2.0 ** -24 * scale * top.max(axis=(2, 3)) + 2.0 ** -20 + L * 2.0 ** -24
        if dtype != "f32":
            delta = delta + 2.0 ** -11 + 2.0 ** -13
        extra[i, 0] = (delta[..., None] * vv.max(axis=1)[:, None]).reshape(Hq, D)
    return half_ulp(out, dtype) * (1 + 1e-6) + extra + 1e-30


def check(got, ref, tol, what):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over the bound at {np.abs(got - ref).max():.3e}"


def run(wl, kernel=0, split_blocks=0, k_scale=K_SCALE, v_scale=V_SCALE, q_gain=None, tree=None,
        keep=None, **more):
    b = W.make_batch(wl)
    if q_gain is not None:
        b.q = W.to_storage(wide(b.q, wl.dtype) * np.float32(q_gain).reshape(1, 1, -1, 1),
                           wl.dtype).reshape(b.q.shape)
    kc, vc = caches_of(b, k_scale, v_scale)
    dk, dv = torch.from_numpy(kc.copy()).to(DEV), torch.from_numpy(vc.copy()).to(DEV)
    kn, vn = dev_tensor(b.k_new, wl.dtype, DEV), dev_tensor(b.v_new, wl.dtype, DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.kv_append_fp4(kn, vn, dk, dv, torch.from_numpy(b.slot_mapping).to(DEV), k_scale, v_scale,
                      error_word=err)
    fp4.append(kc, vc, wide(b.k_new, wl.dtype), wide(b.v_new, wl.dtype), b.slot_mapping, k_scale,
               v_scale)
    np.testing.assert_array_equal(dk.cpu().numpy(), kc)
    np.testing.assert_array_equal(dv.cpu().numpy(), vc)
    q = dev_tensor(b.q, wl.dtype, DEV)
    if wl.num_queries == 1:
        q = q[:, 0].contiguous()
    mask = None if tree is None else torch.from_numpy(tree.view(np.int64)).to(DEV)
    with tuning(**more):
        out = pkv.paged_attention_fp4(q, dk, dv, torch.from_numpy(b.block_table).to(DEV),
                                      torch.from_numpy(b.context_lens).to(DEV), k_scale, v_scale,
                                      scale=wl.softmax_scale, max_context_len=b.max_context_len,
                                      tree_mask=mask, kernel=kernel, split_blocks=split_blocks,
                                      error_word=err)
    torch.cuda.synchronize()
    assert pkv.read_error_word(err) == 0
    qf = wide(b.q, wl.dtype)
    ref = fp4.attention(qf, kc, vc, b.block_table, b.context_lens, wl.softmax_scale, k_scale,
                        v_scale, tree)
    k, v = fp4.unpack(kc, True), fp4.unpack(vc, False)
    tol = bound(qf.astype(np.float64), np.nan_to_num(k) * k_scale, np.nan_to_num(v) * v_scale,
                b.block_table, b.context_lens, wl.softmax_scale, wl.dtype, ref)
    got = host_f64(out if wl.num_queries > 1 else out[:, None], wl.dtype)
    check(got, ref, tol, wl.name)
    if keep is not None:
        keep.update(b=b, dk=dk, dv=dv, q=q, out=out, table=torch.from_numpy(b.block_table).to(DEV),
                    lens=torch.from_numpy(b.context_lens).to(DEV))
    return got, ref


# ---- rows in and out -----------------------------------------------------------------
def new_rows(T, H, D, dtype, seed=1):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x *= (2.0 ** rng.integers(-12, 6, (T, H, 1))).astype(np.float32)
    if T > 3:
        x[0] = 0                                    # a row of zeros
        x[1] = 1e-12                                # scales that round to zero
        x[2, :, ::16] = np.inf                      # saturating blocks
        x[2, :, 1::16] = -np.inf
        x[3, 0, 5] = np.nan                         # one block without values
    return torch.from_numpy(x).to(TORCH_DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H,D", [(1, 1, 64), (7, 3, 64), (33, 2, 128), (16, 5, 128), (9, 2, 256),
                                   (257, 1, 256)])
def test_append_and_load(dtype, T, H, D):
    NB = T // 16 + 3
    k, v = new_rows(T, H, D, dtype, 1), new_rows(T, H, D, dtype, 2)
    rng = np.random.default_rng(T)
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    if T > 4:
        slots[4] = -1
    fill = rng.integers(0, 256, (2,) + pkv.fp4_cache_shape(NB, H, D), dtype=np.uint8)
    kc, vc = fill[0].copy(), fill[1].copy()
    dk, dv = torch.from_numpy(fill[0]).to(DEV), torch.from_numpy(fill[1]).to(DEV)
    ds = torch.from_numpy(slots).to(DEV)
    pkv.kv_append_fp4(k.to(DEV), v.to(DEV), dk, dv, ds, K_SCALE, V_SCALE)
    with np.errstate(all="ignore"):
        fp4.append(kc, vc, k.float().numpy(), v.float().numpy(), slots, K_SCALE, V_SCALE)
    np.testing.assert_array_equal(dk.cpu().numpy(), kc)       # every byte, written or not
    np.testing.assert_array_equal(dv.cpu().numpy(), vc)
    named = np.concatenate([slots, slots[:1], [-5]])           # one slot twice, padding
    for out_t in (torch.float32, torch.bfloat16, torch.float16):
        lk, lv = pkv.kv_load_fp4(dk, dv, torch.from_numpy(named).to(DEV), K_SCALE, V_SCALE,
                                 dtype=out_t)
        for got, cache, scale, keys in ((lk, kc, K_SCALE, True), (lv, vc, V_SCALE, False)):
            want = torch.from_numpy(fp4.load(cache, named, scale, keys)).to(out_t)
            assert torch.equal(torch.nan_to_num(got.cpu(), 77.0), torch.nan_to_num(want, 77.0))


def test_append_of_a_long_prompt_matches_in_every_byte():
    T, H, D = 3001, 4, 128
    k, v = new_rows(T, H, D, "bf16", 3), new_rows(T, H, D, "bf16", 4)
    NB = 200
    slots = np.random.default_rng(5).permutation(NB * 16)[:T].astype(np.int64)
    kc = np.zeros(pkv.fp4_cache_shape(NB, H, D), np.uint8)
    vc = kc.copy()
    dk, dv = torch.from_numpy(kc).to(DEV), torch.from_numpy(vc).to(DEV)
    pkv.kv_append_fp4(k.to(DEV), v.to(DEV), dk, dv, torch.from_numpy(slots).to(DEV), 1.0, 0.37)
    with np.errstate(all="ignore"):
        fp4.append(kc, vc, k.float().numpy(), v.float().numpy(), slots, 1.0, 0.37)
    np.testing.assert_array_equal(dk.cpu().numpy(), kc)
    np.testing.assert_array_equal(dv.cpu().numpy(), vc)


@pytest.mark.parametrize("t", [1.0, 0.0091, 1e-30, 1e30, 2.0 ** -126, 1e-40, 6e34,
                               1.9999998807907104])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_append_over_the_whole_range(t, dtype):
    # magnitudes from subnormal to the largest, blocks of one magnitude and of
    # many, values on and beside the codes' borders, signed zeros
    T, H, D = 48, 2, 64
    rng = np.random.default_rng(11)
    with np.errstate(all="ignore"):
        x = rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-30, 12, (T, H, D // 16)).repeat(
            16, -1) * min(t, 1e37)
        x[:8] = 2.0 ** rng.uniform(-149, 127.9, (8, H, D)) * rng.choice([-1, 1], (8, H, D))
        ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]) * t * 1.125
        x[8:16] = rng.choice(np.concatenate([ties, -ties, [0.0, -0.0]]), (8, H, D))
        x[16:20] = np.nextafter(x[8:12].astype(np.float32), np.float32(0))
        rows = torch.from_numpy(x.astype(np.float32)).to(TORCH_DT[dtype])
    shape = pkv.fp4_cache_shape(4, H, D)
    kc, vc = np.zeros(shape, np.uint8), np.zeros(shape, np.uint8)
    dk, dv = torch.zeros(shape, dtype=torch.uint8, device=DEV), torch.zeros(
        shape, dtype=torch.uint8, device=DEV)
    slots = np.arange(T)
    pkv.kv_append_fp4(rows.to(DEV), (-rows).to(DEV), dk, dv, torch.from_numpy(slots).to(DEV), t, t)
    with np.errstate(all="ignore"):
        fp4.append(kc, vc, rows.float().numpy(), -rows.float().numpy(), slots, t, t)
    np.testing.assert_array_equal(dk.cpu().numpy(), kc)
    np.testing.assert_array_equal(dv.cpu().numpy(), vc)


def test_rows_at_16_byte_alignment():
    T, H, D = 19, 2, 64
    k, v = new_rows(T, H, D, "bf16", 12), new_rows(T, H, D, "bf16", 13)

    def shifted(x):  # the same rows 16 bytes into an allocation
        flat = torch.empty(x.numel() + 8, dtype=x.dtype, device=DEV)
        out = flat[8:].view(x.shape)
        out.copy_(x)
        assert out.data_ptr() % 32 == 16
        return out

    shape = pkv.fp4_cache_shape(3, H, D)
    caches = [torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(4)]
    slots = torch.arange(T, device=DEV)
    pkv.kv_append_fp4(k.to(DEV), v.to(DEV), caches[0], caches[1], slots, 0.02, 0.02)
    pkv.kv_append_fp4(shifted(k), shifted(v), caches[2], caches[3], slots, 0.02, 0.02)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    outs = [shifted(torch.zeros_like(k)), shifted(torch.zeros_like(v))]
    pkv.kv_load_fp4(caches[0], caches[1], slots, 0.02, 0.02, k_out=outs[0], v_out=outs[1])
    want = pkv.kv_load_fp4(caches[0], caches[1], slots, 0.02, 0.02)
    for got, w in zip(outs, want):
        assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(w, 9.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_elements_at_the_ties_between_codes(dtype):
    # the elements nearest to every tie of their block, and the ones beside them, for
    # tensor scales that put ties on, next to and far from 16-bit numbers
    rng = np.random.default_rng(11)
    td = TORCH_DT[dtype]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    scales = [1.0, 0.0091, 1.0 + 2.0 ** -23, 1.0 - 2.0 ** -24, 0.75 + 2.0 ** -24]
    scales += [float(np.float32(x)) for x in rng.uniform(0.5, 2.0, 40)]
    scales += [float(np.float32(a * (1 + e * 2.0 ** -23))) for a in (1.0, 1 / 3, 1 / 5, 1 / 7)
               for e in range(-6, 7)]
    for t in scales:
        rows = []
        for top in np.float32(t) * rng.uniform(0.3, 40.0, 24).astype(np.float32):
            big = torch.tensor(top).to(td)
            _, s = fp4.quantise(np.full((1, 1, 16), big.float().item(), np.float32), t)
            f = np.float32(fp4.SCALE_VALUES[s.item()]) * np.float32(t)
            near = torch.from_numpy(np.concatenate([ties * f, -ties * f])).to(td)
            row = torch.cat([big[None], near, -torch.zeros(1, dtype=td)])
            bits = row.view(torch.int16)
            for step in (-1, 0, 1):
                moved = bits.clone()
                moved[1:15] += step
                rows.append(moved.view(td))
        x = torch.stack(rows).view(-1, 1, 64).contiguous()
        cache = torch.zeros(pkv.fp4_cache_shape(-(-len(x) // 16), 1, 64), dtype=torch.uint8,
                            device=DEV)
        other = torch.zeros_like(cache)
        pkv.kv_append_fp4(x.to(DEV), x.to(DEV), cache, other, torch.arange(len(x), device=DEV), t, t)
        want = np.zeros(cache.shape, np.uint8)
        fp4.write_rows(want, list(range(len(x))), *fp4.quantise(x.float().numpy(), t), True)
        np.testing.assert_array_equal(cache.cpu().numpy(), want)


def test_slots_past_the_cache_are_recorded_and_left_out():
    H, D, NB = 2, 64, 2
    k = new_rows(3, H, D, "f32").to(DEV)
    dk = torch.zeros(pkv.fp4_cache_shape(NB, H, D), dtype=torch.uint8, device=DEV)
    dv = dk.clone()
    slots = torch.tensor([32, 5, 1 << 40], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.kv_append_fp4(k, k, dk, dv, slots, 1.0, 1.0, error_word=err)
    assert pkv.read_error_word(err) == 1
    want = np.zeros(dk.shape, np.uint8)
    fp4.write_rows(want, [5], *fp4.quantise(k[1:2].cpu().numpy(), 1.0), True)
    np.testing.assert_array_equal(dk.cpu().numpy(), want)
    err.zero_()
    lk, _ = pkv.kv_load_fp4(dk, dv, slots, 1.0, 1.0, dtype=torch.float32, error_word=err)
    assert pkv.read_error_word(err) == 1
    assert (lk[[0, 2]] == 0).all() and (lk[1] != 0).any()


def test_no_rows_is_a_no_op():
    dk = torch.zeros(pkv.fp4_cache_shape(2, 1, 64), dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, 1, 64, device=DEV)
    slots = torch.zeros(0, dtype=torch.int64, device=DEV)
    pkv.kv_append_fp4(none, none, dk, dk.clone(), slots, 1.0, 1.0)
    k, v = pkv.kv_load_fp4(dk, dk.clone(), slots, 1.0, 1.0)
    assert k.shape == v.shape == (0, 1, 64)


# ---- attention ------------------------------------------------------------------------
LENS = [1, 15, 16, 17, 33, 250, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Q,Hq,Hkv", [(1, 8, 8), (1, 8, 2), (1, 7, 1), (5, 8, 2), (2, 4, 1),
                                      (3, 9, 3), (10, 8, 2)])
def test_attention(dtype, D, Q, Hq, Hkv):
    lens = [max(n, Q) for n in LENS]
    run(W.Workload(f"fp4 {dtype} D{D} Q{Q} {Hq}/{Hkv}", len(lens), Hq, Hkv, D, dtype,
                   context_lens=lens, num_queries=Q, seed=2000 + D + Q + Hq))


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split_blocks", [1, 3, 16, 1000])
@pytest.mark.parametrize("Q", [1, 4])
def test_splits(kernel, dtype, split_blocks, Q):
    run(W.Workload("fp4 split", 4, 32, 8, 128, dtype, context_lens=[Q, 200, 1500, 3000],
                   num_queries=Q, seed=2100 + split_blocks), kernel=kernel,
        split_blocks=split_blocks)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("rows", [1, 3, 5])
def test_row_chunks(kernel, rows):
    run(W.Workload("fp4 chunks", 3, 12, 2, 128, "f16", context_lens=[7, 64, 517], num_queries=4,
                   seed=2150), kernel=kernel, rows_per_cta=rows)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Q,Hq,Hkv", [(2, 8, 2), (3, 8, 2), (5, 8, 2), (8, 8, 2), (10, 8, 2),
                                      (11, 8, 2), (13, 8, 2), (31, 4, 1), (64, 3, 1)])
@pytest.mark.parametrize("split_blocks", [0, 5])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_column_tile(dtype, D, Q, Hq, Hkv, split_blocks):
    lens = [Q, Q + 1, Q + 40, 333, 1200]
    if dtype == "bf16":
        cap, built = (64, (1, 2, 3, 4, 5, 6, 8)) if D <= 128 else (32, (1, 2, 4))
        rows = Q * Hq // Hkv
        chunks = -(-rows // cap)
        tiles = -(-(-(-rows // chunks)) // 8)
        p = pkv.plan(len(lens), Q, Hq, Hkv, D, max(lens), "fp4", split_blocks=split_blocks)
        assert p["row_chunks"] == chunks and p["warp_tiles"] == min(n for n in built if n >= tiles)
    run(W.Workload("fp4 tiles", len(lens), Hq, Hkv, D, dtype, context_lens=lens, num_queries=Q,
                   seed=2155 + Q), split_blocks=split_blocks)


@pytest.mark.parametrize("Q,Hq", [(1, 8), (2, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_units_at_head_dim_256(dtype, Q, Hq):
    lens = [Q + n for n in [0, 14, 15, 16, 31, 32, 33, 400, 1100, 780] * 4]
    p = pkv.plan(len(lens), Q, Hq, 8, 256, max(lens), "fp4")
    assert p["split_target"] == 4 * p["grid_x"]  # (warps are the workers)
    run(W.Workload("fp4 units", len(lens), Hq, 8, 256, dtype, context_lens=lens, num_queries=Q,
                   seed=2158 + Q))


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("D,Q,dtype", [(128, 1, "bf16"), (64, 3, "f16"), (256, 2, "f32")])
def test_partition_from_the_real_lengths(kernel, D, Q, dtype):
    run(W.Workload("fp4 waves", 5, 8, 2, D, dtype, context_lens=[Q, 40, 2000, 300, 5000],
                   num_queries=Q, seed=2160 + D), kernel=kernel, split_waves=1)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("f32", 128), ("bf16", 256)])
@pytest.mark.parametrize("per_sequence", [False, True])
def test_tree_masks(dtype, D, per_sequence):
    Q, lens = 10, [10, 11, 33, 250, 700]
    masks = W.tree_mask_bits(W.medusa_parents((3, 2)))
    if per_sequence:
        rng = np.random.default_rng(4)
        masks = np.stack([masks & rng.integers(0, 2 ** Q, Q).astype(np.uint64) for _ in lens])
    run(W.Workload("fp4 tree", len(lens), 32, 8, D, dtype, context_lens=lens, num_queries=Q,
                   seed=2170 + D), tree=np.ascontiguousarray(masks))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing_are_zero(dtype):
    # empty sequences, and causal rows before the first cached one (L < Q)
    wl = W.Workload("fp4 empty", 4, 8, 2, 128, dtype, context_lens=[0, 2, 40, 0], num_queries=5,
                    seed=2180)
    got, _ = run(wl)
    assert (got[0] == 0).all() and (got[3] == 0).all() and (got[1, :3] == 0).all()
    assert (got[1, 3:] != 0).any()
    # a tree whose masks leave a node without itself, in a sequence of nothing else
    masks = np.array([1, 0, 5], np.uint64)
    got, _ = run(W.Workload("fp4 tree empty", 2, 4, 4, 64, dtype, context_lens=[3, 20],
                            num_queries=3, seed=2181), tree=masks)
    assert (got[0, 1] == 0).all() and (got[1, 1] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kernel", [0, 1])
def test_query_range(kernel, dtype):
    gains = [3.0e4, 1.0e-6, 1.0, 2.0 ** 40, 2.0 ** -60, 0.0, 7.5, 1.0e8]
    run(W.Workload("fp4 q range", 3, 8, 2, 128, dtype, context_lens=[5, 64, 517], seed=2190),
        kernel=kernel, q_gain=gains)


@pytest.mark.parametrize("k_scale,v_scale", [(1.0, 1.0), (2e-4, 1e-4), (1e3, 1e-6), (1e-20, 1e10)])
def test_tensor_scales(k_scale, v_scale):
    # saturating, underflowing and far-off scales: the codes are what counts
    run(W.Workload("fp4 scales", 3, 8, 2, 128, "f32", context_lens=[10, 90, 300], seed=2200),
        k_scale=k_scale, v_scale=v_scale)


@pytest.mark.parametrize("dtype,kernel", [("bf16", 0), ("f16", 0), ("f32", 0), ("f32", 1)])
@pytest.mark.parametrize("Q,split_blocks", [(1, 0), (1, 100000), (5, 0)])
def test_a_peak_over_a_long_flat_tail(dtype, kernel, Q, split_blocks):
    # one key scores 20 bits above 40000 equal ones, which together weigh 5 % of
    # it: every weight of the tail has to keep its bits (rounded to a multiple of
    # 2^-24 of the peak each would be off by 3 %, the result by 1e-3)
    D, L = 64, 40000
    NB = -(-L // 16)
    k = np.zeros((NB, 1, 16, D), np.float32)
    v = np.ones((NB, 1, 16, D), np.float32)
    k[7, 0, 3, 0] = 6.0
    v[7, 0, 3] = -0.5
    kc, vc = fp4.pack(k, 1.0, True), fp4.pack(v, 1.0, False)
    q = np.zeros((1, Q, 2, D), np.float32)
    scale = 0.125
    q[..., 0] = 19.55 * math.log(2.0) / 6.0 / scale
    qt = torch.from_numpy(q).to(TORCH_DT[dtype])
    table, lens = np.arange(NB, dtype=np.int32)[None], np.array([L], np.int32)
    got = pkv.paged_attention_fp4((qt if Q > 1 else qt[:, 0]).contiguous().to(DEV),
                                  torch.from_numpy(kc).to(DEV), torch.from_numpy(vc).to(DEV),
                                  torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV),
                                  1.0, 1.0, scale=scale, max_context_len=L,
                                  kernel=kernel, split_blocks=split_blocks)
    ref = fp4.attention(qt.float().numpy(), kc, vc, table, lens, scale, 1.0, 1.0)
    got = got.double().cpu().numpy().reshape(ref.shape)
    # the output's rounding, the exponentials' argument (20 bits at 2^-24 relative),
    # the float32 sums, and the weights' 2^-11 (the peak's own)
    tol = half_ulp(ref, dtype) + 20 * 2.0 ** -23
    if dtype == "f32":
        # On CUDA cores a warp adds every fourth block key by key.  Its running numerator is at most
        # 0.5 + 0.013, so each of its L / 4 additions is off by at most 2^-25; its sum of
        # weights is below 2, and gets one addition a block, off by at most 2^-24.
        tol = tol + L / 4 * 2.0 ** -25 + L / 64 * 2.0 ** -24
    else:
        tol = tol + L * 2.0 ** -24 * 0.04 + 2.0 ** -11 * 0.04 + 2.0 ** -14 * 0.5
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_vanishing_scores_average_the_values(dtype):
    # softmax scale times key scale below the smallest float: all weights equal
    wl = W.Workload("fp4 vanishing", 2, 8, 2, 64, dtype, context_lens=[20, 700], seed=2205,
                    scale=1e-30)
    run(wl, k_scale=1e-20, v_scale=0.01)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_blocks_and_lengths_are_recorded(dtype):
    wl = W.Workload("fp4 bad", 3, 8, 2, 128, dtype, context_lens=[40, 40, 40], seed=2210)
    keep = {}
    run(wl, keep=keep)
    b = keep["b"]
    table = b.block_table.copy()
    table[1, 1] = b.num_blocks
    table[2, 0] = -7
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.from_numpy(b.context_lens).to(DEV)
    out = pkv.paged_attention_fp4(keep["q"], keep["dk"], keep["dv"],
                                  torch.from_numpy(table).to(DEV), lens, K_SCALE, V_SCALE,
                                  max_context_len=40, error_word=err)
    assert pkv.read_error_word(err) == 2
    assert torch.equal(out[0], keep["out"][0]) and torch.isfinite(out.float()).all()
    err.zero_()
    lens[0] = 41                                              # over max_context_len
    out = pkv.paged_attention_fp4(keep["q"], keep["dk"], keep["dv"],
                                  torch.from_numpy(b.block_table).to(DEV), lens, K_SCALE, V_SCALE,
                                  max_context_len=40, error_word=err)
    assert pkv.read_error_word(err) == 3
    assert torch.equal(out, keep["out"])


@pytest.mark.parametrize("L", [20, 3000])
@pytest.mark.parametrize("dtype,kernel,split_blocks", [
    ("bf16", 0, 0), ("bf16", 0, 16), ("bf16", 1, 0), ("f32", 0, 16), ("f32", 0, 0)])
def test_a_nan_block_reaches_the_rows_that_see_it(L, dtype, kernel, split_blocks):
    wl = W.Workload("fp4 nan", 2, 4, 2, 128, dtype, context_lens=[L, L], seed=2220)
    keep = {}
    run(wl, keep=keep, kernel=kernel, split_blocks=split_blocks)
    b = keep["b"]
    kn = dev_tensor(b.k_new, dtype, DEV).clone()
    vn = dev_tensor(b.v_new, dtype, DEV)
    kn[0, 1, 3] = float("nan")
    slots = torch.from_numpy(b.slot_mapping).to(DEV)
    pkv.kv_append_fp4(kn, vn, keep["dk"], keep["dv"], slots, K_SCALE, V_SCALE)
    out = pkv.paged_attention_fp4(keep["q"], keep["dk"], keep["dv"],
                                  torch.from_numpy(b.block_table).to(DEV),
                                  torch.from_numpy(b.context_lens).to(DEV), K_SCALE, V_SCALE,
                                  scale=wl.softmax_scale, max_context_len=L, kernel=kernel,
                                  split_blocks=split_blocks)
    assert torch.isnan(out[0, 2:].float()).all()              # heads of KV head 1
    assert torch.equal(out[0, :2], keep["out"][0, :2]) and torch.equal(out[1], keep["out"][1])


@pytest.mark.parametrize("Q,lens", [(1, [0, 300, 5, 4000, 0, 16, 17, 1]), (1, [2000]),
                                    (4, [4, 900, 35, 64])])
@pytest.mark.parametrize("batch", [1, 40])
def test_balanced_partition(Q, lens, batch):
    # ragged and empty sequences, beyond 32 of them, workers CTAs or warps
    wl = W.Workload("fp4 balanced", len(lens) * batch, 16, 16 if Q == 1 else 4, 64, "bf16",
                    context_lens=lens * batch, num_queries=Q, seed=2225)
    p = pkv.plan(wl.batch, Q, 16, wl.num_kv_heads, 64, max(lens), "fp4")
    assert p["stream_k"] == 1 and p["split_target"] % p["grid_x"] == 0
    run(wl)


# ---- as a program uses it ---------------------------------------------------------------
def batch_on_device(wl):
    keep = {}
    run(wl, keep=keep)
    b = keep["b"]
    keep["table"] = torch.from_numpy(b.block_table).to(DEV)
    keep["lens"] = torch.from_numpy(b.context_lens).to(DEV)
    keep["call"] = lambda **kw: pkv.paged_attention_fp4(
        keep["q"], keep["dk"], keep["dv"], keep["table"], keep["lens"], K_SCALE, V_SCALE,
        scale=wl.softmax_scale, max_context_len=b.max_context_len, **kw)
    return keep


def test_side_stream_given_output_and_dirty_workspace():
    keep = batch_on_device(W.Workload("fp4 stream", 2, 32, 8, 128, "bf16",
                                      context_lens=[3000, 5000], seed=2230))
    p = pkv.plan(2, 1, 32, 8, 128, 5000, "fp4")
    assert p["num_splits"] > 1
    need = pkv.workspace_size(2, 1, 32, 8, 128, 5000, "fp4")
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full_like(keep["q"], float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            got = keep["call"](out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out, keep["out"])
    with pytest.raises(pkv.PkvError):
        keep["call"](workspace=ws[: need - 16])


def test_two_streams_at_once():
    # calls that run side by side, a workspace each, give what they give alone
    keeps, alone = [], []
    for i, (dtype, Q) in enumerate([("bf16", 1), ("f32", 3)]):
        keep = {}
        run(W.Workload("fp4 streams", 6, 16, 4, 128, dtype, context_lens=[Q, 900, 2500, 33, 1600, 16],
                       num_queries=Q, seed=2230 + i), keep=keep)
        keeps.append((keep, torch.cuda.Stream()))
        alone.append(keep["out"].clone())
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for keep, stream in keeps:
            b = keep["b"]
            with torch.cuda.stream(stream):
                got.append(pkv.paged_attention_fp4(
                    keep["q"], keep["dk"], keep["dv"], keep["table"], keep["lens"], K_SCALE, V_SCALE,
                    scale=b.wl.softmax_scale, max_context_len=2500))
        torch.cuda.synchronize()
        for g, a in zip(got, alone):
            assert torch.equal(g, a)


@pytest.mark.parametrize("dtype,Q", [("bf16", 1), ("f32", 1), ("f16", 5)])
def test_more_sequences_than_the_balanced_partition_takes(dtype, Q):
    lens = [Q + (37 * i) % 300 for i in range(1100)]
    p = pkv.plan(len(lens), Q, 2, 1, 64, max(lens), "fp4")
    assert p["stream_k"] == 0
    run(W.Workload("fp4 many", len(lens), 2, 1, 64, dtype, context_lens=lens, num_queries=Q,
                   seed=2240 + Q))


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("L", [100, 2000])
def test_a_query_that_is_not_finite_is_its_own_affair(dtype, kernel, L):
    keep = {}
    run(W.Workload("fp4 not finite", 3, 8, 2, 128, dtype, context_lens=[L, L - 7, 40], seed=2250),
        kernel=kernel, keep=keep)
    q = keep["q"].clone()
    flat = q.view(3, 8, 128)
    flat[0, 1, 5], flat[1, 6, 127], flat[2, 3, 0] = float("nan"), float("inf"), float("-inf")
    call = lambda x: pkv.paged_attention_fp4(  # noqa: E731
        x, keep["dk"], keep["dv"], keep["table"], keep["lens"], K_SCALE, V_SCALE,
        scale=keep["b"].wl.softmax_scale, max_context_len=L, kernel=kernel)
    want, got = call(keep["q"]).view(3, 8, 128), call(q).view(3, 8, 128)
    for b in range(3):
        for h in range(8):
            if (b, h) in ((0, 1), (1, 6), (2, 3)):
                assert torch.isnan(got[b, h]).all()
            else:
                assert torch.isfinite(got[b, h]).all()
                # (another reference may be taken: each is within half a bf16 step of the
                # output, 2^-8, and the weights' 2^-11 and 2^-13 of the formula's value)
                far = (got[b, h].float() - want[b, h].float()).abs().max().item()
                near = 2 * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13)
                assert far <= near * want[b].float().abs().max().item()


def test_calls_are_bitwise_repeatable():
    keep = batch_on_device(W.Workload("fp4 repeat", 3, 32, 8, 128, "f16",
                                      context_lens=[900, 5000, 17], num_queries=3, seed=2240))
    for _ in range(5):
        assert torch.equal(keep["call"](), keep["out"])


def test_graphs_with_a_workspace_each_replay_over_new_rows():
    wl = W.Workload("fp4 graph", 2, 32, 8, 128, "bf16", context_lens=[700, 4000], seed=2250)
    keep = batch_on_device(wl)
    b = keep["b"]
    kn, vn = dev_tensor(b.k_new, "bf16", DEV).clone(), dev_tensor(b.v_new, "bf16", DEV).clone()
    slots = torch.from_numpy(b.slot_mapping).to(DEV)

    def step():
        pkv.kv_append_fp4(kn, vn, keep["dk"], keep["dv"], slots, K_SCALE, V_SCALE)
        return keep["call"]()

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for n in range(3):
        kn.normal_(generator=torch.Generator(device=DEV).manual_seed(n))
        vn.normal_(generator=torch.Generator(device=DEV).manual_seed(9 + n))
        for g, out in graphs:
            out.fill_(float("nan"))
            g.replay()
        want = step()
        for _, out in graphs:
            assert torch.equal(out, want)


def test_block_copies_carry_the_tiles():
    keep = batch_on_device(W.Workload("fp4 copy", 1, 8, 2, 128, "bf16", context_lens=[40],
                                      seed=2260))
    owned = keep["table"][0, :3].tolist()
    free = [i for i in range(keep["b"].num_blocks) if i not in owned]
    if not free:
        pad = torch.zeros_like(keep["dk"][:1])
        keep["dk"], keep["dv"] = torch.cat([keep["dk"], pad]), torch.cat([keep["dv"], pad])
        free = [keep["b"].num_blocks]
    pkv.copy_blocks(keep["dk"], keep["dv"], owned[1:2], free[:1])
    keep["dk"][owned[1]] = 255
    keep["dv"][owned[1]] = 255
    keep["table"][0, 1] = free[0]
    assert torch.equal(keep["call"](), keep["out"])


def test_offsets_past_32_bits():
    # a cache of more than 2^32 bytes, its rows at the far end
    H, D, NB = 8, 128, (1 << 32) // (8 * 1152) + 64
    dk = torch.empty(pkv.fp4_cache_shape(NB, H, D), dtype=torch.uint8, device=DEV)
    dv = torch.empty_like(dk)
    blocks = [NB - 1, 3, NB - 2]
    T = 40
    k, v = new_rows(T, H, D, "bf16", 6)[:, :, :].to(DEV), new_rows(T, H, D, "bf16", 7).to(DEV)
    k[:4], v[:4] = k[4:8], v[4:8]                             # finite rows only
    slots = torch.tensor([blocks[i // 16] * 16 + i % 16 for i in range(T)], device=DEV)
    pkv.kv_append_fp4(k, v, dk, dv, slots, 0.02, 0.02)
    lk, lv = pkv.kv_load_fp4(dk, dv, slots, 0.02, 0.02, dtype=torch.float32)
    small_k = torch.zeros(pkv.fp4_cache_shape(3, H, D), dtype=torch.uint8, device=DEV)
    small_v = torch.zeros_like(small_k)
    near = torch.arange(T, device=DEV)
    pkv.kv_append_fp4(k, v, small_k, small_v, near, 0.02, 0.02)
    sk, sv = pkv.kv_load_fp4(small_k, small_v, near, 0.02, 0.02, dtype=torch.float32)
    assert torch.equal(lk, sk) and torch.equal(lv, sv)
    q = torch.randn(1, 32, D, device=DEV, dtype=torch.bfloat16)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    for qq in (q, q.float()):
        far = pkv.paged_attention_fp4(qq, dk, dv, torch.tensor([blocks], dtype=torch.int32,
                                                              device=DEV), lens, 0.02, 0.02,
                                      max_context_len=T)
        here = pkv.paged_attention_fp4(qq, small_k, small_v,
                                       torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV),
                                       lens, 0.02, 0.02, max_context_len=T)
        assert torch.equal(far, here)
        del far, here


def test_refusals_on_the_device():
    keep = batch_on_device(W.Workload("fp4 refuse", 1, 8, 2, 128, "bf16", context_lens=[40],
                                      seed=2270))
    with pytest.raises(ValueError, match="one CUDA device"):
        pkv.paged_attention_fp4(keep["q"], keep["dk"], keep["dv"], keep["table"].cpu(),
                                keep["lens"], K_SCALE, V_SCALE, max_context_len=40)
    with pytest.raises(ValueError):
        keep["call"](out=torch.empty(1, 8, 128, device=DEV))      # another type
    with pytest.raises(pkv.PkvError):
        keep["call"](kernel=pkv.PKV_KERNEL_TC)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_fp4(keep["q"], keep["dk"], keep["dv"], keep["table"], keep["lens"],
                                K_SCALE, V_SCALE, max_context_len=49)   # past the table


def test_append_load_prefill():
    """A chunk's prefill over rows that are kept in 4 bits: load the cached rows
    into a 16-bit cache and attend there; against attention over the codes."""
    H, D, L = 2, 128, 70
    k, v = new_rows(L, H, D, "bf16", 8)[:], new_rows(L, H, D, "bf16", 9)[:]
    k[:4], v[:4] = k[4:8], v[4:8]
    NB = 6
    dk = torch.full(pkv.fp4_cache_shape(NB, H, D), 255, dtype=torch.uint8, device=DEV)
    dv = dk.clone()
    table = torch.tensor([[4, 0, 5, 2, 1]], dtype=torch.int32, device=DEV)
    pos = torch.arange(L, device=DEV)
    slots = table[0].long()[pos // 16] * 16 + pos % 16
    pkv.kv_append_fp4(k.to(DEV), v.to(DEV), dk, dv, slots, 0.02, 0.02)
    lk, lv = pkv.kv_load_fp4(dk, dv, slots, 0.02, 0.02, dtype=torch.float16)
    wk = torch.zeros(NB, H, 16, D, dtype=torch.float16, device=DEV)
    wv = torch.zeros_like(wk)
    pkv.kv_append(lk, lv, wk, wv, slots)
    Q = 12
    q = torch.randn(1, Q, 8, D, device=DEV).half()
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, Q], dtype=torch.int32, device=DEV)
    dense = pkv.paged_prefill_attention(q[0], wk, wv, table, lens, start, max_query_len=Q)
    codes = pkv.paged_attention_fp4(q, dk, dv, table, lens, 0.02, 0.02, max_context_len=L)[0]
    # the loaded rows carry one more rounding (2^-11 each): of a weight's exponent
    # |s| 2^-11, of a value 2^-11; both kernels round their weights to f16
    top = (lk.float().norm(dim=-1).max() * q.float().norm(dim=-1).max()).item() / math.sqrt(D)
    tol = (2 * top + 4) * 2.0 ** -11 * lv.float().abs().max().item()
    assert (dense.float() - codes.float()).abs().max().item() <= tol

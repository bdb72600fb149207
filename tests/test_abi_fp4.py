"""The 4-bit cache's and the row commit's entry points without a GPU: argument
errors return before anything reaches CUDA, and the planner's answers for the
4-bit cache type."""
import ctypes

import pytest
import torch

from paged_kv_cache_18_gb300 import binding, build
from tests.test_abi import tuning


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def rows_call(f, **kw):
    a = dict(k=16, v=16, kc=16, vc=16, slots=16, T=4, Hkv=2, D=128, bs=16, NB=10, dtype=1,
             ks=1.0, vs=1.0, err=None, stream=None)
    a.update(kw)
    return f(*a.values())


BAD_ROWS = [(dict(k=None), 1), (dict(vc=None), 1), (dict(slots=None), 1), (dict(T=-1), 1),
            (dict(Hkv=0), 1), (dict(dtype=3), 1), (dict(dtype=4), 1), (dict(NB=0), 1),
            (dict(ks=0.0), 1), (dict(vs=-1.0), 1), (dict(ks=float("nan")), 1),
            (dict(vs=float("inf")), 1), (dict(D=96), 2), (dict(D=512), 2), (dict(bs=32), 2),
            (dict(k=8), 5), (dict(vc=24), 5), (dict(slots=12), 5), (dict(err=2), 5),
            (dict(T=0, k=None), 0), (dict(T=0, D=80), 2)]


@pytest.mark.parametrize("kw,status", BAD_ROWS)
@pytest.mark.parametrize("name", ["pkv_kv_append_fp4", "pkv_kv_load_fp4"])
def test_row_call_argument_errors(L, name, kw, status):
    assert rows_call(getattr(L, name), **kw) == status


def attend(L, **kw):
    a = dict(out=16, q=16, k=16, v=16, table=16, max_blocks=8, lens=16, max_ctx=100, B=2, Q=1,
             Hq=8, Hkv=2, D=128, bs=16, NB=10, scale=0.1, dtype=1, ks=1.0, vs=1.0, tree=None,
             stride=0, ws=None, ws_bytes=0, opt=None, err=None, stream=None)
    a.update(kw)
    return L.pkv_paged_attention_fp4(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(Hq=7), 1), (dict(Q=0), 1), (dict(D=96), 2),
    (dict(bs=32), 2), (dict(dtype=3), 1), (dict(dtype=4), 1), (dict(max_ctx=129), 1),
    (dict(NB=0), 1), (dict(scale=float("inf")), 1), (dict(ks=0.0), 1), (dict(vs=float("nan")), 1),
    (dict(tree=16, Q=65), 1), (dict(tree=16, Q=3, stride=-1), 1), (dict(tree=12, Q=3), 5),
    (dict(k=8), 5), (dict(B=70000), 2), (dict(B=0, q=None), 0), (dict(max_ctx=-1), 1)])
def test_attention_argument_errors(L, kw, status):
    assert attend(L, **kw) == status


def test_the_type_is_refused_by_the_plain_entry_points(L):
    common = (16, 16, 16, 16, 16, 2, 16, 20, 1)
    assert L.pkv_paged_decode_attention(*common, 4, 4, 128, 16, 10, 0.1, 4, None, 0, None, None,
                                        None) == 1
    assert L.pkv_spec_verify_attention(*common, 2, 4, 4, 128, 16, 10, 0.1, 4, None, 0, None, None,
                                       None) == 1
    assert L.pkv_tree_verify_attention(*common, 2, 4, 4, 128, 16, 10, 0.1, 4, 16, 0, None, 0,
                                       None, None, None) == 1
    assert L.pkv_append_attention(16, 16, 16, 16, 16, 16, 16, 2, 16, 20, 1, 1, 4, 4, 128, 16, 10,
                                  0.1, 4, None, 0, None, None, None) == 1
    assert L.pkv_kv_append(16, 16, 16, 16, 16, 1, 4, 128, 16, 10, 4, None, None) == 1
    assert L.pkv_copy_blocks(16, 16, 16, 16, 1, 4, 72, 16, 10, 4, None, None) == 2   # not a D


@pytest.mark.parametrize("field", ["merge", "stages", "warp_tiles", "blocks_per_iter", "persistent"])
def test_launch_controls_that_do_not_apply_are_refused(L, field):
    opt = binding.Options()
    setattr(opt, field, 1)
    p = binding.Plan()
    assert L.pkv_attention_plan_for(2, 1, 8, 2, 128, 16, 100, 4, ctypes.byref(opt), 152, 0,
                                    ctypes.byref(p)) == 2


@pytest.mark.parametrize("B,Q,Hq,Hkv,D,ctx", [(4, 1, 6, 6, 64, 256), (32, 1, 40, 40, 128, 2048),
                                              (128, 1, 32, 8, 128, 4096), (2, 1, 32, 8, 128, 65536),
                                              (16, 5, 32, 8, 128, 8192), (16, 10, 32, 8, 128, 8192),
                                              (3, 7, 64, 2, 64, 1000), (5, 3, 16, 2, 256, 70),
                                              (1, 1, 1, 1, 64, 0), (1, 64, 64, 1, 128, 333)])
@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("split_blocks", [0, 7])
def test_plan_invariants(B, Q, Hq, Hkv, D, ctx, kernel, split_blocks):
    p = binding.plan_for(B, Q, Hq, Hkv, D, ctx, "fp4", num_sms=152, kernel=kernel,
                         split_blocks=split_blocks)
    rows = Hq // Hkv * Q
    assert p["rows_per_cta"] * p["row_chunks"] >= rows
    assert (p["rows_per_cta"] - 1) * p["row_chunks"] < rows
    assert p["smem_bytes"] <= 227 * 1024
    blocks = -(-ctx // 16)
    if p["split_target"] == 0:
        assert p["num_splits"] * p["split_blocks"] >= blocks
        assert (p["grid_x"], p["grid_y"], p["grid_z"]) == (p["num_splits"],
                                                           Hkv * p["row_chunks"], B)
    assert (p["workspace_bytes"] > 0) == (p["num_splits"] > 1 or p["split_target"] > 0)


def test_tcgen05_kernel_does_not_take_4_bit_caches(L):
    with pytest.raises(binding.PkvError):
        binding.plan_for(2, 1, 8, 2, 128, 100, "fp4", num_sms=152, kernel=binding.PKV_KERNEL_TC)


def commit(L, **kw):
    ptr = ctypes.c_void_p
    a = dict(k=(4096, 1 << 20), v=(2 << 20, 3 << 20), layers=2, table=16, max_blocks=8, lens=1024,
             path=16, max_path=3, path_lens=16, B=2, Q=5, Hkv=2, D=64, bs=16, NB=10, dtype=1,
             new=4096, err=None, stream=None)
    a.update(kw)
    for name in ("k", "v"):
        if a[name] is not None:
            a[name] = (ptr * len(a[name]))(*a[name])
    return L.pkv_commit_rows(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), 1), (dict(layers=513), 2), (dict(B=-1), 1), (dict(Q=0), 1), (dict(Q=65), 1),
    (dict(max_path=0), 1), (dict(max_path=65), 1), (dict(Hkv=0), 1), (dict(D=0), 1),
    (dict(NB=0), 1), (dict(max_blocks=0), 1), (dict(dtype=9), 1), (dict(bs=32), 2),
    (dict(D=4), 2), (dict(D=96, dtype=4), 2), (dict(B=0, table=None), 0), (dict(k=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(path=None), 1), (dict(path_lens=None), 1),
    (dict(path=2), 5), (dict(new=2), 5), (dict(err=3), 5),
    (dict(k=(4096, None)), 1), (dict(k=(4096, (1 << 20) + 8)), 5),
    (dict(new=1024), 1), (dict(new=1028), 1),                    # overlaps the lengths
    (dict(table=8192, new=8192 + 4 * 15), 1), (dict(path=8192, new=8192 + 20), 1),
    (dict(path_lens=8192, new=8196), 1),                         # or what else every warp reads
    (dict(k=(4096, 4096)), 1), (dict(v=(2 << 20, 4096)), 1),     # a tensor named twice
    (dict(k=(4096, 4096 + 10 * 2 * 16 * 64 * 2 - 16)), 1)])      # two that overlap
def test_commit_argument_errors(L, kw, status):
    assert commit(L, **kw) == status


def test_binding_refuses_before_the_library():
    kc = torch.zeros(binding.fp4_cache_shape(3, 2, 64), dtype=torch.uint8)
    rows = torch.zeros(4, 2, 64)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.kv_append_fp4(rows, rows, kc, kc, slots, 1.0, 1.0)
    with pytest.raises(ValueError, match="4-bit caches"):
        binding.kv_append_fp4(rows, rows, kc[..., :32], kc[..., :32], slots, 1.0, 1.0)
    with pytest.raises(ValueError, match="k_new"):
        binding.kv_append_fp4(rows[:, :1], rows[:, :1], kc, kc, slots, 1.0, 1.0)
    with pytest.raises(ValueError, match="slot_mapping"):
        binding.kv_load_fp4(kc, kc, slots.int(), 1.0, 1.0)
    with pytest.raises(ValueError, match="dtype"):
        binding.kv_load_fp4(kc, kc, slots, 1.0, 1.0, dtype=torch.float64)
    q, table, lens = torch.zeros(2, 4, 64), torch.zeros(2, 1, dtype=torch.int32), torch.ones(
        2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.paged_attention_fp4(q, kc, kc, table, lens, 1.0, 1.0)
    with pytest.raises(ValueError, match="q must"):
        binding.paged_attention_fp4(q[..., :32].contiguous(), kc, kc, table, lens, 1.0, 1.0)
    with pytest.raises(ValueError, match="tree_mask"):
        binding.paged_attention_fp4(q, kc, kc, table, lens, 1.0, 1.0,
                                    tree_mask=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="head_dim"):
        binding.fp4_cache_shape(4, 2, 80)
    c = torch.zeros(3, 2, 16, 64)
    p = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="one tensor per layer"):
        binding.commit_rows([c], [], table, lens, p, lens, 5)
    with pytest.raises(ValueError, match="one shape"):
        binding.commit_rows([c], [c.half()], table, lens, p, lens, 5)
    with pytest.raises(ValueError, match="path_lens"):
        binding.commit_rows([c], [c], table, lens, p, lens[:1], 5)
    with pytest.raises(ValueError, match="CUDA"):
        binding.commit_rows([c], [c.clone()], table, lens, p, lens, 5)


def test_split_wave_partition_plans():
    with tuning(split_waves=1):
        p = binding.plan_for(4, 1, 8, 2, 128, 5000, "fp4", num_sms=152)
    assert p["split_target"] > 0 and p["merge_kernel"] == 1

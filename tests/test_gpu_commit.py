"""commit_rows on the GPU: every byte of every cache against host moves."""
import numpy as np
import pytest
import torch

import paged_kv_cache_18_gb300 as pkv
from oracle import fp4
from paged_kv_cache_18_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(kind, layers, NB, H, D, seed):
    """Caches of random bytes: (tensors, host copies as [NB, H, 16, row] views)."""
    rng = np.random.default_rng(seed)
    out = []
    for i in range(2 * layers):
        if kind == "fp4":
            shape, dt = pkv.fp4_cache_shape(NB, H, D), torch.uint8
        else:
            dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
                  "fp8": torch.uint8}[kind]
            shape = (NB, H, 16, D)
        size = torch.tensor([], dtype=dt).element_size()
        raw = rng.integers(0, 256, int(np.prod(shape)) * size, dtype=np.uint8)
        out.append(torch.from_numpy(raw).to(DEV).view(dt).view(shape))
    return out[:layers], out[layers:]


def as_rows(t, kind, keys):
    """Host bytes of the rows: [NB, H, 16, bytes of a row]."""
    NB, H = t.shape[0], t.shape[1]
    raw = t.contiguous().view(torch.uint8).cpu().numpy()
    if kind != "fp4":
        return raw.reshape(NB, H, 16, -1)
    D = t.shape[-1] * 16 // 9
    tiles = raw.reshape(NB, H, 9 * D)
    return np.concatenate([tiles[..., fp4.code_place(D, keys)[:, ::2]],
                           tiles[..., fp4.scale_place(D, keys)]], -1)


def moved(rows, table, lens, paths, Q):
    new = rows.copy()
    for b, path in enumerate(paths):
        for i, node in enumerate(path):
            to, frm = lens[b] - Q + i, lens[b] - Q + node
            new[table[b, to // 16], :, to % 16] = rows[table[b, frm // 16], :, frm % 16]
    return new


def tables(lens, seed, spare=3):
    rng = np.random.default_rng(seed)
    need = [-(-n // 16) for n in lens]
    NB = sum(need) + spare
    perm = rng.permutation(NB).astype(np.int32)
    table = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, NB


def arrays(table, lens, paths, max_path=None):
    m = max_path or max(1, max(len(p) for p in paths))
    path = np.full((len(paths), m), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    return to(table), to(lens), to(path), to([len(p) for p in paths])


@pytest.mark.parametrize("kind,H,D", [("bf16", 2, 128), ("f16", 3, 64), ("f32", 1, 64),
                                      ("fp8", 5, 128), ("fp8", 1, 48), ("f32", 2, 256),
                                      ("fp4", 2, 64), ("fp4", 3, 128), ("fp4", 1, 256)])
@pytest.mark.parametrize("layers", [1, 3])
def test_every_byte(kind, H, D, layers):
    Q, lens = 10, [10, 16, 17, 25, 26, 100, 33]
    paths = [[0, 2, 7], [0], [], list(range(10)), [9], [1, 2, 3, 4, 9], [0, 1, 4]]
    table, NB = tables(lens, 3)
    ks, vs = make(kind, layers, NB, H, D, 4)
    want = [moved(as_rows(t, kind, i < layers), table, lens, paths, Q)
            for i, t in enumerate(ks + vs)]
    dt, dl, dp, dn = arrays(table, lens, paths)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q, fp4=kind == "fp4", error_word=err)
    assert pkv.read_error_word(err) == 0
    assert new.tolist() == [n - Q + len(p) for n, p in zip(lens, paths)]
    for i, t in enumerate(ks + vs):
        np.testing.assert_array_equal(as_rows(t, kind, i < layers), want[i])


@pytest.mark.parametrize("Q", [1, 33, 64])
def test_long_paths(Q):
    rng = np.random.default_rng(Q)
    lens = [Q, Q + 5, 200]
    paths = [sorted(rng.permutation(Q)[:rng.integers(1, Q + 1)].tolist()) for _ in lens]
    paths[0] = list(range(Q))
    paths[2] = list(range(Q // 2, Q))                          # every row moves
    table, NB = tables(lens, 5)
    ks, vs = make("bf16", 2, NB, 2, 64, 6)
    want = [moved(as_rows(t, "bf16", True), table, lens, paths, Q) for t in ks + vs]
    dt, dl, dp, dn = arrays(table, lens, paths, max_path=Q)
    pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q)
    for t, w in zip(ks + vs, want):
        np.testing.assert_array_equal(as_rows(t, "bf16", True), w)


def test_many_layers_take_several_launches():
    Q, lens, paths = 5, [20, 40], [[0, 3], [2, 4]]
    table, NB = tables(lens, 7, spare=0)
    ks, vs = make("fp8", 70, NB, 1, 16, 8)
    want = [moved(as_rows(t, "fp8", True), table, lens, paths, Q) for t in ks + vs]
    dt, dl, dp, dn = arrays(table, lens, paths)
    assert pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q).tolist() == [17, 37]
    for t, w in zip(ks + vs, want):
        np.testing.assert_array_equal(as_rows(t, "fp8", True), w)


def test_latent_caches():
    Q, lens, paths = 6, [30, 7], [[0, 4, 5], [1]]
    table, NB = tables(lens, 9)
    rng = np.random.default_rng(10)
    caches = [torch.from_numpy(rng.integers(0, 2 ** 15, (NB, 16, 576)).astype(np.int16)).to(DEV)
              .view(torch.bfloat16) for _ in range(3)]
    rows = [t.view(torch.uint8).cpu().numpy().reshape(NB, 1, 16, -1) for t in caches]
    dt, dl, dp, dn = arrays(table, lens, paths)
    pkv.commit_rows(caches, None, dt, dl, dp, dn, Q)
    for t, r in zip(caches, rows):
        np.testing.assert_array_equal(t.view(torch.uint8).cpu().numpy().reshape(r.shape),
                                      moved(r, table, lens, paths, Q))


def test_broken_paths_and_lengths_leave_their_sequences_alone():
    Q = 5
    good = [0, 3]
    cases = [([3, 0], 5), ([0, 0], 5), ([0, 5], 5), ([-2, 1], 5)]
    for path, code in cases:
        lens = [20, 20]
        table, NB = tables(lens, 11)
        ks, vs = make("bf16", 1, NB, 2, 64, 12)
        want = [moved(as_rows(t, "bf16", True), table, lens, [[], good], Q) for t in ks + vs]
        dt, dl, dp, dn = arrays(table, lens, [path, good])
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        new = pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q, error_word=err)
        assert pkv.read_error_word(err) == code and new.tolist() == [20, 17]
        for t, w in zip(ks + vs, want):
            np.testing.assert_array_equal(as_rows(t, "bf16", True), w)
    # counts and lengths out of range
    for lens_said, count, code in (([4, 20], 2, 3), ([33, 20], 2, 3), ([20, 20], -1, 5),
                                   ([20, 20], 3, 5)):
        table, NB = tables([20, 20], 13)
        ks, vs = make("bf16", 1, NB, 1, 64, 14)
        want = [moved(as_rows(t, "bf16", True), table, [20, 20], [[], good], Q) for t in ks + vs]
        dt, dl, dp, dn = arrays(table, lens_said, [good, good])
        dn[0] = count
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        new = pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q, error_word=err)
        assert pkv.read_error_word(err) == code and new.tolist() == [lens_said[0], 17]
        for t, w in zip(ks + vs, want):
            np.testing.assert_array_equal(as_rows(t, "bf16", True), w)


def test_rows_in_bad_blocks_are_left_out():
    Q, lens, paths = 5, [34, 34], [[1, 4], [0, 3]]
    table, NB = tables(lens, 15)
    ks, vs = make("f16", 1, NB, 1, 64, 16)
    before = [as_rows(t, "f16", True) for t in ks + vs]
    bad = table.copy()
    bad[0, 2] = NB                                             # rows 32, 33: nodes 3 and 4
    dt, dl, dp, dn = arrays(bad, lens, paths)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q, error_word=err)
    assert pkv.read_error_word(err) == 2 and new.tolist() == [31, 31]
    for t, r in zip(ks + vs, before):
        w = moved(r, table, lens, [[1], paths[1]], Q)          # node 1 still moves
        np.testing.assert_array_equal(as_rows(t, "f16", True), w)


def test_empty_batch():
    ks, vs = make("bf16", 1, 4, 1, 64, 17)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    new = pkv.commit_rows(ks, vs, torch.zeros(0, 2, dtype=torch.int32, device=DEV), none,
                          torch.zeros(0, 2, dtype=torch.int32, device=DEV), none, 5)
    assert new.shape == (0,)


def test_graph_replay_follows_new_paths():
    Q, lens = 6, [40, 25]
    table, NB = tables(lens, 18)
    ks, vs = make("bf16", 2, NB, 2, 64, 19)
    dt, dl, dp, dn = arrays(table, lens, [[0, 1], [0, 1]], max_path=4)
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q, new_lens=new)    # nothing moves
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.commit_rows(ks, vs, dt, dl, dp, dn, Q, new_lens=new)
    for paths in ([[0, 2, 5], [3]], [[1, 2, 3, 4], [0, 5]]):
        before = [as_rows(t, "bf16", True) for t in ks + vs]
        _, _, p, n = arrays(table, lens, paths, max_path=4)
        dp.copy_(p)
        dn.copy_(n)
        g.replay()
        assert new.tolist() == [lens[b] - Q + len(paths[b]) for b in range(2)]
        for t, r in zip(ks + vs, before):
            np.testing.assert_array_equal(as_rows(t, "bf16", True),
                                          moved(r, table, lens, paths, Q))


def test_append_verify_commit_decode_over_4_bit_caches():
    """Two layers of a tree step as a program runs it: the drafts' rows are
    appended, verified, the accepted path committed, and the next token decoded;
    the decode equals one over a cache that never held the rejected rows."""
    H, Hq, D, Q, layers = 2, 8, 128, 10, 2
    prefix = [37, 100]
    lens = [p + Q for p in prefix]
    path = [0, 2, 7]
    table, NB = tables([n + 1 for n in lens], 20)
    masks = torch.from_numpy(W.tree_mask_bits(W.medusa_parents((3, 2))).view(np.int64)).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(21)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    dt = torch.from_numpy(table).to(DEV)

    def slots(b, lo, hi):
        pos = torch.arange(lo, hi, device=DEV)
        return dt[b].long()[pos // 16] * 16 + pos % 16

    def fresh():
        return [torch.full(pkv.fp4_cache_shape(NB, H, D), 255, dtype=torch.uint8, device=DEV)
                for _ in range(2 * layers)]

    got, want = fresh(), fresh()
    new_lens = None
    for layer in range(layers):
        for b, p in enumerate(prefix):
            k, v = rand(p, H, D), rand(p, H, D)
            tk, tv = rand(Q, H, D), rand(Q, H, D)
            for c in (got, want):
                pkv.kv_append_fp4(k, v, c[layer], c[layers + layer], slots(b, 0, p), 0.01, 0.01)
            pkv.kv_append_fp4(tk, tv, got[layer], got[layers + layer], slots(b, p, p + Q), 0.01,
                              0.01)
            pkv.kv_append_fp4(tk[path].contiguous(), tv[path].contiguous(), want[layer],
                              want[layers + layer], slots(b, p, p + len(path)), 0.01, 0.01)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = rand(2, Q, Hq, D)
    tree = [pkv.paged_attention_fp4(q, got[i], got[layers + i], dt, dl, 0.01, 0.01,
                                    max_context_len=max(lens), tree_mask=masks)
            for i in range(layers)]
    dp = torch.tensor([path, path], dtype=torch.int32, device=DEV)
    dn = torch.tensor([3, 3], dtype=torch.int32, device=DEV)
    new_lens = pkv.commit_rows(got[:layers], got[layers:], dt, dl, dp, dn, Q, fp4=True)
    assert new_lens.tolist() == [p + 3 for p in prefix]
    # the path's nodes verified as a chain over the committed rows: the same sums
    for i in range(layers):
        chain = pkv.paged_attention_fp4(q[:, path].contiguous(), want[i], want[layers + i], dt,
                                        new_lens, 0.01, 0.01, max_context_len=max(lens))
        # the masked rows' place in the sums differs: output rounding and f16 weights
        assert (chain.float() - tree[i][:, path].float()).abs().max().item() <= 0.02
    nk, nv, nq = rand(2, H, D), rand(2, H, D), rand(2, Hq, D)
    at = torch.stack([slots(b, p + 3, p + 4)[0] for b, p in enumerate(prefix)])
    for i in range(layers):
        outs = []
        for c in (got, want):
            pkv.kv_append_fp4(nk, nv, c[i], c[layers + i], at, 0.01, 0.01)
            outs.append(pkv.paged_attention_fp4(nq, c[i], c[layers + i], dt, new_lens + 1, 0.01,
                                                0.01, max_context_len=max(lens)))
        assert torch.equal(*outs)
